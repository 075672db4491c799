// Device helpers shared by the translation units: mbarriers and bounded waits,
// 16-bit packing, output stores.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pa_internal.h"

namespace pa {

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ long long global_ns() {
  long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Bounded wait on an mbarrier phase.  Returns false if the CTA is aborting or
// the wait ran out (then it records PA_ERR_TIMEOUT and raises the abort flag).
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                           long long limit_ns, long long* err, int site) {
  if (mbar_try_wait(bar, parity)) return true;
  long long t0 = global_ns();
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (global_ns() - t0 > limit_ns) {
      *abort_flag = 1;
      record_error(err, PA_ERR_TIMEOUT, site);
      return false;
    }
  }
}

// Two fp32 values as a 16-bit pair (a in the low half), rounded to nearest;
// pack_lo packs what rounding left over, so hi + lo carries a to ~2^-17.
template <bool kBf16>
__device__ __forceinline__ uint32_t pack_hi(float a, float b) {
  if (kBf16) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
  }
  __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}
template <bool kBf16>
__device__ __forceinline__ uint32_t pack_lo(float a, float b) {
  if (kBf16) {
    const float ra = a - __bfloat162float(__float2bfloat16_rn(a));
    const float rb = b - __bfloat162float(__float2bfloat16_rn(b));
    __nv_bfloat162 h = __floats2bfloat162_rn(ra, rb);
    return *reinterpret_cast<uint32_t*>(&h);
  }
  const float ra = a - __half2float(__float2half_rn(a));
  const float rb = b - __half2float(__float2half_rn(b));
  __half2 h = __floats2half2_rn(ra, rb);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ void store_out(void* out, long long idx, float x, int out_dtype) {
  if (out_dtype == PA_FP32)
    static_cast<float*>(out)[idx] = x;
  else if (out_dtype == PA_BF16)
    static_cast<__nv_bfloat16*>(out)[idx] = __float2bfloat16_rn(x);
  else
    static_cast<__half*>(out)[idx] = __float2half_rn(x);
}

// Four consecutive outputs starting at an index that is a multiple of 4.
__device__ __forceinline__ void store_out4(void* out, long long idx, float a, float b, float c, float d,
                                           int out_dtype) {
  if (out_dtype == PA_FP32) {
    *reinterpret_cast<float4*>(static_cast<float*>(out) + idx) = make_float4(a, b, c, d);
  } else if (out_dtype == PA_BF16) {
    __nv_bfloat162 h0 = __floats2bfloat162_rn(a, b), h1 = __floats2bfloat162_rn(c, d);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + idx) =
        make_uint2(*reinterpret_cast<uint32_t*>(&h0), *reinterpret_cast<uint32_t*>(&h1));
  } else {
    __half2 h0 = __floats2half2_rn(a, b), h1 = __floats2half2_rn(c, d);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + idx) =
        make_uint2(*reinterpret_cast<uint32_t*>(&h0), *reinterpret_cast<uint32_t*>(&h1));
  }
}

}  // namespace pa
