// The 8-bit pool: its lifetime, and pages: copies inside it, and to and from a
// 16-bit pool.
//
// To 8 bits, a tile (16 rows x 128 of one block, kv head, K or V) gets the
// smallest power of two as its scale that holds its rows' largest magnitude;
// back, a code times the scale, rounded to 16 bits.  Both are bound by memory: 6
// KiB a tile either way (4 + 2), against a comparison, a product and a
// conversion an element.  A warp takes a tile whole, in registers: eight
// 16-byte loads in flight a lane, the largest magnitude by a warp reduction,
// and the codes as 8-byte stores, so each tile is read once and nothing else
// waits for it.
#include <new>

#include "codes8.cuh"
#include "rope_rows.cuh"

namespace pa {

constexpr int kPageWarps = 8;

// Whole-block copy: one CTA per pair; 16-byte vectors, and the exponents.
__global__ void copy_blocks8_kernel(uint4* codes, uint8_t* exps, const int32_t* src, const int32_t* dst, int n,
                                    long long num_blocks, int n_kv_heads, long long* err) {
  const int j = blockIdx.x;
  const long long s = src[j], d = dst[j];
  if (s < 0 || s >= num_blocks || d < 0 || d >= num_blocks) {
    if (threadIdx.x == 0) record_error(err, PA_ERR_DEVICE_CHECK, s < 0 || s >= num_blocks ? s : d);
    return;
  }
  const int vecs = n_kv_heads * (kPair8 / 16);
  const uint4* from = codes + s * vecs;
  uint4* to = codes + d * vecs;
  for (int x = threadIdx.x; x < vecs; x += blockDim.x) to[x] = from[x];
  for (int x = threadIdx.x; x < 2 * n_kv_heads; x += blockDim.x)
    exps[d * 2 * n_kv_heads + x] = exps[s * 2 * n_kv_heads + x];
}

struct PageArgs {
  uint16_t* k;          // 16-bit pool
  uint16_t* v;
  uint8_t* codes;       // 8-bit pool
  uint8_t* exps;
  const int32_t* from;  // [n] blocks
  const int32_t* to;    // [n]
  const int32_t* rows;  // [n] rows that count (to 8 bits), or null: all 16
  long long n_from, n_to;  // blocks of the two pools
  long long tiles;      // n * n_kv_heads * 2
  int n_kv_heads;
  long long* err;
};

// Tile number t of the call: pair j, kv head h, K or V; false if a block is out of range (reported once a pair).
__device__ __forceinline__ bool page_of(const PageArgs& A, long long t, int lane, long long* j, int* hx, long long* from,
                                        long long* to) {
  const int per = 2 * A.n_kv_heads;
  *j = t / per;
  *hx = static_cast<int>(t - *j * per);
  *from = A.from[*j];
  *to = A.to[*j];
  const bool ok_from = *from >= 0 && *from < A.n_from, ok_to = *to >= 0 && *to < A.n_to;
  if ((!ok_from || !ok_to) && *hx == 0 && lane == 0) record_error(A.err, PA_ERR_DEVICE_CHECK, ok_from ? *to : *from);
  return ok_from && ok_to;
}

template <bool kBf16, bool kE4M3>
__global__ void __launch_bounds__(32 * kPageWarps) quantize_kernel(const __grid_constant__ PageArgs A) {
  const int lane = threadIdx.x & 31;
  const long long t = static_cast<long long>(blockIdx.x) * kPageWarps + (threadIdx.x >> 5);
  if (t >= A.tiles) return;
  long long j, from, to;
  int hx;
  int n = A.rows ? A.rows[t / (2 * A.n_kv_heads)] : kBlock;
  if (!page_of(A, t, lane, &j, &hx, &from, &to)) return;
  if (n < 0 || n > kBlock) {
    if (hx == 0 && lane == 0) record_error(A.err, PA_ERR_DEVICE_CHECK, n);
    n = n < 0 ? 0 : kBlock;
  }
  const int h = hx >> 1;
  const uint4* src = reinterpret_cast<const uint4*>(((hx & 1) ? A.v : A.k) + (from * A.n_kv_heads + h) * (kTileBytes / 2));
  // vector 32 i + lane: row 2 i + lane / 16
  uint4 x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    x[i] = 2 * i + (lane >> 4) < n ? __ldcs(src + 32 * i + lane) : make_uint4(0, 0, 0, 0);
  // magnitudes compare as the bits of their 16-bit words; an infinity or a NaN is above them all
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) top = __vmaxu2(top, w[k] & 0x7fff7fffu);
  }
  uint32_t top1 = max(top & 0xffffu, top >> 16);
  top1 = __reduce_max_sync(0xffffffffu, top1);
  const uint32_t amax = kBf16 ? top1 << 16 : (top1 >= 0x7c00u ? 0x7f800000u : __float_as_uint(__half2float(__ushort_as_half(top1))));
  const int e = exponent_for<kE4M3>(amax);
  const float inv = inverse_scale(e);
  uint2* dst = reinterpret_cast<uint2*>(A.codes + ((to * A.n_kv_heads + h) * 2 + (hx & 1)) * kTile8);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float f[8];
    unpack8f<kBf16>(x[i], f);
    if (2 * i + (lane >> 4) < n)
      __stcs(dst + 32 * i + lane, make_uint2(pack_codes<kE4M3>(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                                             pack_codes<kE4M3>(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv)));
  }
  if (lane == 0) A.exps[to * (2 * A.n_kv_heads) + hx] = static_cast<uint8_t>(e);
}

// A value that does not fit in 16 bits (a code rounded up next to the type's
// largest number) becomes that number; NaN stays.
template <bool kBf16>
__device__ __forceinline__ float saturate16(float x) {
  const float top = kBf16 ? __uint_as_float(0x7f7f0000u) : 65504.f;
  return x > top ? top : (x < -top ? -top : x);
}

template <bool kBf16, bool kE4M3>
__global__ void __launch_bounds__(32 * kPageWarps) dequantize_kernel(const __grid_constant__ PageArgs A) {
  const int lane = threadIdx.x & 31;
  const long long t = static_cast<long long>(blockIdx.x) * kPageWarps + (threadIdx.x >> 5);
  if (t >= A.tiles) return;
  long long j, from, to;
  int hx;
  if (!page_of(A, t, lane, &j, &hx, &from, &to)) return;
  const int h = hx >> 1;
  const uint2* src = reinterpret_cast<const uint2*>(A.codes + ((from * A.n_kv_heads + h) * 2 + (hx & 1)) * kTile8);
  const int e = A.exps[from * (2 * A.n_kv_heads) + hx];
  uint2 c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = __ldcs(src + 32 * i + lane);
  const float s = scale_of(e);
  uint4* dst = reinterpret_cast<uint4*>(((hx & 1) ? A.v : A.k) + (to * A.n_kv_heads + h) * (kTileBytes / 2));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float4 a = codes_to_float4<kE4M3>(c[i].x), b = codes_to_float4<kE4M3>(c[i].y);
    float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = saturate16<kBf16>(f[k] * s);
    __stcs(dst + 32 * i + lane, pack8f<kBf16>(f));
  }
}

// Arguments of a page call and its launch; `back`: from 8 bits to 16.
static int pages(pa_pool_t p, pa_pool8_t p8, const int32_t* from, const int32_t* to, const int32_t* rows, int n,
                 bool back, void* stream) {
  if (!p || !p8 || n < 0 || (n > 0 && (!from || !to))) return PA_ERR_INVALID;
  if (p->n_kv_heads != p8->n_kv_heads || p->device != p8->device) return PA_ERR_INVALID;
  if (n == 0) return PA_OK;
  if (!on_pool_device(p8)) return PA_ERR_INVALID;
  PageArgs A{};
  A.k = static_cast<uint16_t*>(p->k);
  A.v = static_cast<uint16_t*>(p->v);
  A.codes = p8->codes;
  A.exps = p8->exps;
  A.from = from;
  A.to = to;
  A.rows = rows;
  A.n_from = back ? p8->num_blocks : p->num_blocks;
  A.n_to = back ? p->num_blocks : p8->num_blocks;
  A.n_kv_heads = p->n_kv_heads;
  A.tiles = 2ll * n * p->n_kv_heads;
  A.err = p8->err;
  const long long ctas = (A.tiles + kPageWarps - 1) / kPageWarps;
  if (ctas > 0x7fffffffll) return PA_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(ctas)), block(32 * kPageWarps);
  cudaStream_t st = as_stream(stream);
  const bool bf16 = p->dtype == PA_BF16, e4m3 = p8->dtype == PA_E4M3;
  if (back) {
    if (bf16)
      e4m3 ? dequantize_kernel<true, true><<<grid, block, 0, st>>>(A) : dequantize_kernel<true, false><<<grid, block, 0, st>>>(A);
    else
      e4m3 ? dequantize_kernel<false, true><<<grid, block, 0, st>>>(A) : dequantize_kernel<false, false><<<grid, block, 0, st>>>(A);
  } else {
    if (bf16)
      e4m3 ? quantize_kernel<true, true><<<grid, block, 0, st>>>(A) : quantize_kernel<true, false><<<grid, block, 0, st>>>(A);
    else
      e4m3 ? quantize_kernel<false, true><<<grid, block, 0, st>>>(A) : quantize_kernel<false, false><<<grid, block, 0, st>>>(A);
  }
  return cuda_status(cudaGetLastError());
}

}  // namespace pa

using namespace pa;

extern "C" {

size_t pa_pool8_bytes(int num_blocks, int block_size, int n_kv_heads, int d_head, int dtype) {
  if (num_blocks <= 0 || n_kv_heads <= 0 || block_size != kBlock || d_head != kHeadDim) return 0;
  if (dtype != PA_E4M3 && dtype != PA_INT8) return 0;
  return static_cast<size_t>(num_blocks) * n_kv_heads * kTile8;
}

int pa_pool8_create(int num_blocks, int block_size, int n_kv_heads, int d_head, int dtype, pa_pool8_t* out) {
  if (!out || num_blocks <= 0 || n_kv_heads <= 0) return PA_ERR_INVALID;
  if (block_size != kBlock || d_head != kHeadDim) return PA_ERR_UNSUPPORTED;
  if (dtype != PA_E4M3 && dtype != PA_INT8) return PA_ERR_UNSUPPORTED;
  // (offsets inside a block are 32-bit ints)
  if (n_kv_heads > PA_MAX_KV_HEADS) return PA_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_blocks) * n_kv_heads * kBlock > 0x7fffffffll) return PA_ERR_UNSUPPORTED;
  *out = nullptr;
  pa_pool8* p = new (std::nothrow) pa_pool8();
  if (!p) return PA_ERR_OOM;
  p->num_blocks = num_blocks;
  p->n_kv_heads = n_kv_heads;
  p->dtype = dtype;
  if (cudaGetDevice(&p->device) != cudaSuccess) { delete p; return PA_ERR_CUDA; }
  const size_t tiles = static_cast<size_t>(num_blocks) * n_kv_heads;
  const size_t claims = static_cast<size_t>(num_blocks) * claim_groups(n_kv_heads) * sizeof(uint32_t);
  int status = PA_OK;
  if (cudaMalloc(&p->codes, tiles * kPair8) != cudaSuccess || cudaMalloc(&p->exps, tiles * 2) != cudaSuccess ||
      cudaMalloc(&p->claims, claims) != cudaSuccess || cudaMalloc(&p->err, 2 * sizeof(long long)) != cudaSuccess)
    status = PA_ERR_OOM;
  else if (cudaMemset(p->codes, 0, tiles * kPair8) != cudaSuccess || cudaMemset(p->exps, 0, tiles * 2) != cudaSuccess ||
           cudaMemset(p->claims, 0, claims) != cudaSuccess ||
           cudaMemset(p->err, 0, 2 * sizeof(long long)) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess ||
           !encode_pool8_map(&p->tmap, p->codes, static_cast<long long>(tiles)))
    status = PA_ERR_CUDA;
  if (status != PA_OK) {
    cudaFree(p->codes);
    cudaFree(p->exps);
    cudaFree(p->claims);
    cudaFree(p->err);
    cudaGetLastError();
    delete p;
    return status;
  }
  *out = p;
  return PA_OK;
}

int pa_pool8_destroy(pa_pool8_t p) {
  if (!p) return PA_OK;
  int prev = 0;
  cudaGetDevice(&prev);
  cudaSetDevice(p->device);
  cudaDeviceSynchronize();
  cudaFree(p->codes);
  cudaFree(p->exps);
  cudaFree(p->claims);
  cudaFree(p->err);
  cudaSetDevice(prev);
  delete p;
  return PA_OK;
}

int pa_pool8_info(pa_pool8_t p, void** codes, void** exponents) {
  if (!p) return PA_ERR_INVALID;
  if (codes) *codes = p->codes;
  if (exponents) *exponents = p->exps;
  return PA_OK;
}

int pa_copy_blocks8(pa_pool8_t p, const int32_t* src, const int32_t* dst, int n, void* stream) {
  if (!p || n < 0 || (n > 0 && (!src || !dst))) return PA_ERR_INVALID;
  if (n == 0) return PA_OK;
  if (!on_pool_device(p)) return PA_ERR_INVALID;
  copy_blocks8_kernel<<<n, 256, 0, as_stream(stream)>>>(reinterpret_cast<uint4*>(p->codes), p->exps, src, dst, n,
                                                        p->num_blocks, p->n_kv_heads, p->err);
  return cuda_status(cudaGetLastError());
}

int pa_quantize_blocks(pa_pool_t pool, const int32_t* src, pa_pool8_t pool8, const int32_t* dst, const int32_t* rows,
                       int n, void* stream) {
  return pages(pool, pool8, src, dst, rows, n, false, stream);
}

int pa_dequantize_blocks(pa_pool8_t pool8, const int32_t* src, pa_pool_t pool, const int32_t* dst, int n, void* stream) {
  return pages(pool, pool8, src, dst, nullptr, n, true, stream);
}

int pa_check8(pa_pool8_t p, void* stream, int64_t* detail) {
  if (!p) return PA_ERR_INVALID;
  return check_error_word(p->err, stream, detail);
}

}  // extern "C"
