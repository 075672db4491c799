// Rows of new tokens on their way into the cache: rotary positions, and RMS
// norms before them.  Shared by the append into a 16-bit pool (all rows) and
// into an 8-bit pool (query rows here, K and V rows by blocks).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pa_internal.h"

namespace pa {

constexpr int kMaxPairs = kHeadDim / 2;
constexpr int kRopeThreads = 128;

struct RopeArgs {
  const uint16_t* q;   // token stride q_stride, heads [n_q_heads][128]
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* q_out;
  uint16_t* k_pool;
  uint16_t* v_pool;
  const int32_t* positions;  // [n_axes][n_tok]
  const float* inv_freq;     // [rot / 2]
  const int64_t* slots;      // [n_tok]
  const uint16_t* q_weight;  // [128] or null: rows are not normed
  const uint16_t* k_weight;
  long long q_stride, k_stride, v_stride, q_out_stride;
  long long n_tok, num_slots;
  int Hq, Hkv, half_vecs;    // half_vecs = rot / 16: lanes of a row that turn
  int interleaved;
  int rows;                  // rows of a token that turn_rows takes: Hq + 2 Hkv, or the Hq query rows alone
  int chunks;                // warps a token's rows are cut into
  float eps;
  long long* err;
  uint32_t axis[kMaxPairs / 16];  // two bits a pair (a byte each would be 32 reads of constant memory a warp)
};

// Angle of position p and frequency f as turns in [-1/2, 1/2], computed in
// two floats: f / (2 pi) = g + g_lo to 2^-48, p = a + b with both parts and
// both products' rounding errors exact, so the turns lost in the reduction
// stay below 2^-23 + |p| 2^-50 for every 32-bit position (a product rounded
// to 32 bits would be off by radians at p = 2^24).
__device__ __forceinline__ float turns(int p, float f) {
  constexpr double kInv2Pi = 0.15915494309189533577;
  constexpr float kHi = static_cast<float>(kInv2Pi);
  constexpr float kLo = static_cast<float>(kInv2Pi - static_cast<double>(kHi));
  const float g = f * kHi;
  const float g_lo = fmaf(f, kLo, fmaf(f, kHi, -g));
  const int hi = p >> 12;  // floor: p = hi * 4096 + lo, 0 <= lo < 4096
  const float a = static_cast<float>(hi) * 4096.f, b = static_cast<float>(p - (hi << 12));
  const float u = a * g, w = b * g;
  const float eu = fmaf(a, g, -u), ew = fmaf(b, g, -w);
  float r = (u - rintf(u)) + (w - rintf(w));
  r += (eu + ew) + (a + b) * g_lo;
  return r - rintf(r);
}

// cos and sin of pair f of token t.
__device__ __forceinline__ float2 cos_sin(const RopeArgs& A, long long t, int f) {
  const uint32_t word = f < 32 ? (f < 16 ? A.axis[0] : A.axis[1]) : (f < 48 ? A.axis[2] : A.axis[3]);
  const int p = A.positions[((word >> (2 * (f & 15))) & 3) * A.n_tok + t];
  float c, s;
  sincospif(2.f * turns(p, A.inv_freq[f]), &s, &c);
  return make_float2(c, s);
}

template <bool kBf16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (kBf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <bool kBf16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if (kBf16) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
  }
  __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}
template <bool kBf16>
__device__ __forceinline__ void unpack8f(const uint4& v, float f[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 x = unpack2<kBf16>(w[k]);
    f[2 * k] = x.x;
    f[2 * k + 1] = x.y;
  }
}
template <bool kBf16>
__device__ __forceinline__ uint4 pack8f(const float f[8]) {
  return make_uint4(pack2<kBf16>(f[0], f[1]), pack2<kBf16>(f[2], f[3]), pack2<kBf16>(f[4], f[5]),
                    pack2<kBf16>(f[6], f[7]));
}

// 1 / rms of a row of 128 whose 8 lanes (an aligned octet) hold 16 elements
// each; every lane of the warp takes part.  The sum of squares is fp32: 128
// terms of one sign, off by at most 2^-20 of itself.
__device__ __forceinline__ float inverse_rms(const float a[8], const float b[8], float eps) {
  float s = 0.f, z = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    s = fmaf(a[k], a[k], s);
    z = fmaf(b[k], b[k], z);
  }
  s += z;
  s += __shfl_xor_sync(0xffffffffu, s, 1);
  s += __shfl_xor_sync(0xffffffffu, s, 2);
  s += __shfl_xor_sync(0xffffffffu, s, 4);
  return rsqrtf(fmaf(s, 1.f / kHeadDim, eps));
}

// x r w for a lane's 16 elements; w0 and w1 are the weights of its two vectors.
template <bool kBf16>
__device__ __forceinline__ void scale_row(float a[8], float b[8], float r, const uint4& w0, const uint4& w1) {
  float w[8];
  unpack8f<kBf16>(w0, w);
#pragma unroll
  for (int k = 0; k < 8; ++k) a[k] = a[k] * r * w[k];
  unpack8f<kBf16>(w1, w);
#pragma unroll
  for (int k = 0; k < 8; ++k) b[k] = b[k] * r * w[k];
}

// Turns a lane's 8 pairs: (a[k], b[k]) in halves, adjacent elements of a and
// then of b interleaved.  cs(k) is the pair's cos and sin.
template <class CosSin>
__device__ __forceinline__ void turn_row(float a[8], float b[8], bool interleaved, CosSin cs) {
  if (interleaved) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 ca = cs(k), cb = cs(4 + k);
      const float x = a[2 * k], y = a[2 * k + 1], u = b[2 * k], w = b[2 * k + 1];
      a[2 * k] = x * ca.x - y * ca.y;
      a[2 * k + 1] = y * ca.x + x * ca.y;
      b[2 * k] = u * cb.x - w * cb.y;
      b[2 * k + 1] = w * cb.x + u * cb.y;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 c = cs(k);
      const float x = a[k], y = b[k];
      a[k] = x * c.x - y * c.y;
      b[k] = y * c.x + x * c.y;
    }
  }
}

// One warp (number w) per (token, chunk of its rows); 8 lanes per row, two
// 16-byte vectors each, so a lane turns the 8 pairs 8j .. 8j + 7 of its row
// (lane j < half_vecs: vectors j and j + half_vecs, or 2j and 2j + 1
// interleaved) or copies vectors 2j and 2j + 1.  U row quads of a warp are
// loaded before the first is turned.  Products and sums are fp32; one rounding
// to 16 bits.  s_cs: the warp's kMaxPairs entries of shared memory.
template <bool kBf16, int U, bool kNorm>
__device__ __forceinline__ void turn_rows(const RopeArgs& A, long long w, float2* s_cs) {
  const int lane = threadIdx.x & 31;
  const long long t = w / A.chunks;
  if (t >= A.n_tok) return;
  const int chunk = static_cast<int>(w - t * A.chunks);
  const int rows = A.rows;
  const int j = lane & 7, sub = lane >> 3;
  const bool turn = j < A.half_vecs;
  const int v0 = turn && !A.interleaved ? j : 2 * j;
  const int v1 = turn && !A.interleaved ? j + A.half_vecs : 2 * j + 1;

  // every row is loaded before the slot is known; a token that keeps out of
  // the cache just does not store its K and V
  const long long slot = A.slots[t];
  uint4 x[U][2];
  const int r0 = chunk * 4 * U + sub;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = r0 + 4 * u;
    if (kNorm) x[u][0] = x[u][1] = make_uint4(0, 0, 0, 0);  // (all lanes take part in the rows' sums)
    if (r >= rows) continue;
    const int h = r < A.Hq ? r : (r < A.Hq + A.Hkv ? r - A.Hq : r - A.Hq - A.Hkv);
    const uint16_t* base = r < A.Hq ? A.q + t * A.q_stride
                                    : (r < A.Hq + A.Hkv ? A.k + t * A.k_stride : A.v + t * A.v_stride);
    const uint4* src = reinterpret_cast<const uint4*>(base + h * kHeadDim);
    x[u][0] = src[v0];
    x[u][1] = src[v1];
  }

  // this token's angles: pair f by lane f % 32
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int f = lane + 32 * e;
    if (f < 8 * A.half_vecs) s_cs[f] = cos_sin(A, t, f);
  }
  __syncwarp();
  float2 cs[8];
  if (turn) {
#pragma unroll
    for (int e = 0; e < 8; ++e) cs[e] = s_cs[8 * j + e];
  }

  const bool to_cache = slot >= 0 && slot < A.num_slots;
  if (slot >= A.num_slots && lane == 0) record_error(A.err, PA_ERR_DEVICE_CHECK, slot);
  const long long row = (slot >> 4) * A.Hkv * kBlock + (slot & 15);  // of kv head 0
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = r0 + 4 * u;
    const bool takes_part = r < rows && (r < A.Hq || to_cache);
    uint16_t* to = r < A.Hq ? A.q_out + t * A.q_out_stride + r * kHeadDim
                            : (r < A.Hq + A.Hkv ? A.k_pool + (row + (r - A.Hq) * kBlock) * kHeadDim
                                                : A.v_pool + (row + (r - A.Hq - A.Hkv) * kBlock) * kHeadDim);
    uint4* dst = reinterpret_cast<uint4*>(to);
    if (kNorm) {
      float a[8], b[8];
      unpack8f<kBf16>(x[u][0], a);
      unpack8f<kBf16>(x[u][1], b);
      const float rr = inverse_rms(a, b, A.eps);
      if (!takes_part) continue;
      if (r < A.Hq + A.Hkv) {
        const uint16_t* weight = r < A.Hq ? A.q_weight : A.k_weight;
        if (weight)
          scale_row<kBf16>(a, b, rr, __ldg(reinterpret_cast<const uint4*>(weight) + v0),
                           __ldg(reinterpret_cast<const uint4*>(weight) + v1));
        if (turn) turn_row(a, b, A.interleaved != 0, [&](int k) { return cs[k]; });
        x[u][0] = pack8f<kBf16>(a);
        x[u][1] = pack8f<kBf16>(b);
      }
      dst[v0] = x[u][0];
      dst[v1] = x[u][1];
      continue;
    }
    if (!takes_part) continue;
    if (turn && r < A.Hq + A.Hkv) {
      float a[8], b[8];
      unpack8f<kBf16>(x[u][0], a);
      unpack8f<kBf16>(x[u][1], b);
      turn_row(a, b, A.interleaved != 0, [&](int k) { return cs[k]; });
      x[u][0] = pack8f<kBf16>(a);
      x[u][1] = pack8f<kBf16>(b);
    }
    dst[v0] = x[u][0];
    dst[v1] = x[u][1];
  }
}

// Checks of the two appends' arguments, which they fill in (rope.cu); a status.
int rope_axes(RopeArgs* A, const uint8_t* axis_of_pair, int n_axes, int rot_dim, int n_q_heads);
int rope_rows(RopeArgs* A, const void* q, int64_t q_stride, int n_q_heads, const void* k_new, int64_t k_stride,
              const void* v_new, int64_t v_stride, int n_kv_heads, const int32_t* positions, const float* inv_freq,
              const int64_t* slot_mapping, int n_tok, void* q_out, int64_t q_out_stride);
inline bool norm_args_ok(const void* q_weight, const void* k_weight, float eps) {
  return eps >= 0.f && eps <= 3.4028234e38f &&
         !((reinterpret_cast<uintptr_t>(q_weight) | reinterpret_cast<uintptr_t>(k_weight)) & 15);
}

}  // namespace pa
