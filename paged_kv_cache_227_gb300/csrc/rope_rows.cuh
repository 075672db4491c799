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
  int rows;                  // rows of a token: Hq + 2 Hkv, or the Hq query rows alone
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

// Packed pairs of fp32: one instruction for two elements.
__device__ __forceinline__ unsigned long long bits2(float2 a) { return *reinterpret_cast<unsigned long long*>(&a); }
__device__ __forceinline__ float2 floats2(unsigned long long a) { return *reinterpret_cast<float2*>(&a); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)));
  return floats2(d);
}
__device__ __forceinline__ float2 sub2(float2 a, float2 b) {
  unsigned long long d;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)));
  return floats2(d);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
  return floats2(d);
}

// Cosines and sines of a row's angles, in shared memory; pair f = 8j + e, of lane
// j, is element e % 4 of vector 8 (e / 4) + j, so that the lanes of a row read 128
// bytes on end.  They are those of turn_rows, to the last bit: 2^-24 off, where the
// hardware's approximations would be 2^-21 (us with those and now: 8,192 tokens 36.2
// and 36.4, 64 tokens 2.62 and 2.71; into 8 bits 7,900 tokens 42.8 and 43.8, 64 tokens
// 5.6 and 5.7).
struct Angles {
  float4 c[kMaxPairs / 4], s[kMaxPairs / 4], minus_s[kMaxPairs / 4];
};

// A lane's part of a row of 128: 8 lanes (an aligned octet) hold it, lane j the 8
// elements from 8 v0 (a) and the 8 from 8 v1 (b).
struct RowPart {
  float2 a[4], b[4];
  template <bool kBf16>
  __device__ __forceinline__ void unpack(const uint4& x, const uint4& y) {
    a[0] = unpack2<kBf16>(x.x), a[1] = unpack2<kBf16>(x.y), a[2] = unpack2<kBf16>(x.z), a[3] = unpack2<kBf16>(x.w);
    b[0] = unpack2<kBf16>(y.x), b[1] = unpack2<kBf16>(y.y), b[2] = unpack2<kBf16>(y.z), b[3] = unpack2<kBf16>(y.w);
  }
  __device__ static __forceinline__ unsigned octet() { return 0xffu << (threadIdx.x & 24); }
  // mean(x^2) + eps of the row, for the lanes of `who` (whole rows).  128 terms of one
  // sign in chains of 8: off by at most 2^-19 of itself.
  __device__ __forceinline__ float mean_square(float eps, unsigned who = 0xffffffffu) const {
    float2 s = mul2(a[0], a[0]);
#pragma unroll
    for (int k = 1; k < 4; ++k) s = fma2(a[k], a[k], s);
#pragma unroll
    for (int k = 0; k < 4; ++k) s = fma2(b[k], b[k], s);
    float t = s.x + s.y;
    t += __shfl_xor_sync(who, t, 1);
    t += __shfl_xor_sync(who, t, 2);
    t += __shfl_xor_sync(who, t, 4);
    return fmaf(t, 1.f / kHeadDim, eps);
  }
  // Where the mean leaves the range in which squares count in full (those below 2^-149
  // are lost: together less than 2^-42 of 2^-100), and its root and the row's products
  // stay in theirs.  Bits of a sum that is not negative compare as numbers.
  __device__ static __forceinline__ bool far(float mean) {
    return __float_as_uint(mean) - 0x0d800000u >= 0x7f800000u - 0x0d800000u;  // not in [2^-100, infinity)
  }
  // Multiplies the row by the power of two that takes the larger one of its largest
  // magnitude and sqrt(eps) to about 1 (none if it is not finite), which leaves
  // x / sqrt(mean(x^2) + eps) as it is with what is returned for eps.
  __device__ __forceinline__ float to_unit_size(float eps) {
    float m = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      m = fmaxf(fmaxf(m, fabsf(a[k].x)), fabsf(a[k].y));
      m = fmaxf(fmaxf(m, fabsf(b[k].x)), fabsf(b[k].y));
    }
    const int e = static_cast<int>(__reduce_max_sync(octet(), __float_as_uint(m)) >> 23);  // exponents of both, biased
    int up = 127 - e;
    if (eps > 0.f) up = min(up, (127 - static_cast<int>(__float_as_uint(eps) >> 23)) >> 1);
    const float r = e == 255 ? 1.f : __int_as_float((127 + max(up, -126)) << 23);
    times(r);
    return eps * r * r;
  }
  __device__ __forceinline__ void times(const RowPart& w) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      a[k] = mul2(a[k], w.a[k]);
      b[k] = mul2(b[k], w.b[k]);
    }
  }
  __device__ __forceinline__ void times(float r) {
    const float2 rr = make_float2(r, r);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      a[k] = mul2(a[k], rr);
      b[k] = mul2(b[k], rr);
    }
  }
  // Turns the lane's 8 pairs: elements k of a and b in halves, adjacent elements of
  // a and then of b interleaved.
  __device__ __forceinline__ void turn(bool interleaved, const Angles& t, int j) {
    const float4 c0 = t.c[j], c1 = t.c[8 + j], s0 = t.s[j], s1 = t.s[8 + j];
    const float2 cc[4] = {{c0.x, c0.y}, {c0.z, c0.w}, {c1.x, c1.y}, {c1.z, c1.w}};
    const float2 ss[4] = {{s0.x, s0.y}, {s0.z, s0.w}, {s1.x, s1.y}, {s1.z, s1.w}};
    if (!interleaved) {
      const float4 m0 = t.minus_s[j], m1 = t.minus_s[8 + j];
      const float2 mm[4] = {{m0.x, m0.y}, {m0.z, m0.w}, {m1.x, m1.y}, {m1.z, m1.w}};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 x = fma2(b[k], mm[k], mul2(a[k], cc[k]));
        b[k] = fma2(a[k], ss[k], mul2(b[k], cc[k]));
        a[k] = x;
      }
      return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // pair k of the lane: element pair k of a, or k - 4 of b
      const float2 x = a[k], y = b[k];
      const float cx = k & 1 ? cc[k >> 1].y : cc[k >> 1].x, sx = k & 1 ? ss[k >> 1].y : ss[k >> 1].x;
      const float cy = k & 1 ? cc[2 + (k >> 1)].y : cc[2 + (k >> 1)].x, sy = k & 1 ? ss[2 + (k >> 1)].y : ss[2 + (k >> 1)].x;
      a[k] = make_float2(x.x * cx - x.y * sx, x.y * cx + x.x * sx);
      b[k] = make_float2(y.x * cy - y.y * sy, y.y * cy + y.x * sy);
    }
  }
};
// A row whose mean is far, and its mean, as to_unit_size leaves them; not inlined, which
// costs the latency of a decode step less (2.76 -> 2.70 us).
struct FarRow {
  RowPart y;
  float mean;
};
static __device__ __noinline__ FarRow far_row(RowPart y, float eps) {
  eps = y.to_unit_size(eps);
  const float mean = y.mean_square(eps, RowPart::octet());
  return {y, mean};
}
template <bool kBf16>
__device__ __forceinline__ uint4 pack_part(const float2 (&x)[4]) {
  return make_uint4(pack2<kBf16>(x[0].x, x[0].y), pack2<kBf16>(x[1].x, x[1].y), pack2<kBf16>(x[2].x, x[2].y),
                    pack2<kBf16>(x[3].x, x[3].y));
}

// kThreads threads (a CTA's, or a warp's) take rows t0 .. t0 + rows - 1.
template <int kThreads>
__device__ __forceinline__ void fill_angles(const RopeArgs& A, Angles* to, long long t0, int rows) {
  const int pairs = 8 * A.half_vecs, thread = threadIdx.x % kThreads;
#pragma unroll 4
  for (int x = thread; x < rows * kMaxPairs; x += kThreads) {
    const int r = x / kMaxPairs, f = x % kMaxPairs;
    if (f >= pairs) continue;
    const uint32_t word = f < 32 ? (f < 16 ? A.axis[0] : A.axis[1]) : (f < 48 ? A.axis[2] : A.axis[3]);
    const int p = A.positions[((word >> (2 * (f & 15))) & 3) * A.n_tok + t0 + r];
    float sine, cosine;
    sincospif(2.f * turns(p, A.inv_freq[f]), &sine, &cosine);
    const int at = 4 * (8 * (f >> 2 & 1) + (f >> 3)) + (f & 3);
    reinterpret_cast<float*>(to[r].c)[at] = cosine;
    reinterpret_cast<float*>(to[r].s)[at] = sine;
    reinterpret_cast<float*>(to[r].minus_s)[at] = -sine;
  }
}

// One warp (number w) per (token, chunk of its rows); 8 lanes per row, two
// 16-byte vectors each, so a lane turns the 8 pairs 8j .. 8j + 7 of its row
// (lane j < half_vecs: vectors j and j + half_vecs, or 2j and 2j + 1
// interleaved) or copies vectors 2j and 2j + 1.  U row quads of a warp are
// loaded before the first is turned.  Products and sums are fp32; one rounding
// to 16 bits.  s_cs: the warp's kMaxPairs entries of shared memory.
template <bool kBf16, int U>
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
    if (f < 8 * A.half_vecs) {
      const uint32_t word = lane < 16 ? A.axis[2 * e] : A.axis[2 * e + 1];
      const int p = A.positions[((word >> (2 * (lane & 15))) & 3) * A.n_tok + t];
      float c, s;
      sincospif(2.f * turns(p, A.inv_freq[f]), &s, &c);
      s_cs[f] = make_float2(c, s);
    }
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
    if (r >= rows || (r >= A.Hq && !to_cache)) continue;
    uint16_t* to = r < A.Hq ? A.q_out + t * A.q_out_stride + r * kHeadDim
                            : (r < A.Hq + A.Hkv ? A.k_pool + (row + (r - A.Hq) * kBlock) * kHeadDim
                                                : A.v_pool + (row + (r - A.Hq - A.Hkv) * kBlock) * kHeadDim);
    uint4* dst = reinterpret_cast<uint4*>(to);
    uint32_t a[4] = {x[u][0].x, x[u][0].y, x[u][0].z, x[u][0].w};
    uint32_t b[4] = {x[u][1].x, x[u][1].y, x[u][1].z, x[u][1].w};
    if (turn && r < A.Hq + A.Hkv) {
      if (A.interleaved) {  // word k of vector e holds pair 8j + 4e + k
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 xa = unpack2<kBf16>(a[k]), xb = unpack2<kBf16>(b[k]);
          const float2 ca = cs[k], cb = cs[4 + k];
          a[k] = pack2<kBf16>(xa.x * ca.x - xa.y * ca.y, xa.y * ca.x + xa.x * ca.y);
          b[k] = pack2<kBf16>(xb.x * cb.x - xb.y * cb.y, xb.y * cb.x + xb.x * cb.y);
        }
      } else {  // word k of both vectors holds pairs 8j + 2k, + 1
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 xa = unpack2<kBf16>(a[k]), xb = unpack2<kBf16>(b[k]);
          const float2 c0 = cs[2 * k], c1 = cs[2 * k + 1];
          a[k] = pack2<kBf16>(xa.x * c0.x - xb.x * c0.y, xa.y * c1.x - xb.y * c1.y);
          b[k] = pack2<kBf16>(xb.x * c0.x + xa.x * c0.y, xb.y * c1.x + xa.y * c1.y);
        }
      }
    }
    dst[v0] = make_uint4(a[0], a[1], a[2], a[3]);
    dst[v1] = make_uint4(b[0], b[1], b[2], b[3]);
  }
}

// turn_rows with norms.  1 / rms comes first: the product with it is in the range of 32
// bits for rows of every size.  Four rows (a quad) go together; quads of query
// rows alone, nearly all of them, take a path whose branches are the warp's, not the
// rows' (the others spend a third of their instructions on those).
// What bounds it is the bytes that a resident warp has on their way (its rows) times
// the warps that its registers leave room for.  So with U > 1 the rows wait in shared
// memory: a lane copies the 32 bytes of each row that it will read (cp.async), needs
// no barrier for its own bytes, and no registers for rows that it has not come to.
// s_rows: 1 KiB a quad; with U = 1 not used.
__device__ __forceinline__ void copy16_async(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ uint4 shared16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
// Waits until at most n of the lane's groups are on their way (n < 8).
__device__ __forceinline__ void wait_async(int n) {
  switch (n) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
    case 6: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 7;" ::: "memory"); break;
  }
}

template <bool kBf16, int U>
__device__ __forceinline__ void norm_rows(const RopeArgs& A, unsigned w, Angles* s_angles, uint32_t s_rows) {
  static_assert(U <= 8, "wait_async");
  const int lane = threadIdx.x & 31;
  const unsigned token = w / static_cast<unsigned>(A.chunks);
  if (token >= A.n_tok) return;
  const int r0 = static_cast<int>(w - token * A.chunks) * 4 * U, kv = A.Hq + A.Hkv;  // the first row
  const long long t = token;
  const int j = lane & 7, sub = lane >> 3;
  const bool turn = j < A.half_vecs;
  const int v0 = turn && !A.interleaved ? j : 2 * j;
  const int v1 = turn && !A.interleaved ? j + A.half_vecs : 2 * j + 1;
  const uint4* const q = reinterpret_cast<const uint4*>(A.q + t * A.q_stride) + (r0 + sub) * (kHeadDim / 8);
  const uint32_t mine = s_rows + 16 * lane;
  uint4 only[2];  // U = 1
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = r0 + 4 * u + sub;
    const uint4* from = q + 4 * u * (kHeadDim / 8);
    if (r0 + 4 * u + 4 > A.Hq && r >= A.Hq)
      from = reinterpret_cast<const uint4*>(r < kv ? A.k + t * A.k_stride + (r - A.Hq) * kHeadDim
                                                   : A.v + t * A.v_stride + (r - kv) * kHeadDim);
    if (U == 1) {
      only[0] = only[1] = make_uint4(0, 0, 0, 0);
      if (r < A.rows) only[0] = from[v0], only[1] = from[v1];
    } else {
      if (r < A.rows) {
        copy16_async(mine + 1024 * u, from + v0);
        copy16_async(mine + 1024 * u + 512, from + v1);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  }
  fill_angles<32>(A, s_angles, t, 1);
  __syncwarp();
  // (an octet whose row is past the end sums what it finds; nothing of it leaves the octet)
  auto row = [&](int u, uint4 (&x)[2]) {
    if (U == 1) {
      x[0] = only[0], x[1] = only[1];
    } else {
      wait_async(U - 1 - u);
      x[0] = shared16(mine + 1024 * u), x[1] = shared16(mine + 1024 * u + 512);
    }
  };
  auto norm_and_turn = [&](RowPart& y, const uint4* weight, float rr) {
    if (weight) {
      RowPart wt;
      wt.unpack<kBf16>(__ldg(weight + v0), __ldg(weight + v1));
      y.times(rr);
      y.times(wt);
    }
    if (turn) y.turn(A.interleaved, *s_angles, j);
  };
  uint4* const q_out = reinterpret_cast<uint4*>(A.q_out + t * A.q_out_stride) + (r0 + sub) * (kHeadDim / 8);
  bool far = false;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (r0 + 4 * u + 4 > A.Hq) break;
    uint4 x[2];
    row(u, x);
    RowPart y;
    y.unpack<kBf16>(x[0], x[1]);
    const float mean = y.mean_square(A.eps);
    far |= RowPart::far(mean);
    norm_and_turn(y, reinterpret_cast<const uint4*>(A.q_weight), rsqrtf(mean));
    q_out[4 * u * (kHeadDim / 8) + v0] = pack_part<kBf16>(y.a);
    q_out[4 * u * (kHeadDim / 8) + v1] = pack_part<kBf16>(y.b);
  }
  // quads that hold K or V rows
  long long at = 0;  // row of kv head 0
  bool to_cache = false;
  // row r, given as x, to its place; `again`: as to_unit_size leaves it, if it is far
  auto any_row = [&](int r, uint4 (&x)[2], bool again) {
    RowPart y;
    y.unpack<kBf16>(x[0], x[1]);
    const uint16_t* const weight = r < A.Hq ? A.q_weight : (r < kv ? A.k_weight : nullptr);
    float mean = y.mean_square(A.eps);
    if (again) {
      if (!weight || !RowPart::far(mean)) return;
      if (U > 1) {
        mean = y.mean_square(y.to_unit_size(A.eps), RowPart::octet());
      } else {
        const FarRow there = far_row(y, A.eps);
        y = there.y;
        mean = there.mean;
      }
    } else {
      far |= weight && RowPart::far(mean);
    }
    if (r >= A.rows || (r >= A.Hq && !to_cache)) return;
    uint4* dst = reinterpret_cast<uint4*>(
        r < A.Hq ? A.q_out + t * A.q_out_stride + r * kHeadDim
                 : (r < kv ? A.k_pool + (at + (r - A.Hq) * kBlock) * kHeadDim : A.v_pool + (at + (r - kv) * kBlock) * kHeadDim));
    if (r < kv) {
      norm_and_turn(y, reinterpret_cast<const uint4*>(weight), rsqrtf(mean));
      x[0] = pack_part<kBf16>(y.a);
      x[1] = pack_part<kBf16>(y.b);
    }
    dst[v0] = x[0];
    dst[v1] = x[1];
  };
  if (r0 + 4 * U > A.Hq) {
    const long long slot = A.slots[t];
    to_cache = slot >= 0 && slot < A.num_slots;
    if (slot >= A.num_slots && lane == 0 && r0 < kv) record_error(A.err, PA_ERR_DEVICE_CHECK, slot);
    at = (slot >> 4) * A.Hkv * kBlock + (slot & 15);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (r0 + 4 * u + 4 <= A.Hq) continue;
      if (r0 + 4 * u >= A.rows) break;
      uint4 x[2];
      row(u, x);
      any_row(r0 + 4 * u + sub, x, false);
    }
  }
  // rows whose squares left 32 bits, once more, apart from the loops above, whose registers
  // they would take (36.5 -> 39.3 us there); they are still here, also where q_out is q
  if (!__any_sync(0xffffffffu, far)) return;
#pragma unroll 1
  for (int u = 0; u < U && r0 + 4 * u < A.rows; ++u) {
    uint4 x[2] = {only[0], only[1]};
    if (U > 1) x[0] = shared16(mine + 1024 * u), x[1] = shared16(mine + 1024 * u + 512);
    any_row(r0 + 4 * u + sub, x, true);
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
