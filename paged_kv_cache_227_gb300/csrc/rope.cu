// Rotary positions with several axes, with the cache write.
//
// A new token n has one position per axis (time, height, width, ...).  The
// first `rot` dims of a head are rot/2 pairs; pair f turns by the angle
//   a = positions[axis(f)][n] * inv_freq[f],
//   (x, y) -> (x cos a - y sin a, y cos a + x sin a),
// where the pair is dims (f, f + rot/2) or, interleaved, (2f, 2f + 1).  Dims
// past rot pass through.  Query rows go to q_out, key rows to the cache slot
// of the token, value rows to the same slot unturned.
//
// Bound: memory.  Every row is read once and written once (512 B), against
// about 3 flops an element.  The angles are the only other work: 64 a token,
// computed by the lanes of a warp together (two each) and shared by all of
// the warp's rows through shared memory.  Measured: 8,192 tokens of 48 heads
// (201 MB) 32.8 us, 6.1 TB/s, 0.90 of this GPU's copy rate; 64 tokens 2.3 us.
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
  long long q_stride, k_stride, v_stride, q_out_stride;
  long long n_tok, num_slots;
  int Hq, Hkv, half_vecs;    // half_vecs = rot / 16: lanes of a row that turn
  int interleaved;
  int chunks;                // warps a token's rows are cut into
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

// One warp per (token, chunk of its rows); 8 lanes per row, two 16-byte
// vectors each, so a lane turns the 8 pairs 8j .. 8j + 7 of its row (lane j <
// half_vecs: vectors j and j + half_vecs, or 2j and 2j + 1 interleaved) or
// copies vectors 2j and 2j + 1.  U row quads of a warp are loaded before the
// first is turned.  Products and sums are fp32; one rounding to 16 bits.
template <bool kBf16, int U>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const __grid_constant__ RopeArgs A) {
  __shared__ float2 s_cs[kRopeThreads / 32][kMaxPairs];
  const int lane = threadIdx.x & 31, wib = threadIdx.x >> 5;
  const long long w = static_cast<long long>(blockIdx.x) * (kRopeThreads / 32) + wib;
  const long long t = w / A.chunks;
  if (t >= A.n_tok) return;
  const int chunk = static_cast<int>(w - t * A.chunks);
  const int rows = A.Hq + 2 * A.Hkv;
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
      s_cs[wib][f] = make_float2(c, s);
    }
  }
  __syncwarp();
  float2 cs[8];
  if (turn) {
#pragma unroll
    for (int e = 0; e < 8; ++e) cs[e] = s_cs[wib][8 * j + e];
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

template <int U>
static int launch_rope(RopeArgs& A, bool bf16, cudaStream_t st) {
  const int rows = A.Hq + 2 * A.Hkv;
  A.chunks = (rows + 4 * U - 1) / (4 * U);
  const long long grid = (A.n_tok * A.chunks + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  if (grid > 0x7fffffffll) return PA_ERR_UNSUPPORTED;
  if (bf16)
    rope_append_kernel<true, U><<<static_cast<unsigned>(grid), kRopeThreads, 0, st>>>(A);
  else
    rope_append_kernel<false, U><<<static_cast<unsigned>(grid), kRopeThreads, 0, st>>>(A);
  return cuda_status(cudaGetLastError());
}

}  // namespace pa

using namespace pa;

static_assert(PA_MAX_ROPE_AXES <= 4, "an axis is two bits");

extern "C" int pa_rope_append(pa_pool_t p, const void* q, int64_t q_stride, int n_q_heads, const void* k_new,
                              int64_t k_stride, const void* v_new, int64_t v_stride, const int32_t* positions,
                              int n_axes, const uint8_t* axis_of_pair, const float* inv_freq, int rot_dim,
                              int interleaved, const int64_t* slot_mapping, int n_tok, void* q_out,
                              int64_t q_out_stride, void* stream) {
  if (!p || n_tok < 0 || n_q_heads <= 0) return PA_ERR_INVALID;
  if (rot_dim <= 0 || rot_dim > kHeadDim || rot_dim % 16) return PA_ERR_UNSUPPORTED;
  if (n_axes < 1 || n_axes > PA_MAX_ROPE_AXES || n_q_heads > PA_MAX_ROPE_HEADS) return PA_ERR_UNSUPPORTED;
  if (!axis_of_pair) return PA_ERR_INVALID;
  RopeArgs A{};
  for (int f = 0; f < rot_dim / 2; ++f) {
    if (axis_of_pair[f] >= n_axes) return PA_ERR_INVALID;
    A.axis[f / 16] |= static_cast<uint32_t>(axis_of_pair[f]) << (2 * (f % 16));
  }
  if (n_tok == 0) return PA_OK;
  if (!q || !k_new || !v_new || !positions || !inv_freq || !slot_mapping || !q_out) return PA_ERR_INVALID;
  // rows are moved as 16-byte vectors; a token's heads are contiguous
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new) |
       reinterpret_cast<uintptr_t>(q_out)) & 15)
    return PA_ERR_INVALID;
  if ((q_stride | k_stride | v_stride | q_out_stride) & 7) return PA_ERR_INVALID;
  const int64_t qw = static_cast<int64_t>(n_q_heads) * kHeadDim, kw = static_cast<int64_t>(p->n_kv_heads) * kHeadDim;
  if (n_tok > 1 && (q_stride < qw || q_out_stride < qw || k_stride < kw || v_stride < kw)) return PA_ERR_INVALID;
  // in place only row for row
  if (q == q_out && n_tok > 1 && q_stride != q_out_stride) return PA_ERR_INVALID;
  if (!on_pool_device(p)) return PA_ERR_INVALID;
  A.q = static_cast<const uint16_t*>(q);
  A.k = static_cast<const uint16_t*>(k_new);
  A.v = static_cast<const uint16_t*>(v_new);
  A.q_out = static_cast<uint16_t*>(q_out);
  A.k_pool = static_cast<uint16_t*>(p->k);
  A.v_pool = static_cast<uint16_t*>(p->v);
  A.positions = positions;
  A.inv_freq = inv_freq;
  A.slots = slot_mapping;
  A.q_stride = q_stride;
  A.k_stride = k_stride;
  A.v_stride = v_stride;
  A.q_out_stride = q_out_stride;
  A.n_tok = n_tok;
  A.num_slots = static_cast<long long>(p->num_blocks) * kBlock;
  A.Hq = n_q_heads;
  A.Hkv = p->n_kv_heads;
  A.half_vecs = rot_dim / 16;
  A.interleaved = interleaved != 0;
  A.err = p->err;
  // rows a warp: 4 while that leaves the GPU partly empty, then 12, which share a
  // token's angles.  us with 4 and with 12 rows, captured calls: 48 rows a token
  // (the switch is at 405 tokens) 64 tokens 2.19 and 2.30, 128 2.43 and 2.35, 400
  // 3.55 and 3.17, 512 4.31 and 3.59, 8,192 49.1 and 33.0; 16 rows a token (1,216)
  // 64 tokens 2.23 and 2.40, 400 2.60 and 2.60, 1,024 3.35 and 3.18, 2,048 5.31
  // and 4.00; 120 rows a token (162) 64 tokens 2.83 and 2.67, 128 3.39 and 3.11
  const long long quads = A.n_tok * ((A.Hq + 2 * A.Hkv + 3) / 4);
  if (quads <= 32ll * sm_count(p->device))
    return launch_rope<1>(A, p->dtype == PA_BF16, as_stream(stream));
  return launch_rope<3>(A, p->dtype == PA_BF16, as_stream(stream));
}
