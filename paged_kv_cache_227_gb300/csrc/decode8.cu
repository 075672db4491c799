// Decode attention over the 8-bit cache.
//
// For sequence i, query head h of kv head g and L = seq_lens[i]:
//   K[t] = 2^(ek - 127) * codes of token t (ek the block's exponent), V likewise,
//   out = softmax(scale * K q) V,
// sums, maxima and weights in fp32.
//
// Bound: memory, 256 bytes a token and kv head, read once for all of the head's
// G query heads (2 G flops a byte).  The tiles (16 tokens: 2 KiB of K, 2 KiB of
// V on end) of all (sequence, kv head) segments, laid end to end, are cut into
// equal ranges, one a warp, so that any length mix loads the GPU evenly; each
// warp streams its range through a ring of its own in shared memory.  A segment
// that a cut divides leaves a record a piece, which a second kernel joins by
// log-sum-exp, in their order.
//
// A lane copies exactly the bytes that it will read (cp.async, 16 bytes each),
// so the ring needs no barrier: the lane's own wait is enough.  Which bytes those
// are follows from the operands of mma.sync m16n8k16, with the query heads as
// the rows of both products:
//   scores  S (heads x tokens) = Q K^T: as an operand, lane (g, c) = (lane / 4,
//           lane % 4) holds token g's dims; any 32 will do as long as Q's lanes
//           hold the same ones, so it takes bytes 16c .. 16c + 15 and 64 + 16c ..
//           of the rows of tokens g and g + 8;
//   values  O (heads x dims) = P V: the scores' fragment, as it comes out, is P's
//           operand; lane (g, c) holds tokens 2c, 2c + 1, 2c + 8, 2c + 9 of
//           column g, and the columns may stand for any dims: dims 16g .. 16g +
//           15, 16 bytes a token.
// A head fills 8 of the product's 16 rows.  In the scores the other 8 stay zero;
// in the values they carry what rounding the weights to 16 bits left, so high
// and low half (23 bits) go through one product.  Codes become fp16 exactly, q in
// bf16 too after a power of two per head (its elements 2^28 below the largest
// lose bits), and the tile's scales are applied in fp32: K's to the scores, V's
// to the tile's 16-token product as it is added to O.
#include <atomic>

#include "codes8.cuh"
#include "device_utils.cuh"

namespace pa {

constexpr int kWarps8 = 16;    // warps of a CTA, one CTA an SM
constexpr int kStages8 = 3;    // tiles in flight of a warp: 192 KiB an SM
constexpr int kSeqs8 = 4096;   // sequences of a call (their prefix lives in shared memory)
constexpr int kMinUnits8 = 2;  // smallest range of a warp
constexpr float kLog2e8 = 1.4426950408889634f;
// The running maximum moves when a score passes it by 2^4; weights are carried
// at 2^11 times their size, below 2^15, so that the low half's smallest step
// (2^-24) is 2^-35 of the row's largest weight.
constexpr float kMove8 = 4.f, kUp8 = 11.f;

// Record of a piece: O as 8 float4 a lane (number k * 32 + lane: head lane / 4,
// dims 32 (lane % 4) + 4 k ..), then the heads' maxima (log2 units) and sums.
constexpr int kRec8 = 8 * 32 * 4 + 2 * 8;

struct Decode8Args {
  const uint8_t* codes;
  const uint8_t* exps;
  const uint16_t* q;          // [B][Hq][128]
  const int32_t* tables;
  const int32_t* seq_lens;
  void* out;
  float* rec;
  long long* err;
  int num_blocks, max_blocks;
  int B, Hq, Hkv, G;
  int out_dtype;
  int units;                  // warps that the ranges are cut for
  float qscale;               // scale * log2(e)
};

// A segment (i, h) is one unit for its start (its query rows, its record) and
// one for each of its tiles; pfx[i] counts the units of one kv head before
// sequence i.
struct Ranges8 {
  long long per;
  __device__ Ranges8(const Decode8Args& A, const int* pfx) {
    per = (static_cast<long long>(A.Hkv) * pfx[A.B] + A.units - 1) / A.units;
    if (per < kMinUnits8) per = kMinUnits8;
  }
};

// pfx[0 .. B] and, with lens, the clamped lengths; a whole CTA.
__device__ void prefix8(const Decode8Args& A, int* pfx, int* lens, bool report) {
  const int lane = threadIdx.x & 31;
  const int cap = A.max_blocks * kBlock;
  for (int i = threadIdx.x; i < A.B; i += blockDim.x) {
    int L = A.seq_lens[i];
    if (L < 0 || L > cap) {
      if (report) record_error(A.err, PA_ERR_DEVICE_CHECK, L);
      L = L < 0 ? 0 : cap;
    }
    lens[i] = L;
    pfx[i + 1] = L ? 1 + (L + kBlock - 1) / kBlock : 0;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    int carry = 0;
    for (int base = 0; base < A.B; base += 32) {
      const int i = base + lane;
      int sum = i < A.B ? pfx[i + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
      }
      if (i < A.B) pfx[i + 1] = carry + sum;
      carry += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) pfx[0] = 0;
  }
  __syncthreads();
}

__device__ __forceinline__ void cp_async16(uint32_t to, const uint8_t* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint4 lds16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A lane's view of 32 units of the warp's range, one a lane: its tile's sequence,
// kv head, number in the sequence (-1: the unit starts a segment, or is past the
// range), place in the pool (-1: none, or out of range) and scales.
struct Window8 {
  int i, h, j, tile;
  float ks, vs;
};
__device__ __forceinline__ Window8 window8(const Decode8Args& A, const int* pfx, long long u, long long end) {
  Window8 w{0, 0, -1, -1, 0.f, 0.f};
  if (u >= end) return w;
  int lo = 0, hi = A.B - 1;  // the last sequence that starts at or before u (never an empty one)
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (static_cast<long long>(A.Hkv) * pfx[mid] <= u) lo = mid; else hi = mid - 1;
  }
  const int r = static_cast<int>(u - static_cast<long long>(A.Hkv) * pfx[lo]), cnt = pfx[lo + 1] - pfx[lo];
  w.i = lo;
  w.h = r / cnt;
  w.j = r - w.h * cnt - 1;
  if (w.j >= 0) {
    const int blk = A.tables[static_cast<long long>(lo) * A.max_blocks + w.j];
    if (blk >= 0 && blk < A.num_blocks) {
      w.tile = blk * A.Hkv + w.h;
      const uint16_t e = reinterpret_cast<const uint16_t*>(A.exps)[w.tile];
      w.ks = scale_of(e & 0xff);
      w.vs = scale_of(e >> 8) * (1.f / (1 << static_cast<int>(kUp8)));
    } else {
      record_error(A.err, PA_ERR_DEVICE_CHECK, blk);
    }
  }
  return w;
}

// The query rows of (i, h) as the scores' operand: lane (g, c) holds head g's dims
// 16c + 4w + {0, 1}, {2, 3} in qa[2w], qa[2w + 1], and from 64 on in qa[8 + ..].
// Returns what the products have to be multiplied by.
template <bool kBf16>
__device__ __forceinline__ float load_q8(const Decode8Args& A, int i, int h, int g, int c, uint32_t (&qa)[16]) {
  uint4 x[4];
  const uint4* src = reinterpret_cast<const uint4*>(A.q + (static_cast<long long>(i) * A.Hq + h * A.G + g) * kHeadDim);
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = g < A.G ? src[8 * (k >> 1) + 2 * c + (k & 1)] : make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    qa[4 * k] = x[k].x;
    qa[4 * k + 1] = x[k].y;
    qa[4 * k + 2] = x[k].z;
    qa[4 * k + 3] = x[k].w;
  }
  if (!kBf16) return A.qscale;
  // bf16: times the power of two that takes the largest finite magnitude to [2^14, 2^15)
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const uint32_t lo = qa[k] << 16 & 0x7fffffffu, hi = qa[k] & 0x7fff0000u;
    if (lo < 0x7f800000u) top = max(top, lo);
    if (hi < 0x7f800000u) top = max(top, hi);
  }
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const int k2 = min(14 + 127 - static_cast<int>(top >> 23), 120);
  const float up = __int_as_float((127 + k2) << 23);
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const __half2 y = __floats2half2_rn(__uint_as_float(qa[k] << 16) * up, __uint_as_float(qa[k] & 0xffff0000u) * up);
    qa[k] = *reinterpret_cast<const uint32_t*>(&y);
  }
  return A.qscale * __int_as_float((127 - k2) << 23);
}

template <bool kBf16, bool kE4M3>
__global__ void __launch_bounds__(kWarps8 * 32, 1) decode8_kernel(const __grid_constant__ Decode8Args A) {
  extern __shared__ __align__(16) uint8_t smem8[];
  int* const pfx = reinterpret_cast<int*>(smem8 + kWarps8 * kStages8 * kPair8);
  int* const lens = pfx + A.B + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  prefix8(A, pfx, lens, blockIdx.x == 0);
  const long long per = Ranges8(A, pfx).per;
  const int unit = warp * gridDim.x + blockIdx.x;
  const long long total = static_cast<long long>(A.Hkv) * pfx[A.B];
  const long long u0 = per * unit, u1 = min(u0 + per, total);
  if (u0 >= u1) return;
  const int n = static_cast<int>(u1 - u0);

  // the lane's bytes of a tile, and its slots of the ring
  const int k_off = g * kRow8 + c * 16, v_off = kTile8 + 2 * c * kRow8 + g * 16;
  const uint32_t ring = smem_addr(smem8) + warp * (kStages8 * kPair8) + lane * 16;
  Window8 now = window8(A, pfx, u0 + lane, u1), next = now;
  auto issue = [&](int x) {  // unit x of the range; x and the windows are the same in all lanes
    const int tile = __shfl_sync(0xffffffffu, next.tile, x & 31);
    if (x < n && tile >= 0) {
      const uint32_t to = ring + (x % kStages8) * kPair8;
      const uint8_t* from = A.codes + static_cast<long long>(tile) * kPair8;
      const uint8_t *k = from + k_off, *v = from + v_off;
      cp_async16(to, k);
      cp_async16(to + 512, k + 64);
      cp_async16(to + 1024, k + 8 * kRow8);
      cp_async16(to + 1536, k + 8 * kRow8 + 64);
      cp_async16(to + 2048, v);
      cp_async16(to + 2560, v + kRow8);
      cp_async16(to + 3072, v + 8 * kRow8);
      cp_async16(to + 3584, v + 9 * kRow8);
    }
    cp_commit();
  };
#pragma unroll
  for (int x = 0; x < kStages8; ++x) issue(x);

  uint32_t qa[16];
  float o[32], m, l, fq = 0.f, mref = 0.f;
  int ci = -1, ch = -1;  // segment of the piece in hand
  auto flush = [&]() {
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    l *= 1.f / (1 << static_cast<int>(kUp8));
    if (g >= A.G) return;
    const int cnt = pfx[ci + 1] - pfx[ci];
    const long long s0 = static_cast<long long>(A.Hkv) * pfx[ci] + static_cast<long long>(ch) * cnt;
    if (s0 + 1 >= u0 && s0 + cnt <= u1) {  // the whole segment
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const long long at = (static_cast<long long>(ci) * A.Hq + ch * A.G + g) * kHeadDim + 32 * c;
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int w = 0; w < 4; ++w)
          store_out4(A.out, at + 16 * e + 4 * w, o[8 * w + e] * inv, o[8 * w + 2 + e] * inv, o[8 * w + 4 + e] * inv,
                     o[8 * w + 6 + e] * inv, A.out_dtype);
      return;
    }
    float* rec = A.rec + (2ll * unit + (s0 > u0)) * kRec8;
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int w = 0; w < 4; ++w)
        reinterpret_cast<float4*>(rec)[(4 * e + w) * 32 + lane] =
            make_float4(o[8 * w + e], o[8 * w + 2 + e], o[8 * w + 4 + e], o[8 * w + 6 + e]);
    if (c == 0) {
      rec[1024 + g] = m;
      rec[1032 + g] = l;
    }
  };

  for (int x = 0; x < n; ++x) {
    if ((x & 31) == 0) now = next;  // (the issues are in this window until the one below)
    const int j = __shfl_sync(0xffffffffu, now.j, x & 31);
    if (j >= 0) {
      const int i = __shfl_sync(0xffffffffu, now.i, x & 31), h = __shfl_sync(0xffffffffu, now.h, x & 31);
      if (i != ci || h != ch) {
        if (ci >= 0) flush();
        ci = i;
        ch = h;
        fq = load_q8<kBf16>(A, i, h, g, c, qa);
        m = -INFINITY;
        mref = 0.f;
        l = 0.f;
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = 0.f;
      }
      cp_wait<kStages8 - 1>();
      if (__shfl_sync(0xffffffffu, now.tile, x & 31) >= 0) {
        const uint32_t at = ring + (x % kStages8) * kPair8;
        const int left = lens[i] - j * kBlock;  // tokens of the tile that count
        // scores of tokens 2c, 2c + 1 (s[0], s[1]) and 8 + 2c, 9 + 2c (s[2], s[3])
        float s[4];
        const float ks = __shfl_sync(0xffffffffu, now.ks, x & 31) * fq;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          float d0[4] = {0.f, 0.f, 0.f, 0.f}, d1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint4 v = lds16(at + 1024 * t + 512 * half);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t b0, b1;
              unpack_codes<kE4M3>(w[k], b0, b1);
              mma_f16(half ? d1 : d0, qa[8 * half + 2 * k], 0u, qa[8 * half + 2 * k + 1], 0u, b0, b1);
            }
          }
          s[2 * t] = (d0[0] + d1[0]) * ks;
          s[2 * t + 1] = (d0[1] + d1[1]) * ks;
        }
        if (left < kBlock) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (8 * (k >> 1) + 2 * c + (k & 1) >= left) s[k] = -INFINITY;
        }
        // running maximum and weights
        float most = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
        if (__any_sync(0xffffffffu, most > m + kMove8)) {
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
          const float to = fmaxf(m, most);
          const float f = to == m ? 1.f : fast_exp2(m - to);
          m = to;
          mref = to == -INFINITY ? 0.f : to - kUp8;
          l *= f;
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] *= f;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) s[k] = fast_exp2(s[k] - mref);
        l += (s[0] + s[1]) + (s[2] + s[3]);
        const uint32_t a0 = pack_hi<false>(s[0], s[1]), a1 = pack_lo<false>(s[0], s[1]);
        const uint32_t a2 = pack_hi<false>(s[2], s[3]), a3 = pack_lo<false>(s[2], s[3]);
        // values
        const float vs = __shfl_sync(0xffffffffu, now.vs, x & 31);
        uint4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = lds16(at + 2048 + 512 * k);
        if (left < kBlock) {  // (a weight of zero times NaN is NaN)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (8 * (k >> 1) + 2 * c + (k & 1) >= left) v[k] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t t0 = w == 0 ? v[0].x : w == 1 ? v[0].y : w == 2 ? v[0].z : v[0].w;
          const uint32_t t1 = w == 0 ? v[1].x : w == 1 ? v[1].y : w == 2 ? v[1].z : v[1].w;
          const uint32_t t2 = w == 0 ? v[2].x : w == 1 ? v[2].y : w == 2 ? v[2].z : v[2].w;
          const uint32_t t3 = w == 0 ? v[3].x : w == 1 ? v[3].y : w == 2 ? v[3].z : v[3].w;
          uint32_t lo[4], hi[4];  // dims 16g + 4w + 0 .. 3 of tokens 2c, 2c + 1 and 2c + 8, 2c + 9
          unpack_codes<kE4M3>(__byte_perm(t0, t1, 0x5140), lo[0], lo[1]);
          unpack_codes<kE4M3>(__byte_perm(t0, t1, 0x7362), lo[2], lo[3]);
          unpack_codes<kE4M3>(__byte_perm(t2, t3, 0x5140), hi[0], hi[1]);
          unpack_codes<kE4M3>(__byte_perm(t2, t3, 0x7362), hi[2], hi[3]);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float d[4] = {0.f, 0.f, 0.f, 0.f};
            mma_f16(d, a0, a1, a2, a3, lo[k], hi[k]);
            o[8 * w + 2 * k] = fmaf(vs, d[0] + d[2], o[8 * w + 2 * k]);
            o[8 * w + 2 * k + 1] = fmaf(vs, d[1] + d[3], o[8 * w + 2 * k + 1]);
          }
        }
      }
    }
    // the stage is free: the unit kStages8 on, from the window it is in
    const int y = x + kStages8;
    if ((y & 31) == 0 && y < n) next = window8(A, pfx, u0 + y + lane, u1);
    issue(y);
  }
  if (ci >= 0) flush();
  cp_wait<0>();
}

// Joins the records of segments that were cut, and writes the zeros of empty
// ones.  A CTA takes a segment at a time; warp k float4 number k of each lane.
__global__ void __launch_bounds__(256) merge8_kernel(const __grid_constant__ Decode8Args A) {
  extern __shared__ __align__(16) uint8_t smem8[];
  int* const pfx = reinterpret_cast<int*>(smem8);
  int* const lens = pfx + A.B + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  prefix8(A, pfx, lens, false);
  const long long per = Ranges8(A, pfx).per;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long segments = static_cast<long long>(A.B) * A.Hkv;
  for (long long s = blockIdx.x; s < segments; s += gridDim.x) {
    const int i = static_cast<int>(s / A.Hkv), h = static_cast<int>(s - static_cast<long long>(i) * A.Hkv);
    const int cnt = pfx[i + 1] - pfx[i];
    const long long at = (static_cast<long long>(i) * A.Hq + h * A.G + g) * kHeadDim + 32 * c + 4 * warp;
    if (cnt == 0) {
      if (g < A.G) store_out4(A.out, at, 0.f, 0.f, 0.f, 0.f, A.out_dtype);
      continue;
    }
    const long long s0 = static_cast<long long>(A.Hkv) * pfx[i] + static_cast<long long>(h) * cnt;
    const long long c0 = (s0 + 1) / per, c1 = (s0 + cnt - 1) / per;
    if (c0 == c1 || g >= A.G) continue;
    const int count = static_cast<int>(c1 - c0 + 1);
    const float* first = A.rec + (2 * c0 + (s0 > c0 * per)) * kRec8;  // the others: slot 0 of their warps
    const float* rest = A.rec + 2 * c0 * kRec8;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kBatch = 8;
    for (int k0 = 0; k0 < count; k0 += kBatch) {
      float rm[kBatch], rl[kBatch];
      float4 ro[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        rm[k] = -INFINITY;
        rl[k] = 0.f;
        ro[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k0 + k < count) {
          const float* r = k0 + k == 0 ? first : rest + 2ll * (k0 + k) * kRec8;
          rm[k] = __ldcg(r + 1024 + g);
          rl[k] = __ldcg(r + 1032 + g);
          ro[k] = __ldcg(reinterpret_cast<const float4*>(r) + warp * 32 + lane);
        }
      }
      float to = m;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) to = fmaxf(to, rm[k]);
      const float f = m == to ? 1.f : fast_exp2(m - to);
      l *= f;
      o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float w = rm[k] == to ? 1.f : fast_exp2(rm[k] - to);
        l = fmaf(w, rl[k], l);
        o.x = fmaf(w, ro[k].x, o.x);
        o.y = fmaf(w, ro[k].y, o.y);
        o.z = fmaf(w, ro[k].z, o.z);
        o.w = fmaf(w, ro[k].w, o.w);
      }
      m = to;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    store_out4(A.out, at, o.x * inv, o.y * inv, o.z * inv, o.w * inv, A.out_dtype);
  }
}

static size_t decode8_records(const pa_pool8* p) {
  return 2 * static_cast<size_t>(sm_count(p->device)) * kWarps8 * kRec8 * sizeof(float);
}

template <bool kBf16, bool kE4M3>
static int launch_decode8(Decode8Args& A, int device, cudaStream_t st) {
  const int sms = sm_count(device);
  const size_t lists = sizeof(int) * (2 * static_cast<size_t>(A.B) + 1);
  const size_t smem = static_cast<size_t>(kWarps8) * kStages8 * kPair8 + lists;
  constexpr int kMaxSmem = kWarps8 * kStages8 * kPair8 + sizeof(int) * (2 * kSeqs8 + 1);
  static_assert(kMaxSmem <= 232448, "shared memory of an SM");
  // once a device, for the largest batch
  static std::atomic<uint64_t> allowed{0};
  const uint64_t bit = device < 64 ? 1ull << device : 0;
  if (!(allowed.load(std::memory_order_relaxed) & bit) || !bit) {
    if (cudaFuncSetAttribute(decode8_kernel<kBf16, kE4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem) !=
        cudaSuccess)
      return PA_ERR_CUDA;
    allowed.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = st;
  cfg.gridDim = dim3(sms);
  cfg.blockDim = dim3(kWarps8 * 32);
  cfg.dynamicSmemBytes = smem;
  if (cudaLaunchKernelEx(&cfg, decode8_kernel<kBf16, kE4M3>, A) != cudaSuccess) return PA_ERR_CUDA;
  const long long segments = static_cast<long long>(A.B) * A.Hkv;
  cfg.gridDim = dim3(static_cast<unsigned>(segments < 8ll * sms ? segments : 8ll * sms));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = lists;
  if (cudaLaunchKernelEx(&cfg, merge8_kernel, A) != cudaSuccess) return PA_ERR_CUDA;
  return PA_OK;
}

}  // namespace pa

using namespace pa;

extern "C" size_t pa_decode8_workspace_bytes(pa_pool8_t p, int num_seqs, int n_q_heads, int max_blocks_per_seq) {
  if (!p || num_seqs <= 0 || n_q_heads <= 0 || max_blocks_per_seq <= 0 || n_q_heads % p->n_kv_heads) return 0;
  if (num_seqs > kSeqs8 || n_q_heads / p->n_kv_heads > PA_MAX_GROUP) return 0;
  return decode8_records(p);
}

extern "C" int pa_decode8(pa_pool8_t p, const void* q, int q_dtype, const int32_t* block_tables, int max_blocks_per_seq,
                          const int32_t* seq_lens, int num_seqs, int n_q_heads, float scale, void* out, int out_dtype,
                          void* workspace, size_t workspace_bytes, void* stream) {
  if (!p || !q || !block_tables || !seq_lens || !out || num_seqs <= 0 || n_q_heads <= 0 || max_blocks_per_seq <= 0)
    return PA_ERR_INVALID;
  if ((q_dtype != PA_FP16 && q_dtype != PA_BF16) || (out_dtype != PA_FP16 && out_dtype != PA_BF16 && out_dtype != PA_FP32))
    return PA_ERR_INVALID;
  if (n_q_heads % p->n_kv_heads || !(scale - scale == 0.f)) return PA_ERR_INVALID;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15) return PA_ERR_INVALID;
  if (n_q_heads / p->n_kv_heads > PA_MAX_GROUP || num_seqs > kSeqs8 || max_blocks_per_seq > kMaxWalkedBlocks)
    return PA_ERR_UNSUPPORTED;
  // units of one kv head, of one sequence and of one warp are counted in 32 bits
  const long long row = max_blocks_per_seq + 1ll;
  if (num_seqs * row >= 0x7fffffffll || p->n_kv_heads * row >= 0x7fffffffll || num_seqs * (p->n_kv_heads * row) >= 1ll << 41)
    return PA_ERR_UNSUPPORTED;
  if (!on_pool_device(p)) return PA_ERR_INVALID;
  if (!workspace || workspace_bytes < decode8_records(p) || (reinterpret_cast<uintptr_t>(workspace) & 255))
    return PA_ERR_INVALID;
  Decode8Args A{};
  A.codes = p->codes;
  A.exps = p->exps;
  A.q = static_cast<const uint16_t*>(q);
  A.tables = block_tables;
  A.seq_lens = seq_lens;
  A.out = out;
  A.rec = static_cast<float*>(workspace);
  A.err = p->err;
  A.num_blocks = p->num_blocks;
  A.max_blocks = max_blocks_per_seq;
  A.B = num_seqs;
  A.Hq = n_q_heads;
  A.Hkv = p->n_kv_heads;
  A.G = n_q_heads / p->n_kv_heads;
  A.out_dtype = out_dtype;
  A.qscale = scale * kLog2e8;
  A.units = sm_count(p->device) * kWarps8;
  cudaStream_t st = as_stream(stream);
  const bool e4m3 = p->dtype == PA_E4M3;
  if (q_dtype == PA_BF16)
    return e4m3 ? launch_decode8<true, true>(A, p->device, st) : launch_decode8<true, false>(A, p->device, st);
  return e4m3 ? launch_decode8<false, true>(A, p->device, st) : launch_decode8<false, false>(A, p->device, st);
}
