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
// equal ranges, one a CTA and SM, so that any length mix loads the GPU evenly, and
// those into equal ranges for the warps; each warp streams its own through a ring
// in shared memory.  Where a cut divides a segment, the warps of a CTA leave
// records in shared memory and join them there; at most one segment goes on from
// one CTA to the next, and a second kernel joins those, by log-sum-exp, always in
// the order of their tiles.  Few or short segments get a CTA each instead.
//
// Measured (captured calls, three inputs in turn; behind a flush of L2): batch 64 of
// chats (108 MB) 26.8 us, 0.60 of the copy rate (29.2); 16 multi-head sequences (276 MB)
// 49.2, 0.83 (51.3); four documents of 8 to 32 thousand tokens (161 MB) 33.2, 0.72 (35);
// four short requests 8.2 (10.3).  Groups of 8 query heads, 64 chats (109 MB) 28.8, 0.56
// (31.7).  Of the 64 chats' 26.8 us 3 are lengths, tables and first tiles, 16 the stream, 5
// what the SMs' ends lie apart and the joins inside them, 3 the second kernel.
//
// A tile is one TMA box, 32 rows of 128 bytes in the 128-byte swizzle, so that the
// operand loads below meet no bank conflict.  Per tile, with mma.sync m16n8k16 (16
// tokens against at most 8 heads are far below what tcgen05 takes) and the codes
// as fp16, which is exact:
//   scores  S (tokens x heads) = K Q^T: ldmatrix hands lane (g, c) = (lane / 4,
//           lane % 4) four codes of token g (g + 8) a matrix, dims 16 j + 4c .. + 3;
//           Q's lanes hold the same dims in the same order.
//   values  O (dims x heads) = V^T P: lane (g, c) reads 16 bytes, dims 16 g .., of tokens
//           2c, 2c + 1, 2c + 8, 2c + 9, pairs the tokens' bytes and has two dims a
//           product as its rows; no transposition but that of P (movmatrix).
// The weights P go in as a high and a low 16-bit half (22 bits): with up to 4 heads
// the columns 4 .. 7 repeat the heads and carry the low halves, with more the
// product is made twice.
// Scales: K's multiplies the scores.  V's, a power of two 2^ev, is carried by O: O
// is kept in units of 2^E, E the largest ev so far, and the weights are multiplied
// by 2^(ev - E) before they are rounded, so the products add up in the accumulators
// themselves; a tile with ev < E - 4, whose weights would lose bits that way,
// is multiplied by itself and added in fp32.
#include <atomic>

#include "codes8.cuh"
#include "device_utils.cuh"

namespace pa {

// One CTA an SM, 12 warps with 3 tiles (4 KiB) in flight each.  us for 64 chats, 16
// multi-head sequences and four documents: 26.7, 49.5, 33.1; 10 warps of 4 tiles 29.1,
// 55.7, 36.4; 8 of 5 29.6, 56.5, 37.9; 11 of 3 27.7, 51.5, 34.4; 13 of 3 (fewer
// registers, spills) 28.1, 52.9, 35.6.
constexpr int kWarps8 = 12;
constexpr int kStages8 = 3;
static_assert(2 * kWarps8 <= 32, "a lane a chain of pieces");
constexpr int kSeqs8 = 4096;   // sequences of a call (their prefix lives in shared memory)
// Smallest range of a CTA.  us with 4, 8, 16, 24: 16 segments of 100 tokens 7.6, 7.0, 7.5,
// 8.3; 16 of about 400 10.6, 10.0, 9.7, 10.4; 80 of about 300 10.9, 10.9, 10.0, 10.6.
constexpr int kMinUnits8 = 8;
// Widest tables of the plan with a CTA a segment, which needs no second kernel but
// waits for its longest segment: for few segments, and for at least kManyWhole8 (the
// balanced split then leaves records in every CTA).  us a call with it and with the
// balanced split, lengths alike: 8 segments of 300, 500, 800 tokens 7.3, 8.2, 10.1 and 8.1,
// 8.2, 8.3; 32 of them 7.8, 8.8, 10.6 and 8.5, 8.7, 9.8; 63 of 300, 800, 1,500 8.3, 11.2,
// 14.6 and 10.4, 11.8, 14.7; 72 of 500, 800, 1,500, 2,500 9.0, 10.9, 14.5, 20.3 and 10.6,
// 12.0, 14.7, 17.6; 128 of 500, 1,500, 4,000 9.8, 15.8, 28.3 and 12.9, 18.3, 29.0.
// Ragged (the longest one in brackets): 32 (376), (753) 8.0, 10.3 and 8.4, 8.7; 72 (537),
// (1,073), (1,530) 9.0, 12.0, 14.7 and 8.9, 10.1, 11.1; 128 (666), (1,331), (1,530) 9.8,
// 13.7, 14.9 and 10.5, 11.5, 13.0.  Batches are ragged, so the limit of many is theirs.
// It is the table's width that a launch knows: a table far wider than its sequences
// gets the balanced split.
constexpr int kFewBlocks8 = 32, kManyBlocks8 = 48, kManyWhole8 = 64;
constexpr float kLog2e8 = 1.4426950408889634f;
// The running maximum moves when a score passes it by 2^4; weights are carried
// at 2^11 times their size, below 2^15, so that the low half's smallest step
// (2^-24) is 2^-35 of the row's largest weight, 2^-31 with V's scales.
constexpr float kMove8 = 4.f, kUp8 = 11.f;
constexpr int kNear8 = 4;

// Record of a piece: O, divided by its sums, as float4 number k * kLanes + r, then the
// heads' maxima (log2 units) and sums.  Lane (g, c) of a warp has k = 4e + q: head 2c +
// e, dims 16g + 4q .. + 3; with up to 4 heads only c < 2 do (kLanes = 16).
template <bool kTwice>
struct Record8 {
  static constexpr int kLanes = kTwice ? 16 : 32;
  static constexpr int kVecs = 8 * kLanes;
  static constexpr int kFloats = 4 * kVecs + 16;
  static constexpr int kBytes = 4 * kFloats;
  static constexpr int kParts = kVecs / 32;  // warps that take a float4 a lane
  float4 o[kVecs];
  float m[8], l[8];
  __device__ static int place(int k, int g, int c) { return k * kLanes + (kTwice ? 2 * g + c : 4 * g + c); }
  __device__ static int head(int f) { return 2 * (f & (kTwice ? 1 : 3)) + (f / kLanes >> 2); }
  __device__ static int dim(int f) { return 16 * ((f % kLanes) / (kTwice ? 2 : 4)) + 4 * (f / kLanes & 3); }
};

struct Decode8Args {
  CUtensorMap tmap;
  const uint8_t* exps;
  const uint16_t* q;          // [B][Hq][128]
  const int32_t* tables;
  const int32_t* seq_lens;
  void* out;
  void* rec;
  long long* err;
  int num_blocks, max_blocks;
  int B, Hq, Hkv, G;
  int out_dtype;
  int whole;                  // a CTA a segment, instead of equal ranges
  float qscale;               // scale * log2(e)
  int hold;                   // self-test: loads of CTA hold - 1 (-1: of all CTAs) do not come, 0: none is held
  long long wait_limit_ns;
};

// A segment (i, h) is one unit for its start (its query rows, its record) and
// one for each of its tiles; pfx[i] counts the units of one kv head before
// sequence i.  A CTA's range is cut into equal ones for its warps.
struct Place8 {
  int i, h, j;  // tile j of the segment, -1: the unit that starts it
};
__device__ __forceinline__ Place8 place8(const Decode8Args& A, const int* pfx, long long u) {
  int lo = 0, hi = A.B - 1;  // the last sequence that starts at or before u (never an empty one)
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (static_cast<long long>(A.Hkv) * pfx[mid] <= u) lo = mid; else hi = mid - 1;
  }
  const int r = static_cast<int>(u - static_cast<long long>(A.Hkv) * pfx[lo]), cnt = pfx[lo + 1] - pfx[lo];
  const int h = r / cnt;
  return {lo, h, r - h * cnt - 1};
}
// Units of segment (i, h): [s0, s0 + cnt).
struct Segment8 {
  long long s0;
  int cnt;
  __device__ Segment8(const Decode8Args& A, const int* pfx, int i, int h)
      : s0(static_cast<long long>(A.Hkv) * pfx[i] + static_cast<long long>(h) * (pfx[i + 1] - pfx[i])),
        cnt(pfx[i + 1] - pfx[i]) {}
};
// Units of a CTA in the balanced split over `ctas` CTAs.
__device__ __forceinline__ long long per_cta8(const Decode8Args& A, const int* pfx, int ctas) {
  const long long per = (static_cast<long long>(A.Hkv) * pfx[A.B] + ctas - 1) / ctas;
  return per < kMinUnits8 ? kMinUnits8 : per;
}

__device__ __forceinline__ int length8(const Decode8Args& A, int i) {
  return min(max(A.seq_lens[i], 0), A.max_blocks * kBlock);
}

// pfx[0 .. B], by a whole CTA.
__device__ void prefix8(const Decode8Args& A, int* pfx, bool report) {
  const int lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < A.B; i += blockDim.x) {
    const int L = length8(A, i);
    if (report && L != A.seq_lens[i]) record_error(A.err, PA_ERR_DEVICE_CHECK, A.seq_lens[i]);
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

__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ uint4 ldmatrix4(uint32_t at) {
  uint4 v;
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t transposed8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The K and V tile number `tile` of the pool into shared memory.  A tile is read once
// for each sequence that holds it, nearly always one, so tiles leave L2 first and push out
// neither records nor tables nor what other kernels read.  With the hint and without, us:
// three inputs in turn, 64 chats 26.9 and 29.2, multi-head 50.0 and 52.4, documents 33.1
// and 35.1; behind a flush 29.2 and 29.3, 51.1 and 51.3, 35.0 and 35.1.  Forks over one
// prefix: 256 behind 1,024 tokens in turn 91.6 and 91.8, behind a flush 93.6 and 92.6; 64
// behind 2,048 51.0 and 51.1, 52.5 and 52.1; 16 behind 8,192 49.0 and 49.2, 51.2 and 50.1.
__device__ __forceinline__ void load_tile8(uint32_t to, const CUtensorMap* map, int tile, uint32_t bar) {
  const int z = 0;
  uint64_t policy;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  mbar_arrive_expect_tx(bar, kPair8);
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %2, %3}],"
      " [%4], %5;" ::"r"(to),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(z), "r"(tile), "r"(bar), "l"(policy)
      : "memory");
}

// A lane's view of 32 units of the warp's range, one a lane: the tile's place in
// the pool (-1: none), K's scale, and packed: how many of its tokens count (0: no
// tile), whether a piece starts with the unit (kNew8) and V's exponent from bit 8 on.
constexpr int kNew8 = 32;
struct Window8 {
  int tile, what;
  float ks;
};
__device__ __forceinline__ Window8 window8(const Decode8Args& A, const int* pfx, long long u, long long u0,
                                           long long end) {
  Window8 w{-1, 0, 0.f};
  if (u >= end) return w;
  const Place8 p = place8(A, pfx, u);
  if (p.j < 0) return w;
  if (p.j == 0 || u == u0) w.what = kNew8;
  const int blk = A.tables[static_cast<long long>(p.i) * A.max_blocks + p.j];
  if (blk >= 0 && blk < A.num_blocks) {
    w.tile = blk * A.Hkv + p.h;
    const int e = reinterpret_cast<const uint16_t*>(A.exps)[w.tile];
    w.ks = scale_of(e & 0xff);
    w.what |= min(length8(A, p.i) - p.j * kBlock, kBlock) | (e & 0xff00);
  } else {
    record_error(A.err, PA_ERR_DEVICE_CHECK, blk);
  }
  // (the first two units of a window: one of them is a tile, and loads behind them are on their way)
  if (A.hold && (A.hold < 0 || A.hold == static_cast<int>(blockIdx.x) + 1) && (threadIdx.x & 31) < 2) w.tile = -1;
  return w;
}

// The query rows of (i, h) as the scores' operand: lane (g, c) holds column g's dims
// 16j + 4c + {0, 1} and {2, 3} in qa[2j] and qa[2j + 1]; column g is head g, or g % 4
// where the columns repeat the heads.  Returns what the column's products have to be
// multiplied by.
template <bool kBf16, bool kTwice>
__device__ __forceinline__ float load_q8(const Decode8Args& A, int i, int h, int g, int c, uint32_t (&qa)[16]) {
  const int head = kTwice ? g & 3 : g;
  const uint2* src = reinterpret_cast<const uint2*>(A.q + (static_cast<long long>(i) * A.Hq + h * A.G + head) * kHeadDim);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint2 x = head < A.G ? src[4 * j + c] : make_uint2(0, 0);
    qa[2 * j] = x.x;
    qa[2 * j + 1] = x.y;
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

// 2^d for d <= 0 (0 below 2^-126).
__device__ __forceinline__ float down2(int d) { return d < -126 ? 0.f : __int_as_float((127 + d) << 23); }

// A running join of records: maximum, sum of weights and four outputs.  Records
// weigh 2^(m - maximum) l; one of -infinity has no weight, but its NaN, if it holds
// one, still counts.  Outputs are means throughout, here and in the records, so that
// the sum of many large values does not leave fp32 where their mean does not.
struct Join8 {
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  template <int N>
  __device__ __forceinline__ void add(const float (&rm)[N], const float (&rl)[N], const float4 (&ro)[N]) {
    float to = m;
#pragma unroll
    for (int k = 0; k < N; ++k) to = fmaxf(to, rm[k]);
    const float had = l * (m == to ? 1.f : fast_exp2(m - to));
    float w[N];
    l = had;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      w[k] = rl[k] * (rm[k] == to ? 1.f : fast_exp2(rm[k] - to));
      l += w[k];
    }
    const float inv = l == 0.f ? 0.f : 1.f / l, f = had * inv;
    o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float a = w[k] * inv;
      o.x = fmaf(a, ro[k].x, o.x);
      o.y = fmaf(a, ro[k].y, o.y);
      o.z = fmaf(a, ro[k].z, o.z);
      o.w = fmaf(a, ro[k].w, o.w);
    }
    m = to;
  }
  __device__ __forceinline__ void store(const Decode8Args& A, int i, int h, int head, int dim) const {
    store_out4(A.out, (static_cast<long long>(i) * A.Hq + h * A.G + head) * kHeadDim + dim, o.x, o.y, o.z, o.w, A.out_dtype);
  }
};

// What follows the pieces of a segment that more than one warp of a CTA took part
// in, noted by the warp of the first one: the last warp, and whether the CTA has the
// whole segment (the result), or a part (a record, in the CTA's slot 0 or 1).
struct Chain8 {
  int i, h, last, kind;  // kind: 0 none, 1 result, 2 and 3 record in slot 0 and 1
};

// What a CTA leaves whose wait ran out: NaN in the rows of each segment that it has
// tiles of, and in its two records, so that a segment which goes on in another CTA gets
// NaN from the second kernel too.
template <bool kTwice>
__device__ __noinline__ void give_up8(const Decode8Args& A, const int* pfx, long long U0, long long U1) {
  using Record = Record8<kTwice>;
  const float nan = __int_as_float(0x7fffffff);
  for (long long u = U0; u < U1;) {
    const Place8 p = place8(A, pfx, u);
    const Segment8 seg(A, pfx, p.i, p.h);
    if (seg.s0 + 1 < U1)  // (not where only its start is here)
      for (int x = threadIdx.x; x < A.G * (kHeadDim / 4); x += blockDim.x)
        store_out4(A.out, (static_cast<long long>(p.i) * A.Hq + p.h * A.G) * kHeadDim + 4 * x, nan, nan, nan, nan, A.out_dtype);
    u = seg.s0 + seg.cnt;
  }
  if (A.whole) return;
  for (int k = 0; k < 2; ++k) {
    Record* rec = static_cast<Record*>(A.rec) + 2 * blockIdx.x + k;
    for (int x = threadIdx.x; x < Record::kVecs; x += blockDim.x) rec->o[x] = make_float4(nan, nan, nan, nan);
    if (threadIdx.x < 8) {
      rec->m[threadIdx.x] = -INFINITY;
      rec->l[threadIdx.x] = nan;
    }
  }
}

// kTwice: at most 4 heads, whose columns are repeated.
template <bool kBf16, bool kE4M3, bool kTwice>
__global__ void __launch_bounds__(kWarps8 * 32, 1) decode8_kernel(const __grid_constant__ Decode8Args A) {
  using Record = Record8<kTwice>;
  extern __shared__ uint8_t smem_raw8[];
  // (the 128-byte swizzle goes by the address)
  uint8_t* const smem8 =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw8) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ __align__(8) unsigned long long s_full[kWarps8][kStages8];
  __shared__ Chain8 s_chain[kWarps8][2];
  __shared__ int s_abort;
  // rings, the warps' first records, the prefix
  Record* const firsts = reinterpret_cast<Record*>(smem8 + kWarps8 * kStages8 * kPair8);
  int* const pfx = reinterpret_cast<int*>(firsts + kWarps8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  if (threadIdx.x == 0) s_abort = 0;
  if (lane < kStages8) mbar_init(smem_addr(&s_full[warp][lane]), 1);
  if (lane < 2) s_chain[warp][lane].kind = 0;
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  if (threadIdx.x == 0) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&A.tmap)) : "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // the tables and the exponents on their way into L2 while the lengths are read: of small
  // pools all (a line a thread; of a pool 10 or 50 times the batch's 7.5 MB that it
  // partly does not need: 64 chats 26.9 us, then 27.5)
  {
    const long long at = 128ll * (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x);
    if (at < 4ll * A.B * A.max_blocks) prefetch_l2(reinterpret_cast<const uint8_t*>(A.tables) + at);
    if (at < 2ll * A.num_blocks * A.Hkv) prefetch_l2(A.exps + at);
  }
  prefix8(A, pfx, blockIdx.x == 0);
  // the CTA's units [U0, U1) and the warp's [u0, u1)
  long long U0, U1, per;
  if (A.whole) {
    const int i = blockIdx.x / A.Hkv;
    const Segment8 seg(A, pfx, i, blockIdx.x - i * A.Hkv);
    U0 = seg.s0;
    U1 = U0 + seg.cnt;
  } else {
    per = per_cta8(A, pfx, gridDim.x);
    U0 = per * blockIdx.x;
    U1 = min(U0 + per, static_cast<long long>(A.Hkv) * pfx[A.B]);
  }
  per = max((U1 - U0 + kWarps8 - 1) / kWarps8, 1ll);
  const long long u0 = U0 + per * warp, u1 = min(u0 + per, U1);
  const int n = static_cast<int>(max(u1 - u0, 0ll));

  const uint32_t ring = smem_addr(smem8) + warp * (kStages8 * kPair8), bars = smem_addr(&s_full[warp][0]);
  // ldmatrix: lane's row of the tile, and its chunk before ^ 2jj; values: dims 16g .. of tokens 2c and 2c + 1
  const uint32_t k_off = ((lane & 7) + (lane & 8)) * kRow8 + (((lane >> 4) ^ (lane & 7)) << 4);
  const uint32_t va_off = kTile8 + 2 * c * kRow8 + ((g ^ (2 * c)) << 4);
  const uint32_t vb_off = kTile8 + (2 * c + 1) * kRow8 + ((g ^ (2 * c + 1)) << 4);
  Window8 now = window8(A, pfx, u0 + lane, u0, u1), next = now;
  uint32_t flying = 0;  // stages with a load on its way
  // unit x of the range into its stage; x and the windows are the same in all lanes
  auto issue = [&](int x, int stage) {
    const int tile = __shfl_sync(0xffffffffu, next.tile, x & 31);
    if (x < n && tile >= 0) {
      flying |= 1u << stage;
      if (lane == 0) load_tile8(ring + stage * kPair8, &A.tmap, tile, bars + 8 * stage);
    }
  };
#pragma unroll
  for (int x = 0; x < kStages8; ++x) issue(x, x);

  // the rows of empty sequences
  for (int i = blockIdx.x; i < A.B; i += gridDim.x)
    if (pfx[i] == pfx[i + 1])
      for (int x = threadIdx.x; x < A.Hq * (kHeadDim / 4); x += blockDim.x)
        store_out4(A.out, (static_cast<long long>(i) * A.Hq * (kHeadDim / 4) + x) * 4, 0.f, 0.f, 0.f, 0.f, A.out_dtype);

  uint32_t qa[16];
  float o[8][4], m[2], l[2], mref[2], fq[2];
  int ci = -1, ch = -1, E = 0;  // the piece in hand
  auto flush = [&]() {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 4);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 8);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 16);
    }
    if (kTwice) {
#pragma unroll
      for (int u = 0; u < 8; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[u][k] += __shfl_xor_sync(0xffffffffu, o[u][k], 2);
    }
    const Segment8 seg(A, pfx, ci, ch);
    const long long rs = seg.s0 + 1, end = seg.s0 + seg.cnt;  // its tiles
    const bool whole = rs >= u0 && end <= u1;                 // all of them are this piece
    const int slot = seg.s0 > u0;
    // (a second record is the last piece's: the ring is done with)
    Record* const rec = slot ? reinterpret_cast<Record*>(smem8 + warp * (kStages8 * kPair8)) : firsts + warp;
    const float unit_of_o = scale_of(E);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int head = 2 * c + e;
      if (kTwice && c >= 2) continue;
      const float f = l[e] == 0.f ? 0.f : 1.f / l[e];
      const long long at = (static_cast<long long>(ci) * A.Hq + ch * A.G + head) * kHeadDim + 16 * g;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float x = o[2 * k][e] * f * unit_of_o, y = o[2 * k][e + 2] * f * unit_of_o;
        const float z = o[2 * k + 1][e] * f * unit_of_o, w = o[2 * k + 1][e + 2] * f * unit_of_o;
        if (!whole)
          rec->o[Record::place(4 * e + k, g, c)] = make_float4(x, y, z, w);
        else if (head < A.G)
          store_out4(A.out, at + 4 * k, x, y, z, w, A.out_dtype);
      }
      if (!whole && g == 0) {
        rec->m[head] = m[e];
        rec->l[head] = l[e];
      }
    }
    if (!whole && lane == 0 && (rs >= u0 || warp == 0)) {
      s_chain[warp][slot] = {ci, ch, static_cast<int>((min(end, U1) - 1 - U0) / per),
                             rs >= U0 && end <= U1 ? 1 : 2 + (seg.s0 > U0)};
    }
  };

  uint32_t parity = 0;  // bit s: phase of stage s
  int stage = 0;
  for (int x = 0; x < n; ++x) {
    if ((x & 31) == 0) now = next;  // (the issues are in this window until the one below)
    const int what = __shfl_sync(0xffffffffu, now.what, x & 31);
    if (what & kNew8) {
      if (ci >= 0) flush();
      const Place8 p = place8(A, pfx, u0 + x);
      ci = p.i;
      ch = p.h;
      const float f = load_q8<kBf16, kTwice>(A, ci, ch, g, c, qa);
      fq[0] = __shfl_sync(0xffffffffu, f, 8 * c);
      fq[1] = __shfl_sync(0xffffffffu, f, 8 * c + 4);
      m[0] = m[1] = -INFINITY;
      mref[0] = mref[1] = l[0] = l[1] = 0.f;
      E = 0;
#pragma unroll
      for (int u = 0; u < 8; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[u][k] = 0.f;
    }
    const int left = what & 31;
    if (left) {
      const bool here = wait_phase(bars + 8 * stage, parity >> stage & 1, &s_abort, A.wait_limit_ns, A.err, 8);
      if (!__all_sync(0xffffffffu, here)) break;
      parity ^= 1u << stage;
      flying &= ~(1u << stage);
      const uint32_t at = ring + stage * kPair8;
      // scores of tokens g (s[0], s[1]) and g + 8 (s[2], s[3]), heads 2c and 2c + 1
      float d0[4] = {0.f, 0.f, 0.f, 0.f}, d1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        const uint4 k = ldmatrix4((at + k_off) ^ (jj << 5));
        uint32_t a0, a1, a2, a3;
        unpack_codes<kE4M3>(k.x, a0, a2);
        unpack_codes<kE4M3>(k.y, a1, a3);
        mma_f16(d0, a0, a1, a2, a3, qa[4 * jj], qa[4 * jj + 1]);
        unpack_codes<kE4M3>(k.z, a0, a2);
        unpack_codes<kE4M3>(k.w, a1, a3);
        mma_f16(d1, a0, a1, a2, a3, qa[4 * jj + 2], qa[4 * jj + 3]);
      }
      const float ks = __shfl_sync(0xffffffffu, now.ks, x & 31);
      float s[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) s[k] = (d0[k] + d1[k]) * (ks * fq[k & 1]);
      if (left < kBlock) {
        if (g >= left) s[0] = s[1] = -INFINITY;
        if (g + 8 >= left) s[2] = s[3] = -INFINITY;
      }
      // running maxima and weights
      const float t0 = fmaxf(s[0], s[2]), t1 = fmaxf(s[1], s[3]);
      if (__any_sync(0xffffffffu, t0 > m[0] + kMove8 || t1 > m[1] + kMove8)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float most = e ? t1 : t0;
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 4));
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 8));
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 16));
          const float to = fmaxf(m[e], most);
          const float f = to == m[e] ? 1.f : fast_exp2(m[e] - to);
          m[e] = to;
          mref[e] = to == -INFINITY ? 0.f : to - kUp8;
          l[e] *= f;
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            o[u][e] *= f;
            o[u][e + 2] *= f;
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) s[k] = fast_exp2(s[k] - mref[k & 1]);
      l[0] += s[0] + s[2];
      l[1] += s[1] + s[3];
      // V's scale
      const int ev = what >> 8;
      if (ev > E && ev != kNanExponent) {
        const float f = down2(E - ev);
        E = ev;
#pragma unroll
        for (int u = 0; u < 8; ++u)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[u][k] *= f;
      }
      const bool near = ev >= E - kNear8;
      if (ev != E) {
        const float f = ev == kNanExponent ? __int_as_float(0x7fffffff) : (near ? down2(ev - E) : 1.f);
#pragma unroll
        for (int k = 0; k < 4; ++k) s[k] *= f;
      }
      uint32_t p0, p1, r0, r1;
      if (kTwice) {
        p0 = transposed8(c < 2 ? pack_hi<false>(s[0], s[1]) : pack_lo<false>(s[0], s[1]));
        p1 = transposed8(c < 2 ? pack_hi<false>(s[2], s[3]) : pack_lo<false>(s[2], s[3]));
      } else {
        p0 = transposed8(pack_hi<false>(s[0], s[1]));
        p1 = transposed8(pack_hi<false>(s[2], s[3]));
        r0 = transposed8(pack_lo<false>(s[0], s[1]));
        r1 = transposed8(pack_lo<false>(s[2], s[3]));
      }
      // values
      uint4 v[4] = {lds16(at + va_off), lds16(at + vb_off), lds16(at + va_off + 8 * kRow8), lds16(at + vb_off + 8 * kRow8)};
      if (left < kBlock) {  // (a weight of zero times NaN is NaN)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (8 * (k >> 1) + 2 * c + (k & 1) >= left) v[k] = make_uint4(0, 0, 0, 0);
      }
      auto values = [&](auto add) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t a = w == 0 ? v[0].x : w == 1 ? v[0].y : w == 2 ? v[0].z : v[0].w;
          const uint32_t b = w == 0 ? v[1].x : w == 1 ? v[1].y : w == 2 ? v[1].z : v[1].w;
          const uint32_t y = w == 0 ? v[2].x : w == 1 ? v[2].y : w == 2 ? v[2].z : v[2].w;
          const uint32_t z = w == 0 ? v[3].x : w == 1 ? v[3].y : w == 2 ? v[3].z : v[3].w;
          uint32_t lo[4], hi[4];  // dims 16g + 4w + 0 .. 3 of tokens 2c, 2c + 1 and 2c + 8, 2c + 9
          unpack_codes<kE4M3>(__byte_perm(a, b, 0x5140), lo[0], lo[1]);
          unpack_codes<kE4M3>(__byte_perm(a, b, 0x7362), lo[2], lo[3]);
          unpack_codes<kE4M3>(__byte_perm(y, z, 0x5140), hi[0], hi[1]);
          unpack_codes<kE4M3>(__byte_perm(y, z, 0x7362), hi[2], hi[3]);
          add(2 * w, lo[0], lo[1], hi[0], hi[1]);
          add(2 * w + 1, lo[2], lo[3], hi[2], hi[3]);
        }
      };
      if (near) {
        values([&](int u, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
          mma_f16(o[u], a0, a1, a2, a3, p0, p1);
          if (!kTwice) mma_f16(o[u], a0, a1, a2, a3, r0, r1);
        });
      } else {
        const float f = down2(ev - E);
        values([&](int u, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
          float d[4] = {0.f, 0.f, 0.f, 0.f};
          mma_f16(d, a0, a1, a2, a3, p0, p1);
          if (!kTwice) mma_f16(d, a0, a1, a2, a3, r0, r1);
#pragma unroll
          for (int k = 0; k < 4; ++k) o[u][k] = fmaf(f, d[k], o[u][k]);
        });
      }
    }
    // the stage is free: the unit kStages8 on, from the window it is in
    __syncwarp();
    const int y = x + kStages8;
    if ((y & 31) == 0 && y < n) next = window8(A, pfx, u0 + y + lane, u0, u1);
    issue(y, stage);
    stage = stage + 1 == kStages8 ? 0 : stage + 1;
  }
  if (flying) {  // a wait ran out: nothing is left on its way into shared memory, with a limit again
    const long long t0 = global_ns();
    for (int k = 0; k < kStages8; ++k)
      while ((flying >> k & 1) && !mbar_try_wait(bars + 8 * k, parity >> k & 1) && global_ns() - t0 < kDrainNs) {
      }
  } else if (ci >= 0) {
    flush();
  }
  __syncthreads();
  if (*static_cast<volatile int*>(&s_abort)) {
    give_up8<kTwice>(A, pfx, U0, U1);
    return;
  }
  // pieces of one segment, joined: a warp a float4 a lane of each
  const Chain8* const chains = &s_chain[0][0];
  uint32_t found = __ballot_sync(0xffffffffu, lane < 2 * kWarps8 && chains[lane < 2 * kWarps8 ? lane : 0].kind != 0);
  for (int t = warp, seen = 0; found; found &= found - 1, seen += Record::kParts) {
    const int number = __ffs(found) - 1, first = number >> 1;
    for (; t < seen + Record::kParts; t += kWarps8) {
      const Chain8 chain = chains[number];
      const int f = (t - seen) * 32 + lane, head = Record::head(f);
      const Record* second = reinterpret_cast<const Record*>(smem8 + first * (kStages8 * kPair8));
      constexpr int kBatch = 4;
      Join8 join;
      for (int w = first; w <= chain.last; w += kBatch) {
        float rm[kBatch], rl[kBatch];
        float4 ro[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          rm[k] = -INFINITY;
          rl[k] = 0.f;
          ro[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (w + k <= chain.last) {
            const Record* rec = w + k == first && (number & 1) ? second : firsts + w + k;
            rm[k] = rec->m[head];
            rl[k] = rec->l[head];
            ro[k] = rec->o[f];
          }
        }
        join.add(rm, rl, ro);
      }
      if (chain.kind == 1) {
        if (head < A.G) join.store(A, chain.i, chain.h, head, Record::dim(f));
      } else {
        Record* rec = static_cast<Record*>(A.rec) + 2 * blockIdx.x + (chain.kind - 2);
        rec->o[f] = join.o;
        if (Record::dim(f) == 0) {
          rec->m[head] = join.m;
          rec->l[head] = join.l;
        }
      }
    }
  }
}

// Joins the records of the segments that CTAs' ranges cut: CTA b has the one that
// goes on behind range b and starts in it, if there is one.
template <bool kTwice>
__global__ void __launch_bounds__(32 * Record8<kTwice>::kParts) merge8_kernel(const __grid_constant__ Decode8Args A) {
  using Record = Record8<kTwice>;
  extern __shared__ uint8_t smem_raw8[];
  int* const pfx = reinterpret_cast<int*>(smem_raw8);
  prefix8(A, pfx, false);
  const long long per = per_cta8(A, pfx, gridDim.x + 1), total = static_cast<long long>(A.Hkv) * pfx[A.B];
  const long long next = per * (blockIdx.x + 1ll);  // the range behind
  int count = 0, i = 0, h = 0;
  bool second = false;
  if (next < total) {
    const Place8 p = place8(A, pfx, next);
    i = p.i;
    h = p.h;
    const Segment8 seg(A, pfx, i, h);
    if (p.j > 0 && (seg.s0 + 1) / per == blockIdx.x) {
      count = static_cast<int>((seg.s0 + seg.cnt - 1) / per - blockIdx.x + 1);
      second = seg.s0 > per * blockIdx.x;
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!count) return;
  const int f = threadIdx.x, head = Record::head(f);
  const Record* rec = static_cast<const Record*>(A.rec) + 2ll * blockIdx.x;
  Join8 join;
  constexpr int kBatch = 8;
  for (int k0 = 0; k0 < count; k0 += kBatch) {
    float rm[kBatch], rl[kBatch];
    float4 ro[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      rm[k] = -INFINITY;
      rl[k] = 0.f;
      ro[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k0 + k < count) {  // (behind the first, a segment's record is slot 0)
        const Record* r = rec + 2 * (k0 + k) + (k0 + k == 0 && second);
        rm[k] = __ldcg(&r->m[head]);
        rl[k] = __ldcg(&r->l[head]);
        ro[k] = __ldcg(&r->o[f]);
      }
    }
    join.add(rm, rl, ro);
  }
  if (head < A.G) join.store(A, i, h, head, Record::dim(f));
}

// Two records a CTA of the balanced split.
static size_t decode8_records(const pa_pool8* p) {
  return 2 * static_cast<size_t>(sm_count(p->device)) * Record8<false>::kBytes;
}

template <bool kBf16, bool kE4M3, bool kTwice>
static int launch_decode8(Decode8Args& A, int device, cudaStream_t st) {
  const int sms = sm_count(device);
  const size_t list = sizeof(int) * (static_cast<size_t>(A.B) + 1);
  static_assert(sizeof(Record8<kTwice>) == Record8<kTwice>::kBytes && sizeof(Record8<kTwice>) <= kStages8 * kPair8, "a record");
  constexpr int kFixed = kWarps8 * (kStages8 * kPair8 + Record8<kTwice>::kBytes) + 1024;  // with room to align it
  constexpr int kMaxSmem = kFixed + sizeof(int) * (kSeqs8 + 1);
  static_assert(kMaxSmem + 1024 <= 232448, "shared memory of an SM, with the static part");
  // once a device, for the largest batch
  static std::atomic<uint64_t> allowed{0};
  const uint64_t bit = device < 64 ? 1ull << device : 0;
  if (!(allowed.load(std::memory_order_relaxed) & bit) || !bit) {
    if (cudaFuncSetAttribute(decode8_kernel<kBf16, kE4M3, kTwice>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem) !=
        cudaSuccess)
      return PA_ERR_CUDA;
    allowed.fetch_or(bit, std::memory_order_relaxed);
  }
  const long long segments = static_cast<long long>(A.B) * A.Hkv;
  A.whole = segments <= sms && A.max_blocks <= (segments >= kManyWhole8 ? kManyBlocks8 : kFewBlocks8);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = st;
  cfg.gridDim = dim3(A.whole ? static_cast<unsigned>(segments) : sms);
  cfg.blockDim = dim3(kWarps8 * 32);
  cfg.dynamicSmemBytes = kFixed + list;
  if (cudaLaunchKernelEx(&cfg, decode8_kernel<kBf16, kE4M3, kTwice>, A) != cudaSuccess) return PA_ERR_CUDA;
  if (A.whole || sms == 1) return PA_OK;
  cfg.gridDim = dim3(sms - 1);
  cfg.blockDim = dim3(32 * Record8<kTwice>::kParts);
  cfg.dynamicSmemBytes = list;
  return cudaLaunchKernelEx(&cfg, merge8_kernel<kTwice>, A) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

template <bool kBf16, bool kE4M3>
static int launch_g8(Decode8Args& A, int device, cudaStream_t st) {
  return A.G <= 4 ? launch_decode8<kBf16, kE4M3, true>(A, device, st) : launch_decode8<kBf16, kE4M3, false>(A, device, st);
}

}  // namespace pa

using namespace pa;

extern "C" size_t pa_decode8_workspace_bytes(pa_pool8_t p, int num_seqs, int n_q_heads, int max_blocks_per_seq) {
  if (!p || num_seqs <= 0 || n_q_heads <= 0 || max_blocks_per_seq <= 0 || n_q_heads % p->n_kv_heads) return 0;
  if (num_seqs > kSeqs8 || n_q_heads / p->n_kv_heads > PA_MAX_GROUP) return 0;
  return decode8_records(p);
}

static int decode8(pa_pool8_t p, const void* q, int q_dtype, const int32_t* block_tables, int max_blocks_per_seq,
                   const int32_t* seq_lens, int num_seqs, int n_q_heads, float scale, void* out, int out_dtype,
                   void* workspace, size_t workspace_bytes, void* stream, int hold, long long limit_ns) {
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
  A.tmap = p->tmap;
  A.exps = p->exps;
  A.q = static_cast<const uint16_t*>(q);
  A.tables = block_tables;
  A.seq_lens = seq_lens;
  A.out = out;
  A.rec = workspace;
  A.err = p->err;
  A.num_blocks = p->num_blocks;
  A.max_blocks = max_blocks_per_seq;
  A.B = num_seqs;
  A.Hq = n_q_heads;
  A.Hkv = p->n_kv_heads;
  A.G = n_q_heads / p->n_kv_heads;
  A.out_dtype = out_dtype;
  A.qscale = scale * kLog2e8;
  A.hold = hold;
  A.wait_limit_ns = limit_ns;
  cudaStream_t st = as_stream(stream);
  const bool e4m3 = p->dtype == PA_E4M3;
  if (q_dtype == PA_BF16) return e4m3 ? launch_g8<true, true>(A, p->device, st) : launch_g8<true, false>(A, p->device, st);
  return e4m3 ? launch_g8<false, true>(A, p->device, st) : launch_g8<false, false>(A, p->device, st);
}

extern "C" int pa_decode8(pa_pool8_t p, const void* q, int q_dtype, const int32_t* block_tables, int max_blocks_per_seq,
                          const int32_t* seq_lens, int num_seqs, int n_q_heads, float scale, void* out, int out_dtype,
                          void* workspace, size_t workspace_bytes, void* stream) {
  return decode8(p, q, q_dtype, block_tables, max_blocks_per_seq, seq_lens, num_seqs, n_q_heads, scale, out, out_dtype,
                 workspace, workspace_bytes, stream, 0, wait_limit_ns());
}

extern "C" int pa_selftest_decode8_timeout(pa_pool8_t p, const void* q, int q_dtype, const int32_t* block_tables,
                                           int max_blocks_per_seq, const int32_t* seq_lens, int num_seqs, int n_q_heads,
                                           float scale, void* out, int out_dtype, void* workspace, size_t workspace_bytes,
                                           int cta, long long limit_ns, void* stream) {
  if (limit_ns <= 0 || limit_ns > 1000000000ll || cta < -1 || cta > 0xffff) return PA_ERR_INVALID;
  return decode8(p, q, q_dtype, block_tables, max_blocks_per_seq, seq_lens, num_seqs, n_q_heads, scale, out, out_dtype,
                 workspace, workspace_bytes, stream, cta < 0 ? -1 : cta + 1, limit_ns);
}
