// Eviction from the cache by accumulated attention weight.
//
// Each kv head of a sequence keeps n = min(keep, L) of its L cached tokens:
// the first n_sink, the last n_recent, and of the rest the n - n_sink -
// n_recent with the largest weight sums (equal sums: the lowest position;
// NaN ranks below every number).  The kept tokens close up in their order:
// token j of the result is position t_j of the old cache, t_0 < t_1 < ..., so
// t_j >= j.  Rotary positions are in the keys already, so a row is moved bit
// for bit, and every head may keep other tokens, since a (block, kv head)
// tile belongs to one head.
//
// Two kernels.  The selection finds the r-th largest sum exactly, by radix
// (the sums as order-preserving 32-bit keys, 11 + 11 + 10 bits, and direct
// ranking as soon as few keys are left), and compacts in position order;
// counts in shared memory only, so the result does not depend on timing.  The
// move copies rows.  Into fresh blocks every row is independent.  In place it
// is safe because batch c (rows j of [a, b)) is written after batches up to c
// are read, and later batches read positions t_j >= j >= b only.
//
// Bound: the move by memory (64 sequences of 8 heads, 1,024 of about 4,000
// tokens kept: 537 MB in 85 us, 6.3 TB/s, 0.93 of this GPU's copy rate), the
// selection by instructions (22 us there, for 8 MB: about 1,300 a warp of 8
// tokens a lane).  The whole call 107 us; 4 sequences of 8-32K tokens to 4,001
// 41 us, in place 54 us.
#include "pa_internal.h"

namespace pa {

// Radix digits of the selection: 11 bits first (sign, exponent and two bits of
// the mantissa: sums of attention weights spread over about 50 bins, so one
// pass mostly leaves few enough keys to rank directly).
constexpr int kBins = 2048;
// Copies of each bin, by lane: equal keys of a warp meet 16 at a time.  That
// does not pay: with one copy (half the counts to clear and read) the whole call
// takes 105.5 us instead of 106.6 for 64 sequences of 4,000, and 103.1 instead of
// 105.8 where all sums are equal.
constexpr int kCopies = 2;
// Keys ranked directly: two warps' work, less than a pass.  64 sequences of 2,000
// tokens: 57.3 us with 32, 56.2 with 64, 55.9 with 128; of 4,000: 106.4, 106.6 and 106.9.
constexpr int kList = 64;
constexpr int kLongBins = 256, kLongCopies = 8;  // the long rows' four passes of 8 bits
constexpr int kMoveThreads = 256;

struct EvictArgs {
  const float* w;            // [B][Hkv][span]
  float* w_out;              // [B][Hkv][span], may be w
  const int32_t* src;        // [B][max_blocks]
  const int32_t* dst;        // [B][dst_blocks]
  const int32_t* seq_lens;   // [B]
  const int32_t* keep;       // [B]
  int32_t* lens_out;         // [B]
  int32_t* kept;             // [B][Hkv][span]
  int B, Hkv, max_blocks, dst_blocks, n_sink, n_recent;
  long long num_blocks;
  long long* err;
};

// Order-preserving key: larger float, larger key; -0 as +0; NaN lowest.
__device__ __forceinline__ uint32_t weight_key(float x) {
  if (isnan(x)) return 0u;
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// What a row keeps: n of its L tokens, those before lo and from hi on always,
// and `r` of the others.
struct EvictRow {
  int L, n, lo, hi, r;
  const float* w;
  float* w_out;
  int32_t* kept;
  __device__ EvictRow(const EvictArgs& A, int i, int h, bool first) {
    const int span = A.max_blocks * kBlock;
    L = A.seq_lens[i];
    n = A.keep[i];
    if (L < 0 || L > span || n < 0) {
      if (first && h == 0) record_error(A.err, PA_ERR_DEVICE_CHECK, L < 0 || L > span ? L : n);
      L = L < 0 ? 0 : (L > span ? span : L);
      n = n < 0 ? 0 : n;
    }
    if (n > L) n = L;
    if (n > A.dst_blocks * kBlock) {  // more rows than the destination holds
      if (first && h == 0) record_error(A.err, PA_ERR_DEVICE_CHECK, n);
      n = A.dst_blocks * kBlock;
    }
    if (first && h == 0) A.lens_out[i] = n;
    const int a = n < A.n_sink ? n : A.n_sink;
    const int b = n - a < A.n_recent ? n - a : A.n_recent;
    lo = a;
    hi = L - b;
    r = n - a - b;
    const long long row = (static_cast<long long>(i) * A.Hkv + h) * span;
    w = A.w + row;
    w_out = A.w_out + row;
    kept = A.kept + row;
  }
  __device__ bool contest() const { return r > 0 && r < hi - lo; }
};

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// `x` of CTA `rank` of this cluster.
__device__ __forceinline__ int remote_int(const int* x, int rank) {
  uint32_t at;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(at)
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(x))), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

// The bin of the r-th key from the top, given thread e's counts c of bins
// N - 1 - e BPT and the BPT - 1 below it (N = THREADS * BPT bins; threads past
// them pass zeros).  found[0] = bin, [1] = keys in higher bins, [2] = keys in
// the bin.  Ends with a block barrier.
template <int BPT>
__device__ __forceinline__ void find_bin(int r, const int (&c)[BPT], int bins, int* s_sums, int* found) {
  const int e = threadIdx.x, lane = e & 31, wid = e >> 5;
  int sum = 0;
#pragma unroll
  for (int q = 0; q < BPT; ++q) sum += c[q];
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_sums[wid] = incl;
  __syncthreads();
  int w = lane < wid ? s_sums[lane] : 0;
  int above = incl - sum + __reduce_add_sync(0xffffffffu, w);
  if (above < r && r <= above + sum) {
#pragma unroll
    for (int q = 0; q < BPT; ++q) {
      if (above < r && r <= above + c[q]) {
        found[0] = bins - 1 - e * BPT - q;
        found[1] = above;
        found[2] = c[q];
      }
      above += c[q];
    }
  }
  __syncthreads();
}

// Rows of up to CL * THREADS * K tokens: a cluster of CL CTAs a row, the keys
// in registers (K a thread at most; the warps share the row's tokens evenly
// and a warp's are contiguous, so ranks grow with lane, warp and CTA).  A thread's tokens are bits of two masks: those that
// stay for sure, and those whose key agrees with the cut so far; a pass costs
// a token only while its bit is in the second.
// (1,024 threads an SM are 64 registers each.  Three CTAs of 256 threads instead
// of four, with more registers, are no faster: 64 sequences of 4,000 tokens, 16 a
// thread, which spill 56 bytes, 333.2 us against 332.4 with nearly all kept; of
// 2,000, 8 a thread, 58.8 against 56.2)
template <int THREADS, int K, int CL>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) evict_select_kernel(const EvictArgs A) {
  constexpr int NW = THREADS / 32;
  constexpr int BPT = kBins / THREADS;
  __shared__ __align__(16) int s_hist[kBins * kCopies];
  __shared__ __align__(16) int s_total[2][CL > 1 ? kBins : 4];
  __shared__ int s_found[3], s_sums[32];
  __shared__ uint2 s_list[kList];  // key, token
  __shared__ uint2 s_all[CL > 1 ? kList : 1];
  __shared__ int s_n;              // entries of s_list
  __shared__ uint32_t s_ranked[NW * K];  // by warp and k: the lanes whose token is ranked in
  __shared__ int s_warp[32];
  __shared__ int s_equal, s_stay;  // this CTA's
  const int rank = CL > 1 ? static_cast<int>(blockIdx.x % CL) : 0;
  const int h = blockIdx.x / CL, tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (the move waits for this grid)
  const EvictRow R(A, blockIdx.y, h, rank == 0 && tid == 0);
  const int used = (R.L + 32 * NW * CL - 1) / (32 * NW * CL);  // tokens a thread, at most K
  const int t0 = (rank * NW + wid) * 32 * used + lane;         // token of bit k: t0 + 32 k
  // the tokens in use, in steps of four (all K in turn would issue the unused)
  auto each = [&](const auto& f) {
#pragma unroll
    for (int k0 = 0; k0 < K; k0 += 4)
      if (k0 < used) {
#pragma unroll
        for (int k = k0; k < k0 + 4; ++k) f(k);
      }
  };
  auto sync = [] {
    if (CL > 1) cluster_barrier(); else __syncthreads();
  };
  // this thread's share of the CTAs' `x` before this one, by warp 0's lanes
  auto before = [&](const int* x) {
    int sum = 0;
#pragma unroll
    for (int c = 0; c < CL - 1; ++c) sum += c < rank ? remote_int(x, c) : 0;
    return sum;
  };
  auto warp_scan = [&](int* own) {  // exclusive over the CTA's warps; *own: the CTA's total
    int v = lane < NW ? s_warp[lane] : 0;
    const int mine = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    if (tid == 31) *own = v;
    return __shfl_sync(0xffffffffu, v - mine, wid);
  };

  float x[K];
  each([&](int k) {
    const int t = t0 + 32 * k;
    x[k] = k < used && t < R.L ? R.w[t] : 0.f;
  });
  uint32_t key[K];
  uint32_t stay = 0, open = 0;
  each([&](int k) {
    const int t = t0 + 32 * k;
    key[k] = weight_key(x[k]);
    const bool inside = k < used && t >= R.lo && t < R.hi;
    stay |= static_cast<uint32_t>(k < used && t < R.L && !inside) << k;
    open |= static_cast<uint32_t>(inside) << k;
  });
  if (R.r == R.hi - R.lo) stay |= open;
  if (R.contest()) {
    int r = R.r;
    for (int e = tid; e < kBins * kCopies / 4; e += THREADS) reinterpret_cast<int4*>(s_hist)[e] = make_int4(0, 0, 0, 0);
    if (tid == 0) s_n = 0;
    __syncthreads();
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t ones = pass < 2 ? 2047 : 1023;
      if (__any_sync(0xffffffffu, open)) {
        each([&](int k) {
          if ((open >> k) & 1)
            atomicAdd(&s_hist[((key[k] >> shift) & ones) * kCopies + (lane & (kCopies - 1))], 1);
        });
      }
      __syncthreads();
      int c[BPT];  // of bins kBins - 1 - BPT tid - q
#pragma unroll
      for (int q = 0; q < BPT; q += 2) {  // two bins, two copies each
        int4* p = reinterpret_cast<int4*>(s_hist + (kBins - 2 - BPT * tid - q) * kCopies);
        const int4 v = *p;
        *p = make_int4(0, 0, 0, 0);
        c[q] = v.z + v.w;
        c[q + 1] = v.x + v.y;
      }
      if (CL > 1) {  // (two buffers: the next pass writes the other one)
        int* total = s_total[pass & 1];
#pragma unroll
        for (int q = 0; q < BPT; ++q) total[q * THREADS + tid] = c[q];
        cluster_barrier();
#pragma unroll
        for (int q = 0; q < BPT; ++q) {
          c[q] = 0;
#pragma unroll
          for (int o = 0; o < CL; ++o) c[q] += remote_int(&total[q * THREADS + tid], o);
        }
      }
      find_bin<BPT>(r, c, kBins, s_sums, s_found);
      const uint32_t bin = s_found[0];
      r -= s_found[1];
      if (__any_sync(0xffffffffu, open)) {
        each([&](int k) {
          const uint32_t digit = (key[k] >> shift) & ones;
          const uint32_t bit = open & (1u << k);
          if (digit > bin) stay |= bit;
          if (digit != bin) open &= ~bit;
        });
      }
      if (s_found[2] == r || s_found[2] <= kList) break;
    }
    const int left = s_found[2];
    if (left == r) {
      stay |= open;  // every key that agrees with the cut stays
    } else if (left <= kList) {
      // few keys left: a thread each counts those that come before it
      for (int e = tid; e < NW * K; e += THREADS) s_ranked[e] = 0;
      if (__any_sync(0xffffffffu, open))
        each([&](int k) {
          if ((open >> k) & 1) s_list[atomicAdd(&s_n, 1)] = make_uint2(key[k], t0 + 32 * k);
        });
      sync();
      const uint2* list = s_list;
      if (CL > 1) {
        int first = 0;
        for (int o = 0; o < CL; ++o) {
          const int n = remote_int(&s_n, o);
          if (tid < n) {
            s_all[first + tid].x = remote_int(reinterpret_cast<const int*>(&s_list[tid].x), o);
            s_all[first + tid].y = remote_int(reinterpret_cast<const int*>(&s_list[tid].y), o);
          }
          first += n;
        }
        list = s_all;
        __syncthreads();
      }
      if (tid < left) {
        const uint2 me = list[tid];
        int ahead = 0;
        for (int e = 0; e < left; ++e) {
          const uint2 y = list[e];
          ahead += y.x > me.x || (y.x == me.x && y.y < me.y);
        }
        const int at = static_cast<int>(me.y) - rank * NW * 32 * used;  // among this CTA's tokens
        if (ahead < r && at >= 0 && at < NW * 32 * used)
          atomicOr(&s_ranked[at / (32 * used) * K + at / 32 % used], 1u << (at & 31));
      }
      __syncthreads();
      each([&](int k) { stay |= ((s_ranked[wid * K + k] >> lane) & 1) << k; });
    } else {  // many equal keys: the first r of them stay
      const int mine = __reduce_add_sync(0xffffffffu, __popc(open));
      if (lane == 0) s_warp[wid] = mine;
      __syncthreads();
      int first = warp_scan(&s_equal);
      sync();
      first += before(&s_equal);
      uint32_t some = 0;
      each([&](int k) {
        const uint32_t m = __ballot_sync(0xffffffffu, (open >> k) & 1);
        if (((open >> k) & 1) && first + __popc(m & ((1u << lane) - 1)) < r) some |= 1u << k;
        first += __popc(m);
      });
      stay |= some;
      __syncthreads();  // s_warp is read
    }
  }

  // the stayers' sums again (a key does not tell -0 from 0 or one NaN from
  // another), read before any is written: w_out may be w
  each([&](int k) { x[k] = (stay >> k) & 1 ? R.w[t0 + 32 * k] : 0.f; });
  const int mine = __reduce_add_sync(0xffffffffu, __popc(stay));
  if (lane == 0) s_warp[wid] = mine;
  __syncthreads();
  int at = warp_scan(&s_stay);
  sync();
  at += before(&s_stay);
  each([&](int k) {
    const bool mine = (stay >> k) & 1;
    const uint32_t m = __ballot_sync(0xffffffffu, mine);
    if (mine) {
      const int j = at + __popc(m & ((1u << lane) - 1));
      R.kept[j] = t0 + 32 * k;
      R.w_out[j] = x[k];
    }
    at += __popc(m);
  });
  for (int t = R.n + rank * THREADS + tid; t < R.L; t += THREADS * CL) R.w_out[t] = 0.f;
  if (CL > 1) cluster_barrier();  // s_stay may still be read by the other CTAs
}

// Longer rows: one CTA a row, which reads the row again for every pass (from
// L2: 128K tokens are 512 KB).
__global__ void __launch_bounds__(1024) evict_select_long_kernel(const EvictArgs A) {
  constexpr int K = 8, TILE = 1024 * K;
  __shared__ __align__(16) int s_hist[kLongBins * kLongCopies];
  __shared__ int s_found[3], s_sums[32];
  __shared__ int2 s_warp[32];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const EvictRow R(A, blockIdx.y, blockIdx.x, tid == 0);
  float x[K];
  auto load = [&](int tile) {  // token k of this lane: tile + 32 (K wid + k) + lane
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int t = tile + 32 * (K * wid + k) + lane;
      x[k] = t < R.L ? R.w[t] : 0.f;
    }
  };
  uint32_t cut = 0;
  int ties = 0;
  const bool contest = R.contest(), all = R.r == R.hi - R.lo;
  if (contest) {
    int r = R.r;
    for (int e = tid; e < kLongBins * kLongCopies; e += 1024) s_hist[e] = 0;
    __syncthreads();
#pragma unroll 1
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int tile = 0; tile < R.L; tile += TILE) {
        load(tile);
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const int t = tile + 32 * (K * wid + k) + lane;
          const uint32_t key = weight_key(x[k]);
          if (t >= R.lo && t < R.hi && (shift == 24 || (key >> (shift + 8)) == cut))
            atomicAdd(&s_hist[((key >> shift) & 255) * kLongCopies + (lane & (kLongCopies - 1))], 1);
        }
      }
      __syncthreads();
      int c[1] = {0};
      if (tid < kLongBins) {
        int4* p = reinterpret_cast<int4*>(s_hist + (kLongBins - 1 - tid) * kLongCopies);
        const int4 u = p[0], v = p[1];
        p[0] = p[1] = make_int4(0, 0, 0, 0);
        c[0] = (u.x + u.y) + (u.z + u.w) + ((v.x + v.y) + (v.z + v.w));
      }
      find_bin<1>(r, c, kLongBins, s_sums, s_found);
      cut = cut << 8 | static_cast<uint32_t>(s_found[0]);
      r -= s_found[1];
    }
    ties = r;
  }
  // rank = stayers before + equal keys before (the first `ties` of them stay);
  // a tile's ranks are at or before its tokens, which are read by then
  const uint32_t below = (1u << lane) - 1;
  int2 carry = make_int2(0, 0);
  for (int tile = 0; tile < R.L; tile += TILE) {
    load(tile);
    uint32_t stay = 0, equal = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int t = tile + 32 * (K * wid + k) + lane;
      const uint32_t key = weight_key(x[k]);
      const bool inside = t >= R.lo && t < R.hi;
      stay |= static_cast<uint32_t>(t < R.L && (!inside || all || (contest && key > cut))) << k;
      equal |= static_cast<uint32_t>(inside && contest && key == cut) << k;
    }
    const int2 mine = make_int2(__reduce_add_sync(0xffffffffu, __popc(stay)),
                                __reduce_add_sync(0xffffffffu, __popc(equal)));
    if (lane == 0) s_warp[wid] = mine;
    __syncthreads();  // (and every token of the tile is read)
    int2 v = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v.x, o), z = __shfl_up_sync(0xffffffffu, v.y, o);
      if (lane >= o) {
        v.x += y;
        v.y += z;
      }
    }
    int sb = carry.x + __shfl_sync(0xffffffffu, v.x, wid) - mine.x;
    int eb = carry.y + __shfl_sync(0xffffffffu, v.y, wid) - mine.y;
    carry.x += __shfl_sync(0xffffffffu, v.x, 31);
    carry.y += __shfl_sync(0xffffffffu, v.y, 31);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const bool s = (stay >> k) & 1, q = (equal >> k) & 1;
      const uint32_t ms = __ballot_sync(0xffffffffu, s), mq = __ballot_sync(0xffffffffu, q);
      const int e = eb + __popc(mq & below);
      if (s || (q && e < ties)) {
        const int j = sb + __popc(ms & below) + (e < ties ? e : ties);
        R.kept[j] = tile + 32 * (K * wid + k) + lane;
        R.w_out[j] = x[k];
      }
      sb += __popc(ms);
      eb += __popc(mq);
    }
    __syncthreads();  // s_warp is read
  }
  for (int t = R.n + tid; t < R.L; t += 1024) R.w_out[t] = 0.f;
}

// CTAs of one (sequence, kv head, K or V) share its rows, 256-byte rows of 16
// lanes: 64 rows a batch and CTA, every CTA its own batches.  A sequence with
// a destination block of its own table has to move batch by batch: its rows
// are cut into 1 << lg slices instead, one CTA a slice, and the other CTAs
// leave.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs A, uint4* k_pool, uint4* v_pool,
                                                                  int lg) {
  constexpr int U = 4;  // rows a thread in flight
  const int i = blockIdx.y;
  uint4* pool = (blockIdx.x & 1) ? v_pool : k_pool;
  const int h = blockIdx.x >> 1;
  const int32_t* kept = A.kept + (static_cast<long long>(i) * A.Hkv + h) * A.max_blocks * kBlock;
  const int32_t* src = A.src + static_cast<long long>(i) * A.max_blocks;
  const int32_t* dst = A.dst + static_cast<long long>(i) * A.dst_blocks;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the selection
  const int n = A.lens_out[i];
  bool ordered = A.src == A.dst;
  if (!ordered) {
    int own = 0;
    const int nb = (n + kBlock - 1) / kBlock;
    for (int j = threadIdx.x; j < nb; j += kMoveThreads) own |= j < A.max_blocks && dst[j] == src[j];
    ordered = __syncthreads_or(own);
  }
  if (!ordered) lg = 0;
  const int lanes = 4 - lg;                          // log2 of a row's lanes
  const int part = ordered ? 0 : blockIdx.z, parts = ordered ? 1 : gridDim.z;
  if (ordered && static_cast<int>(blockIdx.z) >= (1 << lg)) return;
  const int c = (ordered ? blockIdx.z << lanes : 0) + (threadIdx.x & ((1 << lanes) - 1)), rr = threadIdx.x >> lanes;
  const int rpp = kMoveThreads >> lanes, batch = rpp * U;
  int t[U];
  auto indexes = [&](int j0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * rpp + rr;
      t[u] = j < n ? kept[j] : -1;
    }
  };
  indexes(part * batch);
  for (int j0 = part * batch; j0 < n; j0 += batch * parts) {
    uint4 d[U];
    uint4* to[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * rpp + rr;
      to[u] = nullptr;
      if (t[u] < 0) continue;
      const long long sb = __ldg(src + (t[u] >> 4)), db = __ldg(dst + (j >> 4));
      if (sb < 0 || sb >= A.num_blocks || db < 0 || db >= A.num_blocks) {
        record_error(A.err, PA_ERR_DEVICE_CHECK, sb < 0 || sb >= A.num_blocks ? sb : db);
        continue;
      }
      const uint4* from = pool + ((sb * A.Hkv + h) * kBlock + (t[u] & 15)) * 16 + c;
      uint4* at = pool + ((db * A.Hkv + h) * kBlock + (j & 15)) * 16 + c;
      if (from == at) continue;
      d[u] = *from;
      to[u] = at;
    }
    indexes(j0 + batch * parts);
    if (ordered) __syncthreads();  // the batch is read: its rows may be written
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (to[u]) *to[u] = d[u];
  }
}

template <int THREADS, int K, int CL>
static cudaError_t launch_select(const EvictArgs& A, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(A.Hkv) * CL, static_cast<unsigned>(A.B));
  cfg.blockDim = dim3(THREADS);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CL;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CL > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel<THREADS, K, CL>, A);
}

}  // namespace pa

using namespace pa;

extern "C" int pa_evict(pa_pool_t p, const float* weights, float* weights_out, const int32_t* block_tables,
                        int max_blocks_per_seq, const int32_t* dst_tables, int dst_blocks_per_seq,
                        const int32_t* seq_lens, const int32_t* keep, int num_seqs, int n_sink, int n_recent,
                        int32_t* seq_lens_out, int32_t* kept, void* stream) {
  if (!p || num_seqs < 0 || max_blocks_per_seq <= 0 || n_sink < 0 || n_recent < 0) return PA_ERR_INVALID;
  if (dst_tables && dst_blocks_per_seq <= 0) return PA_ERR_INVALID;
  if (max_blocks_per_seq > kMaxWalkedBlocks || dst_blocks_per_seq > kMaxWalkedBlocks) return PA_ERR_UNSUPPORTED;
  if (num_seqs > 65535 || p->n_kv_heads > 65535) return PA_ERR_UNSUPPORTED;  // a grid dimension each
  if (num_seqs == 0) return PA_OK;
  if (!weights || !weights_out || !block_tables || !seq_lens || !keep || !seq_lens_out || !kept) return PA_ERR_INVALID;
  if (seq_lens_out == seq_lens || seq_lens_out == keep) return PA_ERR_INVALID;  // read while it is written
  if (!on_pool_device(p)) return PA_ERR_INVALID;
  EvictArgs A{};
  A.w = weights;
  A.w_out = weights_out;
  A.src = block_tables;
  A.dst = dst_tables ? dst_tables : block_tables;
  A.seq_lens = seq_lens;
  A.keep = keep;
  A.lens_out = seq_lens_out;
  A.kept = kept;
  A.B = num_seqs;
  A.Hkv = p->n_kv_heads;
  A.max_blocks = max_blocks_per_seq;
  A.dst_blocks = dst_tables ? dst_blocks_per_seq : max_blocks_per_seq;
  A.n_sink = n_sink;
  A.n_recent = n_recent;
  A.num_blocks = p->num_blocks;
  A.err = p->err;
  cudaStream_t st = as_stream(stream);
  const int span = max_blocks_per_seq * kBlock;
  cudaError_t e = cudaSuccess;
  // the smallest CTAs that hold a row's keys in registers, 16 a thread at most (64
  // sequences of up to 6,500 tokens, whole calls: 512 threads of 16 106.6 us, 256
  // of 32 111.7, 1,024 of 8 109.6); from 8,192 tokens on a cluster of them (32 rows
  // of up to 32K: 4 CTAs each 17 us; 8 CTAs add 8 us, one CTA that reads its row
  // again for each pass takes 44).  The lengths are on the device: the width of
  // the table stands for them
  if (span <= 256 * 8) e = launch_select<256, 8, 1>(A, st);
  else if (span <= 256 * 16) e = launch_select<256, 16, 1>(A, st);
  else if (span <= 512 * 16) e = launch_select<512, 16, 1>(A, st);
  else if (span <= 512 * 16 * 2) e = launch_select<512, 16, 2>(A, st);
  else if (span <= 512 * 16 * 4) e = launch_select<512, 16, 4>(A, st);
  else if (span <= 512 * 16 * 8) e = launch_select<512, 16, 8>(A, st);
  else evict_select_long_kernel<<<dim3(A.Hkv, A.B), 1024, 0, st>>>(A);
  if (e != cudaSuccess || cudaGetLastError() != cudaSuccess) return PA_ERR_CUDA;
  // CTAs of a row group: about 4,096 in all (64 sequences of 8 heads 106.6 us with
  // 4 a group, 113.6 with 1, 117.4 with 16; 4 long ones, 63 a group, 41.0-41.4 us
  // from 16 a group on), at most one a batch of the longest row.  Slices: about
  // 512 CTAs that move in order (in place, 4 long sequences: 8 slices 53.9 us, 4
  // slices 61.6; 64 sequences: 1 slice 118.6, 2 slices 111.0, which this rule
  // does not take).  Whole calls.
  const long long groups = 2ll * A.Hkv * num_seqs;
  int lg = 0;
  while (lg < 3 && (groups << lg) < 512) ++lg;
  long long parts = 4096 / groups;
  const long long batches = (static_cast<long long>(A.dst_blocks) * kBlock + 63) / 64;
  if (parts > batches) parts = batches;
  if (A.src == A.dst || parts < (1 << lg)) parts = 1 << lg;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2u * A.Hkv, num_seqs, static_cast<unsigned>(parts));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, evict_move_kernel, A, static_cast<uint4*>(p->k), static_cast<uint4*>(p->v), lg) !=
      cudaSuccess)
    return PA_ERR_CUDA;
  return cuda_status(cudaGetLastError());
}
