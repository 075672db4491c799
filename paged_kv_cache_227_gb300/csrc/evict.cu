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
// (the sums as order-preserving 32-bit keys, 11 + 11 + 10 bits), and compacts
// in position order; counts in shared memory only, so the result does not
// depend on timing.  The move copies rows; in place it is safe because batch
// c (rows j of [a, b)) is written after batches up to c are read, and later
// batches read positions t_j >= j >= b only.
#include "pa_internal.h"

namespace pa {

constexpr int kSelThreads = 1024;
constexpr int kBins = 2048;
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

// Inclusive scan over the block of a 64-bit pair of counters.
__device__ __forceinline__ unsigned long long block_scan(unsigned long long v, unsigned long long* s_warp,
                                                         unsigned long long* total) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  if (lane == 31) s_warp[wid] = v;
  __syncthreads();
  if (wid == 0) {
    unsigned long long x = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    s_warp[lane] = x;
  }
  __syncthreads();
  if (wid) v += s_warp[wid - 1];
  *total = s_warp[31];
  __syncthreads();
  return v;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs A) {
  __shared__ int s_hist[kBins];
  __shared__ unsigned long long s_warp[32];
  __shared__ int s_bin, s_above;
  const int i = blockIdx.y, h = blockIdx.x, tid = threadIdx.x;
  const int span = A.max_blocks * kBlock;
  int L = A.seq_lens[i], n = A.keep[i];
  if (L < 0 || L > span || n < 0) {
    if (tid == 0 && h == 0) record_error(A.err, PA_ERR_DEVICE_CHECK, L < 0 || L > span ? L : n);
    L = L < 0 ? 0 : (L > span ? span : L);
    n = n < 0 ? 0 : n;
  }
  if (n > L) n = L;
  if (n > A.dst_blocks * kBlock) {  // more rows than the destination holds
    if (tid == 0 && h == 0) record_error(A.err, PA_ERR_DEVICE_CHECK, n);
    n = A.dst_blocks * kBlock;
  }
  if (tid == 0 && h == 0) A.lens_out[i] = n;
  const int a = n < A.n_sink ? n : A.n_sink;
  const int b = n - a < A.n_recent ? n - a : A.n_recent;
  const int lo = a, hi = L - b;  // the tokens that compete
  int r = n - a - b;             // how many of them stay
  const long long row = (static_cast<long long>(i) * A.Hkv + h) * span;
  const float* w = A.w + row;
  float* w_out = A.w_out + row;
  int32_t* kept = A.kept + row;

  // the r-th largest key `cut`, and how many keys equal to it stay
  uint32_t cut = 0;
  int ties = 0;
  const bool all = r == hi - lo;
  if (!all && r > 0) {
    uint32_t prefix = 0;
    int shift = 32;
    for (int pass = 0; pass < 3; ++pass) {
      const int bits = pass < 2 ? 11 : 10;
      const int above_shift = shift;
      shift -= bits;
      for (int x = tid; x < kBins; x += kSelThreads) s_hist[x] = 0;
      __syncthreads();
      for (int t = lo + tid; t < hi; t += kSelThreads) {
        const uint32_t key = weight_key(w[t]);
        if (pass == 0 || (key >> above_shift) == prefix) atomicAdd(&s_hist[(key >> shift) & ((1u << bits) - 1)], 1);
      }
      __syncthreads();
      // bins from the top: thread tid takes bins kBins - 1 - 2 tid and the one below
      const int c0 = s_hist[kBins - 1 - 2 * tid], c1 = s_hist[kBins - 2 - 2 * tid];
      unsigned long long total;
      const int incl = static_cast<int>(block_scan(c0 + c1, s_warp, &total));
      const int before = incl - c0 - c1;
      if (before < r && r <= before + c0) {
        s_bin = kBins - 1 - 2 * tid;
        s_above = before;
      } else if (before + c0 < r && r <= incl) {
        s_bin = kBins - 2 - 2 * tid;
        s_above = before + c0;
      }
      __syncthreads();
      prefix = (pass == 0 ? 0u : prefix << bits) | static_cast<uint32_t>(s_bin);
      r -= s_above;
      __syncthreads();
    }
    cut = prefix;
    ties = r;
  }

  // compaction: rank = stayers before + equal keys before (the first `ties` stay)
  unsigned long long carry = 0;  // high half: equal keys, low half: other stayers
  for (int base = 0; base < L; base += kSelThreads) {
    const int t = base + tid;
    float x = 0.f;
    bool stays = false, equal = false;
    if (t < L) {
      x = w[t];
      const uint32_t key = weight_key(x);
      const bool open = t >= lo && t < hi && !all;
      stays = !open || (n - a - b > 0 && key > cut);
      equal = open && ties > 0 && key == cut;
    }
    unsigned long long total;
    const unsigned long long mine = (static_cast<unsigned long long>(equal) << 32) | (stays ? 1u : 0u);
    const unsigned long long before = carry + block_scan(mine, s_warp, &total) - mine;
    const int eq = static_cast<int>(before >> 32);
    if (stays || (equal && eq < ties)) {
      const int rank = static_cast<int>(before & 0xffffffffu) + (eq < ties ? eq : ties);
      kept[rank] = t;
      w_out[rank] = x;
    }
    carry += total;
  }
  __syncthreads();
  for (int t = n + tid; t < L; t += kSelThreads) w_out[t] = 0.f;
}

// One CTA per (sequence, kv head, K or V, slice of the row): 16 / slices
// lanes of 16 bytes a row.
template <int kSlices>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs A, uint4* k_pool, uint4* v_pool) {
  constexpr int LPR = 16 / kSlices;          // lanes a row
  constexpr int RPP = kMoveThreads / LPR;    // rows a pass
  constexpr int U = 4;                       // passes a batch
  const int i = blockIdx.y;
  int x = blockIdx.x;
  const int slice = x % kSlices;
  x /= kSlices;
  uint4* pool = (x & 1) ? v_pool : k_pool;
  const int h = x >> 1;
  const int n = A.lens_out[i];
  const int c = slice * LPR + threadIdx.x % LPR, rr = threadIdx.x / LPR;
  const int32_t* kept = A.kept + (static_cast<long long>(i) * A.Hkv + h) * A.max_blocks * kBlock;
  const int32_t* src = A.src + static_cast<long long>(i) * A.max_blocks;
  const int32_t* dst = A.dst + static_cast<long long>(i) * A.dst_blocks;
  for (int j0 = 0; j0 < n; j0 += RPP * U) {
    uint4 d[U];
    uint4* to[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * RPP + rr;
      to[u] = nullptr;
      if (j >= n) continue;
      const int t = kept[j];
      const long long sb = src[t >> 4], db = dst[j >> 4];
      if (sb < 0 || sb >= A.num_blocks || db < 0 || db >= A.num_blocks) {
        record_error(A.err, PA_ERR_DEVICE_CHECK, sb < 0 || sb >= A.num_blocks ? sb : db);
        continue;
      }
      const uint4* from = pool + ((sb * A.Hkv + h) * kBlock + (t & 15)) * 16 + c;
      uint4* at = pool + ((db * A.Hkv + h) * kBlock + (j & 15)) * 16 + c;
      if (from == at) continue;
      d[u] = *from;
      to[u] = at;
    }
    __syncthreads();  // the batch is read: its rows may be written
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (to[u]) *to[u] = d[u];
  }
}

}  // namespace pa

using namespace pa;

extern "C" int pa_evict(pa_pool_t p, const float* weights, float* weights_out, const int32_t* block_tables,
                        int max_blocks_per_seq, const int32_t* dst_tables, int dst_blocks_per_seq,
                        const int32_t* seq_lens, const int32_t* keep, int num_seqs, int n_sink, int n_recent,
                        int32_t* seq_lens_out, int32_t* kept, void* stream) {
  if (!p || num_seqs < 0 || max_blocks_per_seq <= 0 || n_sink < 0 || n_recent < 0) return PA_ERR_INVALID;
  if (dst_tables && dst_blocks_per_seq <= 0) return PA_ERR_INVALID;
  if (max_blocks_per_seq > 0x7fffffff / kBlock || dst_blocks_per_seq > 0x7fffffff / kBlock) return PA_ERR_INVALID;
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
  evict_select_kernel<<<dim3(A.Hkv, num_seqs), kSelThreads, 0, st>>>(A);
  if (cudaGetLastError() != cudaSuccess) return PA_ERR_CUDA;
  uint4 *k = static_cast<uint4*>(p->k), *v = static_cast<uint4*>(p->v);
  evict_move_kernel<4><<<dim3(A.Hkv * 2 * 4, num_seqs), kMoveThreads, 0, st>>>(A, k, v);
  return cuda_status(cudaGetLastError());
}
