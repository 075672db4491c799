// Decode attention of sequences that share long prefixes.
//
// The S members of a group hold the same P blocks at the start of their
// tables.  For one kv head their query heads are R = S * G rows against the
// same K and V, so the prefix is a matrix product with R rows, not S separate
// walks over the cache:
//   S = Q K^T (R x tokens), P = 2^(scale log2(e) S - m), O = P V,
// with the running maximum m and sum l of each row kept online.  Each prefix
// is read once per 256 rows; every sequence's own tokens are attended by the
// ordinary decode (decode.cu), and the two are joined by log-sum-exp:
//   out = sum_k 2^(m_k - M) o_k / sum_k 2^(m_k - M) l_k.
//
// Four kernels in stream order: the plan (checks the groups, lays out the
// work), the decode of the own tokens, the prefix product, the combination.
//
// The prefix product runs on the tcgen05 tensor cores, one CTA an SM:
//  - an item is up to 256 rows of one group; a segment is (item, kv head); a
//    unit is a chunk of 128 prefix tokens of a segment.  The stream of all
//    units is cut into equal ranges, one a CTA, so any mix of groups fills
//    the GPU; what a CTA holds of one segment is a piece, and leaves one
//    record (m, l, unnormalised o of 256 rows).
//  - two softmax warpgroups, one thread a row.  An item of more than 128 rows
//    gives each its own 128 rows and both use every chunk; an item of at most
//    128 rows gives both the same rows, and they take chunks in turn (two
//    half-records of one row, joined like any others).  Either way the tensor
//    cores work for one warpgroup while the other one exponentiates.
//  - per chunk: S_w (128 x 128 fp32 in TMEM) = Q_w K^T; the warpgroup reads it
//    (tcgen05.ld), writes P over it as 16-bit values, and P_w V accumulates in
//    TMEM.  K and V tiles arrive by TMA, block by block through the table, as
//    [half][128 rows][128 bytes] with the 128-byte swizzle: K is the K-major
//    operand; V, whose tokens are rows, the MN-major one, 16 tokens (one cache
//    block) an instruction.
//  - the running maximum moves only when a row's maximum grows by more than
//    2^8 (exact either way: m is whatever the weights were taken against), so
//    O in TMEM is rarely rescaled.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstddef>

#include "device_utils.cuh"
#include "pa_internal.h"

namespace pa {

constexpr int kMaxSharedSeqs = 4096;   // the own-token decode's limit
constexpr int kRows = 128;             // rows of a warpgroup
constexpr int kItemRows = 2 * kRows;
constexpr int kChunkBlocks = 8;        // cache blocks of a chunk: 128 tokens
constexpr int kChunk = kChunkBlocks * kBlock;
constexpr int kTile = kChunk * kRowBytes;  // 32 KiB: K or V of a chunk, Q of a warpgroup
constexpr int kHalf = kTile / 2;           // dims 0-63 | 64-127
constexpr int kStages = 2;
constexpr float kLog2eF = 1.4426950408889634f;
constexpr float kMoveBy = 8.f;         // log2 units the maximum may lag behind

constexpr int kPlanCluster = 8, kPlanThreads = 512;
constexpr int kSoftWarps = 8;
constexpr int kPrefixThreads = (kSoftWarps + 2) * 32;  // + producer warp, + MMA warp
constexpr int kRecFloats = kItemRows * kHeadDim + 2 * kItemRows;  // o, m, l

// Plan of one group (device, written by the plan kernel).
struct GroupPlan {
  long long unit0;  // units before this group
  int item0;        // items before this group
  int rows;         // S * G, 0 for a group that takes no part
  int chunks;       // ceil(P / 8)
  int blocks;       // P
  int member0;      // its first entry in members
};

struct SharedArgs {
  CUtensorMap tmap;               // [K|V][half][rows][64] boxes of 16 rows x 64 elements
  const uint16_t* q;              // [B][Hq][128]
  const int32_t* tables;          // [B][max_blocks]
  const int32_t* seq_lens;        // [B]
  const int32_t* group_start;     // [n_groups + 1]
  const int32_t* members;         // [n_members]
  const int32_t* prefix_blocks;   // [n_groups]
  int B, Hq, Hkv, G, n_groups, n_members, max_blocks;
  float qscale;                   // |scale| * log2(e)
  uint32_t qflip;                 // sign bits to flip in q (negative scale)
  void* out;
  int out_dtype;
  // workspace
  GroupPlan* plan;                // [n_groups + 1]; the last: totals
  int32_t* claims;                // [B]: groups that name the sequence
  int32_t* bad;                   // [n_groups]
  int32_t* place;                 // [B]: entry in members, or -1
  int32_t* group_of;              // [B]
  int32_t* lens_s;                // [B]: own tokens
  int32_t* offs_s;                // [B]: table element where they start
  float* o_s;                     // [B][Hq][128]
  float* lse_s;                   // [B][Hq]
  float* rec;                     // records
  long long num_blocks, n_rec;
  long long* err;
  long long wait_limit_ns;
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// One cluster: checks every group and lays out items and units.  A group that
// breaks a rule, or names a sequence that is named twice, is reported and
// takes no part; its members are decoded without it.
__global__ void __cluster_dims__(kPlanCluster, 1, 1) __launch_bounds__(kPlanThreads) shared_plan_kernel(
    const __grid_constant__ SharedArgs A) {
  const int n_threads = kPlanCluster * kPlanThreads;
  const int tid = blockIdx.x * kPlanThreads + threadIdx.x;
  const int lane = threadIdx.x & 31;
  const int cap = A.max_blocks * kBlock;
  // the decode launched as this grid's dependent waits for it to complete
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int i = tid; i < A.B; i += n_threads) {
    A.claims[i] = 0;
    A.place[i] = -1;
  }
  // group_start runs from 0 to n_members and every group has a member, else
  // no group takes part (every CTA looks at all of it)
  int broken = 0;
  for (int k = threadIdx.x; k < A.n_groups; k += kPlanThreads) {
    const int m0 = A.group_start[k], m1 = A.group_start[k + 1];
    broken |= m0 < 0 || m0 >= m1 || m1 > A.n_members || (k == 0 && m0 != 0) ||
              (k == A.n_groups - 1 && m1 != A.n_members);
  }
  broken = __syncthreads_or(broken);
  for (int k = tid; k < A.n_groups; k += n_threads) {
    const int P = A.prefix_blocks[k];
    A.bad[k] = broken || P < 0 || P > A.max_blocks;
  }
  cluster_sync();
  // members: in range, long enough, on the first member's blocks.  One warp
  // an entry; its group is the last that starts at or before it.
  for (int e = tid >> 5; e < A.n_members; e += n_threads >> 5) {
    int lo = 0, hi = A.n_groups - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (A.group_start[mid] <= e) lo = mid; else hi = mid - 1;
    }
    const int k = lo;
    const int i = A.members[e];
    const bool in = i >= 0 && i < A.B;
    if (lane == 0 && in) atomicAdd(&A.claims[i], 1);
    if (__ldcg(&A.bad[k])) continue;
    const int first = A.members[A.group_start[k]];
    const int P = A.prefix_blocks[k];
    bool fine = in && first >= 0 && first < A.B;
    if (fine) {
      const int L = A.seq_lens[i];
      fine = L <= cap && L >= P * kBlock;
      const int32_t* a = A.tables + static_cast<long long>(i) * A.max_blocks;
      const int32_t* b = A.tables + static_cast<long long>(first) * A.max_blocks;
      if (i != first)
#pragma unroll 8
        for (int x = lane; x < P; x += 32) fine = fine && a[x] == b[x];
    }
    if (!__all_sync(0xffffffffu, fine) && lane == 0) A.bad[k] = 1;
  }
  cluster_sync();
  for (int e = tid; e < A.n_members; e += n_threads) {
    const int i = A.members[e];
    if (i < 0 || i >= A.B || __ldcg(&A.claims[i]) < 2) continue;
    int lo = 0, hi = A.n_groups - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (A.group_start[mid] <= e) lo = mid; else hi = mid - 1;
    }
    A.bad[lo] = 1;
  }
  cluster_sync();
  if (tid < 32) {  // the groups' items and units, in group order
    int item = 0;
    long long unit = 0;
    for (int k0 = 0; k0 < A.n_groups; k0 += 32) {
      const int k = k0 + lane;
      GroupPlan g{};
      int items = 0;
      long long units = 0;
      if (k < A.n_groups) {
        const bool bad = __ldcg(&A.bad[k]) != 0;
        if (bad) record_error(A.err, PA_ERR_DEVICE_CHECK, k);
        g.member0 = A.group_start[k];
        g.blocks = A.prefix_blocks[k];
        g.rows = bad || g.blocks == 0 ? 0 : (A.group_start[k + 1] - g.member0) * A.G;
        g.chunks = (g.blocks + kChunkBlocks - 1) / kChunkBlocks;
        items = (g.rows + kItemRows - 1) / kItemRows;
        units = static_cast<long long>(items) * A.Hkv * g.chunks;
      }
      int ii = items;
      long long uu = units;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, ii, o);
        const long long z = __shfl_up_sync(0xffffffffu, uu, o);
        if (lane >= o) {
          ii += y;
          uu += z;
        }
      }
      g.item0 = item + ii - items;
      g.unit0 = unit + uu - units;
      if (k < A.n_groups) A.plan[k] = g;
      item += __shfl_sync(0xffffffffu, ii, 31);
      unit += __shfl_sync(0xffffffffu, uu, 31);
    }
    if (lane == 0) {
      GroupPlan g{};
      g.unit0 = unit;
      g.item0 = item;
      A.plan[A.n_groups] = g;
    }
  }
  for (int e = tid; e < A.n_members; e += n_threads) {
    const int i = A.members[e];
    if (i < 0 || i >= A.B) continue;
    int lo = 0, hi = A.n_groups - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (A.group_start[mid] <= e) lo = mid; else hi = mid - 1;
    }
    if (!__ldcg(&A.bad[lo]) && A.prefix_blocks[lo] > 0) {
      A.place[i] = e;
      A.group_of[i] = lo;
    }
  }
  cluster_sync();
  for (int i = tid; i < A.B; i += n_threads) {
    const int L = A.seq_lens[i];
    const int P = __ldcg(&A.place[i]) >= 0 ? A.prefix_blocks[__ldcg(&A.group_of[i])] : 0;
    A.lens_s[i] = L - P * kBlock;  // (a length out of range is the decode's to report)
    A.offs_s[i] = i * A.max_blocks + P;
  }
}

// ---------------------------------------------------------------------------
// tcgen05 helpers.
// ---------------------------------------------------------------------------
// Shared-memory operand descriptor, 128-byte swizzle: start address, leading
// and stride byte offsets in 16-byte units, version 1, swizzle mode 2.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
  return static_cast<uint64_t>((addr >> 4) & 0x3fff) | static_cast<uint64_t>((lead >> 4) & 0x3fff) << 16 |
         static_cast<uint64_t>((stride >> 4) & 0x3fff) << 32 | 1ull << 46 | 2ull << 61;
}
// Instruction descriptor: fp32 accumulate, A and B of the pool's type, 128 x
// 128; bit 16: B is MN-major.
__host__ __device__ constexpr uint32_t mma_desc(bool bf16, bool b_mn) {
  return 1u << 4 | (bf16 ? 1u : 0u) << 7 | (bf16 ? 1u : 0u) << 10 | (b_mn ? 1u : 0u) << 16 | (128u / 8) << 17 |
         (128u / 16) << 24;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u)
      : "memory");
}
// Arrives on the mbarrier when every MMA this thread issued so far is done.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// 32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, "
      "%24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, "
      "%24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// One half (64 elements) of one (block, head) tile of K (kv 0) or V (kv 1).
__device__ __forceinline__ void tma_load_half(uint32_t dst, const CUtensorMap* map, int y, int half, int kv,
                                              uint32_t bar) {
  const int z = 0;
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(z), "r"(y), "r"(half), "r"(kv), "r"(bar)
      : "memory");
}

// ---------------------------------------------------------------------------
// Pieces of one CTA: the cut of its unit range by segments.
// ---------------------------------------------------------------------------
struct SharedPiece {
  int group, h;
  int row0, rows;      // the item's rows of the group
  int c0, c1;          // chunks
  int blocks;          // the group's prefix blocks
  int member0;
  long long rec;
  bool both;           // more than 128 rows: every chunk for both warpgroups
};

__device__ __forceinline__ GroupPlan load_plan(const GroupPlan* p) {
  const int4* s = reinterpret_cast<const int4*>(p);
  const int4 a = __ldcg(s), b = __ldcg(s + 1);
  GroupPlan g;
  g.unit0 = static_cast<long long>(static_cast<unsigned>(a.x)) | static_cast<long long>(a.y) << 32;
  g.item0 = a.z;
  g.rows = a.w;
  g.chunks = b.x;
  g.blocks = b.y;
  g.member0 = b.z;
  return g;
}
static_assert(sizeof(GroupPlan) == 32 && offsetof(GroupPlan, item0) == 8 && offsetof(GroupPlan, chunks) == 16,
              "load_plan reads a plan as two 16-byte vectors");

// Smallest range of a CTA, in chunks.
constexpr int kMinUnits = 1;
__device__ __forceinline__ long long units_per_cta(long long units, int ctas) {
  const long long per = (units + ctas - 1) / ctas;
  return per < kMinUnits ? kMinUnits : per;
}

struct SharedPieces {
  const SharedArgs& A;
  long long cur, end;
  int cta, k;
  GroupPlan g;

  __device__ SharedPieces(const SharedArgs& a, int c, int ctas) : A(a), cta(c) {
    const long long total = __ldcg(&A.plan[A.n_groups].unit0);
    const long long per = units_per_cta(total, ctas);
    cur = per * cta;
    end = cur + per < total ? cur + per : total;
    k = -1;
    if (cur < end) {  // the last group that starts at or before cur (warp-wide)
      const int lane = threadIdx.x & 31;
      int count = 0;
      for (int k0 = 0; k0 < A.n_groups; k0 += 32) {
        const bool before = k0 + lane < A.n_groups && __ldcg(&A.plan[k0 + lane].unit0) <= cur;
        const int c = __popc(__ballot_sync(0xffffffffu, before));
        count += c;
        if (c < 32) break;
      }
      k = count - 1;
      g = load_plan(&A.plan[k]);
    }
  }
  __device__ bool next(SharedPiece& p) {
    if (cur >= end) return false;
    auto units = [&] {
      return static_cast<long long>((g.rows + kItemRows - 1) / kItemRows) * A.Hkv * g.chunks;
    };
    while (cur - g.unit0 >= units()) g = load_plan(&A.plan[++k]);  // the next group that has units
    const long long u = cur - g.unit0, seg_units = g.chunks;
    const long long seg = u / seg_units;
    const int item = static_cast<int>(seg / A.Hkv);
    p.group = k;
    p.h = static_cast<int>(seg - static_cast<long long>(item) * A.Hkv);
    p.row0 = item * kItemRows;
    p.rows = g.rows - p.row0 < kItemRows ? g.rows - p.row0 : kItemRows;
    p.both = p.rows > kRows;
    p.c0 = static_cast<int>(u - seg * seg_units);
    const long long left = end - cur;
    p.c1 = seg_units - p.c0 < left ? static_cast<int>(seg_units) : p.c0 + static_cast<int>(left);
    p.blocks = g.blocks;
    p.member0 = g.member0;
    // segment number + CTA number grows with every piece: one record each
    p.rec = static_cast<long long>(g.item0) * A.Hkv + seg + cta;
    cur += p.c1 - p.c0;
    return true;
  }
};

struct __align__(1024) PrefixSmem {
  uint8_t q[2][kTile];
  uint8_t k[kStages][kTile];
  uint8_t v[kStages][kTile];
  unsigned long long kfull[kStages], kfree[kStages], vfull[kStages], vfree[kStages];
  unsigned long long qfull, qfree, sfull[2], pfull[2], ofull[2], drain;
  uint32_t mask[kStages];  // blocks of the chunk that are there
  uint32_t tmem;
  int abort_flag;
};

template <bool kBf16, bool kLo>
__global__ void __launch_bounds__(kPrefixThreads, 1) shared_prefix_kernel(const __grid_constant__ SharedArgs A) {
  extern __shared__ uint8_t smem_raw[];
  PrefixSmem& S = *reinterpret_cast<PrefixSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                 ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kProducer = kSoftWarps, kMma = kSoftWarps + 1;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_addr(&S.kfull[s]), 1);
      mbar_init(smem_addr(&S.kfree[s]), 1);
      mbar_init(smem_addr(&S.vfull[s]), 1);
      mbar_init(smem_addr(&S.vfree[s]), 1);
    }
    mbar_init(smem_addr(&S.qfull), 2 * kRows);
    mbar_init(smem_addr(&S.qfree), 2 * kRows);
    for (int w = 0; w < 2; ++w) {
      mbar_init(smem_addr(&S.sfull[w]), 1);
      mbar_init(smem_addr(&S.pfull[w]), kRows);
      mbar_init(smem_addr(&S.ofull[w]), 1);
    }
    mbar_init(smem_addr(&S.drain), 1);
    S.abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMma) {  // all 512 columns: S and P of both warpgroups, O of both
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&S.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem;
  volatile int* abort_flag = &S.abort_flag;
  const long long limit = A.wait_limit_ns;
  auto wait = [&](unsigned long long& bar, uint32_t parity, int site) {
    return wait_phase(smem_addr(&bar), parity, abort_flag, limit, A.err, site);
  };
  SharedPieces pieces(A, blockIdx.x, gridDim.x);
  SharedPiece p;

  if (warp == kProducer) {
    // ---- loads: K and V of each chunk, lane 2b + half for block b
    int n = 0;
    bool ok = true;
    while (ok && pieces.next(p)) {
      const int32_t* row = A.tables + static_cast<long long>(A.members[p.member0]) * A.max_blocks;
      int blk = 0;
      auto fetch = [&](int c) {  // a chunk's block id, one chunk ahead
        const int b = c * kChunkBlocks + (lane >> 1);
        return lane < 2 * kChunkBlocks && c < p.c1 && b < p.blocks ? row[b] : -2;
      };
      blk = fetch(p.c0);
      for (int c = p.c0; c < p.c1; ++c, ++n) {
        const int s = n % kStages;
        const uint32_t use = static_cast<uint32_t>(n / kStages);
        const int ahead = fetch(c + 1);
        const bool valid = blk >= 0 && blk < A.num_blocks;
        if (!valid && blk != -2 && !(lane & 1)) record_error(A.err, PA_ERR_DEVICE_CHECK, static_cast<long long>(blk));
        const uint32_t both = __ballot_sync(0xffffffffu, valid);
        uint32_t mask = 0;
#pragma unroll
        for (int b = 0; b < kChunkBlocks; ++b) mask |= ((both >> (2 * b)) & 1u) << b;
        const int y = static_cast<int>((static_cast<long long>(blk) * A.Hkv + p.h) * kBlock);
        const uint32_t at = (lane & 1) * kHalf + (lane >> 1) * (kBlock * 128);
        const uint32_t bytes = __popc(mask) * kTileBytes;
        // mask[s] is last read by the weights' product of the stage's previous chunk
        ok = (use == 0) || (wait(S.kfree[s], (use - 1) & 1, 20) && wait(S.vfree[s], (use - 1) & 1, 21));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          S.mask[s] = mask;
          if (bytes) {
            mbar_arrive_expect_tx(smem_addr(&S.kfull[s]), bytes);
            mbar_arrive_expect_tx(smem_addr(&S.vfull[s]), bytes);
          } else {
            mbar_arrive(smem_addr(&S.kfull[s]));
            mbar_arrive(smem_addr(&S.vfull[s]));
          }
        }
        __syncwarp();
        if (valid) {
          tma_load_half(smem_addr(S.k[s]) + at, &A.tmap, y, lane & 1, 0, smem_addr(&S.kfull[s]));
          tma_load_half(smem_addr(S.v[s]) + at, &A.tmap, y, lane & 1, 1, smem_addr(&S.vfull[s]));
        }
        blk = ahead;
      }
    }
    // never leave a load in flight into this CTA's shared memory
    if (lane == 0 && *abort_flag) {
      for (int k = n > kStages ? n - kStages : 0; k < n; ++k) {
        const long long t0 = global_ns();
        while (!(mbar_try_wait(smem_addr(&S.kfull[k % kStages]), (k / kStages) & 1) &&
                 mbar_try_wait(smem_addr(&S.vfull[k % kStages]), (k / kStages) & 1)) &&
               global_ns() - t0 < limit) {
        }
      }
    }
  } else if (warp == kMma) {
    // ---- products.  Step t of a piece serves warpgroup t & 1; S of step
    // t + 2 is issued behind P V of step t, whose P it overwrites (the MMAs of
    // one thread run in order).
    if (lane == 0) {
      constexpr uint32_t kIdS = mma_desc(kBf16, false), kIdO = mma_desc(kBf16, true);
      int n0 = 0;         // chunks of earlier pieces
      int piece_no = 0;
      uint32_t p_phase[2] = {0, 0};
      bool ok = true;
      while (ok && pieces.next(p)) {
        const int nc = p.c1 - p.c0;
        const int steps = p.both ? 2 * nc : nc;
        ok = wait(S.qfull, piece_no & 1, 22);
        ++piece_no;
        bool first[2] = {true, true};
        auto scores = [&](int t) {
          const int w = t & 1, n = n0 + (p.both ? t >> 1 : t), s = n % kStages;
          if (!p.both || w == 0) ok = ok && wait(S.kfull[s], (n / kStages) & 1, 23);
          if (!ok) return;
          tc_fence_after();
          {
            const uint32_t a = smem_addr(S.q[p.both ? w : 0]), b = smem_addr(S.k[s]);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
              const uint32_t off = (ks >> 2) * kHalf + (ks & 3) * 32;
              mma_ss(tmem + w * 128, operand_desc(a + off, 16, 1024), operand_desc(b + off, 16, 1024), kIdS, ks > 0);
            }
            mma_commit(smem_addr(&S.sfull[w]));
            if (!p.both || w == 1) mma_commit(smem_addr(&S.kfree[s]));
          }
        };
        if (ok) scores(0);
        if (ok && steps > 1) scores(1);
        for (int t = 0; ok && t < steps; ++t) {
          const int w = t & 1, n = n0 + (p.both ? t >> 1 : t), s = n % kStages;
          ok = wait(S.pfull[w], p_phase[w], 24);
          p_phase[w] ^= 1;
          if (ok && (!p.both || w == 0)) ok = wait(S.vfull[s], (n / kStages) & 1, 25);
          if (!ok) break;
          tc_fence_after();
          const uint32_t mask = *reinterpret_cast<volatile uint32_t*>(&S.mask[s]);
          {
            const uint32_t b = smem_addr(S.v[s]);
            bool add = !first[w];
            for (int kb = 0; kb < kChunkBlocks; ++kb) {
              if (!((mask >> kb) & 1)) continue;
              // 16 tokens: P's 8 columns, V's 16 rows; halves of the dims kHalf apart
              const uint64_t bd = operand_desc(b + kb * (kBlock * 128), kHalf, 1024);
              mma_ts(tmem + 256 + w * 128, tmem + w * 128 + kb * 8, bd, kIdO, add);
              add = true;
              if (kLo) mma_ts(tmem + 256 + w * 128, tmem + w * 128 + 64 + kb * 8, bd, kIdO, true);
            }
            if (!p.both || w == 1) mma_commit(smem_addr(&S.vfree[s]));
            if (t + 2 >= steps) mma_commit(smem_addr(&S.ofull[w]));
          }
          if (mask) first[w] = false;
          if (t + 2 < steps) scores(t + 2);
        }
        n0 += nc;
      }
      if (!ok) {  // wait for the products in flight before the TMEM goes
        mma_commit(smem_addr(&S.drain));
        const long long t0 = global_ns();
        while (!mbar_try_wait(smem_addr(&S.drain), 0) && global_ns() - t0 < limit) {
        }
      }
    }
    __syncwarp();
  } else {
    // ---- softmax: warpgroup w, one thread a row
    const int w = warp >> 2;
    const int r = threadIdx.x & (kRows - 1);
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lane_base + w * 128, t_o = tmem + lane_base + 256 + w * 128;
    uint32_t s_phase = 0, o_phase = 0;
    int n0 = 0, piece_no = 0;
    bool ok = true;
    while (ok && pieces.next(p)) {
      const int nc = p.c1 - p.c0;
      // Q: rows of this warpgroup, or half the rows of the common tile, once
      // both warpgroups are done with the piece before (its products with it)
      if (piece_no > 0) {
        ok = wait(S.qfree, (piece_no - 1) & 1, 28);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      }
      ++piece_no;
      {
        uint8_t* tile = S.q[p.both ? w : 0];
        const int per = p.both ? 1 : 2;  // threads a row
        const int row = p.both ? r : (w * 64 + (r >> 1));
        const int v0 = p.both ? 0 : (r & 1) * 8;
        const int gr = p.row0 + (p.both ? w * kRows : 0) + row;
        const bool have = gr < p.row0 + p.rows;
        const uint4* src = nullptr;
        if (have) {
          const int i = A.members[p.member0 + gr / A.G];
          src = reinterpret_cast<const uint4*>(
              A.q + (static_cast<long long>(i) * A.Hq + p.h * A.G + gr % A.G) * kHeadDim);
        }
#pragma unroll 8
        for (int x = 0; x < 16 / per; ++x) {
          const int c = v0 + x;
          uint4 v = have ? src[c] : make_uint4(0u, 0u, 0u, 0u);
          v.x ^= A.qflip;
          v.y ^= A.qflip;
          v.z ^= A.qflip;
          v.w ^= A.qflip;
          *reinterpret_cast<uint4*>(tile + (c >> 3) * kHalf + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = v;
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(smem_addr(&S.qfull));

      float m = -INFINITY, l = 0.f;
      const int step = p.both ? 1 : 2;
      const int j0 = p.both ? 0 : w;
      bool any = false;
      for (int j = j0; j < nc; j += step) {
        ok = wait(S.sfull[w], s_phase, 26);
        s_phase ^= 1;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        any = true;
        tc_fence_after();
        const uint32_t mask = *reinterpret_cast<volatile uint32_t*>(&S.mask[(n0 + j) % kStages]);
        uint32_t raw[128];
#pragma unroll
        for (int x = 0; x < 4; ++x) tmem_ld32(t_s + 32 * x, raw + 32 * x);
        tmem_wait_ld();
        float mx = -INFINITY;
        if (mask == 0xffu) {
#pragma unroll
          for (int x = 0; x < 128; ++x) {
            const float v = __uint_as_float(raw[x]) * A.qscale;
            raw[x] = __float_as_uint(v);
            mx = fmaxf(mx, v);
          }
        } else {  // blocks past the prefix or outside the pool weigh nothing
#pragma unroll
          for (int x = 0; x < 128; ++x) {
            const float v = (mask >> (x >> 4)) & 1 ? __uint_as_float(raw[x]) * A.qscale : -INFINITY;
            raw[x] = __float_as_uint(v);
            mx = fmaxf(mx, v);
          }
        }
        const bool move = mx > m + kMoveBy;
        if (__any_sync(0xffffffffu, move)) {
          const float mn = move ? mx : m;
          const float alpha = mn == m ? 1.f : fast_exp2(m - mn);
          l *= alpha;
          m = mn;
          if (j != j0) {  // O holds earlier chunks: their product is done (S came after it)
#pragma unroll 1
            for (int x = 0; x < 4; ++x) {
              uint32_t o[32];
              tmem_ld32(t_o + 32 * x, o);
              tmem_wait_ld();
#pragma unroll
              for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * alpha);
              tmem_st32(t_o + 32 * x, o);
            }
          }
        }
        const float base = m == -INFINITY ? 0.f : m;
        float sum = 0.f;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t hi[32], lo[32];
#pragma unroll
          for (int y = 0; y < 32; ++y) {
            const float a = fast_exp2(__uint_as_float(raw[64 * x + 2 * y]) - base);
            const float b = fast_exp2(__uint_as_float(raw[64 * x + 2 * y + 1]) - base);
            sum += a + b;
            hi[y] = pack_hi<kBf16>(a, b);
            if (kLo) lo[y] = pack_lo<kBf16>(a, b);
          }
          tmem_st32(t_s + 32 * x, hi);
          if (kLo) tmem_st32(t_s + 64 + 32 * x, lo);
        }
        l += sum;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(smem_addr(&S.pfull[w]));
      }
      n0 += nc;
      if (!ok) break;
      // ---- the piece's record
      float* rec = A.rec + p.rec * kRecFloats;
      const bool mine = p.both ? w * kRows + r < p.rows : r < p.rows;
      if (any) {
        ok = wait(S.ofull[w], o_phase, 27);
        o_phase ^= 1;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int x = 0; x < 4; ++x) {
          uint32_t o[32];
          tmem_ld32(t_o + 32 * x, o);
          tmem_wait_ld();
          if (mine) {
            uint4* to = reinterpret_cast<uint4*>(rec + static_cast<long long>(w * kRows + r) * kHeadDim + 32 * x);
#pragma unroll
            for (int y = 0; y < 8; ++y) to[y] = make_uint4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
          }
        }
        tc_fence_before();
      }
      if (mine) {
        rec[kItemRows * kHeadDim + w * kRows + r] = m;
        rec[kItemRows * kHeadDim + kItemRows + w * kRows + r] = l;
      }
      mbar_arrive(smem_addr(&S.qfree));
    }
  }
  __syncthreads();
  tc_fence_after();
  if (warp == kMma) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// One warp per (sequence, query head): its own tokens' normalised output with
// log2-sum-exp e, and its records of the prefix.
__global__ void __launch_bounds__(256) shared_combine_kernel(const __grid_constant__ SharedArgs A, int ctas) {
  const long long wid = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (wid >= static_cast<long long>(A.B) * A.Hq) return;
  const int i = static_cast<int>(wid / A.Hq), hq = static_cast<int>(wid - static_cast<long long>(i) * A.Hq);
  const int place = A.place[i];
  float4 O = reinterpret_cast<const float4*>(A.o_s + wid * kHeadDim)[lane];
  if (place >= 0) {
    const GroupPlan g = load_plan(&A.plan[A.group_of[i]]);
    const long long per = units_per_cta(A.plan[A.n_groups].unit0, ctas);
    const int h = hq / A.G;
    const int row = (place - g.member0) * A.G + (hq - h * A.G);
    const int item = row / kItemRows, ir = row - item * kItemRows;
    const int rows = g.rows - item * kItemRows;
    const int sub = rows > kRows ? 1 : 2;  // half-records of a row
    const long long seg = static_cast<long long>(item) * A.Hkv + h;
    const long long u0 = g.unit0 + seg * g.chunks;
    const long long c0 = u0 / per, c1 = (u0 + g.chunks - 1) / per;
    const int count = static_cast<int>(c1 - c0 + 1) * sub;
    const float* rec0 = A.rec + (static_cast<long long>(g.item0) * A.Hkv + seg + c0) * kRecFloats;
    auto row_of = [&](int x) { return (x % sub) * kRows + ir; };
    auto rec_of = [&](int x) { return rec0 + static_cast<long long>(x / sub) * kRecFloats; };
    const float e = A.lse_s[wid];
    float M = e, Ls = e > -INFINITY ? 1.f : 0.f;
    if (!(e > -INFINITY)) O = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x0 = 0; x0 < count; x0 += 32) {
      const int x = x0 + lane;
      float mk = -INFINITY, lk = 0.f;
      if (x < count) {
        const float* t = rec_of(x) + kItemRows * kHeadDim + row_of(x);
        mk = __ldcg(t);
        lk = __ldcg(t + kItemRows);
      }
      float mx = mk;
#pragma unroll
      for (int msk = 1; msk < 32; msk <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, msk));
      const float mn = fmaxf(M, mx);
      if (mn == -INFINITY) continue;
      const float a = M == mn ? 1.f : fast_exp2(M - mn);
      const float wk = mk == -INFINITY ? 0.f : fast_exp2(mk - mn);
      float lw = wk * lk;
#pragma unroll
      for (int msk = 1; msk < 32; msk <<= 1) lw += __shfl_xor_sync(0xffffffffu, lw, msk);
      Ls = Ls * a + lw;
      O.x *= a; O.y *= a; O.z *= a; O.w *= a;
      M = mn;
      const int n = count - x0 < 32 ? count - x0 : 32;
      constexpr int RB = 8;
      for (int b0 = 0; b0 < n; b0 += RB) {
        float4 ob[RB];
        float wb[RB];
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          wb[b] = __shfl_sync(0xffffffffu, wk, (b0 + b) & 31);
          if (b0 + b >= n) wb[b] = 0.f;
          ob[b] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (wb[b] != 0.f)  // (a record without tokens holds no output)
            ob[b] = __ldcg(reinterpret_cast<const float4*>(rec_of(x0 + b0 + b) + row_of(x0 + b0 + b) * kHeadDim) + lane);
        }
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          O.x = fmaf(wb[b], ob[b].x, O.x);
          O.y = fmaf(wb[b], ob[b].y, O.y);
          O.z = fmaf(wb[b], ob[b].z, O.z);
          O.w = fmaf(wb[b], ob[b].w, O.w);
        }
      }
    }
    const float inv = Ls > 0.f ? 1.f / Ls : (Ls == 0.f ? 0.f : Ls);
    O.x *= inv; O.y *= inv; O.z *= inv; O.w *= inv;
  }
  store_out4(A.out, wid * kHeadDim + 4 * lane, O.x, O.y, O.z, O.w, A.out_dtype);
}

// Workspace pieces, each 256-byte aligned.
struct SharedLayout {
  size_t plan, claims, bad, place, group_of, lens_s, offs_s, o_s, lse_s, dec, rec, total;
  size_t dec_bytes;
  long long n_rec;
};
static bool shared_layout(const pa_pool* p, int B, int Hq, int max_blocks, int n_groups, SharedLayout* L) {
  if (!p || B <= 0 || Hq <= 0 || n_groups < 0 || max_blocks <= 0 || Hq % p->n_kv_heads) return false;
  // table rows are addressed by 32-bit element offsets
  if (static_cast<long long>(B) * max_blocks > 0x7fffffffll) return false;
  if (max_blocks > 0x7fffffff / kBlock) return false;
  const int G = Hq / p->n_kv_heads;
  if (G > PA_MAX_GROUP) return false;
  L->dec_bytes = pa_decode_workspace_bytes(const_cast<pa_pool*>(p), B, Hq, max_blocks, 0);
  if (!L->dec_bytes) return false;
  // a sequence is in one group at most, so the groups have at most
  // n_groups + B G / 256 items; a piece more per CTA
  const long long items = n_groups ? n_groups + static_cast<long long>(B) * G / kItemRows : 0;
  L->n_rec = items * p->n_kv_heads + sm_count(p->device);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) / 256 * 256;
    return at;
  };
  L->plan = take(sizeof(GroupPlan) * (static_cast<size_t>(n_groups) + 1));
  L->claims = take(4 * static_cast<size_t>(B));
  L->bad = take(4 * static_cast<size_t>(n_groups));
  L->place = take(4 * static_cast<size_t>(B));
  L->group_of = take(4 * static_cast<size_t>(B));
  L->lens_s = take(4 * static_cast<size_t>(B));
  L->offs_s = take(4 * static_cast<size_t>(B));
  L->o_s = take(static_cast<size_t>(B) * Hq * kHeadDim * 4);
  L->lse_s = take(static_cast<size_t>(B) * Hq * 4);
  L->dec = take(L->dec_bytes);
  L->rec = take(static_cast<size_t>(L->n_rec) * kRecFloats * 4);
  L->total = off;
  return true;
}

static size_t prefix_smem_bytes() { return sizeof(PrefixSmem) + 1024; }

template <bool kBf16, bool kLo>
static int launch_prefix(const SharedArgs& A, int grid, cudaStream_t st) {
  const size_t bytes = prefix_smem_bytes();
  if (cudaFuncSetAttribute(shared_prefix_kernel<kBf16, kLo>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(bytes)) != cudaSuccess)
    return PA_ERR_CUDA;
  shared_prefix_kernel<kBf16, kLo><<<grid, kPrefixThreads, bytes, st>>>(A);
  return cuda_status(cudaGetLastError());
}

}  // namespace pa

using namespace pa;

extern "C" {

size_t pa_decode_shared_workspace_bytes(pa_pool_t p, int num_seqs, int n_q_heads, int max_blocks_per_seq,
                                        int n_groups) {
  SharedLayout L{};
  return shared_layout(p, num_seqs, n_q_heads, max_blocks_per_seq, n_groups, &L) ? L.total : 0;
}

int pa_decode_shared(pa_pool_t p, const void* q, const int32_t* block_tables, int max_blocks_per_seq,
                     const int32_t* seq_lens, int num_seqs, int n_q_heads, float scale, const int32_t* group_start,
                     const int32_t* members, int n_members, const int32_t* prefix_blocks, int n_groups, void* out,
                     int out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (!p || !q || !block_tables || !seq_lens || !out || num_seqs <= 0 || n_groups < 0 || n_members < 0 ||
      (n_groups > 0 && (!group_start || !members || !prefix_blocks)))
    return PA_ERR_INVALID;
  if (n_members > num_seqs || (n_groups == 0) != (n_members == 0)) return PA_ERR_INVALID;
  if (out_dtype != PA_FP16 && out_dtype != PA_BF16 && out_dtype != PA_FP32) return PA_ERR_INVALID;
  if (num_seqs > kMaxSharedSeqs || n_groups > kMaxSharedSeqs) return PA_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15) return PA_ERR_INVALID;
  SharedLayout L{};
  if (!shared_layout(p, num_seqs, n_q_heads, max_blocks_per_seq, n_groups, &L)) return PA_ERR_INVALID;
  if (!workspace || workspace_bytes < L.total || (reinterpret_cast<uintptr_t>(workspace) & 255))
    return PA_ERR_INVALID;
  if (!on_pool_device(p)) return PA_ERR_INVALID;
  char* ws = static_cast<char*>(workspace);
  SharedArgs A{};
  A.tmap = p->tmap_half;
  A.q = static_cast<const uint16_t*>(q);
  A.tables = block_tables;
  A.seq_lens = seq_lens;
  A.group_start = group_start;
  A.members = members;
  A.prefix_blocks = prefix_blocks;
  A.B = num_seqs;
  A.Hq = n_q_heads;
  A.Hkv = p->n_kv_heads;
  A.G = n_q_heads / p->n_kv_heads;
  A.n_groups = n_groups;
  A.n_members = n_members;
  A.max_blocks = max_blocks_per_seq;
  A.qscale = fabsf(scale) * kLog2eF;
  A.qflip = scale < 0.f ? 0x80008000u : 0u;
  A.out = out;
  A.out_dtype = out_dtype;
  A.plan = reinterpret_cast<GroupPlan*>(ws + L.plan);
  A.claims = reinterpret_cast<int32_t*>(ws + L.claims);
  A.bad = reinterpret_cast<int32_t*>(ws + L.bad);
  A.place = reinterpret_cast<int32_t*>(ws + L.place);
  A.group_of = reinterpret_cast<int32_t*>(ws + L.group_of);
  A.lens_s = reinterpret_cast<int32_t*>(ws + L.lens_s);
  A.offs_s = reinterpret_cast<int32_t*>(ws + L.offs_s);
  A.o_s = reinterpret_cast<float*>(ws + L.o_s);
  A.lse_s = reinterpret_cast<float*>(ws + L.lse_s);
  A.rec = reinterpret_cast<float*>(ws + L.rec);
  A.num_blocks = p->num_blocks;
  A.n_rec = L.n_rec;
  A.err = p->err;
  A.wait_limit_ns = wait_limit_ns();
  cudaStream_t st = as_stream(stream);
  shared_plan_kernel<<<kPlanCluster, kPlanThreads, 0, st>>>(A);
  if (cudaGetLastError() != cudaSuccess) return PA_ERR_CUDA;
  int rc = decode_own_tokens(p, q, block_tables, max_blocks_per_seq, A.lens_s, A.offs_s, num_seqs, n_q_heads, scale,
                             A.o_s, A.lse_s, ws + L.dec, L.dec_bytes, stream);
  if (rc != PA_OK) return rc;
  const int ctas = sm_count(p->device);
  if (n_groups > 0) {
    const bool bf16 = p->dtype == PA_BF16, lo = out_dtype == PA_FP32;
    rc = bf16 ? (lo ? launch_prefix<true, true>(A, ctas, st) : launch_prefix<true, false>(A, ctas, st))
              : (lo ? launch_prefix<false, true>(A, ctas, st) : launch_prefix<false, false>(A, ctas, st));
    if (rc != PA_OK) return rc;
  }
  const long long warps = static_cast<long long>(num_seqs) * n_q_heads;
  shared_combine_kernel<<<static_cast<unsigned>((warps * 32 + 255) / 256), 256, 0, st>>>(A, ctas);
  return cuda_status(cudaGetLastError());
}

}  // extern "C"
