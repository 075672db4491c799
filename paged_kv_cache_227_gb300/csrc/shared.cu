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
// Four kernels, each a programmatic dependent of the one before: the plan
// (checks the groups, lays out the work), the prefix product, the decode of the
// own tokens, and the combination (in decode.cu, with the decode's own merge).
// The product is bound by the tensor cores and the decode by memory, so they
// share the GPU: the plan gives the product as many SMs as its part of the
// work, estimated, and the decode's CTAs take the others, and what the product
// frees.
//
// The prefix product runs on the tcgen05 tensor cores, one CTA an SM:
//  - an item is up to 256 rows of one group; a segment is (item, kv head); a
//    unit is a chunk of 128 prefix tokens of a segment.  The stream of all
//    units is cut into equal ranges, one a CTA, so any mix of groups fills
//    the GPU; what a CTA holds of one segment is a piece, and leaves one
//    record (m, l, unnormalised o of 256 rows).
//  - two teams of 256 softmax threads, two threads a row (64 tokens of a chunk
//    each, the maxima exchanged through shared memory).  An item of more than
//    128 rows gives each team its own 128 rows and both use every chunk; an
//    item of at most 128 rows gives both the same rows, and they take chunks
//    in turn (two half-records of one row, joined like any others).  Either
//    way the tensor cores work for one team while the other one exponentiates.
//  - per chunk: S_w (128 x 128 fp32 in TMEM) = Q_w K^T; the team reads it
//    (tcgen05.ld), writes P over it as 16-bit values, and P_w V accumulates in
//    TMEM.  K and V tiles arrive by TMA, block by block through the table, as
//    [half][128 rows][128 bytes] with the 128-byte swizzle: K is the K-major
//    operand; V, whose tokens are rows, the MN-major one, 16 tokens (one cache
//    block) an instruction.
//  - the running maximum moves only when a row's maximum grows by more than
//    2^8 (exact either way: m is whatever the weights were taken against), so
//    O in TMEM is rarely rescaled.
//  - a weight is rounded to the pool's 16 bits for the value product when the
//    output has 16 bits (half a step of each weight, averaged over the tokens,
//    against half a step of the output); with a 32-bit output it is carried as
//    a high and a low half, in two products.  fp16 has five bits of exponent, so
//    its weights are taken times 2^7: up to 2^15 while the maximum lags, and
//    full steps down to 2^-21 of the maximum's weight (2^-14 without).
//
// Measured (2,070 MHz): a chunk of two tiles takes 3,500 cycles, of which the
// tensor cores could do with 2,048 (8 KB of operands from shared memory each 64
// cycles for the scores is all that it gives, and each hand-over leaves them
// idle for about 100); a piece costs 10 us (its queries, the first load, its
// record).  256 samples of a 16K document, 32 query and 8 kv heads: 125 us for
// 69 GFLOP and 259 MB, the product on 96 SMs for 100 us and the decode of 188 MB
// on the others; 64 chats behind 2,048 tokens: 39 us for 81 MB.  18 warps an SM
// leave 96 registers a thread: the form with two halves and bf16 spills 40 bytes,
// the others 4 to 12.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cmath>
#include <cstddef>
#include <type_traits>

#include "device_utils.cuh"
#include "pa_internal.h"
#include "shared_plan.cuh"

namespace pa {

constexpr int kMaxSharedSeqs = 4096;   // the own-token decode's limit
constexpr int kChunkBlocks = 8;        // cache blocks of a chunk: 128 tokens
constexpr int kChunk = kChunkBlocks * kBlock;
constexpr int kTile = kChunk * kRowBytes;  // 32 KiB: K or V of a chunk, Q of a warpgroup
constexpr int kHalf = kTile / 2;           // dims 0-63 | 64-127
constexpr int kStages = 2;
constexpr float kLog2eF = 1.4426950408889634f;
constexpr float kMoveBy = 8.f;         // log2 units the maximum may lag behind
// log2 of the weight at the maximum (a lagging one adds kMoveBy: below 2^16, where fp16 ends)
template <bool kBf16>
constexpr float kTopWeight = kBf16 ? 0.f : 7.f;
static_assert(kTopWeight<false> + kMoveBy < 16.f, "a weight is past fp16");

constexpr int kPlanCluster = 8, kPlanThreads = 1024, kSmallThreads = 1024;
constexpr int kSoftWarps = 16;
constexpr int kTeam = 256;             // threads of a team: two a row
constexpr int kPrefixThreads = (kSoftWarps + 2) * 32;  // + producer warp, + MMA warp
constexpr int kMasks = 4;              // chunk masks in flight
constexpr long long kDrainNs = 2000000000ll;  // limit of the last waits of a CTA that gives up
// Estimates, in ns, to divide the SMs by: a chunk of the product on its SM, a
// CTA's start and records; a tile of 16 tokens of the decode on one SM, and its
// start.  Measured on 64 chats of 2,048 + about 280 tokens, 16 multi-head
// sequences of two prompts, and 256 samples of a 16K document (a chunk 1.8 us,
// a piece 10 us; tiles 0.16-0.22 us).
constexpr float kChunkNs = 1800.f, kPieceNs = 12000.f, kTileNs = 200.f, kDecodeNs = 4000.f;

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
  // workspace
  GroupPlan* plan;                // [n_groups + 1]; the last: totals
  int32_t* owner;                 // [B]: entry in members + 1 that claimed the sequence, or 0
  int32_t* bad;                   // [n_groups]
  int32_t* place;                 // [B]: entry in members, or -1
  int32_t* group_of;              // [B]
  long long* tiles;               // [kPlanCluster]: each plan CTA's part of sum ceil(L / 16)
  int32_t* lens_s;                // [B]: own tokens
  int32_t* offs_s;                // [B]: table element where they start
  float* rec;                     // records
  long long num_blocks;
  int ctas;                       // of the prefix product: at most this many work
  long long* err;
  long long wait_limit_ns;
  int hold;                       // self-test: nothing is loaded, so that the waits run out
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Checks every group and lays out items and units: CL CTAs of T threads (a
// cluster, for the table comparisons of large batches; else one CTA, which
// keeps its marks in shared memory).  A group that breaks a rule, or names a
// sequence that is named twice, is reported and takes no part; its members
// are decoded without it.
constexpr int kSmallPlan = 512;  // sequences and groups of the one-CTA plan

template <int CL, int T>
__global__ void __launch_bounds__(T) shared_plan_kernel(const __grid_constant__ SharedArgs A) {
  __shared__ long long s_tiles[T / 32];
  __shared__ int s_owner[CL == 1 ? kSmallPlan : 1], s_group[CL == 1 ? kSmallPlan : 1], s_bad[CL == 1 ? kSmallPlan : 1];
  int* const owner = CL == 1 ? s_owner : A.owner;
  int* const group_of = CL == 1 ? s_group : A.group_of;
  int* const bad = CL == 1 ? s_bad : A.bad;
  auto sync = [] {
    if (CL > 1) cluster_sync(); else __syncthreads();
  };
  auto get = [](const int* x) { return CL > 1 ? __ldcg(x) : *const_cast<const volatile int*>(x); };
  constexpr int n_threads = CL * T;
  const int tid = blockIdx.x * T + threadIdx.x;
  const int lane = threadIdx.x & 31;
  const int cap = A.max_blocks * kBlock;
  // the product launched as this grid's dependent waits for it to complete
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  long long tiles = 0;
  for (int i = tid; i < A.B; i += n_threads) {
    owner[i] = 0;
    const int L = A.seq_lens[i];
    tiles += L > 0 ? ((L < cap ? L : cap) + kBlock - 1) / kBlock : 0;
  }
  // group_start runs from 0 to n_members and every group has a member, else
  // no group takes part (every CTA looks at all of it)
  int broken = 0;
  for (int k = threadIdx.x; k < A.n_groups; k += T) {
    const int m0 = A.group_start[k], m1 = A.group_start[k + 1];
    broken |= m0 < 0 || m0 >= m1 || m1 > A.n_members || (k == 0 && m0 != 0) ||
              (k == A.n_groups - 1 && m1 != A.n_members);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) tiles += __shfl_xor_sync(0xffffffffu, tiles, o);
  if (lane == 0) s_tiles[threadIdx.x >> 5] = tiles;
  // (a member entry's loads start before the barrier)
  const int e0 = tid >> 5;
  int i0 = 0, first0 = 0;
  if (e0 < A.n_members) {
    i0 = A.members[e0];
    first0 = A.members[0];
  }
  broken = __syncthreads_or(broken);
  if (threadIdx.x < 32) {
    long long sum = lane < T / 32 ? s_tiles[lane] : 0;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
      if (CL > 1)
        A.tiles[blockIdx.x] = sum;
      else
        s_tiles[0] = sum;
    }
  }
  for (int k = tid; k < A.n_groups; k += n_threads) {
    const int P = A.prefix_blocks[k];
    bad[k] = broken || P < 0 || P > A.max_blocks;
  }
  // a member entry's group: the last that starts at or before it
  auto group_at = [&](int e) {
    int lo = 0, hi = A.n_groups - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (A.group_start[mid] <= e) lo = mid; else hi = mid - 1;
    }
    return lo;
  };
  sync();
  // members: in range, named once, long enough, on the first member's blocks.
  // One warp an entry.
  for (int e = e0; e < A.n_members; e += n_threads >> 5) {
    const int k = group_at(e);
    const int i = e == e0 ? i0 : A.members[e];
    const bool in = i >= 0 && i < A.B;
    if (lane == 0 && in) {
      const int before = atomicExch(&owner[i], e + 1);
      if (before) bad[k] = bad[group_at(before - 1)] = 1;
      group_of[i] = k;  // (either, when named twice: both groups are bad)
    }
    const int m0 = A.group_start[k], P = A.prefix_blocks[k];
    if (broken || P < 0 || P > A.max_blocks) continue;
    const int first = k == 0 ? first0 : A.members[m0];
    bool fine = in && first >= 0 && first < A.B;
    if (fine) {
      const int L = A.seq_lens[i];
      fine = L <= cap && L >= P * kBlock;
      const int32_t* a = A.tables + static_cast<long long>(i) * A.max_blocks;
      const int32_t* b = A.tables + static_cast<long long>(first) * A.max_blocks;
      int other = 0;
      if (i != first) {
        int x = lane;
        if (A.max_blocks % 4 == 0 && reinterpret_cast<uintptr_t>(A.tables) % 16 == 0) {  // 4 entries a load
          const int4 *a4 = reinterpret_cast<const int4*>(a), *b4 = reinterpret_cast<const int4*>(b);
#pragma unroll 4
          for (int y = lane; y < P / 4; y += 32) {
            const int4 u = a4[y], v = b4[y];
            other |= (u.x ^ v.x) | (u.y ^ v.y) | (u.z ^ v.z) | (u.w ^ v.w);
          }
          x += P / 4 * 4;
        }
#pragma unroll 8
        for (; x < P; x += 32) other |= a[x] ^ b[x];
      }
      fine = fine && other == 0;
    }
    if (!__all_sync(0xffffffffu, fine) && lane == 0) bad[k] = 1;
  }
  sync();
  if (blockIdx.x == 0 && threadIdx.x < 32) {  // the groups' items and units, in group order
    int item = 0;
    long long unit = 0, shared_tiles = 0;
    for (int k0 = 0; k0 < A.n_groups; k0 += 32) {
      const int k = k0 + lane;
      GroupPlan g{};
      int items = 0;
      long long units = 0;
      if (k < A.n_groups) {
        const bool out = get(&bad[k]) != 0;
        if (out) record_error(A.err, PA_ERR_DEVICE_CHECK, k);
        g.member0 = A.group_start[k];
        g.blocks = A.prefix_blocks[k];
        const int members = out || g.blocks == 0 ? 0 : A.group_start[k + 1] - g.member0;
        g.rows = members * A.G;
        g.chunks = out ? 0 : (g.blocks + kChunkBlocks - 1) / kChunkBlocks;
        items = (g.rows + kItemRows - 1) / kItemRows;
        units = static_cast<long long>(items) * A.Hkv * g.chunks;
        shared_tiles += static_cast<long long>(members) * g.blocks;
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
    long long own = CL > 1 ? (lane < CL ? __ldcg(&A.tiles[lane]) : 0) : (lane == 0 ? s_tiles[0] : 0);
    own -= shared_tiles;
#pragma unroll
    for (int o = 16; o; o >>= 1) own += __shfl_xor_sync(0xffffffffu, own, o);
    // SMs of the product: those with which the later of the two halves ends
    // first; or all of them, and the decode after it
    const float product = static_cast<float>(unit) * kChunkNs, decode = static_cast<float>(own) * A.Hkv * kTileNs;
    float best = 3e38f;
    int best_n = A.ctas;
    for (int n = 1 + lane; n <= A.ctas; n += 32) {
      const float x = product / n + kPieceNs, y = decode / (A.ctas - n) + kDecodeNs;
      const float time = n < A.ctas ? fmaxf(x, y) : x + decode / n + kDecodeNs;
      if (time < best) {
        best = time;
        best_n = n;
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const float t = __shfl_xor_sync(0xffffffffu, best, o);
      const int n = __shfl_xor_sync(0xffffffffu, best_n, o);
      if (t < best || (t == best && n < best_n)) {
        best = t;
        best_n = n;
      }
    }
    if (lane == 0) {
      GroupPlan g{};
      g.unit0 = unit;
      g.item0 = item;
      g.rows = unit < best_n ? static_cast<int>(unit) : best_n;
      A.plan[A.n_groups] = g;
    }
  }
  for (int i = tid; i < A.B; i += n_threads) {
    const int e = get(&owner[i]) - 1;
    const int k = e >= 0 ? get(&group_of[i]) : 0;
    const int P = e >= 0 && !get(&bad[k]) ? A.prefix_blocks[k] : 0;
    if (CL == 1) A.group_of[i] = k;
    A.place[i] = P > 0 ? e : -1;
    A.lens_s[i] = A.seq_lens[i] - P * kBlock;  // (a length out of range is the decode's to report)
    A.offs_s[i] = i * A.max_blocks + P;
  }
}

// ---------------------------------------------------------------------------
// tcgen05 helpers.
// ---------------------------------------------------------------------------
// Shared-memory operand descriptor, 128-byte swizzle, as two words.  Low: start
// address and leading byte offset; high: stride byte offset (8 rows, 1,024
// bytes), version 1, swizzle mode 2; offsets in 16-byte units.  The issuing
// thread adds constants to the low word only: an MMA takes 64 cycles, and
// descriptors built anew for each one cost more than that to issue.
constexpr uint32_t kDescHigh = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t lead) { return addr >> 4 | (lead >> 4) << 16; }
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// Instruction descriptor: fp32 accumulate, A and B of the pool's type, 128 x
// 128; bit 16: B is MN-major.
__host__ __device__ constexpr uint32_t mma_desc(bool bf16, bool b_mn) {
  return 1u << 4 | (bf16 ? 1u : 0u) << 7 | (bf16 ? 1u : 0u) << 10 | (b_mn ? 1u : 0u) << 16 | (128u / 8) << 17 |
         (128u / 16) << 24;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(add), "r"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(add), "r"(kDescHigh)
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
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(addr)
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
  int h;
  int row0, rows;      // the item's rows of the group
  int c0, c1;          // chunks
  int blocks;          // the group's prefix blocks
  int member0;
  long long rec;
  bool both;           // more than 128 rows: every chunk for both warpgroups
};

// A warp's walk over its CTA's pieces.  It lives in shared memory, written by
// lane 0: in registers it would push the softmax loop into spills, and with
// 200 KB of shared memory a spill goes past L1.
struct SharedPieces {
  long long cur, end;
  GroupPlan g;
  int k, more;
  SharedPiece p;

  // All lanes call; the first piece is p when `more`.
  __device__ void start(const SharedArgs& A, int cta) {
    const GroupPlan all = load_plan(&A.plan[A.n_groups]);
    const long long total = all.unit0, per = units_per_cta(total, all.rows);
    const int lane = threadIdx.x & 31;
    const long long from = per * cta;
    int count = 0;
    if (from < total) {  // the last group that starts at or before it (warp-wide)
      for (int k0 = 0; k0 < A.n_groups; k0 += 32) {
        const bool before = k0 + lane < A.n_groups && __ldcg(&A.plan[k0 + lane].unit0) <= from;
        const int c = __popc(__ballot_sync(0xffffffffu, before));
        count += c;
        if (c < 32) break;
      }
    }
    if (lane == 0) {
      cur = from;
      end = from + per < total ? from + per : total;
      k = count - 1;
      if (count) g = load_plan(&A.plan[k]);
      step(A, cta);
    }
    __syncwarp();
  }
  __device__ void next(const SharedArgs& A, int cta) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) step(A, cta);
    __syncwarp();
  }
  __device__ void step(const SharedArgs& A, int cta) {
    more = cur < end;
    if (!more) return;
    auto units = [&] {
      return static_cast<long long>((g.rows + kItemRows - 1) / kItemRows) * A.Hkv * g.chunks;
    };
    while (cur - g.unit0 >= units()) g = load_plan(&A.plan[++k]);  // the next group that has units
    const long long u = cur - g.unit0, seg_units = g.chunks;
    const long long seg = u / seg_units;
    const int item = static_cast<int>(seg / A.Hkv);
    p.h = static_cast<int>(seg - static_cast<long long>(item) * A.Hkv);
    p.row0 = item * kItemRows;
    p.rows = g.rows - p.row0 < kItemRows ? g.rows - p.row0 : kItemRows;
    p.both = p.rows > kRows;
    p.c0 = static_cast<int>(u - seg * seg_units);
    const long long left = end - cur;
    p.c1 = seg_units - p.c0 < left ? static_cast<int>(seg_units) : p.c0 + static_cast<int>(left);
    p.blocks = g.blocks;
    p.member0 = g.member0;
    p.rec = static_cast<long long>(g.item0) * A.Hkv + seg + cta;
    cur += p.c1 - p.c0;
  }
};

// Barrier of the 256 threads of team w, of the 64 threads of a pair of warps, and
// whether `x` holds for all threads of a barrier.
__device__ __forceinline__ void team_sync(int w) { asm volatile("bar.sync %0, 256;" ::"r"(w + 1) : "memory"); }
__device__ __forceinline__ void pair_sync(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool vote(int id, int threads, bool x) {
  uint32_t y;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(y)
      : "r"(x ? 1u : 0u), "r"(id), "r"(threads)
      : "memory");
  return y != 0;
}

struct __align__(1024) PrefixSmem {
  uint8_t q[2][kTile];
  uint8_t k[kStages][kTile];
  uint8_t v[kStages][kTile];
  unsigned long long kfull[kStages], kfree[kStages], vfull[kStages], vfree[kStages];
  unsigned long long qfull, qfree, sfull[2], pfull[2][2], ofull[2], drain;
  SharedPieces pieces[kSoftWarps + 2];
  float part[2][2][kRows];  // by team and half: a row's maximum, or its sum
  uint32_t mask[kMasks];  // blocks of the chunk that are there
  uint32_t tmem;
  int abort_flag;
  int begun[2];  // K and V loads issued
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
    mbar_init(smem_addr(&S.qfull), 2 * kTeam);
    mbar_init(smem_addr(&S.qfree), 2 * kTeam);
    for (int w = 0; w < 2; ++w) {
      mbar_init(smem_addr(&S.sfull[w]), 1);
      mbar_init(smem_addr(&S.pfull[w][0]), kRows);
      mbar_init(smem_addr(&S.pfull[w][1]), kRows);
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
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = S.tmem;
  volatile int* abort_flag = &S.abort_flag;
  const long long limit = A.wait_limit_ns;
  auto wait = [&](unsigned long long& bar, uint32_t parity, int site) {
    return wait_phase(smem_addr(&bar), parity, abort_flag, limit, A.err, site);
  };
  volatile SharedPieces* const walk = &S.pieces[warp];
  S.pieces[warp].start(A, blockIdx.x);
  const volatile SharedPiece& p = walk->p;

  if (warp == kProducer) {
    // ---- loads: K and V of each chunk, lane 2b + half for block b
    int n = 0, nk = 0, nv = 0;  // chunks, K and V loads issued
    bool ok = true;
    for (; ok && walk->more && !A.hold; S.pieces[warp].next(A, blockIdx.x)) {
      const int c0 = p.c0, c1 = p.c1, blocks = p.blocks, h = p.h;
      const int32_t* row = A.tables + static_cast<long long>(A.members[p.member0]) * A.max_blocks;
      auto fetch = [&](int c) {  // a chunk's block id
        const int b = c * kChunkBlocks + (lane >> 1);
        return lane < 2 * kChunkBlocks && c < c1 && b < blocks ? row[b] : -2;
      };
      int blk = fetch(c0);
      for (int c = c0; c < c1; ++c, ++n) {
        const int s = n % kStages;
        const uint32_t use = static_cast<uint32_t>(n / kStages);
        const int ahead = fetch(c + 1);
        const bool valid = blk >= 0 && blk < A.num_blocks;
        if (!valid && blk != -2 && !(lane & 1)) record_error(A.err, PA_ERR_DEVICE_CHECK, static_cast<long long>(blk));
        const uint32_t both = __ballot_sync(0xffffffffu, valid);
        uint32_t mask = 0;
#pragma unroll
        for (int b = 0; b < kChunkBlocks; ++b) mask |= ((both >> (2 * b)) & 1u) << b;
        const int y = static_cast<int>((static_cast<long long>(blk) * A.Hkv + h) * kBlock);
        const uint32_t at = (lane & 1) * kHalf + (lane >> 1) * (kBlock * 128);
        const uint32_t bytes = __popc(mask) * kTileBytes;
        // (mask[n % 4] was last read for chunk n - 4, whose scores and values
        // came before the scores of chunk n - 2, which free this K stage)
        if (use > 0 && !__all_sync(0xffffffffu, wait(S.kfree[s], (use - 1) & 1, 20))) {
          ok = false;
          break;
        }
        auto load = [&](unsigned long long& full, uint8_t* tile, int kv) {
          if (lane == 0) {
            if (bytes)
              mbar_arrive_expect_tx(smem_addr(&full), bytes);
            else
              mbar_arrive(smem_addr(&full));
          }
          __syncwarp();
          if (valid) tma_load_half(smem_addr(tile) + at, &A.tmap, y, lane & 1, kv, smem_addr(&full));
        };
        if (lane == 0) S.mask[n % kMasks] = mask;
        load(S.kfull[s], S.k[s], 0);
        ++nk;
        if (use > 0 && !__all_sync(0xffffffffu, wait(S.vfree[s], (use - 1) & 1, 21))) {
          ok = false;
          break;
        }
        load(S.vfull[s], S.v[s], 1);
        ++nv;
        blk = ahead;
      }
    }
    if (lane == 0) {
      S.begun[0] = nk;
      S.begun[1] = nv;
    }
  } else if (warp == kMma) {
    // ---- products.  Step t of a piece serves warpgroup t & 1; S of step
    // t + 2 is issued behind P V of step t, whose P it overwrites (the MMAs of
    // one thread run in order).
    // The whole warp runs the loop, so that its values stay uniform; one
    // elected lane issues.
    constexpr uint32_t kIdS = mma_desc(kBf16, false), kIdO = mma_desc(kBf16, true);
    const bool leader = elect_one();
    const uint32_t q_lo = desc_low(smem_addr(S.q[0]), 16), k_lo = desc_low(smem_addr(S.k[0]), 16),
                   v_lo = desc_low(smem_addr(S.v[0]), kHalf);
    int n0 = 0;         // chunks of earlier pieces
    int piece_no = 0;
    uint32_t p_phase = 0;  // bit w
    bool ok = true;
    auto all = [&](bool x) { return __all_sync(0xffffffffu, x); };
    for (; ok && walk->more; S.pieces[warp].next(A, blockIdx.x)) {
      const int nc = p.c1 - p.c0;
      const bool both = p.both;
      const int steps = both ? 2 * nc : nc;
      ok = all(wait(S.qfull, piece_no & 1, 22));
      ++piece_no;
      uint32_t begun = 0;  // bit w: O of w holds something
      auto scores = [&](int t) {
        const int w = t & 1, n = n0 + (both ? t >> 1 : t), s = n % kStages;
        if (!both || w == 0) ok = ok && all(wait(S.kfull[s], (n / kStages) & 1, 23));
        if (!ok) return;
        tc_fence_after();
        const uint32_t a = q_lo + (both ? w * (kTile >> 4) : 0), b = k_lo + s * (kTile >> 4), d = tmem + w * 128;
        if (leader) {
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            const uint32_t off = ((ks >> 2) * kHalf + (ks & 3) * 32) >> 4;
            mma_ss(d, a + off, b + off, kIdS, ks > 0);
          }
          mma_commit(smem_addr(&S.sfull[w]));
          if (!both || w == 1) mma_commit(smem_addr(&S.kfree[s]));
        }
        __syncwarp();
      };
      if (ok) scores(0);
      if (ok && steps > 1) scores(1);
      for (int t = 0; ok && t < steps; ++t) {
        const int w = t & 1, n = n0 + (both ? t >> 1 : t), s = n % kStages;
        const uint32_t phase = (p_phase >> w) & 1;
        p_phase ^= 1u << w;
        // (V first: it came long ago, and what follows P's arrival is on the
        // way of the next products)
        if (!both || w == 0) ok = wait(S.vfull[s], (n / kStages) & 1, 25);
        const uint32_t mask = *reinterpret_cast<volatile uint32_t*>(&S.mask[n % kMasks]);
        ok = all(ok && wait(S.pfull[w][0], phase, 24));
        if (!ok) break;
        tc_fence_after();
        const uint32_t b = v_lo + s * (kTile >> 4), d = tmem + 256 + w * 128, pw = tmem + w * 128;
        // 16 tokens an MMA: P's 8 columns (and 8 for the low halves), V's 16
        // rows; halves of the dims kHalf apart
        auto values = [&](auto half) {
          constexpr int kb0 = decltype(half)::value * (kChunkBlocks / 2);
          if (leader) {
            if (mask == 0xffu) {
#pragma unroll
              for (int kb = kb0; kb < kb0 + kChunkBlocks / 2; ++kb) {
                mma_ts(d, pw + kb * 16, b + kb * (kBlock * 128 >> 4), kIdO, kb > 0 ? 1u : (begun >> w) & 1);
                if (kLo) mma_ts(d, pw + kb * 16 + 8, b + kb * (kBlock * 128 >> 4), kIdO, 1);
              }
            } else {
              uint32_t add = (begun >> w) & 1 || (kb0 && (mask & 15));
              for (int kb = kb0; kb < kb0 + kChunkBlocks / 2; ++kb) {
                if (!((mask >> kb) & 1)) continue;
                mma_ts(d, pw + kb * 16, b + kb * (kBlock * 128 >> 4), kIdO, add);
                add = 1;
                if (kLo) mma_ts(d, pw + kb * 16 + 8, b + kb * (kBlock * 128 >> 4), kIdO, 1);
              }
            }
          }
          __syncwarp();
        };
        values(std::integral_constant<int, 0>{});
        ok = all(wait(S.pfull[w][1], phase, 29));
        if (!ok) break;
        tc_fence_after();
        values(std::integral_constant<int, 1>{});
        if (leader) {
          if (!both || w == 1) mma_commit(smem_addr(&S.vfree[s]));
          if (t + 2 >= steps) mma_commit(smem_addr(&S.ofull[w]));
        }
        __syncwarp();
        if (mask) begun |= 1u << w;
        if (t + 2 < steps) scores(t + 2);
      }
      n0 += nc;
    }
  } else {
    // ---- softmax: team w; row r, tokens 64 hh .. 64 hh + 63 of a chunk
    const int w = warp >> 3, hh = (warp >> 2) & 1;
    const int r = (warp & 3) * 32 + lane;
    const int pair = 3 + (warp & 3) + 4 * w;  // barrier of the two warps of these rows
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lane_base + w * 128, t_o = tmem + lane_base + 256 + w * 128 + 64 * hh;
    uint32_t s_phase = 0, o_phase = 0;
    int n0 = 0, piece_no = 0;
    bool ok = true;
    for (; ok && walk->more; S.pieces[warp].next(A, blockIdx.x)) {
      const int nc = p.c1 - p.c0;
      // Q: rows of this team, or half the rows of the common tile, once both
      // teams are done with the piece before (its products with it)
      // (a wait that ran out in one warp is one for the team: its warps meet in
      // the pair barriers below)
      if (piece_no > 0) ok = vote(w + 1, kTeam, __all_sync(0xffffffffu, wait(S.qfree, (piece_no - 1) & 1, 28)));
      ++piece_no;
      if (ok) {
        const int x = threadIdx.x & (kTeam - 1);
        uint8_t* tile = S.q[p.both ? w : 0];
        const int lg = p.both ? 1 : 2;  // log2 of the threads a row
        const int row = (p.both ? 0 : w * 64) + (x >> lg);
        const int per = 16 >> lg, v0 = (x & ((1 << lg) - 1)) * per;
        const int gr = p.row0 + (p.both ? w * kRows : 0) + row;
        const bool have = gr < p.row0 + p.rows;
        const uint4* src = nullptr;
        if (have) {
          const int i = A.members[p.member0 + gr / A.G];
          src = reinterpret_cast<const uint4*>(
              A.q + (static_cast<long long>(i) * A.Hq + p.h * A.G + gr % A.G) * kHeadDim);
        }
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          if (y >= per) break;
          const int c = v0 + y;
          uint4 v = have ? src[c] : make_uint4(0u, 0u, 0u, 0u);
          v.x ^= A.qflip;
          v.y ^= A.qflip;
          v.z ^= A.qflip;
          v.w ^= A.qflip;
          *reinterpret_cast<uint4*>(tile + (c >> 3) * kHalf + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = v;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        mbar_arrive(smem_addr(&S.qfull));
      }

      float m = -INFINITY, l = 0.f;
      const int step = p.both ? 1 : 2;
      const int j0 = p.both ? 0 : w;
      bool any = false;
      for (int j = j0; ok && j < nc; j += step) {
        ok = __all_sync(0xffffffffu, wait(S.sfull[w], s_phase, 26));
        s_phase ^= 1;
        any = true;
        tc_fence_after();
        uint32_t mask = *reinterpret_cast<volatile uint32_t*>(&S.mask[(n0 + j) % kMasks]);
        mask = (mask >> (4 * hh)) & 15;  // this half's blocks
        float mine = -INFINITY;
        if (ok) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t s[32];
            tmem_ld32(t_s + 64 * hh + 32 * x, s);
            tmem_wait_ld();
            // (blocks past the prefix or outside the pool weigh nothing)
            float m0 = -INFINITY, m1 = -INFINITY;
            if ((mask >> (2 * x)) & 1) {
#pragma unroll
              for (int y = 0; y < 16; y += 2)  // (one three-way maximum)
                m0 = fmaxf(fmaxf(m0, __uint_as_float(s[y])), __uint_as_float(s[y + 1]));
            }
            if ((mask >> (2 * x + 1)) & 1) {
#pragma unroll
              for (int y = 16; y < 32; y += 2) m1 = fmaxf(fmaxf(m1, __uint_as_float(s[y])), __uint_as_float(s[y + 1]));
            }
            mine = fmaxf(mine, fmaxf(m0, m1));
          }
          S.part[w][hh][r] = mine;
        }
        // the row's other half; a wait that ran out in one of the two warps ends both
        ok = vote(pair, 64, ok);
        if (!ok) break;
        const float mx = fmaxf(mine, S.part[w][hh ^ 1][r]) * A.qscale;
        const bool move = mx > m + kMoveBy;  // (a row of masked scores: -inf, or NaN at scale 0)
        if (__any_sync(0xffffffffu, move)) {
          const float mn = move ? mx : m;
          const float alpha = mn == m ? 1.f : fast_exp2(m - mn);
          l *= alpha;
          m = mn;
          if (j != j0) {  // O holds earlier chunks: their product is done (S came after it)
#pragma unroll 1
            for (int x = 0; x < 4; ++x) {
              uint32_t o[16];
              tmem_ld16(t_o + 16 * x, o);
              tmem_wait_ld();
#pragma unroll
              for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * alpha);
              tmem_st16(t_o + 16 * x, o);
            }
            // the first half of the value product adds to all 128 columns of
            // O on the first half's arrivals alone: they come when both warps
            // have rescaled (m and the maximum are the pair's, so is the branch)
            tmem_wait_st();
            tc_fence_before();
            pair_sync(pair);
            tc_fence_after();
          }
        }
        const float base = m == -INFINITY ? 0.f : m - kTopWeight<kBf16>;
        const float2 qs2 = make_float2(A.qscale, A.qscale), mb2 = make_float2(-base, -base);
        float2 sum = make_float2(0.f, 0.f);
        // a block of 16 tokens at a time, read again; P over its columns of S:
        // the high halves in the first 8, the low ones in the others
        uint32_t s[2][16];
        tmem_ld16(t_s + 64 * hh, s[0]);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t hi[8], lo[8];
          tmem_wait_ld();
          if (x < 3) tmem_ld16(t_s + 64 * hh + 16 * (x + 1), s[(x + 1) & 1]);
          const bool there = (mask >> x) & 1;
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const uint32_t* v = s[x & 1] + 2 * y;
            float2 e = __ffma2_rn(make_float2(__uint_as_float(v[0]), __uint_as_float(v[1])), qs2, mb2);
            e.x = there ? fast_exp2(e.x) : 0.f;
            e.y = there ? fast_exp2(e.y) : 0.f;
            sum = __fadd2_rn(sum, e);
            hi[y] = pack_hi<kBf16>(e.x, e.y);
            if constexpr (kLo) lo[y] = pack_lo<kBf16>(e.x, e.y);
          }
          tmem_st8(t_s + 64 * hh + 16 * x, hi);
          if constexpr (kLo) tmem_st8(t_s + 64 * hh + 16 * x + 8, lo);
        }
        l += sum.x + sum.y;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(smem_addr(&S.pfull[w][hh]));
      }
      n0 += nc;
      if (ok && any) ok = __all_sync(0xffffffffu, wait(S.ofull[w], o_phase, 27));
      if (any) o_phase ^= 1;
      // a wait that ran out in one warp ends the team, which meets below
      ok = vote(w + 1, kTeam, ok);
      if (!ok) break;
      // ---- the piece's record: 64 dims of the team's rows at a time, by way
      // of its Q tile (whose products are done; the second team's is free when
      // the tile is common), as one bulk copy of whole rows
      float* rec = A.rec + p.rec * kRecFloats;
      const int rows = p.both && w ? p.rows - kRows : (p.rows < kRows ? p.rows : kRows);
      if (hh) S.part[w][1][r] = l;
      uint8_t* tile = S.q[w];
      float4* to = reinterpret_cast<float4*>(tile) + r * 16;
      tc_fence_after();
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        if (any && hh == half) {
#pragma unroll 1
          for (int x = 0; x < 2; ++x) {
            uint32_t o[32];
            tmem_ld32(t_o + 32 * x, o);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 8; ++c)
              to[(8 * x + c) ^ (r & 15)] = make_float4(__uint_as_float(o[4 * c]), __uint_as_float(o[4 * c + 1]),
                                                       __uint_as_float(o[4 * c + 2]), __uint_as_float(o[4 * c + 3]));
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        team_sync(w);
        if (any && hh == 0 && r == 0) {
          asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                           rec + half * (kItemRows * 64) + w * (kRows * 64)),
                       "r"(smem_addr(tile)), "r"(rows * 256)
                       : "memory");
          asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 0;" ::: "memory");
        }
        team_sync(w);  // the copy has read the tile
      }
      tc_fence_before();
      if (hh == 0 && r < rows) {
        rec[kItemRows * kHeadDim + w * kRows + r] = m - kTopWeight<kBf16>;
        rec[kItemRows * kHeadDim + kItemRows + w * kRows + r] = l + S.part[w][1][r];
      }
      mbar_arrive(smem_addr(&S.qfree));
    }
    if (hh == 0 && r == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  __syncthreads();
  tc_fence_after();
  if (*abort_flag) {  // a wait ran out, in whichever warp: what is in flight here ends before the memory goes
    auto drained = [&](unsigned long long& bar, uint32_t parity) {
      const long long t0 = global_ns();
      while (!mbar_try_wait(smem_addr(&bar), parity) && global_ns() - t0 < kDrainNs) {
      }
    };
    if (warp == kProducer && lane == 0) {
      for (int v = 0; v < 2; ++v) {
        const int issued = S.begun[v];
        for (int k = issued > kStages ? issued - kStages : 0; k < issued; ++k)
          drained(v ? S.vfull[k % kStages] : S.kfull[k % kStages], (k / kStages) & 1);
      }
    }
    if (warp == kMma) {
      if (elect_one()) {  // (the lane that issued the products)
        mma_commit(smem_addr(&S.drain));
        drained(S.drain, 0);
      }
      __syncwarp();
    }
    __syncthreads();
  }
  if (warp == kMma) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// Workspace pieces, each 256-byte aligned.
struct SharedLayout {
  size_t plan, owner, bad, place, group_of, tiles, lens_s, offs_s, o_s, lse_s, dec, rec, total;
  size_t dec_bytes;
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
  const long long n_rec = items * p->n_kv_heads + sm_count(p->device);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) / 256 * 256;
    return at;
  };
  L->plan = take(sizeof(GroupPlan) * (static_cast<size_t>(n_groups) + 1));
  L->owner = take(4 * static_cast<size_t>(B));
  L->bad = take(4 * static_cast<size_t>(n_groups));
  L->place = take(4 * static_cast<size_t>(B));
  L->group_of = take(4 * static_cast<size_t>(B));
  L->tiles = take(8 * kPlanCluster);
  L->lens_s = take(4 * static_cast<size_t>(B));
  L->offs_s = take(4 * static_cast<size_t>(B));
  L->o_s = take(static_cast<size_t>(B) * Hq * kHeadDim * 4);
  L->lse_s = take(static_cast<size_t>(B) * Hq * 4);
  L->dec = take(L->dec_bytes);
  L->rec = take(static_cast<size_t>(n_rec) * kRecFloats * 4);
  L->total = off;
  return true;
}

static size_t prefix_smem_bytes() { return sizeof(PrefixSmem) + 1024; }

template <bool kBf16, bool kLo>
static int launch_prefix(const SharedArgs& A, int device, cudaStream_t st) {
  const size_t bytes = prefix_smem_bytes();
  static std::atomic<long long> ready{0};  // devices (below 64) whose attribute is set
  const long long bit = device < 64 ? 1ll << device : 0;
  if (!(ready.load() & bit)) {
    if (cudaFuncSetAttribute(shared_prefix_kernel<kBf16, kLo>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(bytes)) != cudaSuccess)
      return PA_ERR_CUDA;
    ready |= bit;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(A.ctas));
  cfg.blockDim = dim3(kPrefixThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, shared_prefix_kernel<kBf16, kLo>, A) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa

using namespace pa;

extern "C" {

size_t pa_decode_shared_workspace_bytes(pa_pool_t p, int num_seqs, int n_q_heads, int max_blocks_per_seq,
                                        int n_groups) {
  SharedLayout L{};
  return shared_layout(p, num_seqs, n_q_heads, max_blocks_per_seq, n_groups, &L) ? L.total : 0;
}

}  // extern "C"

// hold_ns: 0, or (self-test) the limit of the product's waits, for loads that do not come.
static int decode_shared(pa_pool_t p, const void* q, const int32_t* block_tables, int max_blocks_per_seq,
                         const int32_t* seq_lens, int num_seqs, int n_q_heads, float scale, const int32_t* group_start,
                         const int32_t* members, int n_members, const int32_t* prefix_blocks, int n_groups, void* out,
                         int out_dtype, void* workspace, size_t workspace_bytes, void* stream, long long hold_ns) {
  if (!p || !q || !block_tables || !seq_lens || !out || num_seqs <= 0 || n_groups < 0 || n_members < 0 ||
      (n_groups > 0 && (!group_start || !members || !prefix_blocks)))
    return PA_ERR_INVALID;
  if (!std::isfinite(scale)) return PA_ERR_INVALID;
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
  A.plan = reinterpret_cast<GroupPlan*>(ws + L.plan);
  A.owner = reinterpret_cast<int32_t*>(ws + L.owner);
  A.tiles = reinterpret_cast<long long*>(ws + L.tiles);
  A.bad = reinterpret_cast<int32_t*>(ws + L.bad);
  A.place = reinterpret_cast<int32_t*>(ws + L.place);
  A.group_of = reinterpret_cast<int32_t*>(ws + L.group_of);
  A.lens_s = reinterpret_cast<int32_t*>(ws + L.lens_s);
  A.offs_s = reinterpret_cast<int32_t*>(ws + L.offs_s);
  A.rec = reinterpret_cast<float*>(ws + L.rec);
  A.num_blocks = p->num_blocks;
  A.ctas = sm_count(p->device);
  A.err = p->err;
  A.wait_limit_ns = hold_ns ? hold_ns : wait_limit_ns();
  A.hold = hold_ns != 0;
  cudaStream_t st = as_stream(stream);
  // one CTA while its warps compare at most 16 K table entries (whole calls with
  // it and with the cluster: 4 sequences 19.3 and 21.5 us, 16 of about 170 blocks
  // 53.3 and 55.4, 64 of about 190 blocks 39.8 and 39.7)
  if (num_seqs <= kSmallPlan && n_groups <= kSmallPlan && static_cast<long long>(n_members) * max_blocks_per_seq <= 16384) {
    shared_plan_kernel<1, kSmallThreads><<<1, kSmallThreads, 0, st>>>(A);
  } else {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kPlanCluster);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kPlanCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, shared_plan_kernel<kPlanCluster, kPlanThreads>, A) != cudaSuccess) return PA_ERR_CUDA;
  }
  if (cudaGetLastError() != cudaSuccess) return PA_ERR_CUDA;
  if (n_groups > 0) {
    const bool bf16 = p->dtype == PA_BF16, lo = out_dtype == PA_FP32;
    const int rc = bf16 ? (lo ? launch_prefix<true, true>(A, p->device, st) : launch_prefix<true, false>(A, p->device, st))
                        : (lo ? launch_prefix<false, true>(A, p->device, st) : launch_prefix<false, false>(A, p->device, st));
    if (rc != PA_OK) return rc;
  }
  PrefixRecords X{A.place, A.group_of, A.plan, A.rec, n_groups};
  return decode_own_and_combine(p, q, block_tables, max_blocks_per_seq, A.lens_s, A.offs_s, num_seqs, n_q_heads, scale,
                                reinterpret_cast<float*>(ws + L.o_s), reinterpret_cast<float*>(ws + L.lse_s), out,
                                out_dtype, X, ws + L.dec, L.dec_bytes, stream);
}

extern "C" {

int pa_decode_shared(pa_pool_t p, const void* q, const int32_t* block_tables, int max_blocks_per_seq,
                     const int32_t* seq_lens, int num_seqs, int n_q_heads, float scale, const int32_t* group_start,
                     const int32_t* members, int n_members, const int32_t* prefix_blocks, int n_groups, void* out,
                     int out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  return decode_shared(p, q, block_tables, max_blocks_per_seq, seq_lens, num_seqs, n_q_heads, scale, group_start,
                       members, n_members, prefix_blocks, n_groups, out, out_dtype, workspace, workspace_bytes, stream,
                       0);
}

int pa_selftest_shared_timeout(pa_pool_t p, const void* q, const int32_t* block_tables, int max_blocks_per_seq,
                               const int32_t* seq_lens, int num_seqs, int n_q_heads, float scale,
                               const int32_t* group_start, const int32_t* members, int n_members,
                               const int32_t* prefix_blocks, int n_groups, void* out, int out_dtype, void* workspace,
                               size_t workspace_bytes, long long limit_ns, void* stream) {
  if (limit_ns <= 0 || limit_ns > 1000000000ll) return PA_ERR_INVALID;
  return decode_shared(p, q, block_tables, max_blocks_per_seq, seq_lens, num_seqs, n_q_heads, scale, group_start,
                       members, n_members, prefix_blocks, n_groups, out, out_dtype, workspace, workspace_bytes, stream,
                       limit_ns);
}

}  // extern "C"
