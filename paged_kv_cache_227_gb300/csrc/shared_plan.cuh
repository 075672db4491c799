// What the kernels of the shared-prefix decode have in common: the plan of a
// group, the cut of the prefix work into CTAs, and the layout of the records.
#pragma once

#include <cstddef>

#include "pa_internal.h"

namespace pa {

constexpr int kRows = 128;                 // rows of a warpgroup
constexpr int kItemRows = 2 * kRows;       // rows of an item
// Record of a piece: o [2 halves of 64 dims][256 rows][64], m [256], l [256]
// (fp32; m in log2 units).  A row's 16 vectors of 4 dims are stored in the order
// c ^ (row & 15), which lets the writer's threads, a row each, go through
// shared memory without bank conflicts.
constexpr int kRecFloats = kItemRows * kHeadDim + 2 * kItemRows;

// Plan of one group; entry [n_groups] holds the totals (unit0, item0, and in
// `rows` the CTAs of the prefix product).
struct GroupPlan {
  long long unit0;  // units before this group
  int item0;        // items before this group
  int rows;         // S * G, 0 for a group that takes no part
  int chunks;       // ceil(P / 8)
  int blocks;       // P
  int member0;      // its first entry in members
};
static_assert(sizeof(GroupPlan) == 32 && offsetof(GroupPlan, item0) == 8 && offsetof(GroupPlan, chunks) == 16,
              "load_plan reads a plan as two 16-byte vectors");

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

// Chunks of one CTA's range.
__device__ __forceinline__ long long units_per_cta(long long units, int ctas) {
  return ctas > 0 ? (units + ctas - 1) / ctas : 1;
}

// Where the combination finds a sequence's prefix records.
struct PrefixRecords {
  const int32_t* place;     // [B]: entry in members, or -1
  const int32_t* group_of;  // [B]
  const GroupPlan* plan;    // [n_groups + 1]
  const float* rec;
  int n_groups;
};

// The records of one query row: `count` of them (half-records of an item of
// at most 128 rows count each).
struct RowRecords {
  const float* rec0 = nullptr;
  int count = 0, sub = 1, row = 0;
  __device__ void find(const PrefixRecords& X, int entry, int group, int h, int g, int G, int Hkv,
                       const GroupPlan& total) {
    const GroupPlan p = load_plan(&X.plan[group]);
    const long long per = units_per_cta(total.unit0, total.rows);
    const int r = (entry - p.member0) * G + g;
    const int item = r / kItemRows;
    row = r - item * kItemRows;
    sub = p.rows - item * kItemRows > kRows ? 1 : 2;
    const long long seg = static_cast<long long>(item) * Hkv + h;
    const long long u0 = p.unit0 + seg * p.chunks;
    const long long c0 = u0 / per, c1 = (u0 + p.chunks - 1) / per;
    count = static_cast<int>(c1 - c0 + 1) * sub;
    // segment number + CTA number grows with every piece: one record each
    rec0 = X.rec + (static_cast<long long>(p.item0) * Hkv + seg + c0) * kRecFloats;
  }
  __device__ const float* rec(int x) const { return rec0 + static_cast<long long>(sub == 2 ? x >> 1 : x) * kRecFloats; }
  __device__ int row_of(int x) const { return sub == 2 ? (x & 1) * kRows + row : row; }
  __device__ const float* m(int x) const { return rec(x) + kItemRows * kHeadDim + row_of(x); }  // l follows at + kItemRows
  // dims 4 c .. 4 c + 3
  __device__ const float4* o(int x, int c) const {
    const int r = row_of(x);
    return reinterpret_cast<const float4*>(rec(x)) + ((c >> 4) * kItemRows + r) * 16 + ((c & 15) ^ (r & 15));
  }
};

}  // namespace pa
