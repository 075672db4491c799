// Cache write in 8 bits: new tokens' K and V rows, with the norms and rotary
// positions of pa_norm_rope_append or as they are.
//
// A run is a stretch of consecutive rows of the call whose slots follow each
// other inside one block.  For every kv head, K and V apart, a run's rows get
// one power-of-two scale, the smallest that holds their largest magnitude, and,
// unless the run starts its block, no smaller one than the block has; where
// the block's scale grows, the codes of its other rows move to it.  Of two runs in
// one block one is skipped and reported.
//
// Bound: memory (512 B read and 256 B written a K or V row; 512 B a query row),
// and latency for the tokens of a decode step.  Two warps take 16 consecutive rows
// of one kv head's K or V, in registers, so a run that fills a block is one pass, and
// so are 16 tokens of 16 sequences: the rows' largest magnitudes meet in shared
// memory, and each run's comes from one segmented reduction over the 16.  A CTA
// has 16 rows of four (kv head, K|V), whose angles are computed once.  Query rows
// go as in the 16-bit appends, in the same launch, with the same bits.
//
// Measured: 7,900 tokens of 32 / 8 / 8 heads in 24 chunks (183 MB) 44 us, 0.61 of the
// copy rate (K and V rows as they are, without query rows, 20); one token of 64 sequences
// 5.6 us: three memory latencies (slots, rows and scales, codes) and the reduction
// between them.  int8 codes: 1 us more for the chunks, 0.4 for a token.
#include "codes8.cuh"
#include "device_utils.cuh"
#include "rope_rows.cuh"

namespace pa {

constexpr int kTok8 = 16;                 // rows of a task
constexpr int kThreads8 = 256;
static_assert(kTasks8 == kThreads8 / 64, "(kv head, K|V) of a CTA");
constexpr int kAngleRows = 2 * kTok8 - 1; // a run that starts in the window ends at most 15 rows behind it

struct Append8Args {
  RopeArgs R;          // rows = query rows; k_pool and v_pool unused
  uint8_t* codes;
  uint8_t* exps;
  uint32_t* claims;
  int groups;          // CTAs that share a window's K and V rows
  unsigned kv_ctas;
};

// The larger magnitude, NaN if one is.
__device__ __forceinline__ float max_abs(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(fabsf(b)));
  return d;
}

// Largest k <= r whose row starts a run (bit k of cont clear).
__device__ __forceinline__ int leader_of(uint32_t cont, int r) { return 31 - __clz(~cont & ((2u << r) - 1)); }

// Two runs of a call in one block would each move the block's rows to a scale of its
// own.  So the run that starts in row r leaves r + 1 in the claim of the block and the
// CTA's four tiles, and of two the later one to come finds the other's there.  Claims
// are not cleared: what an earlier call left counts only where the row that it names has,
// in this call, a slot of the same block and is none of the run's own.  One warp asks for all
// four, before its rows are loaded (64 tokens 5.2 -> 5.4 us, 7,900 42.0 -> 42.4; behind
// the loads 5.6 and 42.7; a claim a tile 5.5 and 43.6).
__device__ __forceinline__ bool another_run(const RopeArgs& R, uint32_t claim, uint32_t row, int behind, int slot) {
  const uint32_t r = claim - 1;
  if (r >= static_cast<uint32_t>(R.n_tok) || r - row <= static_cast<uint32_t>(behind)) return false;
  return R.slots[r] >> 4 == slot >> 4;
}

// kTogether: rows of a lane whose norms are made side by side, 2 where latency counts and
// registers are free, 1 where warps are many (us with 1 and 2: 64 tokens 5.75 and 5.43,
// 7,900 tokens 44.6 and 45.4).
template <bool kBf16, bool kE4M3, bool kNorm, int kTogether>
__device__ __forceinline__ void write_window(const Append8Args& A, Angles* s_angles) {
  __shared__ uint32_t s_top[2][kTasks8][kTok8], s_clash[2];
  const RopeArgs& R = A.R;
  const int lane = threadIdx.x & 31, mine8 = threadIdx.x >> 6, half = threadIdx.x >> 5 & 1;
  const int group = blockIdx.x % A.groups;
  const uint32_t base = blockIdx.x / A.groups * kTok8;
  const int task = group * kTasks8 + mine8;  // K of each head, then V of each head
  const bool active = task < 2 * R.Hkv, is_v = task >= R.Hkv;
  const int h = is_v ? task - R.Hkv : task;
  const int j = lane & 7, sub = lane >> 3;
  const bool turn = !is_v && j < R.half_vecs;
  // (V rows, and dims behind the turned ones: vectors 2j and 2j + 1)
  const bool halves = turn && !R.interleaved;
  const int v0 = halves ? j : 2 * j, v1 = halves ? j + R.half_vecs : 2 * j + 1;

  // slots of rows base - 1 .. base + 30, one a lane (a pool has fewer than 2^31)
  const uint32_t row = base - 1 + lane, n_tok = static_cast<uint32_t>(R.n_tok);
  const long long named = row < n_tok ? R.slots[row] : -1;
  const bool good = named >= 0 && named < R.num_slots;
  if (named >= R.num_slots && lane >= 1 && lane <= kTok8 && task == 0 && half == 0)
    record_error(R.err, PA_ERR_DEVICE_CHECK, named);
  const int slot = good ? static_cast<int>(named) : -1;
  const int before = __shfl_up_sync(0xffffffffu, slot, 1);
  // bit i: row base + i is written; it goes on with the run of the row before it
  const uint32_t goodm = __ballot_sync(0xffffffffu, good) >> 1;
  const uint32_t contm =
      __ballot_sync(0xffffffffu, lane > 0 && good && before >= 0 && slot == before + 1 && (slot & (kBlock - 1)) != 0) >> 1;
  uint32_t todo = goodm & ~contm & 0xffffu;  // first rows of the runs that start in the window

  const uint16_t* from = is_v ? R.v : R.k;
  const long long stride = is_v ? R.v_stride : R.k_stride;
  const uint16_t* weight = !kNorm || is_v || !active ? nullptr : R.k_weight;
  bool angles = R.half_vecs && group * kTasks8 < R.Hkv;  // still to be computed
  const bool claims = threadIdx.x < 32;  // (the first task of a CTA is an active one)
  int pass = 0;
  // (every warp of the CTA goes through the same passes)
  while (todo) {
    const int f = __ffs(todo) - 1;
    // rows f .. f + 15 (bit and row numbers from f on); runs that start among
    // them and end behind them wait for the next pass
    const uint32_t cont = (contm >> f) & 0xffffu;
    uint32_t lead = (todo >> f) & 0xffffu;
    if (f + kTok8 < 32 && ((contm >> (f + kTok8)) & 1)) lead &= (1u << leader_of(cont, kTok8 - 1)) - 1;
    todo &= ~((lead | 1u) << f);  // (a run has at most 16 rows: the first one is never cut)
    const uint32_t part = (goodm >> f) & 0xffffu;
    // row f + l in lane l < 16: its tile, its place in the run and the tile's scale
    const int l = lane & 15;
    const int my_slot = __shfl_sync(0xffffffffu, slot, min(f + l + 1, 31));
    const int first = leader_of(cont, l);
    const bool taken = active && ((part >> l) & 1) && ((lead >> first) & 1);
    const int tile = ((my_slot >> 4) * R.Hkv + h) * 2 + is_v;
    const int off = my_slot & (kBlock - 1), off0 = off - (l - first);
    const int was = taken ? A.exps[tile] : 0;
    const uint32_t next = (~cont & 0xffffu) >> 1 >> l;  // bit i: row l + 1 + i starts a run
    const int last = next ? l + __ffs(next) - 1 : kTok8 - 1;
    const bool heads_run = taken && l == first && lane < kTok8;
    const uint32_t claim =
        claims && heads_run ? atomicExch(A.claims + (my_slot >> 4) * A.groups + group, base + f + l + 1) : 0;
    // this lane's rows: 8 half + sub and 4 behind it
    bool mine[2];
    uint4 x[2][2];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int r = 8 * half + 4 * p + sub;
      mine[p] = active && ((part >> r) & 1) && ((lead >> leader_of(cont, r)) & 1);
      x[p][0] = x[p][1] = make_uint4(0, 0, 0, 0);
      if (mine[p]) {
        const uint4* src = reinterpret_cast<const uint4*>(from + static_cast<long long>(base + f + r) * stride + h * kHeadDim);
        x[p][0] = src[v0];
        x[p][1] = src[v1];
      }
    }
    if (angles) {  // of the window's rows and of the run that leaves it, once, with the first rows on their way
      const int end = kTok8 + __ffs(~(contm >> kTok8)) - 1;  // (bit 31 of contm is clear)
      fill_angles<kThreads8>(R, s_angles, base, static_cast<int>(min(static_cast<uint32_t>(end), n_tok - base)));
      __syncthreads();
      angles = false;
    }
    RowPart y[2];
#pragma unroll
    for (int p0 = 0; p0 < 2; p0 += kTogether) {
#pragma unroll
      for (int p = p0; p < p0 + kTogether; ++p) y[p].unpack<kBf16>(x[p][0], x[p][1]);
      if (weight) {
        const uint4* const at = reinterpret_cast<const uint4*>(weight);
        uint4 w0, w1;
        if (kTogether == 2) w0 = __ldg(at + v0), w1 = __ldg(at + v1);  // (early, where registers are free)
        float mean[2];
        bool any_far = false;
#pragma unroll
        for (int p = p0; p < p0 + kTogether; ++p) any_far |= RowPart::far(mean[p] = y[p].mean_square(R.eps));
        if (any_far) {
#pragma unroll
          for (int p = p0; p < p0 + kTogether; ++p) {
            if (!RowPart::far(mean[p])) continue;
            const FarRow there = far_row(y[p], R.eps);
            y[p] = there.y;
            mean[p] = there.mean;
          }
        }
        if (kTogether == 1) w0 = __ldg(at + v0), w1 = __ldg(at + v1);
        RowPart w;
        w.unpack<kBf16>(w0, w1);
#pragma unroll
        for (int p = p0; p < p0 + kTogether; ++p) {
          y[p].times(rsqrtf(mean[p]));
          y[p].times(w);
        }
      }
#pragma unroll
      for (int p = p0; p < p0 + kTogether; ++p) {
        const int r = 8 * half + 4 * p + sub;
        // (a row that is not taken has no angles)
        if (turn && mine[p]) y[p].turn(R.interleaved, s_angles[f + r], j);
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          m = max_abs(max_abs(m, y[p].a[k].x), y[p].a[k].y);
          m = max_abs(max_abs(m, y[p].b[k].x), y[p].b[k].y);
        }
        // magnitudes compare as their bits, infinities and NaN above all others
        uint32_t t = __float_as_uint(m) & 0x7fffffffu;
        t = max(t, __shfl_xor_sync(0xffffffffu, t, 1));
        t = max(t, __shfl_xor_sync(0xffffffffu, t, 2));
        t = max(t, __shfl_xor_sync(0xffffffffu, t, 4));
        if (j == 0) s_top[pass & 1][mine8][r] = mine[p] ? t : 0;
      }
    }
    if (claims) {
      const bool clash = heads_run && another_run(R, claim, base + f + l, last - l, my_slot);
      if (clash) record_error(R.err, PA_ERR_DEVICE_CHECK, my_slot);
      const uint32_t all = __ballot_sync(0xffffffffu, clash);
      if (lane == 0) s_clash[pass & 1] = all;
    }
    __syncthreads();  // (the next pass writes the other half of s_top)
    const uint32_t clashes = s_clash[pass & 1];
    // the run's magnitude to each of its rows
    uint32_t most = s_top[pass & 1][mine8][l];
    ++pass;
#pragma unroll
    for (int d = 1; d < kTok8; d <<= 1) {
      const uint32_t t = __shfl_up_sync(0xffffffffu, most, d, 16);
      if (l - d >= first) most = max(most, t);
    }
    most = __shfl_sync(0xffffffffu, most, last, 16);
    int e = exponent_for<kE4M3>(most);
    if (off0 > 0 && was > e) e = was;

#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int r = 8 * half + 4 * p + sub;
      const int er = __shfl_sync(0xffffffffu, e, r);
      const int tr = __shfl_sync(0xffffffffu, tile, r);
      const int at = __shfl_sync(0xffffffffu, off, r);
      if (!mine[p] || (clashes >> leader_of(cont, r) & 1)) continue;
      y[p].times(inverse_scale(er));
      uint8_t* dst = A.codes + static_cast<long long>(tr) * kTile8 + at * kRow8;
      const float2 *a = y[p].a, *b = y[p].b;
      const uint2 c0 = make_uint2(pack_codes<kE4M3>(a[0].x, a[0].y, a[1].x, a[1].y),
                                  pack_codes<kE4M3>(a[2].x, a[2].y, a[3].x, a[3].y));
      const uint2 c1 = make_uint2(pack_codes<kE4M3>(b[0].x, b[0].y, b[1].x, b[1].y),
                                  pack_codes<kE4M3>(b[2].x, b[2].y, b[3].x, b[3].y));
      if (halves) {
        *reinterpret_cast<uint2*>(dst + 8 * v0) = c0;
        *reinterpret_cast<uint2*>(dst + 8 * v1) = c1;
      } else {
        *reinterpret_cast<uint4*>(dst + 8 * v0) = make_uint4(c0.x, c0.y, c1.x, c1.y);
      }
    }
    const bool writes = heads_run && !(clashes >> l & 1);
    if (writes && half == 0) A.exps[tile] = static_cast<uint8_t>(e);

    // blocks whose scale grew: the codes of their other rows, half of the tile a warp
    uint32_t grown = __ballot_sync(0xffffffffu, writes && off0 > 0 && e > was && e != kNanExponent);
    while (grown) {
      const int r = __ffs(grown) - 1;
      grown &= grown - 1;
      const int tr = __shfl_sync(0xffffffffu, tile, r);
      const int o0 = __shfl_sync(0xffffffffu, off0, r), o1 = o0 + __shfl_sync(0xffffffffu, last, r) - r;
      const int d = __shfl_sync(0xffffffffu, e - was, r);
      const float ratio = d > 126 ? 0.f : __int_as_float((127 - d) << 23);
      uint4* tile_codes = reinterpret_cast<uint4*>(A.codes + static_cast<long long>(tr) * kTile8);
      uint4 c[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {  // vector 32 (2 half + i) + lane: row 4 (2 half + i) + lane / 8
        const int n = 2 * half + i, rw = 4 * n + sub;
        if (rw < o0 || rw > o1) c[i] = tile_codes[32 * n + lane];
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int n = 2 * half + i, rw = 4 * n + sub;
        if (rw < o0 || rw > o1)
          tile_codes[32 * n + lane] =
              make_uint4(shrink_codes<kE4M3>(c[i].x, ratio), shrink_codes<kE4M3>(c[i].y, ratio),
                         shrink_codes<kE4M3>(c[i].z, ratio), shrink_codes<kE4M3>(c[i].w, ratio));
      }
    }
  }
}

// CTAs below kv_ctas: K and V rows; the others: query rows (U row quads a warp).
template <bool kBf16, bool kE4M3, int U, bool kNorm>
__global__ void __launch_bounds__(kThreads8, U > 1 ? 3 : 2) append8_kernel(const __grid_constant__ Append8Args A) {
  constexpr int kWarps = kThreads8 / 32;
  constexpr int kRows = kNorm && U > 1 ? kWarps * 64 * U : 0;  // vectors of query rows that wait
  // angles of a window, or the query rows' and the rows (128: what a row's lanes read
  // together lies in one line; at 16 the chunks take 44.6 us instead of 43.7)
  constexpr int kQueries = kWarps * sizeof(Angles) + 16 * kRows, kKeys = kAngleRows * sizeof(Angles);
  __shared__ __align__(128) uint8_t s_space[kQueries > kKeys ? kQueries : kKeys];
  Angles* const s_angles = reinterpret_cast<Angles*>(s_space);
  if (blockIdx.x < A.kv_ctas) {
    write_window<kBf16, kE4M3, kNorm, U == 1 ? 2 : 1>(A, s_angles);
    return;
  }
  const int wib = threadIdx.x >> 5;
  const unsigned w = (blockIdx.x - A.kv_ctas) * kWarps + wib;
  if (kNorm)
    norm_rows<kBf16, U>(A.R, w, s_angles + wib, smem_addr(s_space) + kWarps * sizeof(Angles) + wib * 1024 * U);
  else
    turn_rows<kBf16, U>(A.R, w, reinterpret_cast<float2*>(s_angles + wib));
}

template <int U, bool kNorm>
static int launch_append8(Append8Args& A, bool bf16, bool e4m3, cudaStream_t st) {
  const RopeArgs& R = A.R;
  A.R.chunks = (R.rows + 4 * U - 1) / (4 * U);
  A.groups = claim_groups(R.Hkv);
  const long long kv = (R.n_tok + kTok8 - 1) / kTok8 * A.groups;
  const long long q = (R.n_tok * A.R.chunks + kThreads8 / 32 - 1) / (kThreads8 / 32);
  if (kv > 0x3fffffffll || q > 0x1fffffffll) return PA_ERR_UNSUPPORTED;  // (warps of query rows are counted in 32 bits)
  A.kv_ctas = static_cast<unsigned>(kv);
  const unsigned n = static_cast<unsigned>(kv + q);
  if (bf16)
    e4m3 ? append8_kernel<true, true, U, kNorm><<<n, kThreads8, 0, st>>>(A)
         : append8_kernel<true, false, U, kNorm><<<n, kThreads8, 0, st>>>(A);
  else
    e4m3 ? append8_kernel<false, true, U, kNorm><<<n, kThreads8, 0, st>>>(A)
         : append8_kernel<false, false, U, kNorm><<<n, kThreads8, 0, st>>>(A);
  return cuda_status(cudaGetLastError());
}

// The pool's part of the arguments, and the launch; R's rows are checked.
static int launch8(pa_pool8_t p, Append8Args& A, bool bf16, void* stream) {
  A.codes = p->codes;
  A.exps = p->exps;
  A.claims = p->claims;
  A.R.num_slots = static_cast<long long>(p->num_blocks) * kBlock;
  A.R.err = p->err;
  A.R.rows = A.R.Hq;
  const bool e4m3 = p->dtype == PA_E4M3;
  cudaStream_t st = as_stream(stream);
  const long long quads = A.R.n_tok * ((A.R.rows + 3) / 4);
  const long long windows = (A.R.n_tok + kTok8 - 1) / kTok8 * claim_groups(A.R.Hkv);
  // few query rows a warp and 2 CTAs an SM, or 12 (with norms 16) and 3: by the row quads of
  // queries, and by the K and V rows' CTAs, which a call has without query rows too.  us
  // with the one and the other, captured calls, norms: 32 / 8 heads (the switch is at 304
  // tokens) 256 tokens 4.3 and 4.4, 480 5.8 and 5.2, 1,920 20.0 and 13.9; 12 / 2 (810) 480
  // tokens 3.9 and 4.1, 960 4.7 and 4.8, 1,920 7.0 and 5.7; 8 / 8 (1,216) 960 5.3 and 5.7,
  // 1,920 9.0 and 8.0; without norms 32 / 8 256 tokens 4.1 and 4.0, 480 5.3 and 4.1; 12 / 2
  // 480 3.6 and 3.6, 1,920 6.5 and 4.6.  K and V rows alone: 8 heads (3,040) 1,920 tokens
  // 5.6 and 5.7, 3,840 9.8 and 9.0, 7,680 22.5 and 18.5; 40 heads (608) 480 5.9 and 6.1,
  // 960 11.8 and 10.3, 7,680 95 and 74
  const long long sms = sm_count(p->device);
  const bool few = quads <= 16 * sms && windows <= 5 * sms;
  if (A.R.q_weight || A.R.k_weight)
    return few ? launch_append8<1, true>(A, bf16, e4m3, st) : launch_append8<4, true>(A, bf16, e4m3, st);
  return few ? launch_append8<1, false>(A, bf16, e4m3, st) : launch_append8<3, false>(A, bf16, e4m3, st);
}

}  // namespace pa

using namespace pa;

extern "C" int pa_norm_rope_append8(pa_pool8_t p, int dtype, const void* q, int64_t q_stride, int n_q_heads,
                                    const void* k_new, int64_t k_stride, const void* v_new, int64_t v_stride,
                                    const void* q_weight, const void* k_weight, float eps, const int32_t* positions,
                                    int n_axes, const uint8_t* axis_of_pair, const float* inv_freq, int rot_dim,
                                    int interleaved, const int64_t* slot_mapping, int n_tok, void* q_out,
                                    int64_t q_out_stride, void* stream) {
  if (!p || n_tok < 0 || n_q_heads <= 0 || (dtype != PA_FP16 && dtype != PA_BF16)) return PA_ERR_INVALID;
  if (!norm_args_ok(q_weight, k_weight, eps)) return PA_ERR_INVALID;
  Append8Args A{};
  int status = rope_axes(&A.R, axis_of_pair, n_axes, rot_dim, n_q_heads);
  if (status != PA_OK || n_tok == 0) return status;
  status = rope_rows(&A.R, q, q_stride, n_q_heads, k_new, k_stride, v_new, v_stride, p->n_kv_heads, positions, inv_freq,
                     slot_mapping, n_tok, q_out, q_out_stride);
  if (status != PA_OK) return status;
  if (!on_pool_device(p)) return PA_ERR_INVALID;
  A.R.q_weight = static_cast<const uint16_t*>(q_weight);
  A.R.k_weight = static_cast<const uint16_t*>(k_weight);
  A.R.eps = eps;
  A.R.interleaved = interleaved != 0;
  return launch8(p, A, dtype == PA_BF16, stream);
}

extern "C" int pa_cache_append8(pa_pool8_t p, int dtype, const void* k_new, const void* v_new,
                                const int64_t* slot_mapping, int n_tok, void* stream) {
  if (!p || n_tok < 0 || (dtype != PA_FP16 && dtype != PA_BF16)) return PA_ERR_INVALID;
  if (n_tok == 0) return PA_OK;
  if (!k_new || !v_new || !slot_mapping) return PA_ERR_INVALID;
  if ((reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new)) & 15) return PA_ERR_INVALID;
  if (!on_pool_device(p)) return PA_ERR_INVALID;
  Append8Args A{};
  A.R.k = static_cast<const uint16_t*>(k_new);
  A.R.v = static_cast<const uint16_t*>(v_new);
  A.R.k_stride = A.R.v_stride = static_cast<long long>(p->n_kv_heads) * kHeadDim;
  A.R.slots = slot_mapping;
  A.R.n_tok = n_tok;
  A.R.Hkv = p->n_kv_heads;
  return launch8(p, A, dtype == PA_BF16, stream);
}
