// Cache write in 8 bits: new tokens' K and V rows, with the norms and rotary
// positions of pa_norm_rope_append or as they are.
//
// A run is a stretch of consecutive rows of the call whose slots follow each
// other inside one block.  For every kv head, K and V apart, a run's rows get
// one power-of-two scale, the smallest that holds their largest magnitude, and,
// unless the run starts its block, no smaller one than the block has; where
// the block's scale grows, the codes of its other rows move to it.
//
// Bound: memory (512 B read and 256 B written a K or V row; 512 B a query row),
// and latency for the tokens of a decode step.  A warp takes 16 consecutive rows
// of one kv head's K or V, in registers as they were loaded (16 bits), so a
// run that fills a block is one pass, and so are 16 tokens of 16 sequences:
// the runs' largest magnitudes come from one segmented reduction over the rows.
// K rows are normed and turned twice, for the magnitudes and for the codes:
// kept in 32 bits between, they would take 64 registers a thread.  The tokens'
// angles are computed once for a CTA's four heads.  Query rows go by
// (token, chunk of rows) as in the 16-bit append, in the same launch.
#include "codes8.cuh"
#include "rope_rows.cuh"

namespace pa {

constexpr int kTok8 = 16;           // rows of a warp
constexpr int kTasks8 = kRopeThreads / 32;  // (kv head, K|V) of a CTA
constexpr int kAngleRows = 2 * kTok8 - 1;   // a run that starts in the window ends at most 15 rows behind it

struct Append8Args {
  RopeArgs R;          // rows = query rows; k_pool and v_pool unused
  uint8_t* codes;
  uint8_t* exps;
  int groups;          // CTAs that share a window's K and V rows
  unsigned kv_ctas;
};

// Largest k <= r whose row starts a run (bit k of cont clear).
__device__ __forceinline__ int leader_of(uint32_t cont, int r) { return 31 - __clz(~cont & ((2u << r) - 1)); }

template <bool kBf16, bool kE4M3>
__device__ __forceinline__ void write_window(const Append8Args& A, float2 (*s_cs)[kMaxPairs]) {
  const RopeArgs& R = A.R;
  const int lane = threadIdx.x & 31;
  const int group = blockIdx.x % A.groups;
  const long long base = static_cast<long long>(blockIdx.x / A.groups) * kTok8;
  const int task = group * kTasks8 + (threadIdx.x >> 5);  // K of each head, then V of each head
  const bool is_v = task >= R.Hkv;
  const int h = is_v ? task - R.Hkv : task;
  const int j = lane & 7, sub = lane >> 3;
  const bool turn = !is_v && j < R.half_vecs;
  // (V rows, and dims behind the turned ones: vectors 2j and 2j + 1)
  const bool halves = turn && !R.interleaved;
  const int v0 = halves ? j : 2 * j, v1 = halves ? j + R.half_vecs : 2 * j + 1;

  // slots of rows base - 1 .. base + 30, one a lane
  const long long row = base - 1 + lane;
  const long long slot = row >= 0 && row < R.n_tok ? R.slots[row] : -1;
  const bool good = slot >= 0 && slot < R.num_slots;
  if (slot >= R.num_slots && lane >= 1 && lane <= kTok8 && task == 0) record_error(R.err, PA_ERR_DEVICE_CHECK, slot);
  const long long before = __shfl_up_sync(0xffffffffu, slot, 1);
  // bit i: row base + i is written; it goes on with the run of the row before it
  const uint32_t goodm = __ballot_sync(0xffffffffu, good) >> 1;
  const uint32_t contm =
      __ballot_sync(0xffffffffu, lane > 0 && good && before >= 0 && slot == before + 1 && (slot & (kBlock - 1)) != 0) >> 1;
  uint32_t todo = goodm & ~contm & 0xffffu;  // first rows of the runs that start in the window

  // angles of the window's rows and of the run that leaves it
  if (R.half_vecs && group * kTasks8 < R.Hkv) {
    const int end = kTok8 + __ffs(~(contm >> kTok8)) - 1;  // (bit 31 of contm is clear)
    const int pairs = 8 * R.half_vecs;
    for (int x = threadIdx.x; x < end * kMaxPairs; x += kRopeThreads) {
      const int r = x / kMaxPairs, f = x % kMaxPairs;
      if (f < pairs && base + r < R.n_tok) s_cs[r][f] = cos_sin(R, base + r, f);
    }
    __syncthreads();
  }
  if (task >= 2 * R.Hkv) return;

  const uint16_t* from = is_v ? R.v : R.k;
  const long long stride = is_v ? R.v_stride : R.k_stride;
  const uint16_t* weight = is_v ? nullptr : R.k_weight;
  while (todo) {
    const int f = __ffs(todo) - 1;
    // rows f .. f + 15 (bit and row numbers from f on); runs that start among
    // them and end behind them wait for the next pass
    const uint32_t cont = (contm >> f) & 0xffffu;
    uint32_t lead = (todo >> f) & 0xffffu;
    if (f + kTok8 < 32 && ((contm >> (f + kTok8)) & 1)) lead &= (1u << leader_of(cont, kTok8 - 1)) - 1;
    todo &= ~((lead | 1u) << f);  // (a run has at most 16 rows: the first one is never cut)
    const uint32_t part = (goodm >> f) & 0xffffu;
    uint32_t mine = 0;  // rows of the runs taken
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int r = 4 * p + sub;
      if (((part >> r) & 1) && ((lead >> leader_of(cont, r)) & 1)) mine |= 1u << p;
    }

    uint4 x[4][2];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      x[p][0] = x[p][1] = make_uint4(0, 0, 0, 0);
      if (mine >> p & 1) {
        const uint4* src = reinterpret_cast<const uint4*>(from + (base + f + 4 * p + sub) * stride + h * kHeadDim);
        x[p][0] = src[v0];
        x[p][1] = src[v1];
      }
    }
    // row f + l in lane l < 16: its tile, its place in the run and the tile's scale
    const int l = lane & 15;
    const long long my_slot = __shfl_sync(0xffffffffu, slot, min(f + l + 1, 31));
    const int first = leader_of(cont, l);
    const bool taken = ((part >> l) & 1) && ((lead >> first) & 1);
    const long long tile = ((my_slot >> 4) * R.Hkv + h) * 2 + is_v;
    const int off = static_cast<int>(my_slot & (kBlock - 1)), off0 = off - (l - first);
    const int was = taken ? A.exps[tile] : 0;

    float rr[4];
    uint32_t top[4];
    auto values = [&](int p, float a[8], float b[8]) {
      unpack8f<kBf16>(x[p][0], a);
      unpack8f<kBf16>(x[p][1], b);
      if (is_v) return;
      if (weight)
        scale_row<kBf16>(a, b, rr[p], __ldg(reinterpret_cast<const uint4*>(weight) + v0),
                         __ldg(reinterpret_cast<const uint4*>(weight) + v1));
      // (a row that is not taken has no angles)
      if (turn && (mine >> p & 1))
        turn_row(a, b, R.interleaved != 0, [&](int k) { return s_cs[f + 4 * p + sub][8 * j + k]; });
    };
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      float a[8], b[8];
      if (weight) {
        unpack8f<kBf16>(x[p][0], a);
        unpack8f<kBf16>(x[p][1], b);
        rr[p] = inverse_rms(a, b, R.eps);
      }
      values(p, a, b);
      // magnitudes compare as their bits, infinities and NaN above all others
      uint32_t t = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        t = max(t, max(__float_as_uint(a[k]) & 0x7fffffffu, __float_as_uint(b[k]) & 0x7fffffffu));
      t = max(t, __shfl_xor_sync(0xffffffffu, t, 1));
      t = max(t, __shfl_xor_sync(0xffffffffu, t, 2));
      top[p] = max(t, __shfl_xor_sync(0xffffffffu, t, 4));
    }
    // row l's magnitude to lane l, and the run's to each of its rows
    uint32_t most = 0;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const uint32_t t = __shfl_sync(0xffffffffu, top[p], 8 * (l & 3));
      if (l >> 2 == p) most = t;
    }
#pragma unroll
    for (int d = 1; d < kTok8; d <<= 1) {
      const uint32_t t = __shfl_up_sync(0xffffffffu, most, d, 16);
      if (l - d >= first) most = max(most, t);
    }
    const uint32_t next = (~cont & 0xffffu) >> 1 >> l;  // bit i: row l + 1 + i starts a run
    const int last = next ? l + __ffs(next) - 1 : kTok8 - 1;
    most = __shfl_sync(0xffffffffu, most, last, 16);
    int e = exponent_for<kE4M3>(most);
    if (off0 > 0 && was > e) e = was;

#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int r = 4 * p + sub;
      const int er = __shfl_sync(0xffffffffu, e, r);
      const long long tr = __shfl_sync(0xffffffffu, tile, r);
      const int at = __shfl_sync(0xffffffffu, off, r);
      if (!(mine >> p & 1)) continue;
      const float inv = inverse_scale(er);
      float a[8], b[8];
      values(p, a, b);
      uint8_t* dst = A.codes + tr * kTile8 + at * kRow8;
      const uint2 c0 = make_uint2(pack_codes<kE4M3>(a[0] * inv, a[1] * inv, a[2] * inv, a[3] * inv),
                                  pack_codes<kE4M3>(a[4] * inv, a[5] * inv, a[6] * inv, a[7] * inv));
      const uint2 c1 = make_uint2(pack_codes<kE4M3>(b[0] * inv, b[1] * inv, b[2] * inv, b[3] * inv),
                                  pack_codes<kE4M3>(b[4] * inv, b[5] * inv, b[6] * inv, b[7] * inv));
      if (halves) {
        *reinterpret_cast<uint2*>(dst + 8 * v0) = c0;
        *reinterpret_cast<uint2*>(dst + 8 * v1) = c1;
      } else {
        *reinterpret_cast<uint4*>(dst + 8 * v0) = make_uint4(c0.x, c0.y, c1.x, c1.y);
      }
    }
    const bool heads_run = taken && l == first && lane < kTok8;
    if (heads_run) A.exps[tile] = static_cast<uint8_t>(e);

    // blocks whose scale grew: the codes of their other rows
    uint32_t grown = __ballot_sync(0xffffffffu, heads_run && off0 > 0 && e > was && e != kNanExponent);
    while (grown) {
      const int r = __ffs(grown) - 1;
      grown &= grown - 1;
      const long long tr = __shfl_sync(0xffffffffu, tile, r);
      const int o0 = __shfl_sync(0xffffffffu, off0, r), o1 = o0 + __shfl_sync(0xffffffffu, last, r) - r;
      const int d = __shfl_sync(0xffffffffu, e - was, r);
      const float ratio = d > 126 ? 0.f : __int_as_float((127 - d) << 23);
      uint4* tile_codes = reinterpret_cast<uint4*>(A.codes + tr * kTile8);
      uint4 c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // vector 32 i + lane: row 4 i + lane / 8
        const int rw = 4 * i + sub;
        c[i] = rw < o0 || rw > o1 ? tile_codes[32 * i + lane] : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int rw = 4 * i + sub;
        if (rw < o0 || rw > o1)
          tile_codes[32 * i + lane] =
              make_uint4(shrink_codes<kE4M3>(c[i].x, ratio), shrink_codes<kE4M3>(c[i].y, ratio),
                         shrink_codes<kE4M3>(c[i].z, ratio), shrink_codes<kE4M3>(c[i].w, ratio));
      }
    }
  }
}

// CTAs below kv_ctas: K and V rows; the others: query rows (U row quads a warp).
template <bool kBf16, bool kE4M3, int U, bool kNorm>
__global__ void __launch_bounds__(kRopeThreads) append8_kernel(const __grid_constant__ Append8Args A) {
  __shared__ float2 s_cs[kAngleRows][kMaxPairs];
  if (blockIdx.x < A.kv_ctas) {
    write_window<kBf16, kE4M3>(A, s_cs);
  } else {
    const int wib = threadIdx.x >> 5;
    turn_rows<kBf16, U, kNorm>(A.R, static_cast<long long>(blockIdx.x - A.kv_ctas) * (kRopeThreads / 32) + wib, s_cs[wib]);
  }
}

template <int U, bool kNorm>
static int launch_append8(Append8Args& A, bool bf16, bool e4m3, cudaStream_t st) {
  const RopeArgs& R = A.R;
  A.R.chunks = (R.rows + 4 * U - 1) / (4 * U);
  A.groups = (2 * R.Hkv + kTasks8 - 1) / kTasks8;
  const long long kv = (R.n_tok + kTok8 - 1) / kTok8 * A.groups;
  const long long grid = kv + (R.n_tok * A.R.chunks + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  if (grid > 0x7fffffffll) return PA_ERR_UNSUPPORTED;
  A.kv_ctas = static_cast<unsigned>(kv);
  const unsigned n = static_cast<unsigned>(grid);
  if (bf16)
    e4m3 ? append8_kernel<true, true, U, kNorm><<<n, kRopeThreads, 0, st>>>(A)
         : append8_kernel<true, false, U, kNorm><<<n, kRopeThreads, 0, st>>>(A);
  else
    e4m3 ? append8_kernel<false, true, U, kNorm><<<n, kRopeThreads, 0, st>>>(A)
         : append8_kernel<false, false, U, kNorm><<<n, kRopeThreads, 0, st>>>(A);
  return cuda_status(cudaGetLastError());
}

// The pool's part of the arguments, and the launch; R's rows are checked.
static int launch8(pa_pool8_t p, Append8Args& A, bool bf16, void* stream) {
  A.codes = p->codes;
  A.exps = p->exps;
  A.R.num_slots = static_cast<long long>(p->num_blocks) * kBlock;
  A.R.err = p->err;
  A.R.rows = A.R.Hq;
  const bool e4m3 = p->dtype == PA_E4M3;
  cudaStream_t st = as_stream(stream);
  // (query rows a warp: as in the 16-bit append)
  const long long quads = A.R.n_tok * ((A.R.rows + 3) / 4);
  const bool few = quads <= 32ll * sm_count(p->device);
  if (A.R.q_weight) return few ? launch_append8<1, true>(A, bf16, e4m3, st) : launch_append8<3, true>(A, bf16, e4m3, st);
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
