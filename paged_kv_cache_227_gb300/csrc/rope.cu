// Rotary positions with several axes, with the cache write; with norms, the
// RMS norm of each query and key head before them.
//
// A new token n has one position per axis (time, height, width, ...).  The
// first `rot` dims of a head are rot/2 pairs; pair f turns by the angle
//   a = positions[axis(f)][n] * inv_freq[f],
//   (x, y) -> (x cos a - y sin a, y cos a + x sin a),
// where the pair is dims (f, f + rot/2) or, interleaved, (2f, 2f + 1).  Dims
// past rot pass through.  With norms, a query or key row x is first
//   x_d = x_d / sqrt(mean(x^2) + eps) * weight_d
// over its 128 dims.  Query rows go to q_out, key rows to the cache slot
// of the token, value rows to the same slot unturned.
//
// Bound: memory.  Every row is read once and written once (512 B), against
// about 3 flops an element.  The angles are the only other work: 64 a token,
// computed by the lanes of a warp together (two each) and shared by all of
// the warp's rows through shared memory.  Measured: 8,192 tokens of 48 heads
// (201 MB) 32.8 us, 6.1 TB/s, 0.90 of this GPU's copy rate; 64 tokens 2.3 us.
// With norms 35.9 us, 0.83 of the copy rate, and 2.7 us: half of the issue slots go
// to the norms' arithmetic, and its registers leave room for fewer warps.
#include "device_utils.cuh"
#include "rope_rows.cuh"

namespace pa {


template <bool kBf16, int U>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const __grid_constant__ RopeArgs A) {
  __shared__ float2 s_cs[kRopeThreads / 32][kMaxPairs];
  const int wib = threadIdx.x >> 5;
  turn_rows<kBf16, U>(A, static_cast<long long>(blockIdx.x) * (kRopeThreads / 32) + wib, s_cs[wib]);
}

template <bool kBf16, int U>
__global__ void __launch_bounds__(kRopeThreads, 7) norm_append_kernel(const __grid_constant__ RopeArgs A) {
  constexpr int kWarps = kRopeThreads / 32;
  __shared__ Angles s_angles[kWarps];
  __shared__ uint4 s_rows[kWarps][U > 1 ? 64 * U : 1];
  const int wib = threadIdx.x >> 5;
  norm_rows<kBf16, U>(A, blockIdx.x * kWarps + wib, s_angles + wib, smem_addr(s_rows[wib]));
}

template <int U, bool kNorm>
static int launch_rope(RopeArgs& A, bool bf16, cudaStream_t st) {
  A.chunks = (A.rows + 4 * U - 1) / (4 * U);
  const long long grid = (A.n_tok * A.chunks + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  if (grid > (kNorm ? 0x3fffffffll : 0x7fffffffll)) return PA_ERR_UNSUPPORTED;  // (norms count warps in 32 bits)
  const unsigned n = static_cast<unsigned>(grid);
  if constexpr (kNorm)
    bf16 ? norm_append_kernel<true, U><<<n, kRopeThreads, 0, st>>>(A) : norm_append_kernel<false, U><<<n, kRopeThreads, 0, st>>>(A);
  else
    bf16 ? rope_append_kernel<true, U><<<n, kRopeThreads, 0, st>>>(A) : rope_append_kernel<false, U><<<n, kRopeThreads, 0, st>>>(A);
  return cuda_status(cudaGetLastError());
}

int rope_axes(RopeArgs* A, const uint8_t* axis_of_pair, int n_axes, int rot_dim, int n_q_heads) {
  if (rot_dim <= 0 || rot_dim > kHeadDim || rot_dim % 16) return PA_ERR_UNSUPPORTED;
  if (n_axes < 1 || n_axes > PA_MAX_ROPE_AXES || n_q_heads > PA_MAX_ROPE_HEADS) return PA_ERR_UNSUPPORTED;
  if (!axis_of_pair) return PA_ERR_INVALID;
  for (int f = 0; f < rot_dim / 2; ++f) {
    if (axis_of_pair[f] >= n_axes) return PA_ERR_INVALID;
    A->axis[f / 16] |= static_cast<uint32_t>(axis_of_pair[f]) << (2 * (f % 16));
  }
  A->half_vecs = rot_dim / 16;
  return PA_OK;
}

int rope_rows(RopeArgs* A, const void* q, int64_t q_stride, int n_q_heads, const void* k_new, int64_t k_stride,
              const void* v_new, int64_t v_stride, int n_kv_heads, const int32_t* positions, const float* inv_freq,
              const int64_t* slot_mapping, int n_tok, void* q_out, int64_t q_out_stride) {
  if (!q || !k_new || !v_new || !positions || !inv_freq || !slot_mapping || !q_out) return PA_ERR_INVALID;
  // rows are moved as 16-byte vectors; a token's heads are contiguous
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new) |
       reinterpret_cast<uintptr_t>(q_out)) & 15)
    return PA_ERR_INVALID;
  if ((q_stride | k_stride | v_stride | q_out_stride) & 7) return PA_ERR_INVALID;
  const int64_t qw = static_cast<int64_t>(n_q_heads) * kHeadDim, kw = static_cast<int64_t>(n_kv_heads) * kHeadDim;
  if (n_tok > 1 && (q_stride < qw || q_out_stride < qw || k_stride < kw || v_stride < kw)) return PA_ERR_INVALID;
  // in place only row for row
  if (q == q_out && n_tok > 1 && q_stride != q_out_stride) return PA_ERR_INVALID;
  A->q = static_cast<const uint16_t*>(q);
  A->k = static_cast<const uint16_t*>(k_new);
  A->v = static_cast<const uint16_t*>(v_new);
  A->q_out = static_cast<uint16_t*>(q_out);
  A->positions = positions;
  A->inv_freq = inv_freq;
  A->slots = slot_mapping;
  A->q_stride = q_stride;
  A->k_stride = k_stride;
  A->v_stride = v_stride;
  A->q_out_stride = q_out_stride;
  A->n_tok = n_tok;
  A->Hq = n_q_heads;
  A->Hkv = n_kv_heads;
  return PA_OK;
}

// Checks and arguments of both calls; weights may be null.
static int rope_append(pa_pool_t p, const void* q, int64_t q_stride, int n_q_heads, const void* k_new, int64_t k_stride,
                       const void* v_new, int64_t v_stride, const void* q_weight, const void* k_weight, float eps,
                       const int32_t* positions, int n_axes, const uint8_t* axis_of_pair, const float* inv_freq,
                       int rot_dim, int interleaved, const int64_t* slot_mapping, int n_tok, void* q_out,
                       int64_t q_out_stride, void* stream) {
  if (!p || n_tok < 0 || n_q_heads <= 0) return PA_ERR_INVALID;
  RopeArgs A{};
  int status = rope_axes(&A, axis_of_pair, n_axes, rot_dim, n_q_heads);
  if (status != PA_OK || n_tok == 0) return status;
  status = rope_rows(&A, q, q_stride, n_q_heads, k_new, k_stride, v_new, v_stride, p->n_kv_heads, positions, inv_freq,
                     slot_mapping, n_tok, q_out, q_out_stride);
  if (status != PA_OK) return status;
  if (!on_pool_device(p)) return PA_ERR_INVALID;
  A.k_pool = static_cast<uint16_t*>(p->k);
  A.v_pool = static_cast<uint16_t*>(p->v);
  A.q_weight = static_cast<const uint16_t*>(q_weight);
  A.k_weight = static_cast<const uint16_t*>(k_weight);
  A.eps = eps;
  A.num_slots = static_cast<long long>(p->num_blocks) * kBlock;
  A.interleaved = interleaved != 0;
  A.rows = n_q_heads + 2 * p->n_kv_heads;
  A.err = p->err;
  // rows a warp: 4 while that leaves the GPU partly empty, then 12, which share a
  // token's angles.  us with 4 and with 12 rows, captured calls: 48 rows a token
  // (the switch is at 405 tokens) 64 tokens 2.19 and 2.30, 128 2.43 and 2.35, 400
  // 3.55 and 3.17, 512 4.31 and 3.59, 8,192 49.1 and 33.0; 16 rows a token (1,216)
  // 64 tokens 2.23 and 2.40, 400 2.60 and 2.60, 1,024 3.35 and 3.18, 2,048 5.31
  // and 4.00; 120 rows a token (162) 64 tokens 2.83 and 2.67, 128 3.39 and 3.11
  const long long quads = A.n_tok * ((A.rows + 3) / 4);
  const bool few = quads <= 32ll * sm_count(p->device), bf16 = p->dtype == PA_BF16;
  const bool norm = q_weight || k_weight;
  cudaStream_t st = as_stream(stream);
  // with norms: 4 rows a warp, or 16 that wait in shared memory, from the same number of
  // rows on for tokens of many rows, from twice as many for small ones.  us with 4 and with
  // 16, captured calls: 48 rows a token (the switch is at 405 tokens) 200 tokens 3.1 and
  // 3.7, 400 4.6 and 4.0, 1,531 13.1 and 11.0, 6,000 41 and 28; 40 rows (486) 200 3.1 and
  // 3.5, 400 3.7 and 3.8, 800 6.0 and 4.6, 6,000 35 and 24; 28 rows (1,389) 400 3.2 and 3.9,
  // 1,531 7.6 and 5.6; 20 rows (1,945) 800 4.0 and 4.0, 3,000 10.4 and 8.0; 16 rows (2,432)
  // in halves 800 3.4 and 4.3, 1,531 5.1 and 4.6, 3,000 8.5 and 6.0, 6,000 17.8 and 13.8,
  // adjacent pairs 1,531 4.7 and 5.5, 3,000 7.6 and 7.5, 6,000 16.6 and 15.8; 7 rows (4,864)
  // 1,531 3.6 and 4.0, 6,000 8.7 and 7.9
  const bool few_norm = quads <= (A.rows < 32 ? 64ll : 32ll) * sm_count(p->device);
  if (norm) return few_norm ? launch_rope<1, true>(A, bf16, st) : launch_rope<4, true>(A, bf16, st);
  return few ? launch_rope<1, false>(A, bf16, st) : launch_rope<3, false>(A, bf16, st);
}

}  // namespace pa

using namespace pa;

static_assert(PA_MAX_ROPE_AXES <= 4, "an axis is two bits");

extern "C" int pa_rope_append(pa_pool_t p, const void* q, int64_t q_stride, int n_q_heads, const void* k_new,
                              int64_t k_stride, const void* v_new, int64_t v_stride, const int32_t* positions,
                              int n_axes, const uint8_t* axis_of_pair, const float* inv_freq, int rot_dim,
                              int interleaved, const int64_t* slot_mapping, int n_tok, void* q_out,
                              int64_t q_out_stride, void* stream) {
  return rope_append(p, q, q_stride, n_q_heads, k_new, k_stride, v_new, v_stride, nullptr, nullptr, 0.f, positions,
                     n_axes, axis_of_pair, inv_freq, rot_dim, interleaved, slot_mapping, n_tok, q_out, q_out_stride,
                     stream);
}

extern "C" int pa_norm_rope_append(pa_pool_t p, const void* q, int64_t q_stride, int n_q_heads, const void* k_new,
                                   int64_t k_stride, const void* v_new, int64_t v_stride, const void* q_weight,
                                   const void* k_weight, float eps, const int32_t* positions, int n_axes,
                                   const uint8_t* axis_of_pair, const float* inv_freq, int rot_dim, int interleaved,
                                   const int64_t* slot_mapping, int n_tok, void* q_out, int64_t q_out_stride,
                                   void* stream) {
  if (!norm_args_ok(q_weight, k_weight, eps)) return PA_ERR_INVALID;
  return rope_append(p, q, q_stride, n_q_heads, k_new, k_stride, v_new, v_stride, q_weight, k_weight, eps, positions,
                     n_axes, axis_of_pair, inv_freq, rot_dim, interleaved, slot_mapping, n_tok, q_out, q_out_stride,
                     stream);
}
