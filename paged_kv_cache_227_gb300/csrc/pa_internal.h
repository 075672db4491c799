// Internal declarations shared by the library's translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pa.h"

// One pool: K and V arrays [num_blocks][n_kv_heads][16][128] plus a device
// error word.  Fixed-size physical blocks as in "Serving" 23.4.  K and V sit
// in one allocation (V right after K) so that one TMA tensor map covers both:
// it views the pair as a 4-D tensor {64 elements, token rows, 2 row halves,
// K|V} and loads a whole (block, head) tile of K and of V - 16 rows x 128
// elements each - as one box, with the 128-byte swizzle.
struct pa_pool {
  CUtensorMap tmap_kv;  // CUtensorMap carries its own 64-byte alignment
  int num_blocks;
  int n_kv_heads;
  int dtype;          // PA_FP16 | PA_BF16
  int device;
  void* k;            // device
  void* v;            // device
  size_t bytes;       // bytes of one of k / v
  long long* err;     // device: [0] = status code, [1] = detail
  CUtensorMap tmap_half;  // the same view, loaded half a row at a time: boxes of 16 rows x 64 elements
};

// One 8-bit pool: codes [num_blocks][n_kv_heads][K|V][16][128], so that a
// (block, head)'s K and V, which a decode reads together, are 4 KiB on end, and
// exponent bytes [num_blocks][n_kv_heads][K|V].  claims [num_blocks][groups of
// tiles] name the row whose run wrote them last, so that two runs of one call in one
// block show (the cache write).
struct pa_pool8 {
  CUtensorMap tmap;   // a (block, head)'s 32 rows of codes as one box, 128-byte swizzle
  int num_blocks;
  int n_kv_heads;
  int dtype;          // PA_E4M3 | PA_INT8
  int device;
  uint8_t* codes;     // device
  uint8_t* exps;      // device
  uint32_t* claims;   // device
  long long* err;     // device: [0] = status code, [1] = detail
};

namespace pa {

constexpr int kBlock = PA_BLOCK_SIZE;     // tokens per block
constexpr int kHeadDim = PA_HEAD_DIM;     // elements per K/V row
constexpr int kRowBytes = kHeadDim * 2;   // one 16-bit row: 256 B
constexpr int kTileBytes = kBlock * kRowBytes;  // one (block, head) tile: 4 KiB
// Widest table of the operators that walk its positions in steps of up to 2^19
// with 32-bit ints: a step past the end stays below 2^31.
constexpr int kMaxWalkedBlocks = PA_MAX_WALKED_BLOCKS;

inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

// Maps a CUDA error to a status (and clears sticky-free launch errors).
inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? PA_OK : PA_ERR_CUDA; }

// Records the first device-side error: code in err[0] (0 -> code), detail in
// err[1].  Later errors are dropped.
__device__ inline void record_error(long long* err, long long code, long long detail) {
  if (atomicCAS(reinterpret_cast<unsigned long long*>(err), 0ull,
                static_cast<unsigned long long>(code)) == 0ull) {
    atomicExch(reinterpret_cast<unsigned long long*>(err + 1),
               static_cast<unsigned long long>(detail));
  }
}

// Number of SMs of the current device (cached per device).
int sm_count(int device);

// Entry check of every call that launches kernels: the current device must
// be the pool's (kernels launch on the current device and address the pool's
// memory, so a call from another device is refused before anything is
// launched).  It also clears a pending non-sticky error of an earlier runtime
// call, so that the launch checks that follow report this call's launches.
template <class Pool>
inline bool on_pool_device(const Pool* p) {
  (void)cudaGetLastError();
  int cur = -1;
  return cudaGetDevice(&cur) == cudaSuccess && cur == p->device;
}

// The map of an 8-bit pool: {128 bytes, 32 rows, tiles}, boxes {128, 32, 1}.
bool encode_pool8_map(CUtensorMap* map, void* codes, long long tiles);

// pa_check and pa_check8: synchronises the stream, reads and clears an error word.
int check_error_word(long long* err, void* stream, int64_t* detail);

// Wait limit for bounded in-kernel waits, in nanoseconds.
long long wait_limit_ns();

// The fused step's cache write (one new token per sequence at position
// L_i - 1), launched on `stream`; the decode follows as its programmatic
// dependent.
int launch_append_tail(void* k_pool, void* v_pool, int n_kv_heads, long long num_blocks, long long* err,
                       int device, const void* k_new, const void* v_new, const int32_t* tables,
                       int max_blocks, const int32_t* seq_lens, int B, cudaStream_t stream);

// The second half of pa_decode_shared (decode.cu): the split decode of each
// sequence's lens[i] own tokens, whose table starts at element table_offs[i]
// (both written by a kernel that is complete when the kernel before this call
// in the stream has started all of its CTAs), and the combination with the
// prefix's records, which that kernel may still be writing.
struct PrefixRecords;
int decode_own_and_combine(pa_pool* p, const void* q, const int32_t* tables, int max_blocks, const int32_t* lens,
                           const int32_t* table_offs, int B, int Hq, float scale, float* o_s, float* lse_s, void* out,
                           int out_dtype, const PrefixRecords& X, void* ws, size_t ws_bytes, void* stream);

}  // namespace pa
