// Kernel argument blocks and launchers of the serving operators (internal to the library):
// rotate.cu, decode.cu, evict.cu; validated and launched by fp2_serve.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/fp2.h"

namespace fp2 {

// Status of the decode and eviction calls.  The prefill clears one word with a memset and its kernels
// OR into it; at a few microseconds a call, that memset would be a third of a decode step.  Here
// every CTA keeps its bits in shared memory and stores them to a word of its own when it ends, so
// nothing has to be cleared: scratch word 0 is kStatusMore, word 1 holds kStatusMagic and the number of
// CTAs, and their words start at byte FP2_SCRATCH_STATUS_BYTES.  fp2_get_device_status reads both
// forms, and of a word without kStatusMore no more than that word: it may be a lone one (fp2_rotate's).
constexpr uint32_t kStatusMore = 0x80000000u;    // no FP2_DEV_* bit
constexpr uint32_t kStatusMagic = 0x5E000000u;   // low 24 bits: words that follow
constexpr uint32_t kStatusCount = 0x00FFFFFFu;
constexpr int kStatusFirst = 256 / 4;            // FP2_SCRATCH_STATUS_BYTES in words

// Launch in clusters of `cluster` CTAs, with programmatic stream serialization: a serving step is a chain
// of calls of a few microseconds, and the next one's launch and set-up then run under the end of the last.
template <typename... Args>
cudaError_t launch_chained(void (*kernel)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                           int cluster, const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ------------------------------------------------------------------ rotate

struct RotateArgs {
  const void* q;
  const void* k;
  const void* v;
  int64_t q_stride, k_stride, v_stride;  // elements between tokens
  const int32_t* positions;
  const void* q_norm;  // [d] in the input type, or NULL
  const void* k_norm;
  float norm_eps;
  int Hq, Hkv;         // heads rotated as Q (0: no Q) and as K; Hv heads copied as V
  int Hv;
  int rot, interleaved;
  float rope_scale;
  void* q_out;
  void* k_out;
  void* v_out;
  int64_t q_out_stride, kv_out_stride;
  const int64_t* slots;  // NULL: row t
  int64_t num_slots;
  float q_inv, k_inv, v_inv;  // 1 / descale (E4M3 output)
  int64_t tokens;
  int iters;             // steps of a warp
  uint32_t* status;      // may be NULL
  uint64_t phase[64];    // turns per position of pair i, as a fraction of 2^64
};

cudaError_t launch_rotate(int dtype_in, int dtype_out, int D, const RotateArgs& a, cudaStream_t stream);

// ------------------------------------------------------------------ decode

// Query offsets of the batch, passed by value like the prefill's plan.
struct DecodePlan {
  int32_t num_seqs;
  int32_t q_off[FP2_MAX_SEQS + 1];
};

struct DecodeArgs {
  CUtensorMap tm_k;  // [page or sequence][token][Hkv][d], box {128 B, 1, rows, 1}
  CUtensorMap tm_v;
  CUtensorMap tm_q;           // key mass: [token][Hq][d], box {128 B, G, pass_tokens}
  const void* q;
  int64_t q_stride;
  int pass_tokens;            // key mass: tokens of a pass, kMassRows / G
  const int32_t* kv_len;
  int max_kv_len;
  const int32_t* page_table;  // NULL: token j of sequence r is row j of outer index r
  int page_size, page_shift, max_pages, num_pages;
  int box_rows, box_shift;    // rows of a TMA box: 64, or the page size below that
  const uint64_t* mask;       // NULL: causal among the drafted tokens
  int Hq, Hkv, G, T;
  float scale_log2;           // softmax scale * log2(e) * q_descale * k_descale
  float v_descale;
  int groups;                 // CTAs per KV head
  // tree attention
  void* out;                  // [T, Hq, d] bf16, or f32
  int out_f32;
  int join_warps;             // warps that join one row: 1 or 4
  float* lse;                 // [Hq, T] or NULL
  int4* desc;                 // [groups] {slot of the first piece of a split item or -1, sequence, row tile, pieces}
  float2* part_ml;            // [groups * Hkv * 2][rows] running maximum (log2 units) and sum
  float* part_o;              // [groups * Hkv * 2][part_rows][d]
  int part_rows;              // rows of a partial result
  int max_rows;               // most query rows per (sequence, KV head)
  const void* k_ptr;          // the cache without its maps: decode_f32.cu, and (V) values that the wide kernel's
  const void* v_ptr;          // products leave out
  int64_t kv_stride, kv_stride_outer;
  // key mass
  const float* lse_in;
  const float* mass_in;       // NULL: zero
  float* mass_out;
  int64_t mass_stride;
  const int32_t* mass_len;    // keys of each sequence that mass_in holds, or NULL: all
  float decay;
  uint32_t* scratch;          // status words: see StatusWords
  uint64_t wait_limit_ns;
  int withhold;               // testing: the producer skips the load of this local key tile (-1: none)
  int late_v;                 // testing, checked builds, tree_wide.cu: this V tile is loaded after the two behind it (-1: none)
};

// Tree attention kernels: up to kFewRows query rows per (sequence, KV head) decode.cu, above that
// tree_wide.cu; then the join of the items that several groups share (a.groups > 1).
constexpr int kFewRows = 16;
cudaError_t launch_tree_few(int dtype, int D, const DecodeArgs& a, const DecodePlan& P, cudaStream_t stream);
cudaError_t launch_tree_wide(int dtype, int D, const DecodeArgs& a, const DecodePlan& P, cudaStream_t stream);
cudaError_t launch_tree_f32(const DecodeArgs& a, const DecodePlan& P, cudaStream_t stream);
cudaError_t launch_mass_f32(const DecodeArgs& a, const DecodePlan& P, cudaStream_t stream);
cudaError_t launch_tree_join(int D, int max_rows, const DecodeArgs& a, const DecodePlan& P, cudaStream_t stream);
cudaError_t launch_key_mass(int dtype, int D, const DecodeArgs& a, const DecodePlan& P, cudaStream_t stream);
constexpr int kFewTile = 64;     // keys of a tile: decode.cu
constexpr int kWideTile = 64;    // tree_wide.cu, which also counts 128 rows as a row tile
constexpr int kMassTile = 128;   // key_mass.cu: keys of a tile
constexpr int kMassRows = 128;   //   and query rows of a pass over them

// ------------------------------------------------------------------ evict

struct CacheView {
  char* k;
  char* v;
  int64_t stride_tok, stride_outer;  // bytes between tokens, and between pages or sequences
  const int32_t* page_table;         // NULL: outer index r holds sequence r
  int rows, max_pages, num_outer;    // tokens per page (or sequence), pages
};

struct EvictArgs {
  CacheView src, dst;
  const int32_t* kv_len;
  int max_kv_len;
  int num_seqs, Hkv, row_bytes;  // bytes of one (token, head) row
  const float* mass;
  int64_t mass_stride;
  int budget, sink, window;
  float* mass_out;               // [num_seqs, Hkv, budget]
  int32_t* kept;                 // [num_seqs, Hkv, budget]
  int32_t* kv_len_out;
  uint32_t* scratch;             // status words: see StatusWords
};

// CTAs that share one (sequence, KV head): a cluster.
int evict_cluster(const EvictArgs& a);
cudaError_t launch_evict(const EvictArgs& a, int cluster, cudaStream_t stream);

}  // namespace fp2
