// Host side of the serving operators declared in include/fp2.h (fp2_rotate, fp2_tree_attend,
// fp2_key_mass, fp2_evict): argument validation, scratch layout, TMA descriptors and launches.
// Allocates no device memory and never synchronises the caller's stream.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstring>

#include "../../include/fp2.h"
#include "fp2_plan.h"
#include "serve_kernels.h"

namespace fp2_internal {
fp2_status set_error(fp2_status s, const char* msg);
void clear_error();
void* tensor_map_encoder();
uint64_t wait_limit_ns();
int withheld_k_tile();
int late_v_tile();
}  // namespace fp2_internal

namespace {

fp2_status fail(fp2_status s, const char* msg) { return fp2_internal::set_error(s, msg); }
fp2_status invalid(const char* msg) { return fail(FP2_ERR_INVALID_ARG, msg); }
fp2_status unsupported(const char* msg) { return fail(FP2_ERR_UNSUPPORTED, msg); }
fp2_status launched(cudaError_t e) { return e == cudaSuccess ? FP2_OK : fail(FP2_ERR_CUDA, cudaGetErrorString(e)); }

#define FP2_TRY(expr)                      \
  do {                                     \
    const fp2_status try_status = (expr);  \
    if (try_status != FP2_OK) return try_status; \
  } while (0)

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }
int elt_bytes(fp2_dtype t) { return t == FP2_F32 ? 4 : (t == FP2_BF16 ? 2 : 1); }
bool positive(float x) { return x >= FLT_MIN && std::isfinite(x); }  // (1 / x is finite)

int num_sms() {
  int dev = 0, n = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n;
}

bool apart(const void* x, size_t x_bytes, const void* y, size_t y_bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
  return a + x_bytes <= b || b + y_bytes <= a;
}

fp2_status check_scratch(const void* scratch, size_t have, size_t need) {
  if (scratch == nullptr) return invalid("scratch is NULL");
  if ((reinterpret_cast<uintptr_t>(scratch) & (kAlign - 1)) != 0) return invalid("scratch must be 256-byte aligned");
  if (have < need) return fail(FP2_ERR_WORKSPACE_TOO_SMALL, "scratch_bytes is below the workspace query's figure");
  return FP2_OK;
}

fp2_status check_stream(fp2_stream_t stream) {
  return stream == FP2_STREAM_NONE ? invalid("the buffers are not on a GPU") : FP2_OK;
}

fp2_status clear_status(void* scratch, cudaStream_t st) {
  return launched(cudaMemsetAsync(scratch, 0, FP2_SCRATCH_STATUS_BYTES, st));
}

// A cache that holds up to max_len tokens of each of num_seqs sequences.
fp2_status check_cache(const fp2_cache& c, int num_seqs, int64_t max_len, bool need_v) {
  if (c.dtype != FP2_F32 && c.dtype != FP2_BF16 && c.dtype != FP2_E4M3) return invalid("unknown cache dtype");
  if (c.num_kv_heads <= 0) return invalid("num_kv_heads must be positive");
  if (c.num_kv_heads > 65536) return unsupported("more than 65536 heads");
  if (c.head_dim != 64 && c.head_dim != 128) return unsupported("head_dim must be 64 or 128");
  if (c.dtype == FP2_F32 && c.head_dim != 64) return unsupported("an F32 cache needs head_dim 64");
  if (c.dtype == FP2_E4M3 && c.head_dim != 128) return unsupported("an E4M3 cache needs head_dim 128");
  const int elt = elt_bytes(c.dtype);
  if (c.k == nullptr || (need_v && c.v == nullptr)) return invalid("cache k/v must not be NULL");
  if (!aligned16(c.k) || !aligned16(c.v)) return invalid("cache k/v must be 16-byte aligned");
  if (c.num_outer <= 0 || c.rows <= 0) return invalid("cache num_outer and rows must be positive");
  if (c.stride_tok < static_cast<int64_t>(c.num_kv_heads) * c.head_dim || c.stride_tok >= (int64_t(1) << 31))
    return invalid("cache stride_tok must be >= heads * head_dim (and below 2^31)");
  if (c.num_outer > 1 && c.stride_outer < c.rows * c.stride_tok)
    return invalid("cache stride_outer must be >= rows * stride_tok");
  if ((c.stride_tok * elt) % 16 != 0 || (c.stride_outer * elt) % 16 != 0 || c.stride_outer < 0)
    return invalid("cache strides must be multiples of 16 bytes");
  if (c.stride_outer >= (int64_t(1) << 37)) return unsupported("cache stride_outer too large");
  if (c.page_table != nullptr) {
    if (c.rows < 16 || (c.rows & (c.rows - 1)) != 0) return unsupported("page rows must be a power of two >= 16");
    if (!aligned4(c.page_table)) return invalid("page_table must be 4-byte aligned");
    if (c.max_pages_per_seq < (max_len + c.rows - 1) / c.rows)
      return invalid("max_pages_per_seq too small for the longest sequence");
  } else {
    if (c.num_outer < num_seqs) return invalid("a contiguous cache needs num_outer >= num_seqs");
    if (c.rows < max_len) return invalid("a contiguous cache needs rows >= the longest sequence");
  }
  return FP2_OK;
}

// ------------------------------------------------------------------ rotate

fp2_status check_rotation(const fp2_rotation* p) {
  if (p == nullptr) return invalid("rotation must not be NULL");
  if (p->tokens < 0 || p->tokens >= (int64_t(1) << 31)) return invalid("tokens out of range");
  if (p->num_q_heads < 0 || p->num_kv_heads < 0 || p->num_q_heads + static_cast<int64_t>(p->num_kv_heads) == 0)
    return invalid("there must be heads to rotate");
  if (p->num_q_heads > 65536 || p->num_kv_heads > 65536) return unsupported("more than 65536 heads");
  if (p->head_dim != 64 && p->head_dim != 128) return unsupported("head_dim must be 64 or 128");
  if (p->in_dtype != FP2_BF16 && p->in_dtype != FP2_F32) return unsupported("in_dtype must be FP2_BF16 or FP2_F32");
  if (p->out_dtype != p->in_dtype && p->out_dtype != FP2_E4M3)
    return unsupported("out_dtype must be in_dtype or FP2_E4M3");
  if (p->rotary_dim < 0 || p->rotary_dim > p->head_dim || p->rotary_dim % 16 != 0)
    return unsupported("rotary_dim must be a multiple of 16 in [0, head_dim]");
  if (!(p->rope_scale >= 0.f) || !std::isfinite(p->rope_scale)) return invalid("rope_scale must be finite and >= 0");
  if ((p->q_norm != nullptr || p->k_norm != nullptr) && (!(p->norm_eps >= 0.f) || !std::isfinite(p->norm_eps)))
    return invalid("norm_eps must be finite and >= 0");
  if (!positive(p->q_descale) || !positive(p->k_descale) || !positive(p->v_descale))
    return invalid("descale factors must be finite, normal and > 0");
  if (p->out_dtype != FP2_E4M3 && (p->q_descale != 1.f || p->k_descale != 1.f || p->v_descale != 1.f))
    return invalid("descale factors other than 1 need an E4M3 output");
  if (p->rotary_dim > 0) {
    if (p->inv_freq_host == nullptr) return invalid("inv_freq_host is NULL");
    for (int i = 0; i < p->rotary_dim / 2; ++i)
      if (!(std::fabs(p->inv_freq_host[i]) < 1e18)) return invalid("inv_freq must be finite (and below 1e18)");
  }
  if (p->tokens == 0) return FP2_OK;
  if (p->rotary_dim > 0 && (p->positions == nullptr || !aligned4(p->positions)))
    return invalid("positions must be a 4-byte aligned pointer");
  const int ei = elt_bytes(p->in_dtype), eo = elt_bytes(p->out_dtype);
  const int64_t qw = static_cast<int64_t>(p->num_q_heads) * p->head_dim;
  const int64_t kw = static_cast<int64_t>(p->num_kv_heads) * p->head_dim;
  const auto in_ok = [&](const void* x, int64_t stride, int64_t width) {
    return x != nullptr && aligned16(x) && stride >= width && (stride * ei) % 16 == 0;
  };
  const auto out_ok = [&](const void* x, int64_t stride, int64_t width) {
    return x != nullptr && aligned16(x) && stride >= width && (stride * eo) % 16 == 0;
  };
  if (p->num_q_heads > 0 && (!in_ok(p->q, p->q_stride_tok, qw) || !out_ok(p->q_out, p->q_out_stride_tok, qw)))
    return invalid("q and q_out need 16-byte aligned pointers and strides, strides >= heads * head_dim");
  if (p->num_kv_heads > 0) {
    if (!in_ok(p->k, p->k_stride_tok, kw) || !out_ok(p->k_out, p->kv_out_stride_tok, kw))
      return invalid("k and k_out need 16-byte aligned pointers and strides, strides >= heads * head_dim");
    if (p->v != nullptr && (!in_ok(p->v, p->v_stride_tok, kw) || !out_ok(p->v_out, p->kv_out_stride_tok, kw)))
      return invalid("v and v_out need 16-byte aligned pointers and strides, strides >= heads * head_dim");
    if (p->slots != nullptr ? !aligned8(p->slots) || p->num_slots < 0 : p->num_slots < p->tokens)
      return invalid("num_slots must cover every token (or slots be given, 8-byte aligned)");
  }
  // In place every value is read and written by one thread, if it goes to where it came from.
  const auto in_place_ok = [&](const void* x, int64_t stride, const void* out, int64_t out_stride, bool moved) {
    return x != out || (p->out_dtype == p->in_dtype && !moved && (stride == out_stride || p->tokens == 1));
  };
  const bool moved = p->slots != nullptr;
  if ((p->num_q_heads > 0 && !in_place_ok(p->q, p->q_stride_tok, p->q_out, p->q_out_stride_tok, false)) ||
      (p->num_kv_heads > 0 && !in_place_ok(p->k, p->k_stride_tok, p->k_out, p->kv_out_stride_tok, moved)) ||
      (p->num_kv_heads > 0 && p->v != nullptr &&
       !in_place_ok(p->v, p->v_stride_tok, p->v_out, p->kv_out_stride_tok, moved)))
    return invalid("an output in place needs its input's type and stride, and for K and V no slots");
  if (!aligned16(p->q_norm) || !aligned16(p->k_norm)) return invalid("norm weights must be 16-byte aligned");
  return FP2_OK;
}

fp2_status run_rotate(const fp2_rotation* p, uint32_t* status_dev, cudaStream_t st) {
  fp2::RotateArgs a;
  std::memset(&a, 0, sizeof(a));
  a.q = p->q;
  a.k = p->k;
  a.v = p->v;
  a.q_stride = p->q_stride_tok;
  a.k_stride = p->k_stride_tok;
  a.v_stride = p->v_stride_tok;
  a.positions = p->positions;
  a.q_norm = p->num_q_heads > 0 ? p->q_norm : nullptr;
  a.k_norm = p->num_kv_heads > 0 ? p->k_norm : nullptr;
  a.norm_eps = p->norm_eps;
  a.Hq = p->num_q_heads;
  a.Hkv = p->num_kv_heads;
  a.Hv = p->v != nullptr ? p->num_kv_heads : 0;
  a.rot = p->rotary_dim;
  a.interleaved = p->interleaved ? 1 : 0;
  a.rope_scale = p->rope_scale > 0.f ? p->rope_scale : 1.f;
  a.q_out = p->q_out;
  a.k_out = p->k_out;
  a.v_out = p->v_out;
  a.q_out_stride = p->q_out_stride_tok;
  a.kv_out_stride = p->kv_out_stride_tok;
  a.slots = p->slots;
  a.num_slots = p->num_slots;
  a.q_inv = 1.f / p->q_descale;
  a.k_inv = 1.f / p->k_descale;
  a.v_inv = 1.f / p->v_descale;
  a.tokens = p->tokens;
  a.status = status_dev;
  // Turns per position as a fraction of 2^64 (rotate.cu): whole turns drop out (frequencies below 2^60).
  constexpr long double kTurn = 0.15915494309189533576888376337251436203L;  // 1 / 2 pi
  for (int i = 0; i < p->rotary_dim / 2; ++i) {
    const long double turns = static_cast<long double>(p->inv_freq_host[i]) * kTurn;
    const long double part = turns - static_cast<long double>(static_cast<int64_t>(turns));  // in (-1, 1)
    a.phase[i] = static_cast<uint64_t>(static_cast<int64_t>(part * 9223372036854775808.0L)) << 1;
  }
  return launched(fp2::launch_rotate(p->in_dtype, p->out_dtype, p->head_dim, a, st));
}

// ------------------------------------------------------------------ decode

struct DecodeCtx {
  int G = 0, T = 0, max_rows = 0, items = 1;
  bool f32 = false, few = true;         // which tree attention kernel
  int part_rows = 16, groups_tree = 1, groups_mass = 1;
  size_t off_desc = 0, off_ml = 0, off_o = 0, bytes = 0;
  float scale_log2 = 0.f;               // of a score of stored values, in powers of two
};

int groups_for(const fp2_decode* p, int G, int tile, int rows_per_tile, int least_tiles, int ctas) {
  // No more CTAs than the longest possible batch has work for: a small call keeps a small scratch.
  int64_t units = 0;
  const int64_t tiles = std::max<int64_t>(1, (static_cast<int64_t>(p->max_kv_len) + tile - 1) / tile);
  for (int r = 0; r < p->num_seqs; ++r) {
    const int64_t rows = static_cast<int64_t>(p->cu_seqlens_q_host[r + 1] - p->cu_seqlens_q_host[r]) * G;
    units += std::max<int64_t>((rows + rows_per_tile - 1) / rows_per_tile, least_tiles) * tiles;
  }
  const int64_t most = std::max(1, ctas / p->cache.num_kv_heads);
  return static_cast<int>(std::max<int64_t>(1, std::min(most, units)));
}

fp2_status validate(const fp2_decode* p, bool need_v, DecodeCtx& c) {
  if (p == nullptr) return invalid("decode must not be NULL");
  if (p->num_seqs < 1 || p->num_seqs > FP2_MAX_SEQS) return unsupported("num_seqs must be in [1, FP2_MAX_SEQS]");
  if (p->cu_seqlens_q_host == nullptr) return invalid("cu_seqlens_q_host is NULL");
  if (p->max_kv_len < 0) return invalid("max_kv_len must be >= 0");
  if (p->max_kv_len > FP2_MAX_CACHE_LEN) return unsupported("max_kv_len above FP2_MAX_CACHE_LEN");
  FP2_TRY(check_cache(p->cache, p->num_seqs, p->max_kv_len, need_v));
  if (p->num_q_heads <= 0 || p->num_q_heads % p->cache.num_kv_heads != 0)
    return invalid("num_q_heads must be a positive multiple of num_kv_heads");
  c.G = p->num_q_heads / p->cache.num_kv_heads;
  if (c.G > 32) return unsupported("GQA group size above 32");
  if (!(p->softmax_scale >= 0.f) || !std::isfinite(p->softmax_scale))
    return invalid("softmax_scale must be finite and >= 0");
  if (!positive(p->q_descale) || !positive(p->k_descale) || !positive(p->v_descale))
    return invalid("descale factors must be finite, normal and > 0");
  if (p->cu_seqlens_q_host[0] != 0) return invalid("cu_seqlens must start at 0");
  int most = 0;
  for (int r = 0; r < p->num_seqs; ++r) {
    const int64_t n = static_cast<int64_t>(p->cu_seqlens_q_host[r + 1]) - p->cu_seqlens_q_host[r];
    if (n < 0) return invalid("cu_seqlens must be non-decreasing");
    if (n > FP2_MAX_DRAFT) return unsupported("more than FP2_MAX_DRAFT tokens in a sequence");
    if (n > p->max_kv_len) return invalid("max_kv_len is below a sequence's tokens");
    most = std::max(most, static_cast<int>(n));
  }
  c.T = p->cu_seqlens_q_host[p->num_seqs];
  c.max_rows = most * c.G;
  const int D = p->cache.head_dim;
  const float scale =
      p->softmax_scale > 0.f ? p->softmax_scale : static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)));
  c.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634 *
                                    static_cast<double>(p->q_descale) * static_cast<double>(p->k_descale));
  // (a product that is zero would make the scores of keys that no one sees, -infinity, NaN)
  if (!(c.scale_log2 >= FLT_MIN) || !std::isfinite(c.scale_log2) || !std::isfinite(p->v_descale * 256.f))
    return invalid("softmax_scale * q_descale * k_descale must be a normal fp32 number, v_descale below 2^120");
  if (p->kv_len == nullptr || !aligned4(p->kv_len)) return invalid("kv_len must be a 4-byte aligned pointer");
  if (c.T > 0) {
    if (p->q == nullptr || !aligned16(p->q)) return invalid("q must be a 16-byte aligned pointer");
    if (p->q_stride_tok < static_cast<int64_t>(p->num_q_heads) * D || p->q_stride_tok >= (int64_t(1) << 37) ||
        (p->q_stride_tok * elt_bytes(p->cache.dtype)) % 16)
      return invalid("q_stride_tok must be >= heads * head_dim and a multiple of 16 bytes");
    if (!aligned8(p->tree_mask)) return invalid("tree_mask must be 8-byte aligned");
  }
  // Two CTAs of the few-rows kernel share an SM, three of the F32 kernel while rows leave them room, one of the wide
  // kernel fills it.
  const int sms = num_sms();
  c.f32 = p->cache.dtype == FP2_F32;
  c.few = c.f32 || c.max_rows <= fp2::kFewRows;
  c.part_rows = c.few ? fp2::kFewRows : (c.max_rows <= 128 ? 128 : 256);
  c.items = 0;
  for (int r = 0; r < p->num_seqs; ++r)
    c.items += ((p->cu_seqlens_q_host[r + 1] - p->cu_seqlens_q_host[r]) * c.G + c.part_rows - 1) / c.part_rows;
  c.groups_tree = c.few ? groups_for(p, c.G, fp2::kFewTile, fp2::kFewRows, 0, sms * (c.f32 && c.max_rows <= 4 ? 3 : 2))
                        : groups_for(p, c.G, fp2::kWideTile, 128, 0, sms);
  c.groups_mass = c.f32 ? groups_for(p, c.G, fp2::kMassTile, FP2_MAX_DRAFT * c.G, 1, sms * 4)
                        : groups_for(p, c.G, fp2::kMassTile, fp2::kMassRows / c.G * c.G, 1, sms);
  const size_t ctas = static_cast<size_t>(c.groups_tree) * p->cache.num_kv_heads;
  const size_t words = std::max(ctas, static_cast<size_t>(c.groups_mass) * p->cache.num_kv_heads);
  c.off_desc = FP2_SCRATCH_STATUS_BYTES + align_up(words * 4);
  c.off_ml = c.off_desc + align_up(static_cast<size_t>(c.groups_tree) * 16);
  c.off_o = c.off_ml + align_up(ctas * 2 * c.part_rows * 8);
  c.bytes = c.off_o + align_up(ctas * 2 * c.part_rows * D * 4);
  return FP2_OK;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Encodes a map.  The encoder is a driver call, which wants a current context; a thread that has made no runtime call
// yet has none (these calls' maps come before their first launch), and gets its device's then.
template <typename Encode>
fp2_status encode(const Encode& map) {
  const EncodeTiledFn fn = reinterpret_cast<EncodeTiledFn>(fp2_internal::tensor_map_encoder());
  if (fn == nullptr) return fail(FP2_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  CUresult r = map(fn);
  int dev = 0;
  if (r != CUDA_SUCCESS && cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess) r = map(fn);
  return r == CUDA_SUCCESS ? FP2_OK : fail(FP2_ERR_CUDA, "cuTensorMapEncodeTiled failed");
}

int box_rows(const fp2_cache& c) { return c.page_table != nullptr ? std::min(c.rows, 64) : 64; }

// [outer][token][head][d] with boxes of 128 bytes x up to 64 tokens; a box never leaves its page.
fp2_status encode_cache(CUtensorMap* m, const fp2_cache& c, void* base) {
  const int elt = elt_bytes(c.dtype);
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.head_dim), static_cast<cuuint64_t>(c.num_kv_heads),
                              static_cast<cuuint64_t>(c.rows), static_cast<cuuint64_t>(c.num_outer)};
  const cuuint64_t strides[3] = {
      static_cast<cuuint64_t>(c.head_dim) * elt, static_cast<cuuint64_t>(c.stride_tok) * elt,
      static_cast<cuuint64_t>(std::max(c.stride_outer, c.num_outer > 1 ? int64_t(0) : c.stride_tok)) * elt};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(128 / elt), 1u,
                             static_cast<cuuint32_t>(box_rows(c)), 1u};
  const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  return encode([&](EncodeTiledFn fn) {
    return fn(m, c.dtype == FP2_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, base, dims,
              strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  });
}

// [token][head][d] with boxes of 128 bytes x the heads of a group x `tokens`.
fp2_status encode_q(CUtensorMap* m, const fp2_decode* p, int T, int G, int tokens) {
  const fp2_cache& c = p->cache;
  const int elt = elt_bytes(c.dtype);
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(c.head_dim), static_cast<cuuint64_t>(p->num_q_heads),
                              static_cast<cuuint64_t>(T)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(c.head_dim) * elt,
                                 static_cast<cuuint64_t>(p->q_stride_tok) * elt};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / elt), static_cast<cuuint32_t>(G),
                             static_cast<cuuint32_t>(tokens)};
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  return encode([&](EncodeTiledFn fn) {
    return fn(m, c.dtype == FP2_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 3,
              const_cast<void*>(p->q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  });
}

fp2_status fill_decode(const fp2_decode* p, const DecodeCtx& c, void* scratch, fp2::DecodeArgs& a,
                       fp2::DecodePlan& P) {
  std::memset(&a, 0, sizeof(a));
  if (!c.f32) FP2_TRY(encode_cache(&a.tm_k, p->cache, p->cache.k));
  P.num_seqs = p->num_seqs;
  std::memcpy(P.q_off, p->cu_seqlens_q_host, sizeof(int32_t) * (p->num_seqs + 1));
  a.q = p->q;
  a.q_stride = p->q_stride_tok;
  a.kv_len = p->kv_len;
  a.max_kv_len = p->max_kv_len;
  a.page_table = p->cache.page_table;
  a.max_rows = c.max_rows;
  a.k_ptr = p->cache.k;
  a.v_ptr = p->cache.v;
  a.kv_stride = p->cache.stride_tok;
  a.kv_stride_outer = p->cache.stride_outer;
  a.page_size = p->cache.rows;
  while (a.page_table != nullptr && (2 << a.page_shift) <= a.page_size) ++a.page_shift;
  a.box_rows = box_rows(p->cache);
  while ((2 << a.box_shift) <= a.box_rows) ++a.box_shift;
  a.max_pages = p->cache.max_pages_per_seq;
  a.num_pages = p->cache.num_outer;
  a.mask = p->tree_mask;
  a.Hq = p->num_q_heads;
  a.Hkv = p->cache.num_kv_heads;
  a.G = c.G;
  a.T = c.T;
  a.scale_log2 = c.scale_log2;
  a.v_descale = p->v_descale;
  a.scratch = static_cast<uint32_t*>(scratch);
  a.wait_limit_ns = fp2_internal::wait_limit_ns();
  a.withhold = fp2_internal::withheld_k_tile();
  a.late_v = fp2_internal::late_v_tile();
  return FP2_OK;
}

// ------------------------------------------------------------------ evict

fp2::CacheView view(const fp2_cache& c) {
  const int elt = elt_bytes(c.dtype);
  fp2::CacheView v{};
  v.k = static_cast<char*>(c.k);
  v.v = static_cast<char*>(c.v);
  v.stride_tok = c.stride_tok * elt;
  v.stride_outer = c.stride_outer * elt;
  v.page_table = c.page_table;
  v.rows = c.rows;
  v.max_pages = c.max_pages_per_seq;
  v.num_outer = c.num_outer;
  return v;
}

bool overlap(const fp2_cache& x, const void* xp, const fp2_cache& y, const void* yp) {
  const auto bytes = [](const fp2_cache& c) {
    return static_cast<uintptr_t>(((c.num_outer - 1) * c.stride_outer + (c.rows - 1) * c.stride_tok +
                                   static_cast<int64_t>(c.num_kv_heads) * c.head_dim) * elt_bytes(c.dtype));
  };
  const uintptr_t a = reinterpret_cast<uintptr_t>(xp), b = reinterpret_cast<uintptr_t>(yp);
  return a < b + bytes(y) && b < a + bytes(x);
}

fp2_status fill_evict(const fp2_eviction* p, fp2::EvictArgs& a, int& ranks, size_t& bytes) {
  if (p == nullptr) return invalid("eviction must not be NULL");
  if (p->num_seqs < 1 || p->num_seqs > FP2_MAX_SEQS) return unsupported("num_seqs must be in [1, FP2_MAX_SEQS]");
  if (p->max_kv_len < 0) return invalid("max_kv_len must be >= 0");
  if (p->max_kv_len > FP2_MAX_CACHE_LEN) return unsupported("max_kv_len above FP2_MAX_CACHE_LEN");
  if (p->budget < 1 || p->sink < 0 || p->window < 0 || static_cast<int64_t>(p->sink) + p->window > p->budget)
    return invalid("budget must be >= 1, sink and window >= 0 and sink + window <= budget");
  if (p->budget > FP2_MAX_CACHE_LEN) return unsupported("budget above FP2_MAX_CACHE_LEN");
  FP2_TRY(check_cache(p->src, p->num_seqs, p->max_kv_len, true));
  FP2_TRY(check_cache(p->dst, p->num_seqs, std::min(p->budget, p->max_kv_len), true));
  if (p->src.dtype != p->dst.dtype || p->src.num_kv_heads != p->dst.num_kv_heads || p->src.head_dim != p->dst.head_dim)
    return invalid("src and dst must agree in dtype, heads and head_dim");
  if (p->src.page_table == nullptr || p->dst.page_table == nullptr)
    for (const void* s : {p->src.k, p->src.v})
      for (const void* d : {p->dst.k, p->dst.v})
        if (overlap(p->src, s, p->dst, d)) return invalid("src and dst overlap");
  if (p->kv_len == nullptr || p->mass == nullptr || p->mass_out == nullptr || p->kept == nullptr ||
      p->kv_len_out == nullptr)
    return invalid("kv_len, mass, mass_out, kept and kv_len_out must not be NULL");
  if (!aligned4(p->kv_len) || !aligned4(p->mass) || !aligned4(p->mass_out) || !aligned4(p->kept) ||
      !aligned4(p->kv_len_out))
    return invalid("kv_len, mass, mass_out, kept and kv_len_out must be 4-byte aligned");
  if (p->mass_stride < p->max_kv_len) return invalid("mass_stride must be >= max_kv_len");
  // Other CTAs still read the lengths and weights when the first ones write theirs.
  const size_t rows = static_cast<size_t>(p->num_seqs) * p->src.num_kv_heads;
  const size_t mass_bytes = rows * static_cast<size_t>(p->mass_stride) * 4, out_bytes = rows * p->budget * 4;
  const size_t len_bytes = static_cast<size_t>(p->num_seqs) * 4;
  if (!apart(p->kv_len, len_bytes, p->kv_len_out, len_bytes)) return invalid("kv_len_out must not overlap kv_len");
  if (!apart(p->mass, mass_bytes, p->mass_out, out_bytes) || !apart(p->mass, mass_bytes, p->kept, out_bytes) ||
      !apart(p->mass_out, out_bytes, p->kept, out_bytes))
    return invalid("mass, mass_out and kept must not overlap");
  std::memset(&a, 0, sizeof(a));
  a.src = view(p->src);
  a.dst = view(p->dst);
  a.kv_len = p->kv_len;
  a.max_kv_len = p->max_kv_len;
  a.num_seqs = p->num_seqs;
  a.Hkv = p->src.num_kv_heads;
  a.row_bytes = p->src.head_dim * elt_bytes(p->src.dtype);
  a.mass = p->mass;
  a.mass_stride = p->mass_stride;
  a.budget = p->budget;
  a.sink = p->sink;
  a.window = p->window;
  a.mass_out = p->mass_out;
  a.kept = p->kept;
  a.kv_len_out = p->kv_len_out;
  ranks = fp2::evict_cluster(a);
  const int64_t ctas = static_cast<int64_t>(a.num_seqs) * a.Hkv * ranks;
  if (ctas > static_cast<int64_t>(fp2::kStatusCount)) return unsupported("too many (sequence, KV head) rows");
  bytes = FP2_SCRATCH_STATUS_BYTES + align_up(static_cast<size_t>(ctas) * 4);
  return FP2_OK;
}

}  // namespace

extern "C" {

fp2_status fp2_rotate(const fp2_rotation* rotation, uint32_t* status_dev, fp2_stream_t stream) {
  FP2_TRY(check_rotation(rotation));
  if (!aligned4(status_dev)) return invalid("status_dev must be 4-byte aligned");
  if (rotation->tokens == 0) return FP2_OK;
  FP2_TRY(check_stream(stream));
  return run_rotate(rotation, status_dev, static_cast<cudaStream_t>(stream));
}

fp2_status fp2_decode_workspace(const fp2_decode* decode, size_t* scratch_bytes) {
  if (scratch_bytes == nullptr) return invalid("scratch_bytes is NULL");
  DecodeCtx c;
  FP2_TRY(validate(decode, false, c));
  *scratch_bytes = c.bytes;
  fp2_internal::clear_error();
  return FP2_OK;
}

fp2_status fp2_tree_attend(const fp2_decode* decode, void* out, float* lse, void* scratch, size_t scratch_bytes,
                           fp2_stream_t stream) {
  DecodeCtx c;
  FP2_TRY(validate(decode, true, c));
  FP2_TRY(check_scratch(scratch, scratch_bytes, c.bytes));
  if ((c.T > 0 && out == nullptr) || !aligned16(out)) return invalid("out must be a 16-byte aligned pointer");
  if (!aligned4(lse)) return invalid("lse must be 4-byte aligned");
  FP2_TRY(check_stream(stream));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (c.T == 0) return clear_status(scratch, st);
  fp2::DecodeArgs a;
  fp2::DecodePlan P;
  FP2_TRY(fill_decode(decode, c, scratch, a, P));
  if (!c.f32) FP2_TRY(encode_cache(&a.tm_v, decode->cache, decode->cache.v));
  char* base = static_cast<char*>(scratch);
  a.groups = c.groups_tree;
  a.out = out;
  a.lse = lse;
  a.desc = reinterpret_cast<int4*>(base + c.off_desc);
  a.part_ml = reinterpret_cast<float2*>(base + c.off_ml);
  a.part_o = reinterpret_cast<float*>(base + c.off_o);
  a.part_rows = c.part_rows;
  a.out_f32 = c.f32 ? 1 : 0;
  // Few items over many groups have many pieces each: one request of 20K e4m3 keys, 44 rows of one KV head, 148
  // pieces, took 27 us with a warp per row and 22 with four.  With 37 pieces (80K keys, 84 rows, 4 KV heads) the
  // blocks that find nothing to join cost more: 39 and 44 us.
  a.join_warps = c.groups_tree >= 64 * c.items ? 4 : 1;
  if (!c.few && decode->cache.dtype == FP2_E4M3) a.v_descale *= 256.f;  // tree_wide.cu works on V * 2^-8
  const int D = decode->cache.head_dim;
  FP2_TRY(launched(c.f32   ? fp2::launch_tree_f32(a, P, st)
                   : c.few ? fp2::launch_tree_few(decode->cache.dtype, D, a, P, st)
                           : fp2::launch_tree_wide(decode->cache.dtype, D, a, P, st)));
  if (a.groups == 1) return FP2_OK;  // no item is split
  return launched(fp2::launch_tree_join(D, c.max_rows, a, P, st));
}

fp2_status fp2_key_mass(const fp2_decode* decode, const float* lse, const float* mass_in, float* mass_out,
                        int64_t mass_stride, const int32_t* mass_len, float decay, void* scratch,
                        size_t scratch_bytes, fp2_stream_t stream) {
  DecodeCtx c;
  FP2_TRY(validate(decode, false, c));
  FP2_TRY(check_scratch(scratch, scratch_bytes, c.bytes));
  if (mass_stride < decode->max_kv_len) return invalid("mass_stride must be >= max_kv_len");
  if (!std::isfinite(decay)) return invalid("decay must be finite");
  if (!aligned4(lse) || !aligned4(mass_in) || !aligned4(mass_out) || !aligned4(mass_len))
    return invalid("lse, mass_in, mass_out and mass_len must be 4-byte aligned");
  if (mass_out == nullptr || (c.T > 0 && lse == nullptr)) return invalid("lse and mass_out must not be NULL");
  // A CTA reads old weights, LSE and lengths while others write new weights.
  const size_t len_bytes = static_cast<size_t>(decode->num_seqs) * 4;
  const size_t mass_bytes = len_bytes * decode->cache.num_kv_heads * static_cast<size_t>(mass_stride);
  if (mass_in != nullptr && mass_in != mass_out && !apart(mass_in, mass_bytes, mass_out, mass_bytes))
    return invalid("mass_in and mass_out must be the same or not overlap");
  if ((c.T > 0 && !apart(lse, static_cast<size_t>(c.T) * decode->num_q_heads * 4, mass_out, mass_bytes)) ||
      !apart(decode->kv_len, len_bytes, mass_out, mass_bytes) ||
      (mass_len != nullptr && !apart(mass_len, len_bytes, mass_out, mass_bytes)))
    return invalid("mass_out must not overlap lse, kv_len or mass_len");
  FP2_TRY(check_stream(stream));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  fp2::DecodeArgs a;
  fp2::DecodePlan P;
  FP2_TRY(fill_decode(decode, c, scratch, a, P));
  a.groups = c.groups_mass;
  a.pass_tokens = fp2::kMassRows / c.G;
  if (!c.f32 && c.T > 0)
    FP2_TRY(encode_q(&a.tm_q, decode, c.T, c.G, a.pass_tokens));
  else
    a.tm_q = a.tm_k;  // there are no rows to load: see key_mass.cu
  a.lse_in = lse;
  a.mass_in = mass_in;
  a.mass_out = mass_out;
  a.mass_stride = mass_stride;
  a.mass_len = mass_len;
  a.decay = decay;
  if (c.f32) return launched(fp2::launch_mass_f32(a, P, st));
  return launched(fp2::launch_key_mass(decode->cache.dtype, decode->cache.head_dim, a, P, st));
}

fp2_status fp2_evict_workspace(const fp2_eviction* eviction, size_t* scratch_bytes) {
  if (scratch_bytes == nullptr) return invalid("scratch_bytes is NULL");
  fp2::EvictArgs a;
  int ranks = 1;
  FP2_TRY(fill_evict(eviction, a, ranks, *scratch_bytes));
  fp2_internal::clear_error();
  return FP2_OK;
}

fp2_status fp2_evict(const fp2_eviction* eviction, void* scratch, size_t scratch_bytes, fp2_stream_t stream) {
  fp2::EvictArgs a;
  int ranks = 1;
  size_t need = 0;
  FP2_TRY(fill_evict(eviction, a, ranks, need));
  FP2_TRY(check_scratch(scratch, scratch_bytes, need));
  FP2_TRY(check_stream(stream));
  a.scratch = static_cast<uint32_t*>(scratch);
  return launched(fp2::launch_evict(a, ranks, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
