// Tree attention and key mass over an F32 cache (head_dim 64), on the CUDA cores.
//
// The work is cut and joined as in decode.cu: units of (sequence, tile of up to 16 query rows, tile of 64 keys)
// for the attention, tiles of 128 keys for the weights.  The tensor cores would round Q and K to tf32 (half a
// step of 2^-11 in each factor, where an F32 cache promises 2^-24), so the products are fp32 FMAs, two an
// instruction.
//
// Attention, 128 threads: a thread has one key and half the rows for the scores, a warp a quarter of the rows
// for the softmax, a thread one value of d and half the rows for P V.  K and V tiles come by cp.async, the
// next while the current one is worked on; up to 4 rows three CTAs share an SM, above that two.
//
// What bounds it: with up to 4 rows per KV head HBM nearly (537 MB, 16 sequences of 8192 keys, 8 KV heads: 104 to
// 113 us, 4.7 to 5.2 TB/s; the instance for 16 rows took 260 us there, two CTAs with room for 16 rows 146 us, a
// page id read only when its tile is due 114 us).  With more rows the reads of Q, P and K from shared memory, one
// of 16 bytes for two packed FMAs (the FMA pipe is at a quarter of its rate): 193 us for as many bytes and 8 rows,
// 72 us for 134 MB and 16 rows, 245 us for 134 MB and 64 rows, which are four passes over K and V.  The weights:
// 268 MB of K and 4 rows in 81 us (3.3 TB/s); a thread's K row is read 16 bytes at a time, so that L1 serves every
// second access.
#include "decode_device.cuh"

namespace fp2 {

namespace {

constexpr int kD = 64, kRows = kFewRows, kTile = kFewTile, kThreads = 128;
constexpr int kScorePad = kTile + 4;

// NR: the rows of a tile that can be there (4, 8 or 16).  With 4, three CTAs' fit in an SM.
template <int NR>
struct F32Shared {
  float k[2][kTile][kD], v[2][kTile][kD];  // 16-byte chunk c of key j of K lies at c ^ (j & 7)
  float q[NR][kD];
  float p[NR][kScorePad];           // scores, then weights
  float scale[NR];                  // factor of the row's sums so far
  float2 ml[NR];
  long long pre[FP2_MAX_SEQS + 1];
  int len[FP2_MAX_SEQS];
  uint64_t seen[NR];                // keys of the tile that the row sees, where rows differ in that
  uint32_t valid[2][2];             // keys of the tile that are there
  uint32_t status;
};

// Page of key j (below the sequence's length) of sequence r; without pages the sequence itself.
FP2_DEVICE int page_of(const DecodeArgs& a, int r, int j) {
  return a.page_table == nullptr ? r : a.page_table[static_cast<int64_t>(r) * a.max_pages + (j >> a.page_shift)];
}

// Row (of kD values) of key j and KV head g in page `outer`, or NULL for a page id out of range.
FP2_DEVICE const float* cache_at(const DecodeArgs& a, const void* base, int64_t outer, int j, int g, uint32_t* status) {
  int64_t row = j;
  if (a.page_table != nullptr) {
    row = j & (a.page_size - 1);
    if (outer < 0 || outer >= a.num_pages) {
      set_status(status, FP2_DEV_PAGE_OOB);
      return nullptr;
    }
  }
  return static_cast<const float*>(base) + outer * a.kv_stride_outer + row * a.kv_stride + static_cast<int64_t>(g) * kD;
}

FP2_DEVICE void copy16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}

// (x, y) += (a, b) * (c, d): one instruction of two fp32 products.
FP2_DEVICE float2 fma2(float2 m, float2 n, float2 acc) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(*reinterpret_cast<const uint64_t*>(&m)), "l"(*reinterpret_cast<const uint64_t*>(&n)),
        "l"(*reinterpret_cast<const uint64_t*>(&acc)));
  return *reinterpret_cast<const float2*>(&r);
}

template <int NR>
__global__ void __launch_bounds__(kThreads) tree_f32_kernel(const __grid_constant__ DecodeArgs a,
                                                            const __grid_constant__ DecodePlan P) {
  extern __shared__ __align__(16) char smem_raw[];
  F32Shared<NR>& s = *reinterpret_cast<F32Shared<NR>*>(smem_raw);
  constexpr int RT = NR / 2, RW = NR / 4;  // rows of a thread in the products, of a warp in the softmax
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = blockIdx.x % a.Hkv, grp = blockIdx.x / a.Hkv;
  grid_launch_next();
  if (tid == 0) s.status = 0;
  grid_wait();
  __syncthreads();
  scan_units<kTile>(a, P, kRows, 0, s.pre, s.len, &s.status);
  const long long units = s.pre[P.num_seqs];
  const int ng = active_groups(units, a.groups);
  const bool idle = grp >= ng;
  const long long u0 = idle ? 0 : units * grp / ng, u1 = idle ? 0 : units * (grp + 1) / ng;
  if (idle && g == 0 && tid == 0) a.desc[grp] = make_int4(-1, 0, 0, 0);

  int nth = 0;
  for (long long u = u0; u < u1; ++nth) {
    const Piece p = piece_at<kTile>(s.pre, s.len, P.num_seqs, u, u1);
    const int keys = s.len[p.r], t0 = P.q_off[p.r], q_len = P.q_off[p.r + 1] - t0;
    const int row0 = p.rt * kRows, rows = q_len * a.G, base = keys - q_len;
    // Two threads know a key: K's row and V's.  Sixteen lanes copy a row, so that a warp's copies are whole
    // lines.  Rows that are not there are not loaded; their weights are zero.
    // The page id of the tile after is read one tile ahead: a trip to memory that nothing else would cover.
    int page = 0;
    const auto read_page = [&](int t) {
      const int j = t * kTile + (tid & (kTile - 1));
      if (t < p.t1 && j < keys) page = page_of(a, p.r, j);
    };
    const auto load = [&](int t, int b) {
      const int key = tid & (kTile - 1), j = t * kTile + key;
      const bool is_v = tid >= kTile;
      const float* src = j < keys ? cache_at(a, is_v ? a.v_ptr : a.k_ptr, page, j, g, &s.status) : nullptr;
      read_page(t + 1);
      float (*dst)[kD] = (is_v ? s.v[b] : s.k[b]) + (warp & 1) * 32;
#pragma unroll 4
      for (int i = 0; i < 32; i += 2) {
        const int n = i + (lane >> 4), c = lane & 15;
        const float* from =
            reinterpret_cast<const float*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(src), n));
        if (from != nullptr) copy16(&dst[n][4 * (is_v ? c : c ^ (n & 7))], from + 4 * c);
      }
      const uint32_t there = __ballot_sync(0xFFFFFFFFu, src != nullptr);
      if (!is_v && lane == 0) s.valid[b][warp] = there;
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    __syncthreads();  // the piece before is written
    read_page(p.t0);
    load(p.t0, 0);
    for (int i = tid; i < NR * (kD / 4); i += kThreads) {
      const int rr = i / (kD / 4), c = i % (kD / 4), m = row0 + rr;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (m < rows) {
        const int tok = m / a.G, h = g * a.G + (m - tok * a.G);
        x = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) +
                                             (static_cast<int64_t>(t0) + tok) * a.q_stride +
                                             static_cast<int64_t>(h) * kD + 4 * c);
      }
      *reinterpret_cast<float4*>(&s.q[rr][4 * c]) = x;
    }
    const int d = tid & (kD - 1), half = tid >> 6;  // of P V: this thread's value and rows RT half ..
    float o[RT], mx[RW], sum[RW];                   // of the softmax: rows RW warp .., sums of the lane's keys
#pragma unroll
    for (int i = 0; i < RT; ++i) o[i] = 0.f;
#pragma unroll
    for (int i = 0; i < RW; ++i) mx[i] = neg_inf(), sum[i] = 0.f;

    for (int t = p.t0; t < p.t1; ++t) {
      const int b = (t - p.t0) & 1;
      if (t + 1 < p.t1)
        load(t + 1, b ^ 1);
      else
        asm volatile("cp.async.commit_group;" ::: "memory");
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncthreads();
      const uint64_t valid = s.valid[b][0] | (static_cast<uint64_t>(s.valid[b][1]) << 32);
      const bool plain = valid == ~0ull && (t + 1) * kTile <= base;
      {
        const int key = tid & (kTile - 1);
        float2 acc[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) acc[i] = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int c = 0; c < kD / 4; ++c) {
          const float4 k4 = *reinterpret_cast<const float4*>(&s.k[b][key][4 * (c ^ (key & 7))]);
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const float4 q4 = *reinterpret_cast<const float4*>(&s.q[RT * half + i][4 * c]);
            acc[i] = fma2(make_float2(q4.x, q4.y), make_float2(k4.x, k4.y), acc[i]);
            acc[i] = fma2(make_float2(q4.z, q4.w), make_float2(k4.z, k4.w), acc[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < RT; ++i) s.p[RT * half + i][key] = acc[i].x + acc[i].y;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < RW; ++i) {
        const int rr = RW * warp + i, m = row0 + rr;
        float x0 = s.p[rr][lane], x1 = s.p[rr][lane + 32];
        if (!plain) {
          const uint64_t word = m < rows && keys > 0 ? token_mask(a, t0, m / a.G) : 0;
          const auto sees = [&](int key) {
            const int off = t * kTile + key - base;
            return ((valid >> key) & 1) && m < rows && (off < 0 || (off < 64 && ((word >> off) & 1)));
          };
          const bool s0 = sees(lane), s1 = sees(lane + 32);
          if (!s0) x0 = neg_inf();
          if (!s1) x1 = neg_inf();
          const uint32_t low = __ballot_sync(0xFFFFFFFFu, s0), high = __ballot_sync(0xFFFFFFFFu, s1);
          if (lane == 0) s.seen[rr] = low | (static_cast<uint64_t>(high) << 32);
        }
        float now = fmaxf(x0, x1);
#pragma unroll
        for (int o2 = 16; o2; o2 >>= 1) now = fmaxf(now, __shfl_xor_sync(0xFFFFFFFFu, now, o2));
        now = fmaxf(now, mx[i]);
        const float f = now == neg_inf() ? 1.f : fast_exp2((mx[i] - now) * a.scale_log2);
        const float off = now == neg_inf() ? 0.f : -now * a.scale_log2;
        const float e0 = fast_exp2(fmaf(x0, a.scale_log2, off)), e1 = fast_exp2(fmaf(x1, a.scale_log2, off));
        sum[i] = sum[i] * f + e0 + e1;
        mx[i] = now;
        s.p[rr][lane] = e0;
        s.p[rr][lane + 32] = e1;
        if (lane == 0) s.scale[rr] = f;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < RT; ++i) o[i] *= s.scale[RT * half + i];
      // A key that a row does not see has the weight 0 there, and its value may be anything (0 x NaN is NaN): it is
      // left out.  A key that it does see is not, though its weight may have underflowed to 0.
      const auto add = [&](bool check) {
#pragma unroll 4
        for (int j = 0; j < kTile; j += 4) {
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = s.v[b][j + e][d];
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const float4 w = *reinterpret_cast<const float4*>(&s.p[RT * half + i][j]);
            const float we[4] = {w.x, w.y, w.z, w.w};
            const uint32_t in = check ? static_cast<uint32_t>(s.seen[RT * half + i] >> j) : 0u;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!check || ((in >> e) & 1u)) o[i] = fmaf(we[e], x[e], o[i]);
          }
        }
      };
      if (plain)
        add(false);
      else
        add(true);
      __syncthreads();  // K, V and P of this tile are done with
    }

    const bool whole = p.t0 == 0 && p.t1 == p.tiles;
    const int slot = (grp * a.Hkv + g) * 2 + (nth == 0 ? 0 : 1);
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      float x = sum[i];
#pragma unroll
      for (int o2 = 16; o2; o2 >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o2);
      if (lane == 0) s.ml[RW * warp + i] = make_float2(mx[i], x);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int rr = RT * half + i, m = row0 + rr;
      if (m >= rows) continue;
      const float2 ml = s.ml[rr];
      const int tok = m / a.G, h = g * a.G + (m - tok * a.G);
      const int64_t row = static_cast<int64_t>(t0) + tok;
      if (!fp2_check(row < a.T && h < a.Hq, &s.status)) continue;
      if (whole) {
        static_cast<float*>(a.out)[(row * a.Hq + h) * kD + d] = ml.y == 0.f ? 0.f : o[i] * (a.v_descale / ml.y);
        if (d == 0 && a.lse != nullptr)
          a.lse[static_cast<int64_t>(h) * a.T + row] =
              ml.y == 0.f ? neg_inf() : (ml.x * a.scale_log2 + log2f(ml.y)) * kLn2;
      } else {
        a.part_o[(static_cast<int64_t>(slot) * kRows + rr) * kD + d] = o[i];
        if (d == 0)
          a.part_ml[static_cast<int64_t>(slot) * kRows + rr] =
              make_float2(ml.x == neg_inf() ? ml.x : ml.x * a.scale_log2, ml.y);
      }
    }
    u += p.t1 - p.t0;
    if (g == 0 && tid == 0 && u >= u1) {
      int4 dsc = make_int4(-1, 0, 0, 0);
      if (p.t0 == 0 && p.t1 < p.tiles)
        dsc = make_int4(nth == 0 ? 0 : 1, p.r, p.rt, group_of(units, ng, u1 + (p.tiles - p.t1) - 1) - grp + 1);
      a.desc[grp] = dsc;
    }
  }
  store_status(a, &s.status);
}

static_assert(3 * (sizeof(F32Shared<4>) + 1024) <= 227 * 1024, "three CTAs an SM");
static_assert(kThreads == 2 * kTile && kThreads == kMassTile && kRows == 16, "the threads' shares of a tile");

// Key mass: a thread has one key, its K row in registers, and goes through the rows in their order.
struct MassF32Shared {
  float neg_lse[kMassRows];
  uint64_t mask[kMassRows];
  long long pre[FP2_MAX_SEQS + 1];
  int len[FP2_MAX_SEQS];
  uint32_t status;
  alignas(16) float q[kMassRows][kD];  // last: a launch has room for the rows that a pass can have, L1 for the rest
};

__global__ void __launch_bounds__(kThreads) mass_f32_kernel(const __grid_constant__ DecodeArgs a,
                                                            const __grid_constant__ DecodePlan P) {
  extern __shared__ __align__(16) char smem_raw[];
  MassF32Shared& s = *reinterpret_cast<MassF32Shared*>(smem_raw);
  const int tid = threadIdx.x;
  const int g = blockIdx.x % a.Hkv, grp = blockIdx.x / a.Hkv;
  grid_launch_next();
  if (tid == 0) s.status = 0;
  grid_wait();
  __syncthreads();
  scan_units<kMassTile>(a, P, FP2_MAX_DRAFT * a.G, 1, s.pre, s.len, &s.status);
  const long long units = s.pre[P.num_seqs];
  const int ng = active_groups(units, a.groups);
  const long long u0 = grp < ng ? units * grp / ng : 0, u1 = grp < ng ? units * (grp + 1) / ng : 0;
  for (long long u = u0; u < u1;) {
    const Piece p = piece_at<kMassTile>(s.pre, s.len, P.num_seqs, u, u1);
    const int keys = s.len[p.r], t0 = P.q_off[p.r], q_len = P.q_off[p.r + 1] - t0;
    const int rows = q_len * a.G, base = keys - q_len;
    const int had = a.mass_in == nullptr ? 0 : (a.mass_len != nullptr ? a.mass_len[p.r] : keys);
    const int64_t at = (static_cast<int64_t>(p.r) * a.Hkv + g) * a.mass_stride;
    for (int c0 = 0; c0 == 0 || c0 < rows; c0 += kMassRows) {
      const int n = min(kMassRows, rows - c0);
      __syncthreads();
      for (int i = tid; i < n * (kD / 4); i += kThreads) {
        const int rr = i / (kD / 4), c = i % (kD / 4), tok = (c0 + rr) / a.G, h = g * a.G + (c0 + rr - tok * a.G);
        *reinterpret_cast<float4*>(&s.q[rr][4 * c]) = *reinterpret_cast<const float4*>(
            static_cast<const float*>(a.q) + (static_cast<int64_t>(t0) + tok) * a.q_stride +
            static_cast<int64_t>(h) * kD + 4 * c);
      }
      for (int rr = tid; rr < n; rr += kThreads) {
        const int tok = (c0 + rr) / a.G, h = g * a.G + (c0 + rr - tok * a.G);
        const float l = a.lse_in[static_cast<int64_t>(h) * a.T + t0 + tok];
        s.neg_lse[rr] = l == neg_inf() ? neg_inf() : -l * 1.4426950408889634f;
        s.mask[rr] = token_mask(a, t0, tok);
      }
      __syncthreads();
      for (int t = p.t0; t < p.t1; ++t) {
        const int j = t * kMassTile + tid, off = j - base;
        if (j >= keys) continue;
        float k[kD], w = 0.f;
        const float* src = cache_at(a, a.k_ptr, page_of(a, p.r, j), j, g, &s.status);
        if (src != nullptr) {
#pragma unroll
          for (int c = 0; c < kD / 4; ++c) {
            const float4 x = __ldg(reinterpret_cast<const float4*>(src) + c);
            k[4 * c] = x.x, k[4 * c + 1] = x.y, k[4 * c + 2] = x.z, k[4 * c + 3] = x.w;
          }
#pragma unroll 2
          for (int rr = 0; rr < n; ++rr) {
            if (s.neg_lse[rr] == neg_inf() || (off >= 0 && (off >= 64 || !((s.mask[rr] >> off) & 1)))) continue;
            float2 x0 = make_float2(0.f, 0.f), x1 = x0;
#pragma unroll
            for (int c = 0; c < kD / 4; ++c) {
              const float4 q4 = *reinterpret_cast<const float4*>(&s.q[rr][4 * c]);
              x0 = fma2(make_float2(q4.x, q4.y), make_float2(k[4 * c], k[4 * c + 1]), x0);
              x1 = fma2(make_float2(q4.z, q4.w), make_float2(k[4 * c + 2], k[4 * c + 3]), x1);
            }
            w += fast_exp2(fmaf((x0.x + x0.y) + (x1.x + x1.y), a.scale_log2, s.neg_lse[rr]));
          }
        }
        // (after the first pass: this thread's own sum)
        const float old = c0 > 0 ? a.mass_out[at + j] : (j < had ? a.mass_in[at + j] * a.decay : 0.f);
        a.mass_out[at + j] = old + w;
      }
    }
    u += p.t1 - p.t0;
  }
  store_status(a, &s.status);
}

}  // namespace

template <int NR>
static cudaError_t launch_rows(const DecodeArgs& a, const DecodePlan& P, cudaStream_t stream) {
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(tree_f32_kernel<NR>), sizeof(F32Shared<NR>));
  if (e != cudaSuccess) return e;
  return launch_chained(tree_f32_kernel<NR>, dim3(a.groups * a.Hkv), kThreads, sizeof(F32Shared<NR>), stream, 1, a, P);
}

cudaError_t launch_tree_f32(const DecodeArgs& a, const DecodePlan& P, cudaStream_t stream) {
  return a.max_rows <= 4   ? launch_rows<4>(a, P, stream)
         : a.max_rows <= 8 ? launch_rows<8>(a, P, stream)
                           : launch_rows<16>(a, P, stream);
}

cudaError_t launch_mass_f32(const DecodeArgs& a, const DecodePlan& P, cudaStream_t stream) {
  const int rows = a.max_rows < kMassRows ? a.max_rows : kMassRows;
  const size_t bytes = offsetof(MassF32Shared, q) + sizeof(float) * kD * rows;
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(mass_f32_kernel), sizeof(MassF32Shared));
  if (e != cudaSuccess) return e;
  return launch_chained(mass_f32_kernel, dim3(a.groups * a.Hkv), kThreads, bytes, stream, 1, a, P);
}

}  // namespace fp2
