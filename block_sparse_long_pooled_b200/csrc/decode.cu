// Attention of drafted tokens over a KV cache (one token: a decode step) with up to 16 query rows per KV
// head, and the join of what several CTAs have of one sequence.  More rows: tree_wide.cu.
//
// Sequence r has kv_len[r] keys, the last q_len of them its drafted tokens; token i sees every key
// before those and the drafted keys whose bit is set in its mask (no mask: those up to its own).
//
// The cache is read once and little else, so bytes bound it.  The work is one axis of units (sequence, row
// tile, key tile), the same for every KV head; kv_len lives on the device, so each CTA scans it and takes an
// equal share of that axis.  A grid of `groups` x KV heads puts the KV heads of one share side by side in
// time: their rows are neighbours in DRAM.  An (item = sequence, row tile) that several groups share leaves
// partial results in scratch, and join_kernel joins them in group order, so results do not depend on
// timing.  One producer warp brings K/V tiles in by TMA (page by page), four consumer warps run mma.sync on
// them: 16 rows are far below the 128 of a tcgen05 tile, and on that path the same calls were slower (three
// short requests 21 us against 15, a batch of 64 263 us against 247, when that was compared).
//
// Measured: 64 requests of 0.5K to 16K bf16 keys, one token each, 243 to 258 us, 5.6 to 6.0 TB/s (221 us at the
// copy's rate), as many e4m3 keys 217 us (114); three requests of 190 to 1000 keys 11 us, where the trips to
// memory one after another count: lengths, tile, statistics of the pieces, their rows.
#include "decode_device.cuh"

namespace fp2 {

namespace {

FP2_DEVICE void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
FP2_DEVICE void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// c += a (16x16) * b (16x8); bf16 operands, or f16 ones for an e4m3 cache.
template <bool F16>
FP2_DEVICE void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <int N>
FP2_DEVICE void consumer_sync() {  // the N consumer threads only (barrier 1)
  asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory");
}
// ------------------------------------------------------------------ operand fragments

// Address of 16-byte chunk c (of the D * ELT / 16 of a row) of row k in a K/V tile: boxes of 128
// bytes side by side, each with the 128-byte swizzle.
template <int TILE>
FP2_DEVICE uint32_t tile_addr(uint32_t base, int k, int c) {
  return base + (c >> 3) * (TILE * 128) + k * 128 + (((c & 7) ^ (k & 7)) << 4);
}

// e4m3 fragments.  ldmatrix moves units of 16 bits, here two neighbouring values of d.  For QK^T the
// order of d inside a group of 16 is free as long as Q agrees: a thread's four values 4q .. 4q+3
// (q = lane % 4) serve as k = 2q, 2q+1 and 2q+8, 2q+9, and stage_q stores Q in that order.  For PV
// the transposed unit holds d = 2n, 2n+1 of two keys; the bytes are regrouped by key into one
// fragment of the even d and one of the odd d.
FP2_DEVICE void widen_k(uint32_t w, uint32_t& b0, uint32_t& b1) {
  b0 = e4m3x2_to_f16x2(w & 0xFFFFu);
  b1 = e4m3x2_to_f16x2(w >> 16);
}
FP2_DEVICE void widen_v(uint32_t w, uint32_t& even, uint32_t& odd) {
  const uint32_t t = __byte_perm(w, 0, 0x3120);
  even = e4m3x2_to_f16x2(t & 0xFFFFu);
  odd = e4m3x2_to_f16x2(t >> 16);
}

// Query rows [row0, row0 + n) of (tokens from t0, KV head g) into shared memory as 16-bit operands,
// 16-byte chunks swizzled by row; rows from `rows` on are zero.
template <int DT, int D>
FP2_DEVICE uint32_t q_addr(uint32_t base, int row, int c) {
  return base + row * (D * 2) + ((c ^ (row & 7)) << 4);
}
template <int DT, int D, int NTHREADS>
FP2_DEVICE void stage_q(const DecodeArgs& a, char* q_smem, int t0, int g, int row0, int n, int rows, int tid) {
  constexpr int CH = D / 8;  // 16-byte chunks of a 16-bit row
  for (int i = tid; i < n * CH; i += NTHREADS) {
    const int rr = i / CH, c = i - rr * CH, m = row0 + rr;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (m < rows) {
      const int tok = m / a.G, h = g * a.G + (m - tok * a.G);
      const int64_t e = (static_cast<int64_t>(t0) + tok) * a.q_stride + static_cast<int64_t>(h) * D;
      if constexpr (DT == 1) {
        v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + e + 8 * c);
      } else {
        // chunk c holds k = 8 (c % 2) .. + 7 of group c / 2: values 4q + 2 (c % 2), + 1 for q = 0 .. 3
        const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.q) + e + 16 * (c >> 1));
        const uint32_t s = (c & 1) * 16;
        v.x = e4m3x2_to_f16x2((w.x >> s) & 0xFFFFu);
        v.y = e4m3x2_to_f16x2((w.y >> s) & 0xFFFFu);
        v.z = e4m3x2_to_f16x2((w.z >> s) & 0xFFFFu);
        v.w = e4m3x2_to_f16x2((w.w >> s) & 0xFFFFu);
      }
    }
    *reinterpret_cast<uint4*>(q_smem + rr * (D * 2) + ((c ^ (rr & 7)) << 4)) = v;
  }
}

// ------------------------------------------------------------------ tree attention

// Up to 16 rows per KV head in one tile; its 64 keys go to 4 warps, 16 each.
template <int DT, int D>
struct Tree {
  static constexpr int ELT = DT == 1 ? 2 : 1;
  static constexpr bool F16 = DT == 2;
  static constexpr int WN = 4, TILE = kFewTile;
  static constexpr int ROWS = kFewRows;
  static constexpr int CONSUMERS = 32 * WN;
  static constexpr int THREADS = CONSUMERS + 32;
  static constexpr int KV_BYTES = TILE * D * ELT;               // one of K or V
  static constexpr int STAGE_BYTES = 2 * KV_BYTES;
  static constexpr int Q_BYTES = ROWS * D * 2;
  static constexpr int OS = D + 8;                              // row stride of the joined output, floats
  static constexpr int O_BYTES = WN * ROWS * OS * 4;            // of every key warp
  static constexpr int FIXED = 1024 /* alignment */ + Q_BYTES + O_BYTES + WN * ROWS * 8 + (FP2_MAX_SEQS + 1) * 8 +
                               FP2_MAX_SEQS * 4 + 256;
  static constexpr int BUDGET = 113 * 1024;                     // two CTAs per SM
  static constexpr int RAW = (BUDGET - FIXED) / STAGE_BYTES;
  static constexpr int STAGES = RAW > 8 ? 8 : RAW;
  static constexpr int SMEM = FIXED + STAGES * STAGE_BYTES;
  // P is held in bf16 against a bf16 V.  Its rounding (up to 2^-8 of each weight) would be as large as the
  // output's own; few rows leave the tensor cores idle, so a second product adds the remainder
  // P - bf16(P), which costs nothing measurable (a batch of 64 requests: 246.7 us with it, 247.7 without).
  static constexpr bool SPLIT_P = DT == 1;
  // e4m3: P is f16, scaled by 2^8 so that weights down to 2^-22 of the largest keep all 11 bits; the
  // factor leaves with the division by the sum.
  static constexpr float P_BIAS = F16 ? 8.f : 0.f;
};

template <int DT, int D, bool SMALL>
__global__ void __launch_bounds__(Tree<DT, D>::THREADS, 2)
    tree_kernel(const __grid_constant__ DecodeArgs a, const __grid_constant__ DecodePlan P) {
  using C = Tree<DT, D>;
  extern __shared__ char smem_raw[];
  char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  char* stages = smem;
  char* q_smem = stages + C::STAGES * C::STAGE_BYTES;
  float* o_smem = reinterpret_cast<float*>(q_smem + C::Q_BYTES);
  float2* ml_smem = reinterpret_cast<float2*>(reinterpret_cast<char*>(o_smem) + C::O_BYTES);  // [WN][ROWS]
  long long* pre = reinterpret_cast<long long*>(ml_smem + C::WN * C::ROWS);
  int* len = reinterpret_cast<int*>(pre + FP2_MAX_SEQS + 1);
  __shared__ uint64_t full[C::STAGES], empty[C::STAGES], valid[C::STAGES];
  __shared__ int abort_flag;
  __shared__ uint32_t status_word;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = blockIdx.x % a.Hkv, grp = blockIdx.x / a.Hkv;
  grid_launch_next();
  if (tid == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 2);  // K and V
      mbar_init(&empty[s], C::CONSUMERS / 32);
    }
    abort_flag = 0;
    status_word = 0;
    fence_mbar_init();
    tma_prefetch_desc(&a.tm_k);
    tma_prefetch_desc(&a.tm_v);
  }
  grid_wait();
  __syncthreads();
  scan_units<C::TILE>(a, P, C::ROWS, 0, pre, len, &status_word);
  const long long units = pre[P.num_seqs];
  const int ng = active_groups(units, a.groups);
  if (grp >= ng) {
    if (g == 0 && tid == 0) a.desc[grp] = make_int4(-1, 0, 0, 0);
    store_status(a, &status_word);
    return;
  }
  const long long u0 = units * grp / ng, u1 = units * (grp + 1) / ng;

  if (warp == C::CONSUMERS / 32) {
    // ---------------- producer
    Producer<C::TILE, C::ELT, D, SMALL> load;
    int s = 0, it = 0;
    for (long long u = u0; u < u1;) {
      const Piece p = piece_at<C::TILE>(pre, len, P.num_seqs, u, u1);
      for (int t = p.t0; t < p.t1; ++t) {
        if (it >= C::STAGES) {
          // One answer for the warp: lanes that gave up and lanes that did not would wait for each other.
          const bool free = mbar_wait(&empty[s], ((it / C::STAGES) & 1) ^ 1, &abort_flag, &status_word, a.wait_limit_ns);
          if (!__all_sync(0xFFFFFFFFu, free)) goto drain;
        }
        const uint32_t k_at = smem_u32(stages + s * C::STAGE_BYTES);
        load.load(a, &a.tm_k, p.r, len[p.r], g, t * C::TILE, k_at, &full[s], &valid[s], &status_word, it == a.withhold);
        load.load(a, &a.tm_v, p.r, len[p.r], g, t * C::TILE, k_at + C::KV_BYTES, &full[s], &valid[s], &status_word, false);
        ++it;
        if (++s == C::STAGES) s = 0;
      }
      u += p.t1 - p.t0;
    }
  drain:
    // Copies in flight end before the CTA does: the consumers have waited for every tile, unless
    // they gave up, and then the issued ones are waited for here, within a fifth of the limit.
    if (*static_cast<volatile int*>(&abort_flag)) {
      volatile int no_abort = 0;
      for (int i = it > C::STAGES ? it - C::STAGES : 0; i < it; ++i)
        mbar_wait(&full[i % C::STAGES], (i / C::STAGES) & 1, &no_abort, &status_word, a.wait_limit_ns / 5);
    }
    store_status(a, &status_word);
    return;
  }

  // ---------------- consumers
  const int wn = warp;  // of the four key warps
  const uint32_t q_base = smem_u32(q_smem);
  int s = 0, it = 0, nth = 0;
  bool alive = true;
  for (long long u = u0; u < u1; ++nth) {
    const Piece p = piece_at<C::TILE>(pre, len, P.num_seqs, u, u1);
    const int keys = len[p.r], t0 = P.q_off[p.r], q_len = P.q_off[p.r + 1] - t0;
    const int row0 = p.rt * C::ROWS, rows = q_len * a.G;
    const int base = keys - q_len;  // first drafted key
    consumer_sync<C::CONSUMERS>();  // the previous piece is written: q_smem, o_smem and ml_smem are free
    stage_q<DT, D, C::CONSUMERS>(a, q_smem, t0, g, row0, C::ROWS, rows, tid);
    consumer_sync<C::CONSUMERS>();
    uint32_t qf[D / 16][4];  // the query fragments stay in registers
#pragma unroll
    for (int k = 0; k < D / 16; ++k) ldsm4(q_addr<DT, D>(q_base, lane & 15, 2 * k + (lane >> 4)), qf[k]);
    float o[D / 8][4], mx[2], sum[2];
    mx[0] = mx[1] = neg_inf();
    sum[0] = sum[1] = 0.f;
#pragma unroll
    for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;

    for (int t = p.t0; t < p.t1; ++t) {
      if (alive) alive = mbar_wait(&full[s], (it / C::STAGES) & 1, &abort_flag, &status_word, a.wait_limit_ns);
      if (!__all_sync(0xFFFFFFFFu, alive)) {
        alive = false;
        ++it;
        if (++s == C::STAGES) s = 0;
        continue;
      }
      const uint32_t k_at = smem_u32(stages + s * C::STAGE_BYTES), v_at = k_at + C::KV_BYTES;
      const int j0 = t * C::TILE + wn * 16;             // first of this warp's 16 keys
      const uint32_t here = static_cast<uint32_t>(valid[s] >> (wn * 16)) & 0xFFFFu;
      // Rows differ in what they see only from the first drafted key on.
      const bool plain = here == 0xFFFFu && j0 + 16 <= base;

      // S = Q K^T, 16 rows x 16 keys per row tile
      float sc[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        if constexpr (!C::F16) {
          uint32_t b[4];
          ldsm4(tile_addr<C::TILE>(k_at, wn * 16 + (lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)), b);
          mma<false>(sc[0], qf[k], b[0], b[1]);
          mma<false>(sc[1], qf[k], b[2], b[3]);
        } else if ((k & 1) == 0) {
          // matrices: keys 0-7 and 8-15 of chunk k, then of chunk k + 1
          uint32_t b[4];
          ldsm4(tile_addr<C::TILE>(k_at, wn * 16 + (lane & 15), k + (lane >> 4)), b);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t b00, b01, b10, b11;
            widen_k(b[2 * c], b00, b01);
            widen_k(b[2 * c + 1], b10, b11);
            mma<true>(sc[0], qf[k + c], b00, b01);
            mma<true>(sc[1], qf[k + c], b10, b11);
          }
        }
      }

      // Masks, the running maximum and the weights
      uint32_t pf[4], pl[4];
      uint32_t vis[2];
      vis[0] = vis[1] = here;
      if (!plain) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = row0 + (lane >> 2) + 8 * i;
          vis[i] = row < rows && keys > 0 ? here & seen16(token_mask(a, t0, row / a.G), j0, base) : 0u;
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (!((vis[i] >> (8 * n + 2 * (lane & 3) + e)) & 1u)) sc[n][2 * i + e] = neg_inf();
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float v = fmaxf(fmaxf(sc[0][2 * i], sc[0][2 * i + 1]), fmaxf(sc[1][2 * i], sc[1][2 * i + 1]));
        v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
        v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
        const float now = fmaxf(mx[i], v);
        if (__any_sync(0xFFFFFFFFu, now > mx[i])) {
          // exp2(-inf) = 0 clears a row that had seen nothing; a row that still has keeps its zeros.
          const float f = now == neg_inf() ? 1.f : fast_exp2((mx[i] - now) * a.scale_log2);
          sum[i] *= f;
#pragma unroll
          for (int n = 0; n < D / 8; ++n) {
            o[n][2 * i] *= f;
            o[n][2 * i + 1] *= f;
          }
          mx[i] = now;
        }
        const float off = now == neg_inf() ? 0.f : C::P_BIAS - now * a.scale_log2;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float e0 = fast_exp2(fmaf(sc[n][2 * i], a.scale_log2, off));
          const float e1 = fast_exp2(fmaf(sc[n][2 * i + 1], a.scale_log2, off));
          sum[i] += e0 + e1;
          const uint32_t w = C::F16 ? pack_f16x2(e0, e1) : pack_bf16x2(e0, e1);
          pf[2 * n + i] = w;
          if constexpr (C::SPLIT_P)
            pl[2 * n + i] = pack_bf16x2(e0 - __uint_as_float(w << 16), e1 - __uint_as_float(w & 0xFFFF0000u));
        }
      }

      // O += P V.  Rows of V that hold no key are cleared (0 x NaN is NaN).  A drafted key's row that
      // is not finite would reach rows that do not see it the same way: its values are cleared too and
      // added afterwards to the rows that do see the key.
      uint32_t clr[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
      if (!plain) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t two = here >> (2 * (lane & 3) + 8 * i);
          clr[i] = ((two & 1u) ? 0xFFFFu : 0u) | ((two & 2u) ? 0xFFFF0000u : 0u);
        }
      }
      const auto pv = [&](int n, uint32_t b0, uint32_t b1) {  // accumulator n, keys 0-7 and 8-15 of the warp's 16
        if (!plain) {
          b0 &= clr[0];
          b1 &= clr[1];
          constexpr uint32_t EXP = C::F16 ? 0x7C00u : 0x7F80u;
          const uint32_t b[2] = {b0, b1};
          uint32_t bad[4];
          bool any = false;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t h = (b[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
            bad[e] = (h & EXP) == EXP ? h : 0u;
            any |= bad[e] != 0;
          }
          if (__any_sync(0xFFFFFFFFu, any)) {
            // How many seen keys of each row hold +inf, -inf or NaN, as products of 0/1 operands.
            constexpr uint32_t ONE = C::F16 ? 0x3C00u : 0x3F80u;
            if (bad[0]) b0 &= 0xFFFF0000u;
            if (bad[1]) b0 &= 0xFFFFu;
            if (bad[2]) b1 &= 0xFFFF0000u;
            if (bad[3]) b1 &= 0xFFFFu;
#pragma unroll
            for (int kind = 0; kind < 3; ++kind) {
              uint32_t f[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                f[e] = (kind == 0 ? bad[e] == EXP : kind == 1 ? bad[e] == (EXP | 0x8000u) : (bad[e] & 0x7FFFu) > EXP)
                           ? ONE : 0u;
              uint32_t va[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t two = vis[e & 1] >> (2 * (lane & 3) + 8 * (e >> 1));
                va[e] = ((two & 1u) ? ONE : 0u) | ((two & 2u) ? ONE << 16 : 0u);
              }
              float cnt[4] = {0.f, 0.f, 0.f, 0.f};
              mma<C::F16>(cnt, va, f[0] | (f[1] << 16), f[2] | (f[3] << 16));
              const float add = kind == 0 ? pos_inf() : kind == 1 ? neg_inf() : __uint_as_float(0x7FFFFFFFu);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (cnt[e] > 0.f) o[n][e] += add;
            }
          }
        }
        mma<C::F16>(o[n], pf, b0, b1);
        if constexpr (C::SPLIT_P) mma<C::F16>(o[n], pl, b0, b1);
      };
      if constexpr (!C::F16) {
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
          uint32_t b[4];
          ldsm4t(tile_addr<C::TILE>(v_at, wn * 16 + (lane & 15), 2 * n + (lane >> 4)), b);
          pv(2 * n, b[0], b[1]);
          pv(2 * n + 1, b[2], b[3]);
        }
      } else {
        // a 16-byte chunk is 16 values of d: accumulator 2c takes its even ones, 2c + 1 its odd ones
#pragma unroll
        for (int n = 0; n < D / 32; ++n) {
          uint32_t b[4], even[4], odd[4];
          ldsm4t(tile_addr<C::TILE>(v_at, wn * 16 + (lane & 15), 2 * n + (lane >> 4)), b);
#pragma unroll
          for (int e = 0; e < 4; ++e) widen_v(b[e], even[e], odd[e]);
          pv(4 * n, even[0], even[1]);
          pv(4 * n + 1, odd[0], odd[1]);
          pv(4 * n + 2, even[2], even[3]);
          pv(4 * n + 3, odd[2], odd[3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
      ++it;
      if (++s == C::STAGES) s = 0;
    }

    // The four key warps lay down what they have of each row; whoever writes the row adds it up.  (Adding
    // it up in shared memory warp by warp cost four barriers more, 0.6 us of a decode step's 6.)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float x = sum[i];
      x += __shfl_xor_sync(0xFFFFFFFFu, x, 1);
      x += __shfl_xor_sync(0xFFFFFFFFu, x, 2);
      const int row = (lane >> 2) + 8 * i;
      if ((lane & 3) == 0) ml_smem[wn * C::ROWS + row] = make_float2(mx[i], x);
      if (row0 + row >= rows) continue;
      float* dst = o_smem + (wn * C::ROWS + row) * C::OS;
      if constexpr (!C::F16) {
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
          *reinterpret_cast<float2*>(dst + 8 * n + 2 * (lane & 3)) = make_float2(o[n][2 * i], o[n][2 * i + 1]);
      } else {
        // columns 2q, 2q+1 of the even and odd accumulators are d = 4q, 4q+2 and 4q+1, 4q+3
#pragma unroll
        for (int n = 0; n < D / 16; ++n)
          *reinterpret_cast<float4*>(dst + 16 * n + 4 * (lane & 3)) =
              make_float4(o[2 * n][2 * i], o[2 * n + 1][2 * i], o[2 * n][2 * i + 1], o[2 * n + 1][2 * i + 1]);
      }
    }
    consumer_sync<C::CONSUMERS>();

    // Out: the whole item, or this group's part of it.
    const bool whole = p.t0 == 0 && p.t1 == p.tiles;
    const int slot = (grp * a.Hkv + g) * 2 + (nth == 0 ? 0 : 1);
    constexpr int LANES = D / 4;  // threads of a row, four values each
    for (int i = tid; i < C::ROWS * LANES; i += C::CONSUMERS) {
      const int rr = i / LANES, c = (i - rr * LANES) * 4, m = row0 + rr;
      if (m >= rows) continue;
      float top = neg_inf(), total = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < C::WN; ++w) top = fmaxf(top, ml_smem[w * C::ROWS + rr].x);
#pragma unroll
      for (int w = 0; w < C::WN; ++w) {
        const float2 x = ml_smem[w * C::ROWS + rr];
        // a warp that saw nothing has the sum 0; one whose scores are all NaN has the maximum -inf too
        if (x.y == 0.f) continue;
        const float f = fast_exp2((x.x - top) * a.scale_log2);
        const float4 part = *reinterpret_cast<const float4*>(o_smem + (w * C::ROWS + rr) * C::OS + c);
        total += x.y * f;
        v.x += part.x * f;
        v.y += part.y * f;
        v.z += part.z * f;
        v.w += part.w * f;
      }
      if (whole) {
        const int tok = m / a.G, h = g * a.G + (m - tok * a.G);
        const float f = total == 0.f ? 0.f : a.v_descale / total;
        const int64_t row = static_cast<int64_t>(t0) + tok;
        if (fp2_check(row < a.T && h < a.Hq, &status_word)) {
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + (row * a.Hq + h) * D + c) =
              make_uint2(pack_bf16x2(v.x * f, v.y * f), pack_bf16x2(v.z * f, v.w * f));
          if (c == 0 && a.lse != nullptr)
            a.lse[static_cast<int64_t>(h) * a.T + row] =
                total == 0.f ? neg_inf() : (top * a.scale_log2 - C::P_BIAS + log2f(total)) * kLn2;
        }
      } else {
        *reinterpret_cast<float4*>(a.part_o + (static_cast<int64_t>(slot) * C::ROWS + rr) * D + c) = v;
        if (c == 0)
          a.part_ml[static_cast<int64_t>(slot) * C::ROWS + rr] =
              make_float2(top == neg_inf() ? top : top * a.scale_log2 - C::P_BIAS, total);
      }
    }
    // The group that holds an item's first piece tells join_kernel how many follow.
    u += p.t1 - p.t0;
    if (g == 0 && tid == 0 && u >= u1) {
      int4 d = make_int4(-1, 0, 0, 0);
      if (p.t0 == 0 && p.t1 < p.tiles) {
        d = make_int4(nth == 0 ? 0 : 1, p.r, p.rt, group_of(units, ng, u1 + (p.tiles - p.t1) - 1) - grp + 1);
      }
      a.desc[grp] = d;
    }
  }
  store_status(a, &status_word);
}

// Joins the pieces of an item that several groups worked on, in group order,
// o = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i: WARPS warps per row, each an equal run of the pieces; the
// first then adds up what the others have.
template <int D, int WARPS>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ DecodeArgs a,
                                                   const __grid_constant__ DecodePlan P) {
  grid_launch_next();
  grid_wait();
  const int g = blockIdx.x % a.Hkv, grp = blockIdx.x / a.Hkv;
  const int4 d = a.desc[grp];
  if (d.x < 0) return;
  constexpr int ROWS = 4 / WARPS;  // of a block
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rr = blockIdx.y * ROWS + warp / WARPS, part = warp % WARPS;
  const int t0 = P.q_off[d.y], rows = (P.q_off[d.y + 1] - t0) * a.G, m = d.z * a.part_rows + rr;
  if (m >= rows) return;
  const auto at = [&](int i) {  // row of piece i in the partial buffers
    const int64_t slot = (static_cast<int64_t>(grp + i) * a.Hkv + g) * 2 + (i == 0 ? d.x : 0);
    return slot * a.part_rows + rr;
  };
  constexpr int V = D / 32;
  float acc[V], total = 0.f, top = neg_inf();
  bool some = false;  // a piece so far saw a key of this row
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = 0.f;
  // Up to 32 pieces at a time, lane i with the statistics of piece i; all their rows are on their way
  // together, 16 at a time.
  const int first = d.w * part / WARPS, last = d.w * (part + 1) / WARPS;
  for (int i0 = first; i0 < last; i0 += 32) {
    const int n = min(32, last - i0);
    const float2 ml = lane < n ? a.part_ml[at(i0 + lane)] : make_float2(neg_inf(), 0.f);
    float x[16][V];
    const auto fetch = [&](int i1) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (i1 + i >= n) break;
        const float* src = a.part_o + at(i0 + i1 + i) * D + lane * V;
        if constexpr (V == 4) {
          const float4 v = *reinterpret_cast<const float4*>(src);
          x[i][0] = v.x, x[i][1] = v.y, x[i][2] = v.z, x[i][3] = v.w;
        } else {
          const float2 v = *reinterpret_cast<const float2*>(src);
          x[i][0] = v.x, x[i][1] = v.y;
        }
      }
    };
    fetch(0);
    float now = ml.x;
#pragma unroll
    for (int o = 16; o; o >>= 1) now = fmaxf(now, __shfl_xor_sync(0xFFFFFFFFu, now, o));
    now = fmaxf(now, top);
    // What came before, if anything did: a piece whose scores were all NaN has a sum but no maximum, and one whose
    // factor underflows to 0 still hands on an infinity or a NaN of a value (0 x NaN).
    const float f = some ? fast_exp2(top - now) : 0.f;
    total = some ? total * f : 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = some ? acc[e] * f : 0.f;
    top = now;
    // a piece that saw nothing of the row has the sum 0 and may not even have written its part_o
    const bool saw = !(ml.y == 0.f);
    const float w = saw ? fast_exp2(ml.x - top) : 0.f;
    float sum = saw ? w * ml.y : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    total += sum;
    const uint32_t seen = __ballot_sync(0xFFFFFFFFu, saw);
    some |= seen != 0;
    for (int i1 = 0; i1 < n; i1 += 16) {
      if (i1 > 0) fetch(i1);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (i1 + i >= n) break;
        const float wi = __shfl_sync(0xFFFFFFFFu, w, i1 + i);
        const bool use = (seen >> (i1 + i)) & 1u;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] += use ? wi * x[i][e] : 0.f;
      }
    }
  }
  if constexpr (WARPS > 1) {
    __shared__ float sums[WARPS][D], tops[WARPS], totals[WARPS];
#pragma unroll
    for (int e = 0; e < V; ++e) sums[part][lane * V + e] = acc[e];
    if (lane == 0) tops[part] = top, totals[part] = total;
    __syncthreads();  // (a block has one row: all its warps come here or none)
    if (part != 0) return;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) top = fmaxf(top, tops[w]);
    total = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      if (totals[w] == 0.f) continue;
      const float f = fast_exp2(tops[w] - top);
      total += totals[w] * f;
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] += sums[w][lane * V + e] * f;
    }
  }
  const int tok = m / a.G, h = g * a.G + (m - tok * a.G);
  const int64_t row = static_cast<int64_t>(t0) + tok;
  const float f = total == 0.f ? 0.f : a.v_descale / total;
  // the word of the attention CTA with this index, written before this kernel went on
  if (!fp2_check(row < a.T && h < a.Hq, a.scratch + kStatusFirst + blockIdx.x)) return;
  const int64_t to = (row * a.Hq + h) * D + lane * V;
  if (a.out_f32) {
#pragma unroll
    for (int e = 0; e < V; ++e) static_cast<float*>(a.out)[to + e] = acc[e] * f;
  } else {
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + to);
#pragma unroll
    for (int e = 0; e < V / 2; ++e) dst[e] = pack_bf16x2(acc[2 * e] * f, acc[2 * e + 1] * f);
  }
  if (lane == 0 && a.lse != nullptr)
    a.lse[static_cast<int64_t>(h) * a.T + row] = total == 0.f ? neg_inf() : (top + log2f(total)) * kLn2;
}

template <int DT, int D>
cudaError_t run_tree(const DecodeArgs& a, const DecodePlan& P, cudaStream_t stream) {
  using C = Tree<DT, D>;
  static_assert(C::STAGES >= 2, "tiles must fit twice");
  const auto kernel = a.box_rows < 64 ? tree_kernel<DT, D, true> : tree_kernel<DT, D, false>;
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_chained(kernel, dim3(a.groups * a.Hkv), C::THREADS, C::SMEM, stream, 1, a, P);
}

}  // namespace

cudaError_t launch_tree_few(int dtype, int D, const DecodeArgs& a, const DecodePlan& P, cudaStream_t stream) {
  if (dtype == FP2_BF16 && D == 128) return run_tree<1, 128>(a, P, stream);
  if (dtype == FP2_BF16 && D == 64) return run_tree<1, 64>(a, P, stream);
  if (dtype == FP2_E4M3 && D == 128) return run_tree<2, 128>(a, P, stream);
  return cudaErrorInvalidValue;
}

cudaError_t launch_tree_join(int D, int max_rows, const DecodeArgs& a, const DecodePlan& P, cudaStream_t stream) {
  const int rows = max_rows < a.part_rows ? max_rows : a.part_rows;
  const dim3 grid(a.groups * a.Hkv, a.join_warps == 4 ? rows : (rows + 3) / 4);
  const auto kernel = D == 128 ? (a.join_warps == 4 ? join_kernel<128, 4> : join_kernel<128, 1>)
                               : (a.join_warps == 4 ? join_kernel<64, 4> : join_kernel<64, 1>);
  return launch_chained(kernel, grid, 128, 0, stream, 1, a, P);
}

}  // namespace fp2
