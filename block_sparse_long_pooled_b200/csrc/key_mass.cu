// The attention weight that each cached key receives from a call's tokens (fp2_key_mass):
//   mass'[r, g, j] = decay * mass[r, g, j] + sum over the rows that see key j of exp(q . k_j scale - lse).
//
// Keys are the M side: S^T = K Q^T puts a key in a lane of tensor memory and its up to 128 query rows in
// the columns, so that the sum over rows stays inside one thread: no shuffles, no atomics, one order.  K
// is read once, the weights once and written once; bytes bound the call up to some 200 rows per KV head,
// above that the exponentials (128 x 128 of them take the SM 1024 cycles, its share of a bf16 K tile
// 1400).  A pass has the whole tokens that fit into 128 rows (their heads of the group side by side, as
// a TMA box of Q brings them); more tokens take several passes over a CTA's keys, which come from L2 then.
//
// Units as in decode.cu: (sequence, key tile of 128), weighted by the sequence's passes.  Warps: 0-3 and
// 4-7 take the even and the odd tiles out of tensor memory; 8 loads K; 9 issues the products; 10 and 11
// bring Q, -lse and the masks of the next pass into the second of two buffers while the current one is
// worked on.  Measured: 32 tokens by 4 heads over 64K bf16 keys, 8 KV heads, 35 us (21 us of bytes);
// one token of 32 sequences over 200 to 8K e4m3 keys 28 us (14 us of bytes), of which 17 in the tiles at
// 5.3 TB/s and the rest before the first and after the last.
#include "decode_device.cuh"

namespace fp2 {

namespace {

template <int DT, int D>
struct Mass {
  static constexpr bool E4 = DT == 2;
  static constexpr int ELT = E4 ? 1 : 2;
  static constexpr int TILE = kMassTile, ROWS = kMassRows;
  static constexpr int KCH = 128 / ELT;                 // elements of a 128-byte swizzled row
  static constexpr int KIND = E4 ? 2 : 1, UK = 32 / ELT;
  static constexpr uint32_t FMT = E4 ? 0u : 1u;
  static constexpr int Q_BYTES = ROWS * D * ELT, K_BYTES = TILE * D * ELT;
  static constexpr int STAGES = E4 || D == 64 ? 8 : 4;
  static constexpr int OFF_Q = 0;                       // [2]
  static constexpr int OFF_K = 2 * Q_BYTES;             // [STAGES]
  static constexpr int OFF_LSE = OFF_K + STAGES * K_BYTES;            // [2][ROWS] -lse in log2 units
  static constexpr int OFF_MASK = OFF_LSE + 2 * ROWS * 4;             // [2][ROWS]
  static constexpr int OFF_PRE = OFF_MASK + 2 * ROWS * 8;
  static constexpr int OFF_LEN = OFF_PRE + (FP2_MAX_SEQS + 1) * 8;
  static constexpr int SMEM_RAW = OFF_LEN + FP2_MAX_SEQS * 4 + 1024;
  static constexpr int SMEM = SMEM_RAW > 116 * 1024 ? SMEM_RAW : 116 * 1024;   // one CTA per SM
  static_assert(SMEM <= 226 * 1024, "shared memory");
};
constexpr int kMassThreads = 384;

// Key tiles [t0, t1) of sequence r; a unit is (key tile, pass).
struct MassPiece {
  int r, passes, t0, t1;
  long long next;
};
FP2_DEVICE MassPiece mass_piece(const long long* pre, const int* len, const DecodeArgs& a, const DecodePlan& P,
                                long long u, long long u1) {
  int lo = 0, hi = P.num_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= u) lo = mid; else hi = mid - 1;
  }
  MassPiece p;
  p.r = lo;
  const int tiles = len[lo] <= 0 ? 1 : (len[lo] + kMassTile - 1) / kMassTile;
  p.passes = max(1, (P.q_off[lo + 1] - P.q_off[lo] + a.pass_tokens - 1) / a.pass_tokens);
  const int off = static_cast<int>(u - pre[lo]);
  const long long left = u1 - u;
  const int end = tiles * p.passes - off <= left ? tiles * p.passes : off + static_cast<int>(left);
  p.t0 = (off + p.passes - 1) / p.passes;
  p.t1 = (end + p.passes - 1) / p.passes;
  p.next = u + (end - off);
  return p;
}

FP2_DEVICE void ld16_now(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

FP2_DEVICE void ld32_now(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

template <int DT, int D, bool SMALL>
__global__ void __launch_bounds__(kMassThreads, 1)
    mass_kernel(const __grid_constant__ DecodeArgs a, const __grid_constant__ DecodePlan P) {
  using C = Mass<DT, D>;
  extern __shared__ char smem_raw[];
  char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = smem_u32(smem);
  float* neg_lse = reinterpret_cast<float*>(smem + C::OFF_LSE);
  uint64_t* masks = reinterpret_cast<uint64_t*>(smem + C::OFF_MASK);
  long long* pre = reinterpret_cast<long long*>(smem + C::OFF_PRE);
  int* len = reinterpret_cast<int*>(smem + C::OFF_LEN);
  __shared__ uint64_t k_full[C::STAGES], k_empty[C::STAGES], q_full[2], l_full[2], q_empty[2], s_full[4], s_free[4], all_done;
  // Which rows of a K tile hold keys.  Read after its stage is released: then the products of tile
  // x - STAGES are issued, so each half of the warps is past the tile three of its own before that one.
  constexpr int VALID = 16;
  static_assert(VALID >= C::STAGES + 7, "ring of masks");
  __shared__ uint64_t valid[VALID][2];
  __shared__ int any_empty[2];                // some row of the buffer saw nothing
  __shared__ int abort_flag;
  __shared__ uint32_t status_word, tmem_slot;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = blockIdx.x % a.Hkv, grp = blockIdx.x / a.Hkv;
  grid_launch_next();
  if (tid == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&q_full[b], 1);
      mbar_init(&l_full[b], 2);
      mbar_init(&q_empty[b], 9);   // the MMA warp and eight warps that read -lse and masks
    }
    for (int b = 0; b < 4; ++b) {  // [half of the warps][buffer]
      mbar_init(&s_full[b], 1);
      mbar_init(&s_free[b], 4);
    }
    mbar_init(&all_done, 1);
    abort_flag = 0;
    status_word = 0;
    fence_mbar_init();
    tma_prefetch_desc(&a.tm_k);
    tma_prefetch_desc(&a.tm_q);
  }
  if (warp == 8) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  grid_wait();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  // A sequence without tokens counts as one pass: its weights still decay.
  scan_units<C::TILE>(a, P, a.pass_tokens * a.G, 1, pre, len, &status_word);
  const long long units = pre[P.num_seqs];
  const int ng = active_groups(units, a.groups);
  const bool idle = grp >= ng;
  const long long u0 = idle ? 0 : units * grp / ng, u1 = idle ? 0 : units * (grp + 1) / ng;
  const int pass_rows = a.pass_tokens * a.G;
  const auto wait = [&](uint64_t* bar, uint32_t parity) {  // one answer for the warp
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, &abort_flag, &status_word, a.wait_limit_ns));
  };

  if (warp == 8) {
    // ---------------------------------------------------------------- producer
    Producer<C::TILE, C::ELT, D, SMALL> load;
    int it = 0;
    bool alive = true;
    for (long long u = u0; u < u1 && alive;) {
      const MassPiece p = mass_piece(pre, len, a, P, u, u1);
      for (int pass = 0; pass < p.passes && alive; ++pass)
        for (int t = p.t0; t < p.t1; ++t, ++it) {
          const int st = it % C::STAGES, round = it / C::STAGES;
          if (round > 0 && !(alive = wait(&k_empty[st], (round - 1) & 1))) break;
          load.load(a, &a.tm_k, p.r, len[p.r], g, t * C::TILE, sbase + C::OFF_K + st * C::K_BYTES, &k_full[st],
                    valid[it % VALID], &status_word, it == a.withhold);
        }
      u = p.next;
    }
    // Copies in flight end before the CTA does.
    if (*static_cast<volatile int*>(&abort_flag)) {
      volatile int no_abort = 0;
      for (int i = max(0, it - C::STAGES); i < it; ++i)
        mbar_wait(&k_full[i % C::STAGES], (i / C::STAGES) & 1, &no_abort, &status_word, a.wait_limit_ns / 5);
    }
  } else if (warp == 9) {
    // ---------------------------------------------------------------- MMA issuer
    int it = 0, nq = 0, uses[2] = {0, 0};
    bool alive = true;
    for (long long u = u0; u < u1 && alive;) {
      const MassPiece p = mass_piece(pre, len, a, P, u, u1);
      const int rows = (P.q_off[p.r + 1] - P.q_off[p.r]) * a.G;
      for (int pass = 0; pass < p.passes && alive && p.t0 < p.t1; ++pass, ++nq) {
        const int qb = nq & 1, n = min(pass_rows, rows - pass * pass_rows);
        if (!(alive = wait(&q_full[qb], (nq >> 1) & 1))) break;
        tc_fence_after();
        const uint64_t qd = smem_desc_sw128(sbase + C::OFF_Q + qb * C::Q_BYTES, 16, 1024);
        const uint32_t idesc = make_idesc(C::FMT, C::FMT, 0, 0, 128, max(16, (n + 15) / 16 * 16));
        for (int t = p.t0; t < p.t1; ++t, ++it) {
          const int st = it % C::STAGES, use = uses[t & 1]++, b = 2 * (t & 1) + (use & 1);
          if (!(alive = wait(&k_full[st], (it / C::STAGES) & 1))) break;
          if (use >= 2 && !(alive = wait(&s_free[b], ((use >> 1) - 1) & 1))) break;
          tc_fence_after();
          const uint64_t kd = smem_desc_sw128(sbase + C::OFF_K + st * C::K_BYTES, 16, 1024);
#pragma unroll
          for (int k = 0; k < D / C::UK; ++k) {
            const uint64_t off =
                static_cast<uint64_t>(((k * C::UK / C::KCH) * (128 * 128) + (k * C::UK % C::KCH) * C::ELT) >> 4);
            umma_ss_warp<C::KIND>(tmem + b * 128, kd + off, qd + off, idesc, k > 0 ? 1u : 0u);
          }
          umma_commit_warp(&s_full[b]);
          umma_commit_warp(&k_empty[st]);
        }
        umma_commit_warp(&q_empty[qb]);
      }
      u = p.next;
    }
    // No product in flight when the CTA ends.
    umma_commit_warp(&all_done);
    volatile int no_abort = 0;
    mbar_wait(&all_done, 0, &no_abort, &status_word, a.wait_limit_ns / 5);
  } else if (warp >= 10) {
    // ---------------------------------------------------------------- Q, -lse and masks of a pass
    const int t64 = tid - 320;
    int nq = 0;
    bool alive = true;
    for (long long u = u0; u < u1 && alive;) {
      const MassPiece p = mass_piece(pre, len, a, P, u, u1);
      const int tok0 = P.q_off[p.r], rows = (P.q_off[p.r + 1] - tok0) * a.G;
      for (int pass = 0; pass < p.passes && p.t0 < p.t1; ++pass, ++nq) {
        const int qb = nq & 1, row0 = pass * pass_rows, n = min(pass_rows, rows - row0);
        if (nq >= 2 && !(alive = wait(&q_empty[qb], ((nq >> 1) - 1) & 1))) break;
        // Rows past the sequence's tokens are other tokens' (or zeros past Q's end): columns nobody reads.
        if (t64 == 0 && n <= 0) mbar_arrive(&q_full[qb]);
        if (t64 == 0 && n > 0) {
          mbar_arrive_expect_tx(&q_full[qb], pass_rows * D * C::ELT);
#pragma unroll
          for (int b = 0; b < D / C::KCH; ++b)
            tma_load_3d(smem + C::OFF_Q + qb * C::Q_BYTES + b * (C::ROWS * 128), &a.tm_q, &q_full[qb], b * C::KCH, g * a.G,
                        tok0 + pass * a.pass_tokens);
        }
        bool empty = false;
#pragma unroll
        for (int i = 0; i < C::ROWS / 64; ++i) {
          const int rr = t64 + 64 * i;
          float x = neg_inf();  // rows that are none, or saw nothing
          uint64_t m = 0;
          if (rr < n) {
            const int tok = (row0 + rr) / a.G, h = g * a.G + (row0 + rr - tok * a.G);
            const float l = a.lse_in[static_cast<int64_t>(h) * a.T + tok0 + tok];
            m = token_mask(a, tok0, tok);
            if (l != neg_inf()) x = -l * 1.4426950408889634f;
            empty |= x == neg_inf();
          }
          neg_lse[qb * C::ROWS + rr] = x;
          masks[qb * C::ROWS + rr] = m;
        }
        // each of the two warps has half of the word
        const uint32_t some = __any_sync(0xFFFFFFFFu, empty);
        if (lane == 0) reinterpret_cast<uint16_t*>(&any_empty[qb])[warp - 10] = some ? 1 : 0;
        __syncwarp();
        if (lane == 0) mbar_arrive(&l_full[qb]);
      }
      u = p.next;
    }
    // Q's last copies, if nobody waited for them
    if (t64 == 0 && *static_cast<volatile int*>(&abort_flag)) {
      volatile int no_abort = 0;
      for (int i = max(0, nq - 2); i < nq; ++i)
        mbar_wait(&q_full[i & 1], (i >> 1) & 1, &no_abort, &status_word, a.wait_limit_ns / 5);
    }
  } else {
    // ---------------------------------------------------------------- thread = key: weights of a tile
    const int half = warp >> 2, kt = tid & 127;
    const uint32_t s_at = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + half * 256;
    int it = 0, nq = 0, use = 0;
    bool alive = true;
    for (long long u = u0; u < u1;) {
      const MassPiece p = mass_piece(pre, len, a, P, u, u1);
      const int keys = len[p.r], q_len = P.q_off[p.r + 1] - P.q_off[p.r], rows = q_len * a.G, base = keys - q_len;
      const int had = a.mass_in == nullptr ? 0 : min(keys, a.mass_len != nullptr ? a.mass_len[p.r] : keys);
      const int64_t at = (static_cast<int64_t>(p.r) * a.Hkv + g) * a.mass_stride;
      for (int pass = 0; pass < p.passes && p.t0 < p.t1; ++pass, ++nq) {
        const int qb = nq & 1, n = min(pass_rows, rows - pass * pass_rows);
        // Old weights (after the first pass: this thread's own sums) are loaded a tile ahead.
        const auto old_weight = [&](int t) {
          const int j = t * C::TILE + kt;
          if (t >= p.t1 || j >= (pass > 0 ? keys : had)) return 0.f;
          return pass > 0 ? a.mass_out[at + j] : a.mass_in[at + j];
        };
        const float decay = pass > 0 ? 1.f : a.decay;
        const int first = p.t0 + ((p.t0 ^ half) & 1);
        float ahead = old_weight(first);
        if (alive) alive = wait(&l_full[qb], (nq >> 1) & 1);
        const bool whole_rows = n > 0 && any_empty[qb] == 0;
        const float* off = neg_lse + qb * C::ROWS;
        const uint64_t* mk = masks + qb * C::ROWS;
        for (int t = first; t < p.t1; t += 2, ++use) {
          const int j = t * C::TILE + kt, b = use & 1;
          const float old = ahead;
          ahead = old_weight(t + 2);
          if (alive) alive = wait(&s_full[2 * half + b], (use >> 1) & 1);
          if (!alive) continue;
          tc_fence_after();
          const bool plain = whole_rows && (t + 1) * C::TILE <= base;
          const bool here = (valid[(it + t - p.t0) % VALID][kt >> 6] >> (kt & 63)) & 1;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
          int c0 = 0;
          if (plain) {
#pragma unroll 1
            for (; c0 + 32 <= n; c0 += 32) {
              uint32_t v[32];
              ld32_now(s_at + b * 128 + c0, v);
              const float2 s2 = make_float2(a.scale_log2, a.scale_log2);
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 o = *reinterpret_cast<const float4*>(off + c0 + e);
                const float2 x = __ffma2_rn(make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), s2,
                                            make_float2(o.x, o.y));
                const float2 y = __ffma2_rn(make_float2(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])), s2,
                                            make_float2(o.z, o.w));
                sum[0] += fast_exp2(x.x);
                sum[1] += fast_exp2(x.y);
                sum[2] += fast_exp2(y.x);
                sum[3] += fast_exp2(y.y);
              }
            }
          }
#pragma unroll 1
          for (; c0 < n; c0 += 16) {
            uint32_t v[16];
            ld16_now(s_at + b * 128 + c0, v);
            if (plain) {
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (c0 + e < n) sum[e & 3] += fast_exp2(fmaf(__uint_as_float(v[e]), a.scale_log2, off[c0 + e]));
            } else {
              // Rows that saw nothing, and keys that not every token sees: first which, then their weights.
              const int d = j - base;
              uint32_t sees = 0;
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const uint32_t bit = d < 0 ? 1u : static_cast<uint32_t>(mk[c0 + e] >> (d & 63)) & 1u;
                if (off[c0 + e] != neg_inf()) sees |= bit << e;  // (columns of no row are -inf too)
              }
              if (d >= 64) sees = 0;
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float x = fast_exp2(fmaf(__uint_as_float(v[e]), a.scale_log2, off[c0 + e]));
                sum[e & 3] += (sees >> e) & 1u ? x : 0.f;
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_free[2 * half + b]);
          // A key of a page that is not there keeps its weight; its status bit is set.
          if (j < keys) a.mass_out[at + j] = old * decay + (here ? (sum[0] + sum[1]) + (sum[2] + sum[3]) : 0.f);
        }
        it += p.t1 - p.t0;
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_empty[qb]);
      }
      u = p.next;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, 512);
  store_status(a, &status_word);
}

template <int DT, int D>
cudaError_t run_mass(const DecodeArgs& a, const DecodePlan& P, cudaStream_t stream) {
  using C = Mass<DT, D>;
  const auto kernel = a.box_rows < 64 ? mass_kernel<DT, D, true> : mass_kernel<DT, D, false>;
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_chained(kernel, dim3(a.groups * a.Hkv), kMassThreads, C::SMEM, stream, 1, a, P);
}

}  // namespace

cudaError_t launch_key_mass(int dtype, int D, const DecodeArgs& a, const DecodePlan& P, cudaStream_t stream) {
  if (dtype == FP2_BF16 && D == 128) return run_mass<1, 128>(a, P, stream);
  if (dtype == FP2_BF16 && D == 64) return run_mass<1, 64>(a, P, stream);
  if (dtype == FP2_E4M3 && D == 128) return run_mass<2, 128>(a, P, stream);
  return cudaErrorInvalidValue;
}

}  // namespace fp2
