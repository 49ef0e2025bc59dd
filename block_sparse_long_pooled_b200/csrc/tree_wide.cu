// Tree attention with more than 16 query rows per KV head, on the tcgen05 tensor cores.
//
// The work is cut as in decode.cu (units on one axis, equal shares, partial results joined in group
// order); only the tile differs.  An M tile is 128 packed rows (token-major, the heads of the group
// inside) and a key tile 128 keys.  A CTA runs two streams, each with its own S, O and softmax
// warpgroup, so that the tensor pipe works for one while the other is at its exponentials:
//   rows left > 128   ("pair")    stream s has M tile s; both use every key tile that is loaded;
//   rows left <= 128  ("parity")  both streams have the one M tile, stream s the key tiles with
//                                 index s mod 2, and their results are merged in shared memory.
// A pair takes twice a parity tile's time, so a unit is an (M tile, key tile).
//
// Per key tile and stream: S = Q K^T into TMEM; one thread per row reads the row's 128 scores,
// masks them, raises the running maximum only when it grew by more than 2^8 (then O is
// rescaled in TMEM), and writes P over S in TMEM; O += P V.  Each step needs the one before, hence
// the two streams.
//
// P in bf16 would be off by up to 2^-9 of each weight, as much as the output's own rounding; with at
// most 128 rows the cache's bytes bound the call, so there a second product adds P - bf16(P), for
// which S has the columns.  e4m3: P is f16, and V is widened to f16 in shared memory by a warpgroup
// of its own (the products of kind f16 want both operands of one type, and e4m3 weights would keep 4
// bits).  That warpgroup also clears the rows of V that hold no key, and the elements of a drafted
// key that are not finite (0 x NaN is NaN for rows that do not see the key); the epilogue adds those
// back to the rows that do.
//
// Warps: 0-3 and 4-7 softmax of stream 0 and 1; 8 producer; 9, 10 MMA issuers of stream 0 and 1;
// 12-15 V.  TMEM: S0 | S1 | O0 | O1, 128 columns each.
#include "decode_device.cuh"

namespace fp2 {

namespace {

template <int DT, int D, bool SPLIT_>
struct Wide {
  static constexpr bool E4 = DT == 2;
  static constexpr bool SPLIT = SPLIT_ && !E4;
  static constexpr int ELT = E4 ? 1 : 2;
  static constexpr int TILE = 128;
  static constexpr int KCH = 128 / ELT;           // elements of a 128-byte swizzled row
  static constexpr int Q_BYTES = 128 * D * ELT;   // one M tile
  static constexpr int KV_BYTES = TILE * D * ELT; // one K or V tile
  static constexpr int V16_BYTES = E4 ? TILE * D * 2 : 0;
  static constexpr int STAGES = E4 ? 3 : (D == 64 ? 4 : 2);
  static constexpr int KIND_QK = E4 ? 2 : 1, UK = 32 / ELT;
  static constexpr uint32_t FMT_QK = E4 ? 0u : 1u, FMT_PV = E4 ? 0u : 1u;  // e4m3 / bf16; f16 / bf16
  static constexpr uint32_t IDESC_S = make_idesc(FMT_QK, FMT_QK, 0, 0, 128, 128);
  static constexpr uint32_t IDESC_PV = make_idesc(FMT_PV, FMT_PV, 0, 1, 128, D);
  static constexpr float LAZY = 8.f;
  // f16 holds 2^-14 with all its bits: a factor of 2^4 keeps small weights away from the subnormals,
  // and 2^(4 + LAZY) far below the largest value.
  static constexpr float P_BIAS = E4 ? 4.f : 0.f;
  static constexpr int OFF_Q = 0;                              // [2] M tiles
  static constexpr int OFF_K = 2 * Q_BYTES;                    // [STAGES]
  static constexpr int OFF_V = OFF_K + STAGES * KV_BYTES;      // [STAGES]
  static constexpr int OFF_V16 = OFF_V + STAGES * KV_BYTES;    // [2]
  static constexpr int OFF_ML = OFF_V16 + 2 * V16_BYTES;       // [128] float2: maximum and sum of stream 1
  static constexpr int OFF_PRE = OFF_ML + 128 * 8;
  static constexpr int OFF_LEN = OFF_PRE + (FP2_MAX_SEQS + 1) * 8;
  static constexpr int OFF_BAR = (OFF_LEN + FP2_MAX_SEQS * 4 + 15) / 16 * 16;
  static constexpr int SMEM_RAW = OFF_BAR + 512 + 1024;
  // One CTA per SM: it holds all of TMEM.
  static constexpr int SMEM = SMEM_RAW > 116 * 1024 ? SMEM_RAW : 116 * 1024;
  static_assert(SMEM <= 226 * 1024, "shared memory");
  // Columns of stream 1's O that fit into the unused second Q tile during a merge.
  static constexpr int MERGE = Q_BYTES / (128 * 4);
  static_assert(MERGE % 32 == 0 && D % MERGE == 0, "merge rounds");
};
constexpr int kWideThreads = 512;

// Weighted pieces: an item (sequence, pair of M tiles) spans w * tiles units, w = its M tiles.
struct WidePiece {
  int r, rt, w, t0, t1, tiles, end;  // key tiles [t0, t1) of `tiles`; `end`: offset in the item at which it ends
  long long next;                    // first unit after the piece
};
FP2_DEVICE WidePiece wide_piece(const long long* pre, const int* len, const DecodeArgs& a, const DecodePlan& P,
                                long long u, long long u1) {
  int lo = 0, hi = P.num_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= u) lo = mid; else hi = mid - 1;
  }
  WidePiece p;
  p.r = lo;
  p.tiles = len[lo] <= 0 ? 1 : (len[lo] + 127) / 128;
  const int mt = ((P.q_off[lo + 1] - P.q_off[lo]) * a.G + 127) / 128;
  const int rem = static_cast<int>(u - pre[lo]);
  p.rt = rem / (2 * p.tiles);
  const int off = rem - p.rt * 2 * p.tiles;
  p.w = min(2, mt - 2 * p.rt);
  const long long left = u1 - u;
  p.end = p.tiles * p.w - off <= left ? p.tiles * p.w : off + static_cast<int>(left);
  p.t0 = (off + p.w - 1) / p.w;
  p.t1 = (p.end + p.w - 1) / p.w;  // a piece of one unit in the middle of a pair's tile is empty
  p.next = u + (p.end - off);
  return p;
}

FP2_DEVICE void tmem_ld32_now(uint32_t taddr, uint32_t (&r)[32]) {
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

// Address of 16-byte chunk c of row k in a tile of 128 rows: 128-byte boxes side by side, swizzled.
FP2_DEVICE uint32_t box_addr(int k, int c) { return (c >> 3) * (128 * 128) + k * 128 + (((c & 7) ^ (k & 7)) << 4); }

FP2_DEVICE uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
FP2_DEVICE void sts16(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Clears the halves of a word (bf16, exponent all ones) or the bytes (e4m3, 0x7F) that are not finite.
template <bool E4>
FP2_DEVICE uint32_t finite_only(uint32_t w, bool& bad) {
  uint32_t keep = 0xFFFFFFFFu;
  if constexpr (E4) {
#pragma unroll
    for (int b = 0; b < 4; ++b)
      if (((w >> (8 * b)) & 0x7Fu) == 0x7Fu) keep &= ~(0xFFu << (8 * b));
  } else {
#pragma unroll
    for (int b = 0; b < 2; ++b)
      if (((w >> (16 * b)) & 0x7F80u) == 0x7F80u) keep &= ~(0xFFFFu << (16 * b));
  }
  bad |= keep != 0xFFFFFFFFu;
  return w & keep;
}

template <int DT, int D, bool SPLIT>
__global__ void __launch_bounds__(kWideThreads, 1)
    tree_wide_kernel(const __grid_constant__ DecodeArgs a, const __grid_constant__ DecodePlan P) {
  using C = Wide<DT, D, SPLIT>;
  extern __shared__ char smem_raw[];
  char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = smem_u32(smem);
  float2* ml_smem = reinterpret_cast<float2*>(smem + C::OFF_ML);
  long long* pre = reinterpret_cast<long long*>(smem + C::OFF_PRE);
  int* len = reinterpret_cast<int*>(smem + C::OFF_LEN);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* k_full = bars;                    // the K tile has landed
  uint64_t* k_empty = k_full + C::STAGES;     // both streams are done with it
  uint64_t* v_full = k_empty + C::STAGES;
  uint64_t* v_empty = v_full + C::STAGES;     // bf16: by the MMA issuers; e4m3: by the V warps
  uint64_t* v_ready = v_empty + C::STAGES;    // V (e4m3: its f16 copy, two of them) can be multiplied
  uint64_t* v_used = v_ready + C::STAGES;     // [2] e4m3: the copy is free again
  uint64_t* q_ready = v_used + 2;             // [2] stream s may start the piece's products
  uint64_t* s_full = q_ready + 2;             // [2]
  uint64_t* p_full = s_full + 2;              // [2]
  uint64_t* pv_done = p_full + 2;             // [2]
  uint64_t* all_done = pv_done + 2;           // [2]
  // Which rows of a tile hold keys: valid_v goes with the V stage.  The softmax reads valid_k later than
  // its K stage is released; when tile x is loaded every stream is past tile x - STAGES - 2.
  constexpr int VALID = 8;
  static_assert(VALID >= C::STAGES + 2, "ring of masks");
  __shared__ uint64_t valid_k[VALID][2], valid_v[C::STAGES][2];
  __shared__ int abort_flag;
  __shared__ int bad_v;                       // some drafted key of this CTA's has a value that is not finite
  __shared__ uint32_t status_word, tmem_slot;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = blockIdx.x % a.Hkv, grp = blockIdx.x / a.Hkv;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 2);
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], C::E4 ? 4 : 2);
      mbar_init(&v_ready[s], 4);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&v_used[s], 2);
      mbar_init(&q_ready[s], 4);
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], 4);
      mbar_init(&pv_done[s], 1);
      mbar_init(&all_done[s], 1);
    }
    abort_flag = 0;
    bad_v = 0;
    status_word = 0;
    fence_mbar_init();
    tma_prefetch_desc(&a.tm_k);
    tma_prefetch_desc(&a.tm_v);
  }
  if (warp == 8) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  scan_units<C::TILE>(a, P, 128, 0, pre, len, &status_word);
  const long long units = pre[P.num_seqs];
  const int ng = active_groups(units, a.groups);
  const bool idle = grp >= ng;
  const long long u0 = idle ? 0 : units * grp / ng, u1 = idle ? 0 : units * (grp + 1) / ng;
  if (idle && g == 0 && tid == 0) a.desc[grp] = make_int4(-1, 0, 0, 0);
  const auto wait = [&](uint64_t* bar, uint32_t parity) {  // one answer for the warp
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, &abort_flag, &status_word, a.wait_limit_ns));
  };

  if (warp >= 8) {
    if (warp == 8) {
      // ---------------------------------------------------------------- producer
      Producer<C::TILE, C::ELT, D> load;
      int it = 0;
      bool alive = true;
      for (long long u = u0; u < u1 && alive;) {
        const WidePiece p = wide_piece(pre, len, a, P, u, u1);
        for (int t = p.t0; t < p.t1; ++t) {
          const int st = it % C::STAGES, round = it / C::STAGES;
          if (round > 0 && !(alive = wait(&k_empty[st], (round - 1) & 1))) break;
          load.load(a, &a.tm_k, p.r, len[p.r], g, t * C::TILE, sbase + C::OFF_K + st * C::KV_BYTES, &k_full[st],
                    valid_k[it % VALID], &status_word, it == a.withhold);
          if (round > 0 && !(alive = wait(&v_empty[st], (round - 1) & 1))) {
            ++it;
            break;
          }
          load.load(a, &a.tm_v, p.r, len[p.r], g, t * C::TILE, sbase + C::OFF_V + st * C::KV_BYTES, &v_full[st],
                    valid_v[st], &status_word, false);
          ++it;
        }
        u = p.next;
      }
      // Copies in flight end before the CTA does.
      if (*static_cast<volatile int*>(&abort_flag)) {
        volatile int no_abort = 0;
        for (int i = max(0, it - C::STAGES); i < it; ++i) {
          mbar_wait(&k_full[i % C::STAGES], (i / C::STAGES) & 1, &no_abort, &status_word, a.wait_limit_ns / 5);
          mbar_wait(&v_full[i % C::STAGES], (i / C::STAGES) & 1, &no_abort, &status_word, a.wait_limit_ns / 5);
        }
      }
    } else if (warp == 9 || warp == 10) {
      // ---------------------------------------------------------------- MMA issuer of stream s
      const int s = warp - 9;
      const uint32_t s_col = tmem + s * 128, o_col = tmem + 256 + s * 128;
      int base = 0, cs = 0, nq = 0;  // tiles before this piece; tiles, and pieces with any, of this stream
      bool alive = true;
      for (long long u = u0; u < u1 && alive;) {
        const WidePiece p = wide_piece(pre, len, a, P, u, u1);
        const int n = p.t1 - p.t0;
        const bool pair = p.w == 2;
        u = p.next;
        if (n <= (pair ? 0 : s)) {
          base += n;
          continue;
        }
        if (!(alive = wait(&q_ready[s], nq++ & 1))) break;
        tc_fence_after();
        const uint64_t qd = smem_desc_sw128(sbase + C::OFF_Q + (pair ? s : 0) * C::Q_BYTES, 16, 1024);
        const int step = pair ? 1 : 2;
        for (int i = pair ? 0 : s, j = 0; i < n; i += step, ++j, ++cs) {
          const int it = base + i, st = it % C::STAGES, ph = (it / C::STAGES) & 1;
          if (!(alive = wait(&k_full[st], ph))) break;
          // P(j - 1), which S(j) overwrites, has been used
          if (j > 0 && !(alive = wait(&pv_done[s], (cs - 1) & 1))) break;
          tc_fence_after();
          const uint64_t kd = smem_desc_sw128(sbase + C::OFF_K + st * C::KV_BYTES, 16, 1024);
#pragma unroll
          for (int k = 0; k < D / C::UK; ++k) {
            const uint64_t off = ((k * C::UK / C::KCH) * (128 * 128) + (k * C::UK % C::KCH) * C::ELT) >> 4;
            umma_ss_warp<C::KIND_QK>(s_col, qd + off, kd + off, C::IDESC_S, k > 0 ? 1u : 0u);
          }
          umma_commit_warp(&s_full[s]);
          umma_commit_warp(&k_empty[st]);
          if (!pair) umma_commit_warp(&k_empty[st]);
          const int vs = C::E4 ? it & 1 : st;
          if (!(alive = wait(&v_ready[vs], C::E4 ? (it >> 1) & 1 : ph))) break;
          if (!(alive = wait(&p_full[s], cs & 1))) break;
          tc_fence_after();
          const uint64_t vd = smem_desc_sw128(
              sbase + (C::E4 ? C::OFF_V16 + vs * C::V16_BYTES : C::OFF_V + st * C::KV_BYTES), C::TILE * 128, 1024);
#pragma unroll
          for (int part = 0; part < (C::SPLIT ? 2 : 1); ++part) {
#pragma unroll
            for (int k = 0; k < C::TILE / 16; ++k)
              umma_ts_warp<1>(o_col, s_col + part * 64 + k * 8, vd + static_cast<uint64_t>((k * 16 * 128) >> 4),
                              C::IDESC_PV, (part > 0 || k > 0 || j > 0) ? 1u : 0u);
          }
          uint64_t* used = C::E4 ? &v_used[vs] : &v_empty[st];
          umma_commit_warp(used);
          if (!pair) umma_commit_warp(used);
          umma_commit_warp(&pv_done[s]);
        }
        base += n;
      }
      // No product in flight when the CTA ends.
      umma_commit_warp(&all_done[s]);
      volatile int no_abort = 0;
      mbar_wait(&all_done[s], 0, &no_abort, &status_word, a.wait_limit_ns / 5);
    } else if (warp >= 12) {
      // ---------------------------------------------------------------- V: thread = key of the tile
      const int row = tid - 12 * 32;
      int it = 0;
      bool alive = true;
      for (long long u = u0; u < u1 && alive;) {
        const WidePiece p = wide_piece(pre, len, a, P, u, u1);
        const int keys = len[p.r], base = keys - (P.q_off[p.r + 1] - P.q_off[p.r]);
        for (int t = p.t0; t < p.t1; ++t, ++it) {
          const int st = it % C::STAGES, ph = (it / C::STAGES) & 1;
          if (!(alive = wait(&v_full[st], ph))) break;
          const bool here = (valid_v[st][row >> 6] >> (row & 63)) & 1;
          const bool drafted = t * C::TILE + row >= base;
          const uint32_t v_at = sbase + C::OFF_V + st * C::KV_BYTES;
          bool bad = false;
          if constexpr (C::E4) {
            if (it >= 2 && !(alive = wait(&v_used[it & 1], ((it >> 1) - 1) & 1))) break;
            const uint32_t out = sbase + C::OFF_V16 + (it & 1) * C::V16_BYTES;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              uint4 x = here ? lds16(v_at + box_addr(row, c)) : make_uint4(0, 0, 0, 0);
              if (drafted) {
                x.x = finite_only<true>(x.x, bad);
                x.y = finite_only<true>(x.y, bad);
                x.z = finite_only<true>(x.z, bad);
                x.w = finite_only<true>(x.w, bad);
              }
              sts16(out + box_addr(row, 2 * c),
                    make_uint4(e4m3x2_to_f16x2(x.x & 0xFFFFu), e4m3x2_to_f16x2(x.x >> 16),
                               e4m3x2_to_f16x2(x.y & 0xFFFFu), e4m3x2_to_f16x2(x.y >> 16)));
              sts16(out + box_addr(row, 2 * c + 1),
                    make_uint4(e4m3x2_to_f16x2(x.z & 0xFFFFu), e4m3x2_to_f16x2(x.z >> 16),
                               e4m3x2_to_f16x2(x.w & 0xFFFFu), e4m3x2_to_f16x2(x.w >> 16)));
            }
          } else {
            if (!here) {
#pragma unroll
              for (int c = 0; c < D / 8; ++c) sts16(v_at + box_addr(row, c), make_uint4(0, 0, 0, 0));
            } else if (drafted) {
#pragma unroll
              for (int c = 0; c < D / 8; ++c) {
                uint4 x = lds16(v_at + box_addr(row, c));
                bool cut = false;
                x.x = finite_only<false>(x.x, cut);
                x.y = finite_only<false>(x.y, cut);
                x.z = finite_only<false>(x.z, cut);
                x.w = finite_only<false>(x.w, cut);
                if (cut) sts16(v_at + box_addr(row, c), x);
                bad |= cut;
              }
            }
          }
          if (bad) *static_cast<volatile int*>(&bad_v) = 1;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if constexpr (C::E4) {
              mbar_arrive(&v_empty[st]);
              mbar_arrive(&v_ready[it & 1]);
            } else {
              mbar_arrive(&v_ready[st]);
            }
          }
        }
        u = p.next;
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax of stream s, thread = row
    const int s = warp >> 2, rt = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + s * 128, o_at = tmem + lanes + 256 + s * 128;
    const float s2 = a.scale_log2;
    int base_it = 0, cs = 0, nth = 0;
    bool alive = true;
    for (long long u = u0; u < u1; ++nth) {
      const WidePiece p = wide_piece(pre, len, a, P, u, u1);
      const bool pair = p.w == 2;
      const int keys = len[p.r], tok0 = P.q_off[p.r], q_len = P.q_off[p.r + 1] - tok0;
      const int rows = q_len * a.G, base = keys - q_len;
      const int row = p.rt * 256 + (pair ? s * 128 : 0) + rt;    // packed row of the sequence
      const bool mine = row < rows;
      const int tok = mine ? row / a.G : 0, h = g * a.G + (mine ? row - tok * a.G : 0);
      const bool busy = __any_sync(0xFFFFFFFFu, mine);
      const int n = p.t1 - p.t0;

      // Q: each row by the thread that owns it (parity: by stream 0's).  The row before has been
      // used: this thread has seen the last product of the piece before.
      if (pair || s == 0) {
        const uint32_t q_at = sbase + C::OFF_Q + (pair ? s : 0) * C::Q_BYTES;
        const char* src = static_cast<const char*>(a.q) +
                          ((static_cast<int64_t>(tok0) + tok) * a.q_stride + static_cast<int64_t>(h) * D) * C::ELT;
#pragma unroll 8
        for (int c = 0; c < D * C::ELT / 16; ++c)
          sts16(q_at + box_addr(rt, c),
                mine ? __ldg(reinterpret_cast<const uint4*>(src) + c) : make_uint4(0, 0, 0, 0));
        fence_proxy_async_smem();
      }
      if (pair)
        __syncwarp();
      else
        asm volatile("bar.sync 1, 256;" ::: "memory");  // stream 0's rows are there, stream 1 has come this far
      if (n > (pair ? 0 : s) && lane == 0) mbar_arrive(&q_ready[s]);

      float m_run = neg_inf(), l_run = 0.f;
      const uint64_t mask = mine ? token_mask(a, tok0, tok) : 0;
      int done = 0;
      for (int i = pair ? 0 : s; i < n; i += pair ? 1 : 2, ++cs, ++done) {
        const uint64_t* valid = valid_k[(base_it + i) % VALID];
        if (alive) alive = wait(&s_full[s], cs & 1);
        if (!alive) continue;
        tc_fence_after();
        if (busy) {
          const int j0 = (p.t0 + i) * C::TILE;
          // Twice through the row, 32 scores at a time: all 128 at once would leave the 16 warps' registers.
          const bool tail = j0 + C::TILE > base || valid[0] != ~0ull || valid[1] != ~0ull;
          const auto scores = [&](int c, uint32_t (&v)[32]) {
            tmem_ld32_now(s_at + 32 * c, v);
            if (tail) {
              const uint32_t here = static_cast<uint32_t>(valid[c >> 1] >> (32 * (c & 1)));
              const uint32_t vis = here & (seen16(mask, j0 + 32 * c, base) | (seen16(mask, j0 + 32 * c + 16, base) << 16));
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((vis >> e) & 1u)) v[e] = 0xFF800000u;
            }
          };
          float top[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32];
            scores(c, v);
#pragma unroll
            for (int e = 0; e < 32; e += 8)
#pragma unroll
              for (int x = 0; x < 4; ++x)
                top[x] = fmax3(top[x], __uint_as_float(v[e + 2 * x]), __uint_as_float(v[e + 2 * x + 1]));
          }
          const float m_new = fmaxf(m_run, fmax3(top[0], top[1], fmaxf(top[2], top[3])) * s2);
          // The maximum is raised, and O rescaled, when it grew by more than 2^8.
          const bool need = m_new > m_run + C::LAZY;
          if (done > 0 && __any_sync(0xFFFFFFFFu, need)) {
            const float f = need ? fast_exp2(m_run - m_new) : 1.f;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32_now(o_at + 32 * c, o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st32(o_at + 32 * c, o);
            }
          }
          if (need) {
            l_run = m_run == neg_inf() ? 0.f : l_run * fast_exp2(m_run - m_new);
            m_run = m_new;
          }
          const float off = m_run == neg_inf() ? 0.f : C::P_BIAS - m_run;
          const float2 s22 = make_float2(s2, s2), off2 = make_float2(off, off);
          float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          // P's columns 16 c .. of chunk c lie on scores that have been read; the remainders' do not yet.
          [[maybe_unused]] uint32_t lo[64];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32], hi[16];
            scores(c, v);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 x = __ffma2_rn(make_float2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), s22, off2);
              const float2 w = make_float2(fast_exp2(x.x), fast_exp2(x.y));
              acc[e & 1] = __fadd2_rn(acc[e & 1], w);
              hi[e] = C::E4 ? pack_f16x2(w.x, w.y) : pack_bf16x2(w.x, w.y);
              if constexpr (C::SPLIT)
                lo[16 * c + e] =
                    pack_bf16x2(w.x - __uint_as_float(hi[e] << 16), w.y - __uint_as_float(hi[e] & 0xFFFF0000u));
            }
            tmem_st16(s_at + 16 * c, hi);
          }
          if constexpr (C::SPLIT) {
            tmem_st32(s_at + 64, *reinterpret_cast<const uint32_t(*)[32]>(&lo[0]));
            tmem_st32(s_at + 96, *reinterpret_cast<const uint32_t(*)[32]>(&lo[32]));
          }
          l_run += (acc[0].x + acc[1].x) + (acc[0].y + acc[1].y);
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[s]);
      }
      if (done > 0 && alive) alive = wait(&pv_done[s], (cs - 1) & 1);
      tc_fence_after();
      base_it += n;

      // ---------------- epilogue
      const bool any_tile = done > 0 && alive && busy;
      // Values of drafted keys that V's warps cleared come back here, for the rows that see the key.
      const bool fix = *static_cast<volatile int*>(&bad_v) != 0 && n > 0 && keys > 0 && p.t1 * C::TILE > base && mine;
      const auto add_cleared = [&](uint32_t (&o)[32], int c0) {
        for (int b = 0; b < q_len; ++b) {
          const int j = base + b, t = j / C::TILE;
          if (!((mask >> b) & 1) || t < p.t0 || t >= p.t1 || (!pair && ((t - p.t0) & 1) != s)) continue;
          int64_t outer = p.r, at = j;
          if (a.page_table != nullptr) {
            outer = a.page_table[static_cast<int64_t>(p.r) * a.max_pages + j / a.page_size];
            at = j % a.page_size;
            if (outer < 0 || outer >= a.num_pages) continue;
          }
          const char* src = static_cast<const char*>(a.v_ptr) +
                            (outer * a.kv_stride_outer + at * a.kv_stride + static_cast<int64_t>(g) * D + c0) * C::ELT;
#pragma unroll 1
          for (int q = 0; q < 32 * C::ELT / 4; ++q) {
            const uint32_t word = reinterpret_cast<const uint32_t*>(src)[q];
            bool bad = false;
            finite_only<C::E4>(word, bad);
            if (!bad) continue;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              if (e * C::ELT / 4 != q) continue;
              const uint32_t x = C::E4 ? (word >> (8 * (e & 3))) & 0xFFu : (word >> (16 * (e & 1))) & 0xFFFFu;
              const bool nonfinite = C::E4 ? (x & 0x7Fu) == 0x7Fu : (x & 0x7F80u) == 0x7F80u;
              if (nonfinite) o[e] = __float_as_uint(__uint_as_float(o[e]) + __uint_as_float(C::E4 ? 0x7FFFFFFFu : x << 16));
            }
          }
        }
      };
      const bool whole = p.t0 == 0 && p.t1 == p.tiles;
      const int slot = (grp * a.Hkv + g) * 2 + (nth == 0 ? 0 : 1);
      const int64_t part_row = static_cast<int64_t>(slot) * a.part_rows + (pair ? s * 128 : 0) + rt;
      const int64_t out_row = static_cast<int64_t>(tok0) + tok;
      const bool store = mine && fp2_check(out_row < a.T && h < a.Hq, &status_word);
      const auto write = [&](uint32_t (&o)[32], int c0, float f) {  // 32 values of this thread's row
        if (whole) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + (out_row * a.Hq + h) * D + c0);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[e] = pack_bf16x2(__uint_as_float(o[8 * q + 2 * e]) * f, __uint_as_float(o[8 * q + 2 * e + 1]) * f);
            dst[q] = make_uint4(x[0], x[1], x[2], x[3]);
          }
        } else {
          uint4* dst = reinterpret_cast<uint4*>(a.part_o + part_row * D + c0);
#pragma unroll
          for (int q = 0; q < 8; ++q) dst[q] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
        }
      };
      const auto write_stats = [&](float top, float total) {
        if (whole) {
          if (a.lse != nullptr)
            a.lse[static_cast<int64_t>(h) * a.T + out_row] =
                total == 0.f ? neg_inf() : (top - C::P_BIAS + log2f(total)) * kLn2;
        } else {
          a.part_ml[part_row] = make_float2(top == neg_inf() ? top : top - C::P_BIAS, total);
        }
      };
      if (pair) {
        const float f = l_run == 0.f ? 0.f : a.v_descale / l_run;
        if (busy) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
            if (any_tile) tmem_ld32_now(o_at + 32 * c, o);
            if (fix) add_cleared(o, 32 * c);
            if (store && (n > 0 || whole)) write(o, 32 * c, f);
          }
          if (store) write_stats(m_run, l_run);
        }
      } else {
        // Stream 1 hands its sums and O to stream 0 through the second Q tile, MERGE columns at a time.
        float* buf = reinterpret_cast<float*>(smem + C::OFF_Q + C::Q_BYTES);
        if (s == 1) ml_smem[rt] = make_float2(m_run, l_run);
        asm volatile("bar.sync 1, 256;" ::: "memory");
        float top = m_run, total = l_run, f0 = 1.f, f1 = 0.f;
        if (s == 0) {
          const float2 other = ml_smem[rt];
          top = fmaxf(m_run, other.x);
          f0 = l_run == 0.f ? 0.f : fast_exp2(m_run - top);
          f1 = other.y == 0.f ? 0.f : fast_exp2(other.x - top);
          total = l_run * f0 + other.y * f1;
          if (l_run == 0.f) total = other.y * f1;
          if (other.y == 0.f) total = l_run * f0;
        }
        const float f = total == 0.f ? 0.f : a.v_descale / total;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += C::MERGE) {
          if (s == 1 && busy) {
#pragma unroll 1
            for (int c = 0; c < C::MERGE; c += 32) {
              uint32_t o[32];
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = 0u;
              if (any_tile) tmem_ld32_now(o_at + c0 + c, o);
              if (fix) add_cleared(o, c0 + c);
#pragma unroll
              for (int e = 0; e < 32; ++e) buf[(c + e) * 128 + rt] = __uint_as_float(o[e]);
            }
          }
          asm volatile("bar.sync 1, 256;" ::: "memory");
          if (s == 0 && busy) {
#pragma unroll 1
            for (int c = 0; c < C::MERGE; c += 32) {
              uint32_t o[32];
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = 0u;
              if (any_tile) tmem_ld32_now(o_at + c0 + c, o);
              if (fix) add_cleared(o, c0 + c);
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                // a stream that saw nothing of the row leaves zeros
                float x = l_run == 0.f ? 0.f : __uint_as_float(o[e]) * f0;
                if (f1 != 0.f) x += buf[(c + e) * 128 + rt] * f1;
                o[e] = __float_as_uint(x);
              }
              if (store) write(o, c0 + c, f);
            }
          }
          asm volatile("bar.sync 1, 256;" ::: "memory");  // (the last one: the buffer is Q's again)
        }
        if (s == 0 && store) write_stats(top, total);
      }
      tc_fence_before();
      // The group that holds an item's first piece tells join_kernel how many follow.
      u = p.next;
      if (g == 0 && tid == 0 && u >= u1) {
        int4 d = make_int4(-1, 0, 0, 0);
        if (p.t0 == 0 && p.t1 < p.tiles) {
          const long long last = u1 + (p.w * p.tiles - p.end) - 1;  // the item's last unit
          int e = grp + 1;
          while (units * (e + 1) / ng <= last) ++e;
          d = make_int4(nth == 0 ? 0 : 1, p.r, p.rt, e - grp + 1);
        }
        a.desc[grp] = d;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, 512);
  store_status(a, &status_word);
}

template <int DT, int D, bool SPLIT>
cudaError_t run(const DecodeArgs& a, const DecodePlan& P, cudaStream_t stream) {
  using C = Wide<DT, D, SPLIT>;
  const auto kernel = tree_wide_kernel<DT, D, SPLIT>;
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), C::SMEM);
  if (e != cudaSuccess) return e;
  kernel<<<a.groups * a.Hkv, kWideThreads, C::SMEM, stream>>>(a, P);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_wide(int dtype, int D, const DecodeArgs& a, const DecodePlan& P, cudaStream_t stream) {
  const bool split = a.part_rows <= 128;
  if (dtype == FP2_BF16 && D == 128) return split ? run<1, 128, true>(a, P, stream) : run<1, 128, false>(a, P, stream);
  if (dtype == FP2_BF16 && D == 64) return split ? run<1, 64, true>(a, P, stream) : run<1, 64, false>(a, P, stream);
  if (dtype == FP2_E4M3 && D == 128) return run<2, 128, false>(a, P, stream);
  return cudaErrorInvalidValue;
}

}  // namespace fp2
