// Tree attention with more than 16 query rows per KV head, on the tcgen05 tensor cores.
//
// The work is cut as in decode.cu (units on one axis, equal shares, partial results joined in group
// order); only the tile differs.  An M tile is 128 packed rows (token-major, the heads of the group
// inside) and a key tile 64 keys.  A CTA runs two streams, each with its own O and softmax warpgroup:
//   rows left > 128   ("pair")    stream s has M tile s; both use every key tile that is loaded;
//   rows left <= 128  ("parity")  both streams have the one M tile, stream s the key tiles with
//                                 index s mod 2, and their results are merged in shared memory.
// A pair takes twice a parity tile's time, so a unit is an (M tile, key tile).
//
// Per key tile and stream: S = Q K^T into TMEM; one thread per row takes the row's 64 scores into registers, masks
// them, raises the running maximum only when it grew by more than 2^8 (then O is rescaled in TMEM), and writes P
// over S in TMEM; O += P V.  A stream has two buffers of 64 columns: S(j + 1) is computed while the softmax works
// on S(j).  With one buffer of 128 keys the exponentials stood still for the products of every tile: 299 us for
// eight trees of 33 to 64 tokens by 8 heads on an e4m3 cache of 9K to 33K keys, now 137 to 157 (620 to 710
// TFLOP/s).  A pair's tile takes about 2,800 cycles of it.  The exponentials (16 a cycle and SM) would need 1,024
// of them and the products 900; taking either away saves little, and half of them on the FMA pipe cost 10 us.
// What bounds it is the chain: some 1,600 cycles in which a stream's issuing warp waits, issues and commits S and
// O, and the softmax's loads, votes and barriers around its arithmetic.  With few rows the cache's bytes bound the
// call: 7 tokens by 4 heads at 128K bf16 keys 96 to 116 us, 82 of them in the tiles.
//
// P in bf16 is off by up to 2^-8 of each weight, as much as the output's own rounding.  For sequences of up to 128
// rows, where the cache's bytes bound the call, a second product adds P - bf16(P) (2^-16), for which S has the
// columns: 7 tokens by 4 heads at 128K bf16 keys take 96 us with it, 91 without.  Above 128 rows, where products
// and softmax do, P stays single: eight trees of 33 to 64 tokens by 8 heads on a bf16 cache of 9K to 33K keys take
// 147 us, 161 with both.  The choice goes by the sequence's own rows: by the batch's longest draft, a sequence's
// precision would depend on its neighbours.  e4m3: P is f16, and V is widened to f16 in shared memory by a
// warpgroup of its own (the products of kind f16 want both operands of one type, and e4m3 weights would keep 4
// bits).  That warpgroup also clears the rows of V that hold no key, and the elements of a drafted key that are
// not finite (0 x NaN is NaN for rows that do not see the key); the epilogue adds those back to the rows that do.
//
// Warps: 0-3 and 4-7 softmax of stream 0 and 1; 8 producer; 9, 10 MMA issuers of stream 0 and 1;
// 12-15 V.  TMEM: S0 | S1 | O0 | O1, 128 columns each.
#include "decode_device.cuh"

namespace fp2 {

namespace {

template <int DT, int D>
struct Wide {
  static constexpr bool E4 = DT == 2;
  static constexpr int ELT = E4 ? 1 : 2;
  static constexpr int TILE = kWideTile;
  static constexpr int KCH = 128 / ELT;           // elements of a 128-byte swizzled row
  static constexpr int Q_BYTES = 128 * D * ELT;   // one M tile
  static constexpr int KV_BYTES = TILE * D * ELT; // one K or V tile
  static constexpr int V16_BYTES = E4 ? TILE * D * 2 : 0;
  // Rings.  A wait names its phase by parity alone, so whoever waits on a barrier has to have seen the phase before
  // it end; loads land in any order, so only a waiter's own earlier waits tell it that.
  //   K: the issuers wait.  In parity a stream meets every second tile: an even ring gives it both phases of a stage,
  //      in an odd one the stages would belong to the streams in turn.
  //   V: the four V warps wait, each for every fourth tile: the ring is a multiple of four, or a warp would meet a
  //      stage in some of its phases only.  The same for the copies.
  static constexpr int K_STAGES = E4 || D == 64 ? 6 : 4;
  static constexpr int V_STAGES = E4 || D == 64 ? 8 : 4;
  static constexpr int COPIES = 4;                // of V in f16
  static constexpr int V_WARPS = 4;
  static_assert(K_STAGES % 2 == 0 && V_STAGES % V_WARPS == 0 && COPIES % V_WARPS == 0, "rings and their waiters");
  static constexpr int KIND_QK = E4 ? 2 : 1, UK = 32 / ELT;
  static constexpr uint32_t FMT_QK = E4 ? 0u : 1u, FMT_PV = E4 ? 0u : 1u;  // e4m3 / bf16; f16 / bf16
  static constexpr uint32_t IDESC_S = make_idesc(FMT_QK, FMT_QK, 0, 0, 128, TILE);
  static constexpr uint32_t IDESC_PV = make_idesc(FMT_PV, FMT_PV, 0, 1, 128, D);
  static constexpr float LAZY = 8.f;
  // f16 holds 2^-14 with all its bits and 2^16 not at all: a factor of 2^7 keeps weights down to 2^-21 of the largest
  // away from the subnormals, and 2^(7 + LAZY), the most a weight can be, below the end.  (With 2^4, weights of
  // 2^-27 beside a large one whose value is 0 were off by 1 %.)
  static constexpr float P_BIAS = E4 ? 7.f : 0.f;
  static_assert(P_BIAS + LAZY <= 15.f, "weights are f16");
  static constexpr int OFF_Q = 0;                              // [2] M tiles
  static constexpr int OFF_K = 2 * Q_BYTES;                    // [K_STAGES]
  static constexpr int OFF_V = OFF_K + K_STAGES * KV_BYTES;    // [V_STAGES]
  static constexpr int OFF_V16 = OFF_V + V_STAGES * KV_BYTES;  // [COPIES]
  static constexpr int OFF_ML = OFF_V16 + COPIES * V16_BYTES;       // [128] float2: maximum and sum of stream 1
  static constexpr int OFF_PRE = OFF_ML + 128 * 8;
  static constexpr int OFF_LEN = OFF_PRE + (FP2_MAX_SEQS + 1) * 8;
  static constexpr int OFF_BAR = (OFF_LEN + FP2_MAX_SEQS * 4 + 15) / 16 * 16;
  static constexpr int BARS = 2 * K_STAGES + 3 * V_STAGES + COPIES + 16;
  static constexpr int SMEM_RAW = OFF_BAR + BARS * 8 + 1024;
  // One CTA per SM: it holds all of TMEM.
  static constexpr int SMEM = SMEM_RAW > 116 * 1024 ? SMEM_RAW : 116 * 1024;
  static_assert(SMEM <= 226 * 1024, "shared memory");
  // Columns of stream 1's O that fit into the unused second Q tile during a merge.
  static constexpr int MERGE = Q_BYTES / (128 * 4);
  static_assert(MERGE % 32 == 0 && D % MERGE == 0, "merge rounds");
};
constexpr int kWideThreads = 512;

// bf16: whether the weights of a sequence of so many rows go to the tensor cores as hi + lo.
__host__ FP2_DEVICE bool split_weights(int rows) { return rows > 0 && rows <= 128; }

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
  p.tiles = len[lo] <= 0 ? 1 : (len[lo] + kWideTile - 1) / kWideTile;
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

FP2_DEVICE void tmem_ld64_now(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, "
      "%22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, "
      "%42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, "
      "%62, %63 }, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]),
        "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]),
        "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]),
        "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]),
        "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr)
      : "memory");
}

FP2_DEVICE void tmem_ld16_now(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// Address of 16-byte chunk c of row k in a tile of ROWS rows: 128-byte boxes side by side, swizzled.
template <int ROWS>
FP2_DEVICE uint32_t box_addr(int k, int c) {
  return (c >> 3) * (ROWS * 128) + k * 128 + (((c & 7) ^ (k & 7)) << 4);
}

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

// e4m3 to f16 by moving bits: sign, 4 and 3 bits of e4m3 one place lower in a half's top byte are an
// f16 of 2^-8 times the value, subnormals included (the factor leaves with v_descale).  Three
// instructions of the integer pipe for two values, where cvt.f16x2.e4m3x2 took 0.9 us a tile of 64 x
// 128 for the SM's four V warps.  0x7F, NaN in e4m3, becomes a number: those bytes are looked for.
FP2_DEVICE uint32_t widen_pair(uint32_t t) { return (t & 0x80008000u) | ((t >> 1) & 0x3F803F80u); }
FP2_DEVICE uint32_t widen_lo(uint32_t w) { return widen_pair(__byte_perm(w, 0, 0x1404)); }
FP2_DEVICE uint32_t widen_hi(uint32_t w) { return widen_pair(__byte_perm(w, 0, 0x3424)); }
FP2_DEVICE uint32_t nan_bytes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }  // bit 7 of each

// Clears the halves of a word (bf16, exponent all ones) or the bytes (e4m3, 0x7F) that are not finite.
template <bool E4>
FP2_DEVICE uint32_t finite_only(uint32_t w) {
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
  return w & keep;
}

// Adds what finite_only cleared of the drafted keys in [j0, j1) to one row's result (f32 partial or bf16
// output), where the row sees the key.  Out of line: it hardly ever runs.
template <int DT, int D>
__device__ __noinline__ void add_cleared(const DecodeArgs& a, int r, int g, int base, int q_len, uint64_t mask, int j0,
                                         int j1, float* part, uint16_t* out) {
  for (int b = 0; b < q_len; ++b) {
    const int j = base + b;
    if (!((mask >> b) & 1) || j < j0 || j >= j1) continue;
    int64_t outer = r, at = j;
    if (a.page_table != nullptr) {
      outer = a.page_table[static_cast<int64_t>(r) * a.max_pages + j / a.page_size];
      at = j % a.page_size;
      if (outer < 0 || outer >= a.num_pages) continue;
    }
    const int64_t e = outer * a.kv_stride_outer + at * a.kv_stride + static_cast<int64_t>(g) * D;
    for (int d = 0; d < D; ++d) {
      float v;
      if constexpr (DT == 2) {
        if ((static_cast<const uint8_t*>(a.v_ptr)[e + d] & 0x7Fu) != 0x7Fu) continue;
        v = __uint_as_float(0x7FFFFFFFu);
      } else {
        v = __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(a.v_ptr)[e + d]) << 16);
        if (isfinite(v)) continue;
      }
      if (part != nullptr)
        part[d] += v;
      else
        out[d] = static_cast<uint16_t>(pack_bf16x2(__uint_as_float(static_cast<uint32_t>(out[d]) << 16) + v, 0.f));
    }
  }
}

// SPLIT: the batch has sequences whose weights come as hi + lo (split_weights).
template <int DT, int D, bool SPLIT, bool SMALL>
__global__ void __launch_bounds__(kWideThreads, 1)
    tree_wide_kernel(const __grid_constant__ DecodeArgs a, const __grid_constant__ DecodePlan P) {
  using C = Wide<DT, D>;
  extern __shared__ char smem_raw[];
  char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sbase = smem_u32(smem);
  float2* ml_smem = reinterpret_cast<float2*>(smem + C::OFF_ML);
  long long* pre = reinterpret_cast<long long*>(smem + C::OFF_PRE);
  int* len = reinterpret_cast<int*>(smem + C::OFF_LEN);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* k_full = bars;                    // the K tile has landed
  uint64_t* k_empty = k_full + C::K_STAGES;   // both streams are done with it
  uint64_t* v_full = k_empty + C::K_STAGES;
  uint64_t* v_empty = v_full + C::V_STAGES;   // bf16: by the MMA issuers; e4m3: by the V warps
  uint64_t* v_ready = v_empty + C::V_STAGES;  // V (e4m3: copy it % COPIES) can be multiplied
  uint64_t* v_used = v_ready + C::V_STAGES;   // [COPIES] e4m3: the copy is free again
  uint64_t* q_ready = v_used + C::COPIES;     // [2] stream s may start the piece's products
  uint64_t* s_full = q_ready + 2;             // [stream][buffer], as the next two
  uint64_t* p_full = s_full + 4;
  uint64_t* pv_done = p_full + 4;
  uint64_t* all_done = pv_done + 4;           // [2]
  // Which rows of a tile hold keys: valid_v goes with the V stage.  The softmax reads valid_k later than
  // its K stage is released: S(x - K_STAGES) is issued then, whose buffer the stream's tile two before had
  // (in parity four tiles before), so everything up to tile x - K_STAGES - 5 has been read.
  constexpr int VALID = 16;
  static_assert(VALID >= C::K_STAGES + 5, "ring of masks");
  __shared__ uint64_t valid_k[VALID], valid_v[C::V_STAGES];
  __shared__ int abort_flag;
  __shared__ int bad_v;                       // some drafted key of this CTA's has a value that is not finite
  __shared__ uint32_t status_word, tmem_slot;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = blockIdx.x % a.Hkv, grp = blockIdx.x / a.Hkv;
  grid_launch_next();
  if (tid == 0) {
    for (int s = 0; s < C::K_STAGES; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 2);
    }
    for (int s = 0; s < C::V_STAGES; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], C::E4 ? 1 : 2);
      mbar_init(&v_ready[s], 1);
    }
    for (int s = 0; s < C::COPIES; ++s) mbar_init(&v_used[s], 2);
    for (int s = 0; s < 4; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], 4);
      mbar_init(&pv_done[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&q_ready[s], 4);
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
  grid_wait();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  scan_units<C::TILE>(a, P, 128, 0, pre, len, &status_word);
  const long long units = pre[P.num_seqs];
  // Partial results of 256 rows cost as much as four units: fewer CTAs then.
  const int ng = active_groups(a.max_rows > 128 ? (units + 3) / 4 : units, a.groups);
  const bool idle = grp >= ng;
  const long long u0 = idle ? 0 : units * grp / ng, u1 = idle ? 0 : units * (grp + 1) / ng;
  if (idle && g == 0 && tid == 0) a.desc[grp] = make_int4(-1, 0, 0, 0);
  const auto wait = [&](uint64_t* bar, uint32_t parity) {  // one answer for the warp
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, &abort_flag, &status_word, a.wait_limit_ns));
  };

  if (warp >= 8) {
    if (warp == 8 || warp == 11) {
      // ---------------------------------------------------------------- producers: K, V
      const bool is_k = warp == 8;
      uint64_t* full = is_k ? k_full : v_full;
      uint64_t* empty = is_k ? k_empty : v_empty;
      const uint32_t ring = sbase + (is_k ? C::OFF_K : C::OFF_V);
      const int stages = is_k ? C::K_STAGES : C::V_STAGES;
      Producer<C::TILE, C::ELT, D, SMALL> load;
      int it = 0, st = 0, round = 0;
      [[maybe_unused]] int late_t = -1, late_st = 0;
      bool alive = true;
      for (long long u = u0; u < u1 && alive;) {
        const WidePiece p = wide_piece(pre, len, a, P, u, u1);
        for (int t = p.t0; t < p.t1; ++t, ++it) {
          if (round > 0 && !(alive = wait(&empty[st], (round - 1) & 1))) break;
          const auto bring = [&](int t, int st) {
            load.load(a, is_k ? &a.tm_k : &a.tm_v, p.r, len[p.r], g, t * C::TILE, ring + st * C::KV_BYTES, &full[st],
                      is_k ? &valid_k[it % VALID] : &valid_v[st], &status_word, is_k && it == a.withhold);
          };
          if constexpr (FP2_CHECKED) {   // testing: one V tile follows the next two of its piece
            const bool held = !is_k && it == a.late_v && t + 2 < p.t1;
            if (held) late_t = t, late_st = st;
            else bring(t, st);
            if (late_t >= 0 && it == a.late_v + 2) {
              __nanosleep(50000);
              bring(late_t, late_st);
              late_t = -1;
            }
          } else {
            bring(t, st);
          }
          if (++st == stages) st = 0, ++round;
        }
        u = p.next;
      }
      // Copies in flight end before the CTA does.
      if (*static_cast<volatile int*>(&abort_flag)) {
        volatile int no_abort = 0;
        for (int i = max(0, it - stages); i < it; ++i)
          mbar_wait(&full[i % stages], (i / stages) & 1, &no_abort, &status_word, a.wait_limit_ns / 5);
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
        const int ns = pair ? n : (n + 1 - s) / 2;  // tiles of this stream
        const int parts = SPLIT && split_weights((P.q_off[p.r + 1] - P.q_off[p.r]) * a.G) ? 2 : 1;
        if (ns > 0) {
          if (!(alive = wait(&q_ready[s], nq++ & 1))) break;
          tc_fence_after();
        }
        const uint64_t qd = smem_desc_sw128(sbase + C::OFF_Q + (pair ? s : 0) * C::Q_BYTES, 16, 1024);
        // S(j), then O += P(j - 1) V
        for (int j = 0; j <= ns && ns > 0; ++j) {
          if (j < ns) {
            const int it = base + (pair ? j : 2 * j + s), st = it % C::K_STAGES, c = cs + j, b = c & 1;
            if (!(alive = wait(&k_full[st], (it / C::K_STAGES) & 1))) break;
            // P(j - 2), which S(j) overwrites, has been used
            if (j > 1 && !(alive = wait(&pv_done[2 * s + b], ((c >> 1) - 1) & 1))) break;
            tc_fence_after();
            const uint64_t kd = smem_desc_sw128(sbase + C::OFF_K + st * C::KV_BYTES, 16, 1024);
#pragma unroll
            for (int k = 0; k < D / C::UK; ++k) {
              const int box = k * C::UK / C::KCH, in = (k * C::UK % C::KCH) * C::ELT;
              umma_ss_warp<C::KIND_QK>(s_col + b * 64, qd + static_cast<uint64_t>((box * (128 * 128) + in) >> 4),
                                       kd + static_cast<uint64_t>((box * (C::TILE * 128) + in) >> 4), C::IDESC_S,
                                       k > 0 ? 1u : 0u);
            }
            umma_commit_warp(&s_full[2 * s + b]);
            umma_commit_warp(&k_empty[st]);
            if (!pair) umma_commit_warp(&k_empty[st]);
          }
          if (j > 0) {
            const int it = base + (pair ? j - 1 : 2 * (j - 1) + s), st = it % C::V_STAGES, c = cs + j - 1, b = c & 1;
            const int vs = C::E4 ? it % C::COPIES : st;
            if (!(alive = wait(&v_ready[vs], (C::E4 ? it / C::COPIES : it / C::V_STAGES) & 1))) break;
            if (!(alive = wait(&p_full[2 * s + b], (c >> 1) & 1))) break;
            tc_fence_after();
            const uint64_t vd = smem_desc_sw128(
                sbase + (C::E4 ? C::OFF_V16 + vs * C::V16_BYTES : C::OFF_V + st * C::KV_BYTES), C::TILE * 128, 1024);
#pragma unroll
            for (int part = 0; part < (SPLIT ? 2 : 1); ++part) {
              if (part >= parts) break;
#pragma unroll
              for (int k = 0; k < C::TILE / 16; ++k)
                umma_ts_warp<1>(o_col, s_col + b * 64 + part * 32 + k * 8,
                                vd + static_cast<uint64_t>((k * 16 * 128) >> 4), C::IDESC_PV,
                                (part > 0 || k > 0 || j > 1) ? 1u : 0u);
            }
            uint64_t* used = C::E4 ? &v_used[vs] : &v_empty[st];
            umma_commit_warp(used);
            if (!pair) umma_commit_warp(used);
            umma_commit_warp(&pv_done[2 * s + b]);
          }
        }
        cs += ns;
        base += n;
      }
      // No product in flight when the CTA ends.
      umma_commit_warp(&all_done[s]);
      volatile int no_abort = 0;
      mbar_wait(&all_done[s], 0, &no_abort, &status_word, a.wait_limit_ns / 5);
    } else if (warp >= 12) {
      // ---------------------------------------------------------------- V: a warp per tile, a lane per two keys
      // (A warp's barriers and fence then wait while the others work.)  The loop is kept small: with its 16
      // chunks unrolled the warps of this CTA thrashed the instruction cache, 177 us instead of 150.
      int it = 0;
      bool alive = true;
      for (long long u = u0; u < u1 && alive;) {
        const WidePiece p = wide_piece(pre, len, a, P, u, u1);
        const int keys = len[p.r], base = keys - (P.q_off[p.r + 1] - P.q_off[p.r]);
        for (int t = p.t0; t < p.t1; ++t, ++it) {
          if (it % C::V_WARPS != warp - 12) continue;
          const int st = it % C::V_STAGES;
          if (!(alive = wait(&v_full[st], (it / C::V_STAGES) & 1))) break;
          const uint64_t valid = valid_v[st];
          const uint32_t v_at = sbase + C::OFF_V + st * C::KV_BYTES;
          bool bad = false;
          if constexpr (C::E4) {
            const int copy = it % C::COPIES, turn = it / C::COPIES;
            if (turn > 0 && !(alive = wait(&v_used[copy], (turn - 1) & 1))) break;
            const uint32_t out = sbase + C::OFF_V16 + copy * C::V16_BYTES;
            const auto widen = [&](int row, int c, uint4 x) {
              sts16(out + box_addr<C::TILE>(row, 2 * c), make_uint4(widen_lo(x.x), widen_hi(x.x), widen_lo(x.y), widen_hi(x.y)));
              sts16(out + box_addr<C::TILE>(row, 2 * c + 1),
                    make_uint4(widen_lo(x.z), widen_hi(x.z), widen_lo(x.w), widen_hi(x.w)));
            };
            uint32_t nan = 0;
            if (valid == ~0ull && (t + 1) * C::TILE <= base) {
#pragma unroll 1
              for (int i = 0; i < 2 * (D / 32); ++i) {
                const int row = lane + 32 * (i & 1), c = i & ~1;
                const uint4 x = lds16(v_at + box_addr<C::TILE>(row, c)), y = lds16(v_at + box_addr<C::TILE>(row, c + 1));
                widen(row, c, x);
                widen(row, c + 1, y);
                nan |= nan_bytes(x.x) | nan_bytes(x.y) | nan_bytes(x.z) | nan_bytes(x.w);
                nan |= nan_bytes(y.x) | nan_bytes(y.y) | nan_bytes(y.z) | nan_bytes(y.w);
              }
            } else {
              nan = 1;
            }
            if (__any_sync(0xFFFFFFFFu, nan != 0)) {
              // With the tile's end, drafted keys or a NaN: row by row.
#pragma unroll 1
              for (int i = 0; i < 2 * (D / 16); ++i) {
                const int row = lane + 32 * (i & 1), c = i >> 1;
                const bool drafted = t * C::TILE + row >= base;
                uint4 x = (valid >> row) & 1 ? lds16(v_at + box_addr<C::TILE>(row, c)) : make_uint4(0, 0, 0, 0);
                const uint32_t m[4] = {nan_bytes(x.x), nan_bytes(x.y), nan_bytes(x.z), nan_bytes(x.w)};
                const bool any = (m[0] | m[1] | m[2] | m[3]) != 0;
                bad |= any && drafted;
                if (any && drafted) {
                  x.x = finite_only<true>(x.x);
                  x.y = finite_only<true>(x.y);
                  x.z = finite_only<true>(x.z);
                  x.w = finite_only<true>(x.w);
                }
                widen(row, c, x);
                if (any && !drafted) {
#pragma unroll 1
                  for (int e = 0; e < 16; ++e)
                    if ((m[e >> 2] >> (8 * (e & 3) + 7)) & 1)
                      asm volatile("st.shared.u16 [%0], %1;" ::"r"(out + box_addr<C::TILE>(row, 2 * c + (e >> 3)) + 2 * (e & 7)),
                                   "h"(static_cast<uint16_t>(0x7FFF))
                                   : "memory");
                }
              }
            }
          } else if (valid != ~0ull || (t + 1) * C::TILE > base) {
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              const int row = lane + 32 * h;
              if (!((valid >> row) & 1)) {
#pragma unroll 1
                for (int c = 0; c < D / 8; ++c) sts16(v_at + box_addr<C::TILE>(row, c), make_uint4(0, 0, 0, 0));
              } else if (t * C::TILE + row >= base) {
#pragma unroll 1
                for (int c = 0; c < D / 8; ++c) {
                  const uint32_t at = v_at + box_addr<C::TILE>(row, c);
                  const uint4 x0 = lds16(at);
                  const uint4 x = make_uint4(finite_only<false>(x0.x), finite_only<false>(x0.y), finite_only<false>(x0.z),
                                             finite_only<false>(x0.w));
                  const bool cut = x.x != x0.x || x.y != x0.y || x.z != x0.z || x.w != x0.w;
                  if (cut) sts16(at, x);
                  bad |= cut;
                }
              }
            }
          }
          if (bad) *static_cast<volatile int*>(&bad_v) = 1;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if constexpr (C::E4) {
              mbar_arrive(&v_empty[st]);
              mbar_arrive(&v_ready[it % C::COPIES]);
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
      // Parity with up to 64 rows: they lie in the M tile twice, and stream 1 takes the copy in rows 64 on,
      // which other schedulers' warps read.
      const int left = rows - p.rt * 256, shift = !pair && left <= 64 ? 64 : 0;
      const int local = pair ? s * 128 + rt : rt - s * shift;    // row of the item that this thread has
      const int row = p.rt * 256 + local;                        // packed row of the sequence
      const bool mine = local >= 0 && row < rows;
      const int tok = mine ? row / a.G : 0, h = g * a.G + (mine ? row - tok * a.G : 0);
      const bool busy = __any_sync(0xFFFFFFFFu, mine);
      [[maybe_unused]] const bool split = SPLIT && split_weights(rows);
      const int n = p.t1 - p.t0;

      // Q: the warp's 32 rows, RPL of them at a time with their chunks side by side in the lanes, every load
      // on its way at once (parity: by stream 0).  The rows before have been used: this warp has seen the
      // last product of the piece before.
      if (pair || s == 0) {
        constexpr int CH = D * C::ELT / 16, RPL = 32 / CH;
        const uint32_t q_at = sbase + C::OFF_Q + (pair ? s : 0) * C::Q_BYTES;
        const int ch = lane % CH, r0 = (warp & 3) * 32 + lane / CH;  // this lane's chunk and first row
        const int from0 = p.rt * 256 + (pair ? s * 128 : 0) + (shift ? r0 & 63 : r0);
        int ft = from0 / a.G, fh = from0 - ft * a.G;                 // token and head go along by steps of RPL rows
        const int step_t = RPL / a.G, step_h = RPL - step_t * a.G;
        const char* src = static_cast<const char*>(a.q) +
                          (static_cast<int64_t>(tok0) * a.q_stride + static_cast<int64_t>(g) * a.G * D) * C::ELT + 16 * ch;
        uint4 v[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          v[i] = make_uint4(0, 0, 0, 0);
          if (from0 + i * RPL < rows) v[i] = __ldg(reinterpret_cast<const uint4*>(src + (ft * a.q_stride + fh * D) * C::ELT));
          ft += step_t;
          fh += step_h;
          if (fh >= a.G) {
            fh -= a.G;
            ++ft;
          }
        }
#pragma unroll
        for (int i = 0; i < CH; ++i) sts16(q_at + box_addr<128>(r0 + i * RPL, ch), v[i]);
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
        const int b = cs & 1;
        if (alive) alive = wait(&s_full[2 * s + b], (cs >> 1) & 1);
        if (!alive) continue;
        tc_fence_after();
        if (busy) {
          const uint64_t valid = valid_k[(base_it + i) % VALID];
          const int j0 = (p.t0 + i) * C::TILE;
          uint32_t v[64];
          tmem_ld64_now(s_at + 64 * b, v);
          if (j0 + C::TILE > base || valid != ~0ull) {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const uint32_t vis = static_cast<uint32_t>(valid >> (32 * w)) &
                                   (seen16(mask, j0 + 32 * w, base) | (seen16(mask, j0 + 32 * w + 16, base) << 16));
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((vis >> e) & 1u)) v[32 * w + e] = 0xFF800000u;
            }
          }
          float top[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) top[e] = fmaxf(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
#pragma unroll
          for (int e = 8; e < 64; e += 8)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              top[x] = fmax3(top[x], __uint_as_float(v[e + 2 * x]), __uint_as_float(v[e + 2 * x + 1]));
          const float m_new = fmaxf(m_run, fmax3(top[0], top[1], fmaxf(top[2], top[3])) * s2);
          // The maximum is raised, and O rescaled, when it grew by more than 2^8.
          const bool need = m_new > m_run + C::LAZY;
          if (done > 0 && __any_sync(0xFFFFFFFFu, need)) {
            // O is whole: the products of the tile before have ended
            alive = wait(&pv_done[2 * s + (b ^ 1)], ((cs - 1) >> 1) & 1);
            tc_fence_after();
            const float f = need ? fast_exp2(m_run - m_new) : 1.f;
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              tmem_ld16_now(o_at + 16 * c, o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st16(o_at + 16 * c, o);
            }
          }
          if (need) {
            l_run *= fast_exp2(m_run - m_new);  // (no maximum yet: 0 x 0, or NaN when the scores were NaN)
            m_run = m_new;
          }
          const float off = m_run == neg_inf() ? 0.f : C::P_BIAS - m_run;
          const float2 s22 = make_float2(s2, s2), off2 = make_float2(off, off);
          float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t hi[16];
            float2 w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 x = __ffma2_rn(
                  make_float2(__uint_as_float(v[32 * c + 2 * e]), __uint_as_float(v[32 * c + 2 * e + 1])), s22, off2);
              w[e] = make_float2(fast_exp2(x.x), fast_exp2(x.y));
              acc[e & 1] = __fadd2_rn(acc[e & 1], w[e]);
              hi[e] = C::E4 ? pack_f16x2(w[e].x, w[e].y) : pack_bf16x2(w[e].x, w[e].y);
            }
            tmem_st16(s_at + 64 * b + 16 * c, hi);
            if (SPLIT && split) {
              uint32_t lo[16];
#pragma unroll
              for (int e = 0; e < 16; ++e)
                lo[e] = pack_bf16x2(w[e].x - __uint_as_float(hi[e] << 16), w[e].y - __uint_as_float(hi[e] & 0xFFFF0000u));
              tmem_st16(s_at + 64 * b + 32 + 16 * c, lo);
            }
          }
          l_run += (acc[0].x + acc[1].x) + (acc[0].y + acc[1].y);
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * s + b]);
      }
      if (done > 0 && alive) alive = wait(&pv_done[2 * s + ((cs - 1) & 1)], ((cs - 1) >> 1) & 1);
      tc_fence_after();
      base_it += n;

      // ---------------- epilogue
      const bool any_tile = done > 0 && alive && busy;
      const bool whole = p.t0 == 0 && p.t1 == p.tiles;
      const int slot = (grp * a.Hkv + g) * 2 + (nth == 0 ? 0 : 1);
      const int64_t part_row = static_cast<int64_t>(slot) * a.part_rows + local;
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
            if (store && (n > 0 || whole)) write(o, 32 * c, f);
          }
          if (store) write_stats(m_run, l_run);
        }
      } else {
        // Stream 1 hands its sums and O to stream 0 through the second Q tile, MERGE columns at a time.
        float* buf = reinterpret_cast<float*>(smem + C::OFF_Q + C::Q_BYTES);
        if (s == 1 && mine) ml_smem[local] = make_float2(m_run, l_run);
        asm volatile("bar.sync 1, 256;" ::: "memory");
        float top = m_run, total = l_run, f0 = 1.f, f1 = 0.f;
        bool saw1 = false;  // stream 1 saw a key of the row: its factor may be 0 and its O infinite or NaN
        if (s == 0) {
          const float2 other = mine ? ml_smem[local] : make_float2(neg_inf(), 0.f);
          top = fmaxf(m_run, other.x);
          f0 = l_run == 0.f ? 0.f : fast_exp2(m_run - top);
          saw1 = other.y != 0.f;
          f1 = saw1 ? fast_exp2(other.x - top) : 0.f;
          total = l_run * f0 + other.y * f1;
          if (l_run == 0.f) total = other.y * f1;
          if (!saw1) total = l_run * f0;
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
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (mine) buf[(c + e) * 128 + local] = __uint_as_float(o[e]);
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
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                // a stream that saw nothing of the row leaves zeros
                float x = l_run == 0.f ? 0.f : __uint_as_float(o[e]) * f0;
                if (saw1) x += buf[(c + e) * 128 + local] * f1;
                o[e] = __float_as_uint(x);
              }
              if (store) write(o, c0 + c, f);
            }
          }
          asm volatile("bar.sync 1, 256;" ::: "memory");  // (the last one: the buffer is Q's again)
        }
        if (s == 0 && store) write_stats(top, total);
      }
      // Values of drafted keys that V's warps cleared come back now, for the rows that see the key.
      if (*static_cast<volatile int*>(&bad_v) != 0 && keys > 0 && p.t1 * C::TILE > base && store && n > 0 &&
          (pair || s == 0))
        add_cleared<DT, D>(a, p.r, g, base, q_len, mask, p.t0 * C::TILE, p.t1 * C::TILE,
                           whole ? nullptr : a.part_o + part_row * D,
                           whole ? static_cast<uint16_t*>(a.out) + (out_row * a.Hq + h) * D : nullptr);
      tc_fence_before();
      // The group that holds an item's first piece tells join_kernel how many follow.
      u = p.next;
      if (g == 0 && tid == 0 && u >= u1) {
        int4 d = make_int4(-1, 0, 0, 0);
        if (p.t0 == 0 && p.t1 < p.tiles) {
          d = make_int4(nth == 0 ? 0 : 1, p.r, p.rt, group_of(units, ng, u1 + (p.w * p.tiles - p.end) - 1) - grp + 1);
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
  using C = Wide<DT, D>;
  const auto kernel = a.box_rows < 64 ? tree_wide_kernel<DT, D, SPLIT, true> : tree_wide_kernel<DT, D, SPLIT, false>;
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_chained(kernel, dim3(a.groups * a.Hkv), kWideThreads, C::SMEM, stream, 1, a, P);
}

}  // namespace

cudaError_t launch_tree_wide(int dtype, int D, const DecodeArgs& a, const DecodePlan& P, cudaStream_t stream) {
  bool split = false;
  for (int r = 0; r < P.num_seqs; ++r) split |= split_weights((P.q_off[r + 1] - P.q_off[r]) * a.G);
  if (dtype == FP2_BF16 && D == 128) return split ? run<1, 128, true>(a, P, stream) : run<1, 128, false>(a, P, stream);
  if (dtype == FP2_BF16 && D == 64) return split ? run<1, 64, true>(a, P, stream) : run<1, 64, false>(a, P, stream);
  if (dtype == FP2_E4M3 && D == 128) return run<2, 128, false>(a, P, stream);
  return cudaErrorInvalidValue;
}

}  // namespace fp2
