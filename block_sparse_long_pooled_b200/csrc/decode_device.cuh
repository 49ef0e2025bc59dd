// What the kernels that read a KV cache share: the axis of units that balances a ragged batch, the TMA
// producer that walks its pages, and the masks of drafted tokens.
#pragma once

#include "fp2_device.cuh"
#include "fp2_kernels.h"
#include "serve_kernels.h"

namespace fp2 {

namespace {

constexpr float kLn2 = 0.6931471805599453f;

// ------------------------------------------------------------------ small PTX wrappers

FP2_DEVICE void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
      "[%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
FP2_DEVICE float neg_inf() { return __uint_as_float(0xFF800000u); }
FP2_DEVICE float pos_inf() { return __uint_as_float(0x7F800000u); }

// ------------------------------------------------------------------ the axis of units

// Keys of sequence r, or -1 when its length is no valid one (below its drafted tokens, above
// max_kv_len): such a sequence has one empty tile and its rows see nothing.
FP2_DEVICE int seq_keys(const DecodeArgs& a, const DecodePlan& P, int r) {
  const int n = a.kv_len[r];
  return (n < P.q_off[r + 1] - P.q_off[r] || n > a.max_kv_len) ? -1 : n;
}

// Lengths into len[] and the exclusive prefix of the units per sequence into pre[0 .. num_seqs]:
// units = row tiles (at least least_tiles) * max(1, key tiles).  The whole block reads the lengths at once (one trip to
// memory whatever the batch), one warp adds up.  Ends with the block synchronised.
template <int TILE>
FP2_DEVICE void scan_units(const DecodeArgs& a, const DecodePlan& P, int rows_per_tile, int least_tiles, long long* pre,
                           int* len, uint32_t* status) {
  for (int r = threadIdx.x; r < P.num_seqs; r += blockDim.x) {
    len[r] = seq_keys(a, P, r);
    if (len[r] < 0) set_status(status, FP2_DEV_LEN_OOB);
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    long long run = 0;
    for (int base = 0; base < P.num_seqs; base += 32) {
      const int r = base + lane;
      long long u = 0;
      if (r < P.num_seqs) {
        const int rows = (P.q_off[r + 1] - P.q_off[r]) * a.G;
        const int tiles = len[r] <= 0 ? 1 : (len[r] + TILE - 1) / TILE;
        u = static_cast<long long>(max((rows + rows_per_tile - 1) / rows_per_tile, least_tiles)) * tiles;
      }
      long long inc = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += v;
      }
      if (r < P.num_seqs) pre[r] = run + inc - u;
      run += __shfl_sync(0xFFFFFFFFu, inc, 31);
    }
    if (lane == 0) pre[P.num_seqs] = run;
  }
  __syncthreads();
}

// Groups that get a share: no more than there are units.
FP2_DEVICE int active_groups(long long units, int groups) {
  return static_cast<int>(units < 1 ? 1 : (units < groups ? units : groups));
}

// The group that works on unit u: shares begin at units * group / groups.
FP2_DEVICE int group_of(long long units, int groups, long long u) {
  return static_cast<int>(((u + 1) * groups - 1) / units);
}

struct Piece {  // key tiles [t0, t1) of one item
  int r, rt, t0, t1, tiles;
};

// The piece that starts at unit u (u < u1 <= pre[num_seqs]).
template <int TILE>
FP2_DEVICE Piece piece_at(const long long* pre, const int* len, int num_seqs, long long u, long long u1) {
  int lo = 0, hi = num_seqs - 1;  // the last r with pre[r] <= u: sequences without rows have no units
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= u) lo = mid; else hi = mid - 1;
  }
  Piece p;
  p.r = lo;
  p.tiles = len[lo] <= 0 ? 1 : (len[lo] + TILE - 1) / TILE;
  const int rem = static_cast<int>(u - pre[lo]);
  p.rt = rem / p.tiles;
  p.t0 = rem - p.rt * p.tiles;
  const long long left = u1 - u;
  p.t1 = p.tiles - p.t0 <= left ? p.tiles : p.t0 + static_cast<int>(left);
  return p;
}

// The CTA's status bits go to a word of its own in scratch (see serve_kernels.h); every thread
// calls it, with nothing of the CTA's left to do.
FP2_DEVICE void store_status(const DecodeArgs& a, const uint32_t* status) {
  __syncthreads();
  if (threadIdx.x == 0) {
    a.scratch[kStatusFirst + blockIdx.x] = *status;
    if (blockIdx.x == 0) *reinterpret_cast<uint2*>(a.scratch) = make_uint2(kStatusMore, kStatusMagic | gridDim.x);
  }
}

// ------------------------------------------------------------------ producer

// Brings one tile of TILE keys (from key j0) of K or V into shared memory, page by page, in boxes of
// 128 bytes x up to 64 rows, and completes `bar`.  Called by a whole warp: lane l looks after box l, and
// the ids of 32 pages at a time sit in the lanes.  `valid` (64 bits a word) tells which rows hold a key of
// the sequence: rows past its end and rows of a page id out of range do not, and are not loaded.
// The warp's instructions follow each other at some five cycles apiece, so their number sets the pace of
// the whole kernel once a tile takes less than they do: a lane walking the boxes twice, with divisions by
// the page size, took 1,800 cycles a tile, the general form below still 1,100; whole tiles go a short way
// of their own.  SMALL is for pages below 64 rows: one form for all made a batch of 64 requests 1 % slower, and
// without it, in pages of 16, 15 requests of 8K e4m3 keys took key mass 55 us instead of 40, and a tree of 28
// rows at 128K bf16 keys 118 us instead of 103.
template <int TILE, int ELT, int D, bool SMALL>
struct Producer {
  static constexpr int HALVES = D * ELT / 128;            // boxes side by side
  int page_base = -1, page_id = -1, seq = -1;             // lanes hold pages page_base .. + 31 of sequence seq

  FP2_DEVICE void fetch_pages(const DecodeArgs& a, int r, int keys, int first) {
    const int mine = first + static_cast<int>(threadIdx.x & 31);
    seq = r;
    page_base = first;
    page_id = mine <= (keys - 1) >> a.page_shift ? a.page_table[static_cast<int64_t>(r) * a.max_pages + mine] : -1;
  }

  FP2_DEVICE void load(const DecodeArgs& a, const CUtensorMap* map, int r, int keys, int g, int j0, uint32_t dst,
                       uint64_t* bar, uint64_t* valid, uint32_t* status, bool withhold) {
    const int lane = threadIdx.x & 31;
    const bool paged = a.page_table != nullptr;
    if (!SMALL && a.box_rows == 64 && j0 + TILE <= keys) {
      const int j = j0 + (lane & (TILE / 64 - 1)) * 64;
      int outer = r, row = j;
      if (paged) {
        if (seq != r || (j0 >> a.page_shift) < page_base || ((j0 + TILE - 1) >> a.page_shift) >= page_base + 32)
          fetch_pages(a, r, keys, j0 >> a.page_shift);
        outer = __shfl_sync(0xFFFFFFFFu, page_id, (j >> a.page_shift) - page_base);
        row = j & (a.page_size - 1);
      }
      if (__all_sync(0xFFFFFFFFu, !paged || static_cast<unsigned>(outer) < static_cast<unsigned>(a.num_pages))) {
        if (lane == 0) {
#pragma unroll
          for (int w = 0; w < TILE / 64; ++w) valid[w] = ~0ull;
          mbar_arrive_expect_tx(bar, TILE * D * ELT);
        }
        __syncwarp();
        if (lane < TILE / 64 && !withhold) {
#pragma unroll
          for (int h = 0; h < HALVES; ++h)
            tma_load_4d(dst + h * (TILE * 128) + lane * (64 * 128), map, bar, h * (128 / ELT), g, row, outer);
        }
        return;
      }
    }
    if (SMALL && j0 + TILE <= keys) {                     // the same for smaller pages
      const int boxes = TILE >> a.box_shift, j = j0 + ((lane & (boxes - 1)) << a.box_shift);
      if (seq != r || (j0 >> a.box_shift) < page_base || ((j0 + TILE - 1) >> a.box_shift) >= page_base + 32)
        fetch_pages(a, r, keys, j0 >> a.box_shift);
      const int outer = __shfl_sync(0xFFFFFFFFu, page_id, (j >> a.box_shift) - page_base);
      if (__all_sync(0xFFFFFFFFu, static_cast<unsigned>(outer) < static_cast<unsigned>(a.num_pages))) {
        if (lane == 0) {
#pragma unroll
          for (int w = 0; w < TILE / 64; ++w) valid[w] = ~0ull;
          mbar_arrive_expect_tx(bar, TILE * D * ELT);
        }
        __syncwarp();
        if (lane < boxes && !withhold) {
#pragma unroll
          for (int h = 0; h < HALVES; ++h)
            tma_load_4d(dst + h * (TILE * 128) + (lane << a.box_shift) * 128, map, bar, h * (128 / ELT), g, 0, outer);
        }
        return;
      }
    }
    const int step = a.box_rows;                          // a power of two: 64, or the page size below that
    const int j = j0 + lane * step;
    bool there = lane * step < TILE && j < keys;
    int outer = r, row = j;
    if (paged) {
      const int first = j0 >> a.page_shift, last = (min(j0 + TILE, keys) - 1) >> a.page_shift;
      if (keys > j0 && (seq != r || first < page_base || last >= page_base + 32)) fetch_pages(a, r, keys, first);
      const int pg = j >> a.page_shift;
      row = j - (pg << a.page_shift);
      outer = __shfl_sync(0xFFFFFFFFu, page_id, there ? pg - page_base : 0);
      if (there && (outer < 0 || outer >= a.num_pages)) {
        set_status(status, FP2_DEV_PAGE_OOB);
        there = false;
      }
    }
    const uint32_t boxes = __ballot_sync(0xFFFFFFFFu, there);
    if (lane == 0) {
      const uint64_t box = step == 64 ? ~0ull : (1ull << step) - 1;
#pragma unroll
      for (int w = 0; w < TILE / 64; ++w) {
        uint64_t ok = 0;
        for (int b = 0; b < 64; b += step)
          if ((boxes >> ((64 * w + b) >> a.box_shift)) & 1u) ok |= box << b;
        const int end = keys - (j0 + 64 * w);             // rows of this word before the sequence's end
        valid[w] = end >= 64 ? ok : (end <= 0 ? 0 : ok & ((1ull << end) - 1));
      }
      if (boxes != 0)
        mbar_arrive_expect_tx(bar, __popc(boxes) * step * D * ELT);
      else
        mbar_arrive(bar);
    }
    __syncwarp();  // armed before the first byte arrives
    if (there && !withhold) {
#pragma unroll
      for (int h = 0; h < HALVES; ++h)
        tma_load_4d(dst + h * (TILE * 128) + lane * step * 128, map, bar, h * (128 / ELT), g, row, outer);
    }
  }
};

// Which of the 16 keys from key j a token sees, bit by bit: all below `base` (the first drafted
// key), of the drafted ones those in its mask.
FP2_DEVICE uint32_t seen16(uint64_t mask, int j, int base) {
  const int off = j - base;
  if (off >= 0) return off < 64 ? static_cast<uint32_t>(mask >> off) & 0xFFFFu : 0u;
  if (off <= -16) return 0xFFFFu;
  return static_cast<uint32_t>((mask << -off) | ((1ull << -off) - 1)) & 0xFFFFu;
}
FP2_DEVICE uint64_t token_mask(const DecodeArgs& a, int t0, int i) {
  return a.mask != nullptr ? a.mask[static_cast<int64_t>(t0) + i] : (i >= 63 ? ~0ull : (2ull << i) - 1);
}

}  // namespace

}  // namespace fp2
