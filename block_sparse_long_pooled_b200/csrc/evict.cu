// Eviction from a KV cache by accumulated attention weight.
//
// Per (sequence, KV head) with n keys and a budget B: all keys when n <= B, else the first `sink`,
// the last `window` and, of the others, the B - sink - window heaviest (ties: lowest index).  The
// kept keys go, in ascending order, to rows 0 .. N-1 of another cache, with their weights and old
// indexes.
//
// The weights are read, the kept rows of K and V read and written: bytes bound it, and for short
// caches the number of dependent steps.  One launch does both parts.  A cluster of 1 to 16 CTAs owns
// one (sequence, KV head), each rank an equal range of its keys.  Selection is a radix select on the
// weights' bits in order-preserving form: up to three histograms (11, 11 and 10 bits) of the keys that
// agree with the digits found so far give the weight of the last key to keep and how many of its equals
// are kept; it ends early when a digit's keys are all kept.  Each rank publishes its histogram and the
// sums of 64 groups of 32 bins; warp q of every rank reads rank q's groups, then its 32 bins of the one
// group that matters: one cluster barrier a digit, little traffic, one trip to another SM at a time.
// (Adding the histograms up in rank 0 cost 6 us a digit for 16 ranks, one warp reading all ranks 5.)
// Weights of zero, in earnest the most frequent one, are counted by ballot: one shared-memory add a
// warp instead of one a key on the same word.  Up to 16 keys a thread stay in registers in between
// (8,192 a rank); longer ranges are read again from L2.  Ballots in index order then give every kept key
// its row: what the ranks before keep follows from their histograms, so nothing depends on timing.  After
// that the rows are moved, each rank an equal share of the output rows whatever range they came from: the
// addresses of 512 rows at a time are looked up first, so that the copies themselves wait only for their
// data.
//
// Measured: 128K keys of 8 KV heads to 8K, bf16: 37 us (11 us of bytes): 3 for the weights, 3 to 4 a
// digit, 5 for the rows' places, 7 to 9 for the rows themselves.  24 sequences of 0.9K to 32K to 2K, e4m3,
// 33 us (14 us of bytes); five of up to 2K to 512 14 us.
#include <cooperative_groups.h>

#include <cstddef>

#include "fp2_device.cuh"
#include "serve_kernels.h"

namespace fp2 {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2048, kGroups = kBins / 32, kMaxRanks = 16;
constexpr int kHeld = 16;         // keys a thread holds
constexpr int kChunk = kThreads;  // rows whose addresses are looked up at a time

// Weights in an order that unsigned comparison follows.  -0 equals 0; NaN counts as the heaviest.
FP2_DEVICE uint32_t ordered(float f) {
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
  if ((u << 1) == 0u) return 0x80000000u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct EvictShared {
  alignas(16) uint32_t bins[3][kBins];  // this rank's histograms, read 16 bytes at a time
  uint32_t groups[3][kGroups];
  uint32_t got[kMaxRanks][kGroups];  // groups, then bins, of every rank
  uint32_t got_bins[kMaxRanks][32];
  uint32_t warp_sel[kWarps], warp_eq[kWarps];
  int64_t from[kChunk], to[kChunk];
  uint32_t status;
};
static_assert(alignof(EvictShared) >= 16 && kBins * sizeof(uint32_t) % 16 == 0 && kBins == 4 * kThreads, "uint4 of bins");
static_assert(offsetof(EvictShared, groups) % 8 == 0 && offsetof(EvictShared, got) % 8 == 0, "uint2 of groups");

// Byte offset of (token j, KV head g) of sequence r, or -1 for a page id out of range.
FP2_DEVICE int64_t row_offset(const CacheView& c, int r, int j, int g, int row_bytes, uint32_t* status) {
  int64_t outer = r, row = j;
  if (c.page_table != nullptr) {
    const int pg = j / c.rows;
    outer = c.page_table[static_cast<int64_t>(r) * c.max_pages + pg];
    row = j - pg * c.rows;
    if (outer < 0 || outer >= c.num_outer) {
      set_status(status, FP2_DEV_PAGE_OOB);
      return -1;
    }
  }
  return outer * c.stride_outer + row * c.stride_tok + static_cast<int64_t>(g) * row_bytes;
}

template <int LANES>  // 16-byte pieces of a row
__global__ void __launch_bounds__(kThreads, 2) evict_kernel(const __grid_constant__ EvictArgs a) {
  __shared__ EvictShared s;
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int row = blockIdx.x / ranks, r = row / a.Hkv, g = row - r * a.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_launch_next();
  grid_wait();

  int n = a.kv_len[r];
  const bool bad = n < 0 || n > a.max_kv_len;
  if (bad) n = 0;  // such a sequence keeps nothing
  const int N = n < a.budget ? n : a.budget;
  const float* mass = a.mass + static_cast<int64_t>(row) * a.mass_stride;
  int32_t* kept = a.kept + static_cast<int64_t>(row) * a.budget;
  float* mass_out = a.mass_out + static_cast<int64_t>(row) * a.budget;
  const int free0 = a.sink, free1 = n - a.window;  // the keys that compete, when some are dropped

  if (tid == 0) s.status = bad && g == 0 ? FP2_DEV_LEN_OOB : 0u;
  if (g == 0 && rank == 0 && tid == 0) a.kv_len_out[r] = N;
  for (int i = N + rank * kThreads + tid; i < a.budget; i += ranks * kThreads) {
    kept[i] = -1;
    mass_out[i] = 0.f;
  }

  const auto sync = [&] {
    if (ranks > 1)
      cluster.sync();
    else
      __syncthreads();
  };
  if (N == n) {
    // nothing is dropped
    __syncthreads();
    for (int i = rank * kThreads + tid; i < N; i += ranks * kThreads) {
      kept[i] = i;
      mass_out[i] = mass[i];
    }
  } else {
    // Ranges of 32-key steps: of this rank, and in it of this warp.
    const int steps = (n + 31) / 32;
    const int first = static_cast<int>(static_cast<int64_t>(steps) * rank / ranks);
    const int last = static_cast<int>(static_cast<int64_t>(steps) * (rank + 1) / ranks);
    const int w0 = first + static_cast<int>(static_cast<int64_t>(last - first) * warp / kWarps);
    const int w1 = first + static_cast<int>(static_cast<int64_t>(last - first) * (warp + 1) / kWarps);
    const bool held = w1 - w0 <= kHeld;  // every key of this warp's stays in registers

    uint32_t u[kHeld];
    const auto fetch = [&](int t0) {  // steps t0 .. of this warp, all loads on their way at once
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        const int j = (t0 + i) * 32 + lane;
        u[i] = t0 + i < w1 && j < n ? __float_as_uint(__ldg(mass + j)) : 0u;
      }
#pragma unroll
      for (int i = 0; i < kHeld; ++i) u[i] = ordered(__uint_as_float(u[i]));
    };
    fetch(w0);
    for (int i = tid; i < 3 * kBins; i += kThreads) (&s.bins[0][0])[i] = 0;
    uint32_t need = static_cast<uint32_t>(a.budget - a.sink - a.window);  // of the competing keys
    uint32_t prefix = 0, mask = 0;
    // What the ranks before this one keep: first of the keys that do not compete.
    const int low_keys = min(first * 32, n);
    uint32_t sel_before = static_cast<uint32_t>(min(low_keys, free0) + max(low_keys - free1, 0)), eq_before = 0;
    __syncthreads();
    // need == 0: no competing key stays, and no key's order value exceeds this threshold.
    bool done = need == 0;
    if (done) prefix = 0xFFFFFFFFu;
#pragma unroll 1
    for (int pass = 0; pass < 3 && !done; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
      const uint32_t digit = pass == 2 ? 1023u : 2047u;
      uint32_t* mine = s.bins[pass];
#pragma unroll 1
      for (int t0 = w0; t0 < w1; t0 += kHeld) {
        if (!held) fetch(t0);
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
          if (t0 + i >= w1) break;
          const int j = (t0 + i) * 32 + lane;
          const bool counts = j >= free0 && j < free1 && (u[i] & mask) == prefix;
          const bool zero = counts && u[i] == 0x80000000u;
          const uint32_t zeros = __ballot_sync(0xFFFFFFFFu, zero);
          if (counts && (!zero || (zeros & ((1u << lane) - 1)) == 0))
            atomicAdd(&mine[(u[i] >> shift) & digit], zero ? static_cast<uint32_t>(__popc(zeros)) : 1u);
        }
      }
      __syncthreads();
      {
        // thread t: bins 4t .. 4t + 3; eight threads a group
        const uint4 four = *reinterpret_cast<const uint4*>(mine + 4 * tid);
        uint32_t sum = (four.x + four.y) + (four.z + four.w);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if ((lane & 7) == 0) s.groups[pass][tid >> 3] = sum;
      }
      sync();
      // From the heaviest down: lane l has groups 63 - 2l and 62 - 2l, then bin 31 - l of the group.  Every
      // warp comes to the same answer from all ranks' counts.
      const auto before = [&](uint32_t x) {  // sum of the lanes below
        uint32_t inc = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
          if (lane >= o) inc += v;
        }
        return inc - x;
      };
      if (ranks > 1 && warp < ranks)
        *reinterpret_cast<uint2*>(&s.got[warp][2 * lane]) =
            *reinterpret_cast<const uint2*>(cluster.map_shared_rank(&s.groups[pass][2 * lane], warp));
      if (ranks > 1) __syncthreads();
      uint32_t g0 = 0, g1 = 0, low0 = 0, low1 = 0;  // low: of the ranks before this one
#pragma unroll 4
      for (int q = 0; q < ranks; ++q) {
        const uint2 x = *reinterpret_cast<const uint2*>(ranks > 1 ? &s.got[q][kGroups - 2 - 2 * lane]
                                                                  : &s.groups[pass][kGroups - 2 - 2 * lane]);
        g0 += x.y;
        g1 += x.x;
        if (q == rank - 1) low0 = g0, low1 = g1;
      }
      uint32_t above = before(g0 + g1);
      // The one group, then the one bin, in which the need-th key lies (need is at most all of them).
      const int from = __ffs(__ballot_sync(0xFFFFFFFFu, above < need && above + g0 + g1 >= need)) - 1;
      const bool second = __shfl_sync(0xFFFFFFFFu, above + g0 < need, from);
      const uint32_t left = need - __shfl_sync(0xFFFFFFFFu, second ? above + g0 : above, from);
      const int group = kGroups - 1 - 2 * from - (second ? 1 : 0);
      if (ranks > 1) {
        if (warp < ranks) s.got_bins[warp][lane] = *cluster.map_shared_rank(&mine[group * 32 + lane], warp);
        __syncthreads();
      }
      uint32_t x = 0, low = 0;
#pragma unroll 4
      for (int q = 0; q < ranks; ++q) {
        x += ranks > 1 ? s.got_bins[q][31 - lane] : mine[group * 32 + 31 - lane];
        if (q == rank - 1) low = x;
      }
      above = before(x);
      const int at = __ffs(__ballot_sync(0xFFFFFFFFu, above < left && above + x >= left)) - 1;
      // Keys of the ranks before this one: above the bin (they stay), and in it.
      const int first_group = kGroups - 1 - 2 * lane;
      sel_before += __reduce_add_sync(0xFFFFFFFFu, (first_group > group ? low0 : 0u) + (first_group - 1 > group ? low1 : 0u) +
                                                       (lane < at ? low : 0u));
      eq_before = __shfl_sync(0xFFFFFFFFu, low, at);
      prefix |= static_cast<uint32_t>(group * 32 + 31 - at) << shift;
      mask |= digit << shift;
      need = left - __shfl_sync(0xFFFFFFFFu, above, at);
      if (need == __shfl_sync(0xFFFFFFFFu, x, at)) {
        // All keys with these digits stay: the threshold is the value before them (no weight maps to 0).
        prefix -= 1;
        need = 0;
        done = true;
        sel_before += eq_before;
        eq_before = 0;
      }
    }
    // Keys above `prefix` stay, and of those equal to it the first `need`.
    const auto classify = [&](int i, int t, bool& keep, bool& tie) {
      const int j = t * 32 + lane;
      const bool competes = j >= free0 && j < free1;
      keep = j < n && (!competes || u[i] > prefix);
      tie = competes && u[i] == prefix;
    };
    uint32_t sel = 0, eq = 0;
#pragma unroll 1
    for (int t0 = w0; t0 < w1; t0 += kHeld) {
      if (!held) fetch(t0);
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        if (t0 + i >= w1) break;
        bool keep, tie;
        classify(i, t0 + i, keep, tie);
        sel += __popc(__ballot_sync(0xFFFFFFFFu, keep));
        eq += __popc(__ballot_sync(0xFFFFFFFFu, tie));
      }
    }
    if (lane == 0) {
      s.warp_sel[warp] = sel;
      s.warp_eq[warp] = eq;
    }
    __syncthreads();
    sel_before += __reduce_add_sync(0xFFFFFFFFu, lane < warp ? s.warp_sel[lane & (kWarps - 1)] : 0u);
    eq_before += __reduce_add_sync(0xFFFFFFFFu, lane < warp ? s.warp_eq[lane & (kWarps - 1)] : 0u);
    const uint32_t below = (1u << lane) - 1;
#pragma unroll 1
    for (int t0 = w0; t0 < w1; t0 += kHeld) {
      if (!held) fetch(t0);
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        if (t0 + i >= w1) break;
        bool keep, tie;
        classify(i, t0 + i, keep, tie);
        const uint32_t ks = __ballot_sync(0xFFFFFFFFu, keep), es = __ballot_sync(0xFFFFFFFFu, tie);
        const uint32_t eq_at = eq_before + __popc(es & below);
        const uint32_t pos = sel_before + __popc(ks & below) + min(eq_at, need);  // (ties kept before this key)
        if ((keep || (tie && eq_at < need)) && fp2_check(pos < static_cast<uint32_t>(a.budget), &s.status)) {
          const int j = (t0 + i) * 32 + lane;
          kept[pos] = j;
          // the weight back from its order (no load to wait for; a NaN's own bits are read again)
          mass_out[pos] = u[i] == 0xFFFFFFFFu ? __ldg(mass + j)
                                              : __uint_as_float(u[i] & 0x80000000u ? u[i] & 0x7FFFFFFFu : ~u[i]);
        }
        sel_before += __popc(ks);
        eq_before += __popc(es);
      }
    }
  }
  sync();  // kept[] is complete, and no rank reads another's shared memory from here on

  const int i0 = static_cast<int>(static_cast<int64_t>(N) * rank / ranks);
  const int i1 = static_cast<int>(static_cast<int64_t>(N) * (rank + 1) / ranks);
  constexpr int ROWS = kThreads / LANES;  // rows that the block copies at a time
  constexpr int U = 4;
  const int c = (tid % LANES) * 16, lead = tid / LANES;
  for (int base = i0; base < i1; base += kChunk) {
    const int rows = min(kChunk, i1 - base);
    __syncthreads();
    if (tid < rows) {
      // written by this kernel, so not through the read-only path
      const int j = __ldcg(kept + base + tid);
      int64_t from = row_offset(a.src, r, j, g, a.row_bytes, &s.status);
      const int64_t to = row_offset(a.dst, r, base + tid, g, a.row_bytes, &s.status);
      s.from[tid] = to < 0 ? -1 : from;
      s.to[tid] = to;
    }
    __syncthreads();
    for (int i = lead; i < rows; i += U * ROWS) {
      uint4 k[U], v[U];
#pragma unroll
      for (int e = 0; e < U; ++e) {
        const int x = i + e * ROWS;
        if (x < rows && s.from[x] >= 0) {
          k[e] = __ldcs(reinterpret_cast<const uint4*>(a.src.k + s.from[x] + c));
          v[e] = __ldcs(reinterpret_cast<const uint4*>(a.src.v + s.from[x] + c));
        }
      }
#pragma unroll
      for (int e = 0; e < U; ++e) {
        const int x = i + e * ROWS;
        if (x < rows && s.from[x] >= 0) {
          *reinterpret_cast<uint4*>(a.dst.k + s.to[x] + c) = k[e];
          *reinterpret_cast<uint4*>(a.dst.v + s.to[x] + c) = v[e];
        }
      }
    }
  }
  __syncthreads();
  if (tid == 0) {
    a.scratch[kStatusFirst + blockIdx.x] = s.status;
    if (blockIdx.x == 0) *reinterpret_cast<uint2*>(a.scratch) = make_uint2(kStatusMore, kStatusMagic | gridDim.x);
  }
}

}  // namespace

// Ranks per cluster: so many that the threads can hold a rank's keys (16 x 512), and more for few rows,
// as long as a rank keeps five hundred keys.  More than 8 need the attribute for clusters beyond the
// portable size.
int evict_cluster(const EvictArgs& a) {
  const int64_t rows = static_cast<int64_t>(a.num_seqs) * a.Hkv;
  int c = 1;
  while (c < kMaxRanks && (a.max_kv_len > c * kHeld * kThreads || (rows * c < 148 && a.max_kv_len >= 1024 * c))) c *= 2;
  return c;
}

cudaError_t launch_evict(const EvictArgs& a, int ranks, cudaStream_t stream) {
  const auto kernel = a.row_bytes == 128 ? evict_kernel<8> : evict_kernel<16>;
  if (a.row_bytes != 128 && a.row_bytes != 256) return cudaErrorInvalidValue;
  if (ranks > 8) {
    const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                               cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  return launch_chained(kernel, dim3(static_cast<unsigned>(a.num_seqs) * a.Hkv * ranks), kThreads, 0, stream, ranks, a);
}

}  // namespace fp2
