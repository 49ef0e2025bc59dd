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
// weights' bits in order-preserving form: three histograms (11, 11 and 10 bits) of the keys that
// agree with the digits found so far, added up in rank 0's shared memory through the cluster, give
// the exact weight of the last key to keep and how many of its equals are kept.  The weights are
// read once from HBM and four more times from L2, which costs less than holding them would (a rank's
// share does not fit in registers at 128K keys).  Ballots in index order then give every kept key
// its row; ranks know the counts of the ranks before them, so nothing depends on timing.  After that
// the rows are moved, each rank an equal share of the output rows whatever range they came from:
// the addresses of 512 rows at a time are looked up first, so that the copies themselves wait only
// for their data.
#include <cooperative_groups.h>

#include "fp2_device.cuh"
#include "serve_kernels.h"

namespace fp2 {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kChunk = kThreads;  // rows whose addresses are looked up at a time

// Weights in an order that unsigned comparison follows.  -0 equals 0; NaN counts as the heaviest.
FP2_DEVICE uint32_t ordered(float f) {
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
  if ((u << 1) == 0u) return 0x80000000u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct EvictShared {
  uint32_t local[kBins];      // this rank's histogram
  uint32_t total[3][kBins];   // the cluster's, in rank 0
  uint32_t scan[kWarps];
  uint32_t found[2];          // digit, and how many of the keys above it are still wanted
  uint32_t count[2];          // of this rank: keys kept outright, keys equal to the threshold
  uint32_t warp_sel[kWarps], warp_eq[kWarps];
  int64_t from[kChunk], to[kChunk];
  uint32_t status;
};

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

    for (int i = tid; i < 3 * kBins; i += kThreads) (&s.total[0][0])[i] = 0;
    uint32_t need = static_cast<uint32_t>(a.budget - a.sink - a.window);  // of the competing keys
    uint32_t prefix = 0, mask = 0;
    cluster.sync();
    // need == 0: no competing key stays, and no key's order value exceeds this threshold.
    if (need == 0) prefix = 0xFFFFFFFFu;
    if (need != 0) {
#pragma unroll 1
      for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
        const uint32_t digit = pass == 2 ? 1023u : 2047u;
        for (int i = tid; i < kBins; i += kThreads) s.local[i] = 0;
        __syncthreads();
        const int j1 = min(last * 32, free1);
#pragma unroll 4
        for (int j = max(first * 32, free0) + tid; j < j1; j += kThreads) {
          const uint32_t u = ordered(__ldg(mass + j));
          if ((u & mask) == prefix) atomicAdd(&s.local[(u >> shift) & digit], 1u);
        }
        __syncthreads();
        uint32_t* total = cluster.map_shared_rank(&s.total[pass][0], 0);
        for (int i = tid; i < kBins; i += kThreads)
          if (s.local[i] != 0) atomicAdd(total + i, s.local[i]);
        cluster.sync();
        // Bins from the heaviest down: thread t holds bins 2047 - 4t .. 2044 - 4t.
        uint32_t c[4], sum = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          c[e] = total[kBins - 1 - 4 * tid - e];
          sum += c[e];
        }
        uint32_t inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
          if (lane >= o) inc += v;
        }
        if (lane == 31) s.scan[warp] = inc;
        __syncthreads();
        uint32_t before = inc - sum;
        for (int w = 0; w < warp; ++w) before += s.scan[w];
        // The one bin in which the need-th key lies (need is at most the number of keys counted).
        if (before < need && before + sum >= need) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (before < need && before + c[e] >= need) {
              s.found[0] = kBins - 1 - 4 * tid - e;
              s.found[1] = need - before;
            }
            before += c[e];
          }
        }
        __syncthreads();
        prefix |= s.found[0] << shift;
        mask |= digit << shift;
        need = s.found[1];
        __syncthreads();
      }
    }
    // Keys above `prefix` stay, and of those equal to it the first `need`.
    const auto classify = [&](int j, bool& keep, bool& tie) {
      keep = tie = false;
      if (j >= n) return;
      if (j < free0 || j >= free1) {
        keep = true;
        return;
      }
      const uint32_t u = ordered(__ldg(mass + j));
      keep = u > prefix;
      tie = u == prefix;
    };
    uint32_t sel = 0, eq = 0;
#pragma unroll 4
    for (int t = w0; t < w1; ++t) {
      bool keep, tie;
      classify(t * 32 + lane, keep, tie);
      sel += __popc(__ballot_sync(0xFFFFFFFFu, keep));
      eq += __popc(__ballot_sync(0xFFFFFFFFu, tie));
    }
    if (lane == 0) {
      s.warp_sel[warp] = sel;
      s.warp_eq[warp] = eq;
    }
    __syncthreads();
    if (tid == 0) {
      uint32_t x = 0, y = 0;
      for (int w = 0; w < kWarps; ++w) {
        x += s.warp_sel[w];
        y += s.warp_eq[w];
      }
      s.count[0] = x;
      s.count[1] = y;
    }
    cluster.sync();
    uint32_t sel_before = 0, eq_before = 0;
    for (int q = lane; q < rank; q += 32) {
      const uint32_t* c = cluster.map_shared_rank(&s.count[0], q);
      sel_before += c[0];
      eq_before += c[1];
    }
    for (int w = lane; w < warp; w += 32) {
      sel_before += s.warp_sel[w];
      eq_before += s.warp_eq[w];
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      sel_before += __shfl_xor_sync(0xFFFFFFFFu, sel_before, o);
      eq_before += __shfl_xor_sync(0xFFFFFFFFu, eq_before, o);
    }
    const uint32_t below = (1u << lane) - 1;
#pragma unroll 2
    for (int t = w0; t < w1; ++t) {
      const int j = t * 32 + lane;
      bool keep, tie;
      classify(j, keep, tie);
      const uint32_t ks = __ballot_sync(0xFFFFFFFFu, keep), es = __ballot_sync(0xFFFFFFFFu, tie);
      const uint32_t eq_at = eq_before + __popc(es & below);
      const uint32_t taken = eq_at < need ? eq_at : need;  // ties kept before this key
      const uint32_t pos = sel_before + __popc(ks & below) + taken;
      if ((keep || (tie && eq_at < need)) && fp2_check(pos < static_cast<uint32_t>(a.budget), &s.status)) {
        kept[pos] = j;
        mass_out[pos] = mass[j];
      }
      sel_before += __popc(ks);
      eq_before += __popc(es);
    }
  }
  cluster.sync();  // kept[] is complete, and no rank reads another's shared memory from here on

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
    if (blockIdx.x == 0) *reinterpret_cast<uint2*>(a.scratch) = make_uint2(0u, kStatusMagic | gridDim.x);
  }
}

}  // namespace

// Ranks per cluster: enough that the rows fill the GPU twice over (two CTAs fit on an SM), as long as
// a rank keeps a thousand keys to look through or to move.
int evict_cluster(const EvictArgs& a) {
  const int64_t rows = static_cast<int64_t>(a.num_seqs) * a.Hkv;
  int c = 1;
  while (c < 8 && rows * c < 2 * 148 && a.max_kv_len / (2 * c) >= 1024) c *= 2;
  return c;
}

cudaError_t launch_evict(const EvictArgs& a, int ranks, cudaStream_t stream) {
  const auto kernel = a.row_bytes == 128 ? evict_kernel<8> : evict_kernel<16>;
  if (a.row_bytes != 128 && a.row_bytes != 256) return cudaErrorInvalidValue;
  return launch_chained(kernel, dim3(static_cast<unsigned>(a.num_seqs) * a.Hkv * ranks), kThreads, 0, stream, ranks, a);
}

}  // namespace fp2
