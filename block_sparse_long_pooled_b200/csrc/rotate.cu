// Per-head RMS norm, rotary positions, conversion and cache append of one projection's Q, K and V.
//
// For a head x of d values: x <- w x / sqrt(mean(x^2) + eps) when a norm weight is given, then pair
// i of the first rot values, (x[i], x[i + rot/2]) or (x[2i], x[2i+1]), turns by the angle
// pos * inv_freq[i]; K and V go to the rows of a cache that `slots` names.  One rounding, at the end.
//
// Angles.  pos * inv_freq reaches 1e5 radians, where an fp32 product has lost the angle to 1e-2.
// Each frequency comes as a 64-bit fraction of a turn, so pos * phase wraps modulo 2^64, which is
// modulo one turn: the reduction is the integer product itself, exact to pos * 2^-64 turns.  The
// nearest quarter turn is taken off as an integer too, so the fp32 argument of sincospi is at most
// an eighth of a turn and keeps 2^-28 of one.
//
// One pass over memory: a thread owns 16 values of a head as two vectors of 8 that hold whole pairs
// ((8c.., rot/2 + 8c..) in the half layout, 16 neighbours in the interleaved one), so no value
// crosses threads and in-place calls are safe; d / 16 threads share a head's norm by shuffles.  A
// warp walks the heads of a token, first Q's, then K's, then V's.  Bytes should bound it, but at 335
// million values the instructions count as much: norm weight, cosine and sine are multiplied once per
// token into four factors a pair, so that a head costs a thread two products, two fused ones and the
// norm's factor for each pair, in packed fp32 pairs; and the values come four steps ahead through shared
// memory, as loads into registers left the SM waiting (250 and 220 us).  With many tokens, or few heads,
// each group of d / 16 lanes has a token of its own, so that a warp's work on one token (angles, factors,
// addresses) serves two to eight; with few tokens the heads are spread over more warps instead (run_rotate).
//
// Measured: 64K tokens of 32 + 4 + 4 heads, norms, bf16 to e4m3 pages: 193 us, 5.2 TB/s (154 us at the copy's
// rate; on one machine 166, where a token a warp took 178).  32K of them bf16 to bf16: 104 us (102).  Eight
// tokens: 2.9 us in a graph, 4 us by call, which is the host's time.  f32 heads and interleaved bf16 pairs take
// 1.8 to 2 times the bytes' time (61K tokens of 3 f32 heads 29 us, 14.5 of bytes): a lane's 8 values are 32 bytes,
// or half of its 32, copied and stored 16 at a time, so that every sector moves twice.
#include "fp2_device.cuh"
#include "serve_kernels.h"

namespace fp2 {

namespace {

constexpr int kRotThreads = 128;
// Blocks per SM that the registers are cut for: 7 of bf16 (72 registers; 6 or 8 were 1 and 4 % slower on the
// prompt below), 6 with several tokens a warp, whose factors take more shared memory (5 and 7: 4 and 2 % slower),
// 4 of f32 (with 5 an odd chunk of 1537 tokens took 7.2 us instead of 6.2).
constexpr int blocks_per_sm(int din, bool many) { return din == 0 ? 4 : (many ? 6 : 7); }

// Eight values from four words of two bf16, or eight floats.
template <int DIN>
FP2_DEVICE void unpack8(uint4 a, uint4 b, float (&x)[8]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if constexpr (DIN == 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(w[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(w[e] << 16);
      x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
  }
}
template <int DIN>
FP2_DEVICE void load8(const char* p, float (&x)[8]) {
  const uint4* v = reinterpret_cast<const uint4*>(p);
  unpack8<DIN>(v[0], DIN == 0 ? v[1] : make_uint4(0, 0, 0, 0), x);
}
FP2_DEVICE uint32_t four_e4m3(float a, float b, float c, float d) {  // a in the lowest byte, saturating
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
template <int DOUT>
FP2_DEVICE void store8(char* p, const float (&x)[8]) {
  if constexpr (DOUT == 0) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else if constexpr (DOUT == 1) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                              pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  } else {
    *reinterpret_cast<uint2*>(p) = make_uint2(four_e4m3(x[0], x[1], x[2], x[3]), four_e4m3(x[4], x[5], x[6], x[7]));
  }
}

FP2_DEVICE void copy16(uint32_t to, const char* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
FP2_DEVICE uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
FP2_DEVICE float4 lds_f4(uint32_t addr) {
  const uint4 v = lds16(addr);
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}

// DIN / DOUT: 0 f32, 1 bf16, 2 e4m3.  MANY: a warp has several tokens, a group of D / 16 lanes each; else one, and
// its groups of lanes have one head each.
template <int DIN, int DOUT, int D, bool INTER, bool MANY>
__global__ void __launch_bounds__(kRotThreads, blocks_per_sm(DIN, MANY))
    rotate_kernel(const __grid_constant__ RotateArgs a) {
  grid_launch_next();
  grid_wait();
  constexpr int TPH = D / 16;                          // threads per head
  constexpr int GROUPS = 32 / TPH;                     // of lanes
  constexpr int HPW = MANY ? 1 : GROUPS;               // heads of a token per step
  constexpr int FL = MANY ? 32 : TPH;                  // lanes with factors of their own
  // Four factors a pair: in shared memory, as 32 registers more would halve the warps per SM.
  __shared__ __align__(16) float factors[kRotThreads / 32][4][2][FL][4];
  constexpr int EIN = DIN == 0 ? 4 : 2, EOUT = DOUT == 0 ? 4 : (DOUT == 1 ? 2 : 1);
  const int lane = threadIdx.x & 31;
  const int p = lane % TPH, group = lane / TPH;
  const int head0 = MANY ? 0 : group;                  // of this lane in a step
  int64_t t = static_cast<int64_t>(blockIdx.x) * (kRotThreads / 32) + (threadIdx.x >> 5);
  if constexpr (MANY) t = t * GROUPS + group;
  const bool mine = t < a.tokens;
  if (!__any_sync(0xFFFFFFFFu, mine)) return;
  if (!mine) t = a.tokens - 1;                         // (such lanes load what another does and store nothing)
  const int half = a.rot >> 1;
  // The two vectors of 8 values: whole pairs of the rotated part, or 16 values of the rest.
  const bool rotated = 16 * p < a.rot;
  const bool split = rotated && !INTER;
  const int e0 = split ? 8 * p : 16 * p, e1 = split ? half + 8 * p : 16 * p + 8;

  // Steps of this warp: HPW heads each, Q's first.
  const int sq = (a.Hq + HPW - 1) / HPW, sk = (a.Hkv + HPW - 1) / HPW, sv = (a.Hv + HPW - 1) / HPW;
  const int begin = blockIdx.y * a.iters, end = min(begin + a.iters, sq + sk + sv);

  // Values come through shared memory, AHEAD steps before they are needed and across Q, K and V: in
  // registers, one step ahead, the loads left the SM waiting.  Every lane reads back what it copied.
  constexpr int AHEAD = 4, VECS = EIN / 2;             // 16-byte copies of a vector of 8
  __shared__ __align__(16) char ring[kRotThreads / 32][AHEAD][2 * VECS][32][16];
  constexpr uint32_t VEC = 32 * 16, SLOT = 2 * VECS * VEC;
  const uint32_t ring_at = smem_u32(ring[threadIdx.x >> 5][0][0][lane]);
  uint32_t ask_slot = ring_at, get_slot = ring_at;
  // The next step to ask for: its section's end, this lane's head in it, and its two vectors.
  int ask = begin, ask_end = 0, ask_head = 0, ask_heads = 0;
  const char *ask0 = nullptr, *ask1 = nullptr;
  const auto request = [&]() {
    if (ask < end) {
      if (ask >= ask_end) {
        const int which = ask < sq ? 0 : (ask < sq + sk ? 1 : 2);
        const int base = which == 0 ? 0 : (which == 1 ? sq : sq + sk);
        ask_end = which == 0 ? sq : (which == 1 ? sq + sk : sq + sk + sv);
        ask_heads = which == 0 ? a.Hq : a.Hkv;
        ask_head = (ask - base) * HPW + head0;
        const char* at = static_cast<const char*>(which == 0 ? a.q : (which == 1 ? a.k : a.v)) +
                         (t * (which == 0 ? a.q_stride : (which == 1 ? a.k_stride : a.v_stride)) +
                          static_cast<int64_t>(ask_head) * D) * EIN;
        ask0 = at + (which == 2 ? 16 * p : e0) * EIN;
        ask1 = at + (which == 2 ? 16 * p + 8 : e1) * EIN;
      }
      // (a lane past the last head works on what its slot holds and stores nothing)
      if (ask_head < ask_heads) {
#pragma unroll
        for (int v = 0; v < VECS; ++v) {
          copy16(ask_slot + v * VEC, ask0 + 16 * v);
          copy16(ask_slot + (VECS + v) * VEC, ask1 + 16 * v);
        }
      }
      ++ask;
      ask_slot = ask_slot == ring_at + (AHEAD - 1) * SLOT ? ring_at : ask_slot + SLOT;
      ask_head += HPW;
      ask0 += HPW * D * EIN;
      ask1 += HPW * D * EIN;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");  // (an empty one keeps the count)
  };
#pragma unroll 1
  for (int i = 0; i < AHEAD; ++i) request();
  const auto arrived = [&](float (&x)[8], float (&y)[8]) {
    asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD - 1) : "memory");
    const uint4 zero = make_uint4(0, 0, 0, 0);
    unpack8<DIN>(lds16(get_slot), DIN == 0 ? lds16(get_slot + VEC) : zero, x);
    unpack8<DIN>(lds16(get_slot + VECS * VEC), DIN == 0 ? lds16(get_slot + 3 * VEC) : zero, y);
    get_slot = get_slot == ring_at + (AHEAD - 1) * SLOT ? ring_at : get_slot + SLOT;
  };

  // The TPH lanes of every head need the same 8 pairs' cosines and sines: each of the HPW groups of
  // lanes works out 8 / HPW of them and the others take them over.
  constexpr int MINE = 8 / HPW;
  float cs[8], sn[8];
  if (begin < sq + sk && a.rot > 0) {
    const int64_t pos = a.positions[t];
    float cm[MINE], sm[MINE];
#pragma unroll
    for (int m = 0; m < MINE; ++m) {
      const int i = head0 * MINE + m;
      const uint64_t phase = rotated ? a.phase[8 * p + i] : 0;
      const uint32_t turn = static_cast<uint32_t>((static_cast<uint64_t>(pos) * phase) >> 32);
      const uint32_t quarter = (turn + 0x20000000u) >> 30;
      const int32_t rest = static_cast<int32_t>(turn - (quarter << 30));
      float s, c;
      sincospif(static_cast<float>(rest) * 4.656612873077393e-10f, &s, &c);  // 2^-31: turns to half turns
      const float c1 = (quarter & 1u) ? s : c, s1 = (quarter & 1u) ? c : s;
      cm[m] = ((quarter == 1u || quarter == 2u) ? -c1 : c1) * a.rope_scale;
      sm[m] = ((quarter >= 2u) ? -s1 : s1) * a.rope_scale;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cs[i] = MANY ? cm[i % MINE] : __shfl_sync(0xFFFFFFFFu, cm[i % MINE], (i / MINE) * TPH + p);
      sn[i] = MANY ? sm[i % MINE] : __shfl_sync(0xFFFFFFFFu, sm[i % MINE], (i / MINE) * TPH + p);
    }
  }
  int64_t row = t;
  bool put = mine;
  if (a.slots != nullptr && end > sq) {
    row = a.slots[t];
    put = mine && row >= 0 && row < a.num_slots;
    if (row >= a.num_slots && a.status != nullptr && lane == TPH * group * MANY && mine && end == sq + sk + sv)
      set_status(a.status, FP2_DEV_SLOT_OOB);
  }

#pragma unroll 1
  for (int which = 0; which < 3; ++which) {
    const int base = which == 0 ? 0 : (which == 1 ? sq : sq + sk), steps = which == 0 ? sq : (which == 1 ? sk : sv);
    const int heads = which == 0 ? a.Hq : (which == 1 ? a.Hkv : a.Hv);
    const int s0 = max(begin - base, 0), s1 = min(end - base, steps);
    // (K and V without a place are the last steps)
    if (s0 >= s1 || (which > 0 && !__any_sync(0xFFFFFFFFu, put))) continue;
    const bool store = which > 0 ? put : mine;
    char* dst = static_cast<char*>(which == 0 ? a.q_out : (which == 1 ? a.k_out : a.v_out)) +
                (which == 0 ? t * a.q_out_stride : row * a.kv_out_stride) * EOUT;
    const float inv = DOUT == 2 ? (which == 0 ? a.q_inv : (which == 1 ? a.k_inv : a.v_inv)) : 1.f;
    if (which == 2) {
      // V passes through: 16 neighbours a thread, whatever Q's layout.
      int h = s0 * HPW + head0;
      char* to = dst + (static_cast<int64_t>(h) * D + 16 * p) * EOUT;
#pragma unroll 1
      for (int s = s0; s < s1; ++s) {
        float x[8], y[8];
        arrived(x, y);
        request();
        if (DOUT == 2 && inv != 1.f) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] *= inv, y[i] *= inv;
        }
        if (h < heads && store) {
          store8<DOUT>(to, x);
          store8<DOUT>(to + 8 * EOUT, y);
        }
        to += HPW * D * EOUT;
        h += HPW;
      }
      continue;
    }
    const void* w = which == 0 ? a.q_norm : a.k_norm;
    const bool turns = rotated;
    // Pair (x1, x2) becomes r (x1 f1 - x2 f2, x2 f3 + x1 f4); values that do not turn r (x f1), r (x f3).
    float f1[8], f2[8], f3[8], f4[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f1[i] = f3[i] = 1.f, f2[i] = f4[i] = 0.f;
    if (w != nullptr) {
      load8<DIN>(static_cast<const char*>(w) + e0 * EIN, f1);
      load8<DIN>(static_cast<const char*>(w) + e1 * EIN, f3);
    }
    if constexpr (INTER) {  // first and second values of the pairs from vectors of 8 neighbours each
      float first[8], second[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        first[i] = f1[2 * i], second[i] = f1[2 * i + 1];
        first[4 + i] = f3[2 * i], second[4 + i] = f3[2 * i + 1];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) f1[i] = first[i], f3[i] = second[i];
    }
    if (turns) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float w1 = f1[i], w2 = f3[i];
        f1[i] = w1 * cs[i];
        f2[i] = -(w2 * sn[i]);
        f3[i] = w2 * cs[i];
        f4[i] = w1 * sn[i];
      }
    }

    __syncwarp();
    float (*fac)[2][FL][4] = factors[threadIdx.x >> 5];
    const int fl = MANY ? lane : p;
    if (lane < FL) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        *reinterpret_cast<float4*>(fac[0][q][fl]) = make_float4(f1[4 * q], f1[4 * q + 1], f1[4 * q + 2], f1[4 * q + 3]);
        *reinterpret_cast<float4*>(fac[1][q][fl]) = make_float4(f2[4 * q], f2[4 * q + 1], f2[4 * q + 2], f2[4 * q + 3]);
        *reinterpret_cast<float4*>(fac[2][q][fl]) = make_float4(f3[4 * q], f3[4 * q + 1], f3[4 * q + 2], f3[4 * q + 3]);
        *reinterpret_cast<float4*>(fac[3][q][fl]) = make_float4(f4[4 * q], f4[4 * q + 1], f4[4 * q + 2], f4[4 * q + 3]);
      }
    }
    __syncwarp();

    int h = s0 * HPW + head0;
    char* to = dst + (static_cast<int64_t>(h) * D + e0) * EOUT;
    const int apart = (e1 - e0) * EOUT;
    const uint32_t fac_at = smem_u32(fac[0][0][fl]);
#pragma unroll 1
    for (int s = s0; s < s1; ++s) {
      float v0[8], v1[8], x1[8], x2[8];
      arrived(v0, v1);
      request();
      float r = inv;
      if (w != nullptr) {
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          ss = __ffma2_rn(make_float2(v0[i], v0[i + 1]), make_float2(v0[i], v0[i + 1]), ss);
          ss = __ffma2_rn(make_float2(v1[i], v1[i + 1]), make_float2(v1[i], v1[i + 1]), ss);
        }
        float sum = ss.x + ss.y;
#pragma unroll
        for (int o = 1; o < TPH; o <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        r *= rsqrtf(sum * (1.f / D) + a.norm_eps);
      }
      if constexpr (!INTER) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x1[i] = v0[i], x2[i] = v1[i];
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x1[i] = v0[2 * i], x2[i] = v0[2 * i + 1];
          x1[4 + i] = v1[2 * i], x2[4 + i] = v1[2 * i + 1];
        }
      }
      const float2 r2 = make_float2(r, r);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float4 g1 = lds_f4(fac_at + q * (FL * 16)), g3 = lds_f4(fac_at + (4 + q) * (FL * 16));
        const float4 g2 = lds_f4(fac_at + (2 + q) * (FL * 16)), g4 = lds_f4(fac_at + (6 + q) * (FL * 16));
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = 4 * q + 2 * e;
          const float2 a1 = make_float2(x1[i], x1[i + 1]), a2 = make_float2(x2[i], x2[i + 1]);
          float2 y1 = __fmul2_rn(a1, e ? make_float2(g1.z, g1.w) : make_float2(g1.x, g1.y));
          float2 y2 = __fmul2_rn(a2, e ? make_float2(g3.z, g3.w) : make_float2(g3.x, g3.y));
          if (turns) {
            y1 = __ffma2_rn(a2, e ? make_float2(g2.z, g2.w) : make_float2(g2.x, g2.y), y1);
            y2 = __ffma2_rn(a1, e ? make_float2(g4.z, g4.w) : make_float2(g4.x, g4.y), y2);
          }
          y1 = __fmul2_rn(y1, r2);
          y2 = __fmul2_rn(y2, r2);
          x1[i] = y1.x, x1[i + 1] = y1.y;
          x2[i] = y2.x, x2[i + 1] = y2.y;
        }
      }
      if constexpr (!INTER) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v0[i] = x1[i], v1[i] = x2[i];
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v0[2 * i] = x1[i], v0[2 * i + 1] = x2[i];
          v1[2 * i] = x1[4 + i], v1[2 * i + 1] = x2[4 + i];
        }
      }
      if (h < heads && store) {
        store8<DOUT>(to, v0);
        store8<DOUT>(to + apart, v1);
      }
      to += HPW * D * EOUT;
      h += HPW;
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int DIN, int DOUT, int D, bool MANY>
cudaError_t run_layout(RotateArgs& a, int chunks, cudaStream_t stream) {
  constexpr int GROUPS = 32 / (D / 16), HPW = MANY ? 1 : GROUPS, PER_BLOCK = kRotThreads / 32 * (MANY ? GROUPS : 1);
  const int steps = (a.Hq + HPW - 1) / HPW + (a.Hkv + HPW - 1) / HPW + (a.Hv + HPW - 1) / HPW;
  if (chunks > steps) chunks = steps;
  a.iters = (steps + chunks - 1) / chunks;
  const dim3 grid(static_cast<unsigned>((a.tokens + PER_BLOCK - 1) / PER_BLOCK), (steps + a.iters - 1) / a.iters);
  const auto kernel =
      a.interleaved ? rotate_kernel<DIN, DOUT, D, true, MANY> : rotate_kernel<DIN, DOUT, D, false, MANY>;
  return launch_chained(kernel, grid, kRotThreads, 0, stream, 1, a);
}

template <int DIN, int DOUT, int D>
cudaError_t run_rotate(RotateArgs a, cudaStream_t stream) {
  // A warp with one token spends 1.3 ns of the GPU on every one, whatever its heads, and lanes without a head; a
  // warp with several needs tokens enough to fill the GPU, and its loads are single heads.  Tokens 600, 2400,
  // 9600, 40000 (us, one | several):  3 heads bf16 to bf16, d 128  5, 8, 16, 53 | 4, 5, 8, 19;  8 heads  5, 8, 16, 56 |
  // 6, 7, 12, 36;  24 heads, d 64  4, 8, 16, 63 | 10, 10, 22, 54;  40 heads bf16 to e4m3  8, 14, 33, 111 | 15, 20, 38,
  // 106;  48 heads bf16 to bf16, bound by its 25 KB a token  8, 16, 42, 149 | 17, 24, 52, 165.
  constexpr int HEAD = D * ((DIN == 0 ? 4 : 2) + (DOUT == 0 ? 4 : (DOUT == 1 ? 2 : 1)));  // bytes of a head
  const int heads = a.Hq + a.Hkv + a.Hv;
  if (heads <= 8 ? a.tokens >= 148 * 16 : a.tokens >= 16384 && static_cast<int64_t>(heads) * HEAD < 20480)
    return run_layout<DIN, DOUT, D, true>(a, 1, stream);
  // A warp walks all heads of its token when there are tokens enough to fill the GPU (148 SMs x 16
  // warps); below that the steps are spread over the grid's y, at the price of more sines.
  const int64_t want = (148 * 16 + a.tokens - 1) / a.tokens;
  return run_layout<DIN, DOUT, D, false>(a, static_cast<int>(want < 1 ? 1 : want), stream);
}

}  // namespace

cudaError_t launch_rotate(int dtype_in, int dtype_out, int D, const RotateArgs& a, cudaStream_t stream) {
  if (D == 128) {
    if (dtype_in == FP2_BF16 && dtype_out == FP2_BF16) return run_rotate<1, 1, 128>(a, stream);
    if (dtype_in == FP2_BF16 && dtype_out == FP2_E4M3) return run_rotate<1, 2, 128>(a, stream);
    if (dtype_in == FP2_F32 && dtype_out == FP2_F32) return run_rotate<0, 0, 128>(a, stream);
    if (dtype_in == FP2_F32 && dtype_out == FP2_E4M3) return run_rotate<0, 2, 128>(a, stream);
  } else if (D == 64) {
    if (dtype_in == FP2_BF16 && dtype_out == FP2_BF16) return run_rotate<1, 1, 64>(a, stream);
    if (dtype_in == FP2_BF16 && dtype_out == FP2_E4M3) return run_rotate<1, 2, 64>(a, stream);
    if (dtype_in == FP2_F32 && dtype_out == FP2_F32) return run_rotate<0, 0, 64>(a, stream);
    if (dtype_in == FP2_F32 && dtype_out == FP2_E4M3) return run_rotate<0, 2, 64>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace fp2
