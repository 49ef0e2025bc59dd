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
// warp walks the heads of one token, so the eight sines and cosines of a thread serve all of them;
// with few tokens the heads are spread over more warps instead (launch_rotate).
#include "fp2_device.cuh"
#include "serve_kernels.h"

namespace fp2 {

namespace {

constexpr int kRotThreads = 128;

FP2_DEVICE void load8(const void* p, bool f32, float (&x)[8]) {
  if (f32) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(w[e] << 16);
      x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
  }
}

template <int DOUT>
FP2_DEVICE void store8(void* p, const float (&x)[8], float inv) {
  if constexpr (DOUT == 0) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else if constexpr (DOUT == 1) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                              pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  } else {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_e4m3x4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                                              pack_e4m3x4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv));
  }
}

// DIN / DOUT: 0 f32, 1 bf16, 2 e4m3.
template <int DIN, int DOUT, int D>
__global__ void __launch_bounds__(kRotThreads) rotate_kernel(const __grid_constant__ RotateArgs a) {
  grid_launch_next();
  grid_wait();
  constexpr int TPH = D / 16;                          // threads per head
  constexpr int HPW = 32 / TPH;                        // heads per warp step
  constexpr int EIN = DIN == 0 ? 4 : 2, EOUT = DOUT == 0 ? 4 : (DOUT == 1 ? 2 : 1);
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kRotThreads / 32) + (threadIdx.x >> 5);
  if (t >= a.tokens) return;
  const int p = lane % TPH;
  const int half = a.rot >> 1;
  // The two vectors of 8 values: whole pairs of the rotated part, or 16 values of the rest.
  const bool rotated = 16 * p < a.rot;
  const bool split = rotated && !a.interleaved;
  const int e0 = split ? 8 * p : 16 * p, e1 = split ? half + 8 * p : 16 * p + 8;

  float cs[8], sn[8];
  if (rotated) {
    const int64_t pos = a.positions[t];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t turn = static_cast<uint32_t>((static_cast<uint64_t>(pos) * a.phase[8 * p + i]) >> 32);
      const uint32_t quarter = (turn + 0x20000000u) >> 30;
      const int32_t rest = static_cast<int32_t>(turn - (quarter << 30));
      float s, c;
      sincospif(static_cast<float>(rest) * 4.656612873077393e-10f, &s, &c);  // 2^-31: turns to half turns
      const float c1 = (quarter & 1u) ? s : c, s1 = (quarter & 1u) ? c : s;
      cs[i] = (quarter == 1u || quarter == 2u) ? -c1 : c1;
      sn[i] = (quarter >= 2u) ? -s1 : s1;
      cs[i] *= a.rope_scale;
      sn[i] *= a.rope_scale;
    }
  }
  int64_t row = t;
  bool put = true;
  if (a.slots != nullptr && (a.Hkv > 0 || a.Hv > 0)) {
    row = a.slots[t];
    put = row >= 0 && row < a.num_slots;
    if (row >= a.num_slots && a.status != nullptr && lane == 0 && blockIdx.y == 0) set_status(a.status, FP2_DEV_SLOT_OOB);
  }

  const int heads = a.Hq + a.Hkv + a.Hv;
  const int h_begin = blockIdx.y * a.iters * HPW;
  // Warp-uniform trip count: the shuffles of the norm need every lane.
#pragma unroll 2
  for (int it = 0; it < a.iters; ++it) {
    const int h0 = h_begin + it * HPW;
    if (h0 >= heads) break;
    const int h = h0 + lane / TPH;
    const int which = h < a.Hq ? 0 : (h < a.Hq + a.Hkv ? 1 : 2);
    const int hh = which == 0 ? h : (which == 1 ? h - a.Hq : h - a.Hq - a.Hkv);
    const bool live = h < heads && (which == 0 || put);
    float x[8], y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = y[i] = 0.f;
    if (live) {
      const char* src = static_cast<const char*>(which == 0 ? a.q : (which == 1 ? a.k : a.v));
      const int64_t stride = which == 0 ? a.q_stride : (which == 1 ? a.k_stride : a.v_stride);
      src += (t * stride + static_cast<int64_t>(hh) * D) * EIN;
      load8(src + e0 * EIN, DIN == 0, x);
      load8(src + e1 * EIN, DIN == 0, y);
    }
    if (a.q_norm != nullptr || a.k_norm != nullptr) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += x[i] * x[i] + y[i] * y[i];
#pragma unroll
      for (int o = 1; o < TPH; o <<= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
      const void* w = which == 0 ? a.q_norm : (which == 1 ? a.k_norm : nullptr);
      if (w != nullptr && live) {
        const float r = rsqrtf(ss * (1.f / D) + a.norm_eps);
        float w0[8], w1[8];
        load8(static_cast<const char*>(w) + e0 * EIN, DIN == 0, w0);
        load8(static_cast<const char*>(w) + e1 * EIN, DIN == 0, w1);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= r * w0[i], y[i] *= r * w1[i];
      }
    }
    if (rotated && which != 2) {
      if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x1 = x[2 * i], x2 = x[2 * i + 1], y1 = y[2 * i], y2 = y[2 * i + 1];
          x[2 * i] = x1 * cs[i] - x2 * sn[i];
          x[2 * i + 1] = x2 * cs[i] + x1 * sn[i];
          y[2 * i] = y1 * cs[4 + i] - y2 * sn[4 + i];
          y[2 * i + 1] = y2 * cs[4 + i] + y1 * sn[4 + i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x1 = x[i], x2 = y[i];
          x[i] = x1 * cs[i] - x2 * sn[i];
          y[i] = x2 * cs[i] + x1 * sn[i];
        }
      }
    }
    if (live) {
      char* dst = static_cast<char*>(which == 0 ? a.q_out : (which == 1 ? a.k_out : a.v_out));
      const int64_t at = which == 0 ? t * a.q_out_stride : row * a.kv_out_stride;
      dst += (at + static_cast<int64_t>(hh) * D) * EOUT;
      const float inv = which == 0 ? a.q_inv : (which == 1 ? a.k_inv : a.v_inv);
      store8<DOUT>(dst + e0 * EOUT, x, inv);
      store8<DOUT>(dst + e1 * EOUT, y, inv);
    }
  }
}

template <int DIN, int DOUT, int D>
cudaError_t run_rotate(RotateArgs a, cudaStream_t stream) {
  constexpr int HPW = 32 / (D / 16);
  const int heads = a.Hq + a.Hkv + a.Hv;
  const int steps = (heads + HPW - 1) / HPW;
  // A warp walks all heads of its token when there are tokens enough to fill the GPU (148 SMs x 16
  // warps); below that the steps are spread over the grid's y, at the price of more sines.
  const int64_t want = (148 * 16 + a.tokens - 1) / a.tokens;
  const int chunks = static_cast<int>(want < 1 ? 1 : (want > steps ? steps : want));
  a.iters = (steps + chunks - 1) / chunks;
  const dim3 grid(static_cast<unsigned>((a.tokens + kRotThreads / 32 - 1) / (kRotThreads / 32)),
                  (steps + a.iters - 1) / a.iters);
  return launch_chained(rotate_kernel<DIN, DOUT, D>, grid, kRotThreads, 0, stream, 1, a);
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
