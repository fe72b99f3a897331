// q8_rope.cu -- RMSNorm of every query and key head and the rotation by position, one pass.
//
// The attention half of the hybrid models that "CUDA inference engine for running
// Qwen3.5/3.6 hybrid models on mining cards (CMP 100-210)" (news.hada.io topic 29953) runs
// norms its query and key heads and turns their channels by the token's position between
// the projections and the attention.  Per head: z = x r w, r = 1 / sqrt(mean x^2 + eps); pair
// (a, b) of the first rot channels becomes (a cos t - b sin t, a sin t + b cos t),
// t = position * inv_freq[i].
//
// Bound: bytes (each input once, each bfloat16 output once).
//  - A team of d / 16 lanes (rounded up to a power of two) owns a head, each lane the two
//    8-channel chunks whose channels pair up, so the rotation needs no exchange and every
//    access is 16 bytes; the sum of squares is a shuffle tree in a fixed order.
//  - A team walks several heads of one token, so that one set of 8 sines and cosines a lane
//    serves them all; with few tokens every head gets a team of its own.
//  - Angles: the fraction of a turn that one position advances is formed once a lane as a
//    64-bit fixed-point number; position * step modulo 2^64 is then the exact fraction of a
//    turn at any position, and only its top 32 bits become binary32.  Binary64 arithmetic
//    would cost more than the memory traffic on this GPU.
#include <cuda_bf16.h>

#include <algorithm>

#include "q8_internal.h"
#include "q8_quant_dev.cuh"

namespace q8 {
namespace {

constexpr int kThreads = 256;

struct RopeParams {
  const void* x[2];        // q, k
  int64_t x_stride[2];     // elements between tokens
  const float* w[2];       // [d] or nullptr
  uint16_t* out[2];
  int64_t out_stride[2];
  int heads[2];
  const int32_t* positions;
  const double* inv_freq;
  float eps, inv_d;
  int64_t T;
  int d, rot;
  int teams_per_token;     // a token's heads are dealt to this many teams in turn
};

// inv_freq / (2 pi) as a fraction of a turn in units of 2^-64, modulo whole turns, from the
// bits of the binary64 value m 2^e: m 2^11 times the leading 64 bits of 2 / pi, shifted.
__device__ __forceinline__ uint64_t turn_step(double f) {
  const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(f));
  const int ex = static_cast<int>((bits >> 52) & 0x7FF);
  if (ex == 0) return 0;  // zero; a subnormal frequency turns by less than 2^-64
  const uint64_t m = (bits & 0xFFFFFFFFFFFFFull) | 0x10000000000000ull;
  const uint64_t x = __umul64hi(m << 11, 0xA2F9836E4E441529ull);  // floor(m (2 / pi) 2^11)
  const int sh = ex - 1075 + 51;  // f / (2 pi) 2^64 = x 2^(ex - 1075 + 51)
  const uint64_t s = sh <= -64 ? 0 : sh < 0 ? x >> -sh : sh < 64 ? x << sh : 0;
  return (bits >> 63) != 0 ? 0 - s : s;
}

template <bool kF32>
__device__ __forceinline__ void load8(const void* x, int64_t at, float (&v)[8]) {
  if constexpr (kF32) {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
    const float4 a = f[0], b = f[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    bf16x8_to_f32(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at), v);
  }
}

__device__ __forceinline__ void store8(uint16_t* out, const float (&v)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(out) = make_uint4(u[0], u[1], u[2], u[3]);
}

template <int kLanes, bool kF32, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const RopeParams p) {
  const int lane = threadIdx.x % kLanes;
  const int64_t team = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) / kLanes;
  const int64_t nteams = static_cast<int64_t>(gridDim.x) * kThreads / kLanes;
  const bool active = 16 * lane < p.d;
  const bool turns = 16 * lane < p.rot;  // this lane's pairs are rotated
  // chunks (of 8 channels) a and b
  const int ca = !kInterleaved && turns ? lane : 2 * lane;
  const int cb = !kInterleaved && turns ? lane + p.rot / 16 : 2 * lane + 1;
  uint64_t step[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) step[i] = turns ? turn_step(p.inv_freq[8 * lane + i]) : 0;
  // the lane's weights of a query head and of a key head (1 where heads are not normalised)
  float w[2][16];
#pragma unroll
  for (int part = 0; part < 2; ++part)
#pragma unroll
    for (int i = 0; i < 16; ++i)
      w[part][i] = p.w[part] != nullptr && active ? p.w[part][8 * (i < 8 ? ca : cb) + (i & 7)] : 1.0f;
  const bool norm_q = p.w[0] != nullptr, norm_k = p.w[1] != nullptr;
  const int nh = p.heads[0] + p.heads[1];
  const int64_t work = p.T * p.teams_per_token;
  const int64_t rounds = (work + nteams - 1) / nteams;  // the same for every lane
  for (int64_t it = 0; it < rounds; ++it) {
    const int64_t item = it * nteams + team;
    const bool on = active && item < work;
    const int64_t t = item < work ? item / p.teams_per_token : 0;
    const int first = static_cast<int>(item - t * p.teams_per_token);
    float cs[8], sn[8];
    const int64_t pos = on ? p.positions[t] : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int32_t frac = static_cast<int32_t>((static_cast<uint64_t>(pos) * step[i]) >> 32);
      sincospif(static_cast<float>(frac) * 4.656612873077392578125e-10f, &sn[i], &cs[i]);  // 2^-31
    }
    for (int h0 = 0; h0 < nh; h0 += p.teams_per_token) {
      const int h = h0 + first;
      const bool here = on && h < nh;
      const int part = h < p.heads[0] ? 0 : 1;
      const int64_t hd = static_cast<int64_t>(part == 0 ? h : h - p.heads[0]) * p.d;
      float a[8] = {}, b[8] = {};
      if (here) {
        const int64_t row = t * p.x_stride[part] + hd;
        load8<kF32>(p.x[part], row + 8 * ca, a);
        load8<kF32>(p.x[part], row + 8 * cb, b);
      }
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(a[i], a[i], fmaf(b[i], b[i], ss));
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
      const float r = (part == 0 ? norm_q : norm_k) ? __frsqrt_rn(fmaf(ss, p.inv_d, p.eps)) : 1.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] *= r * (part == 0 ? w[0][i] : w[1][i]);
        b[i] *= r * (part == 0 ? w[0][8 + i] : w[1][8 + i]);
      }
      if (turns) {
        if constexpr (kInterleaved) {  // pairs inside a chunk: a holds pairs 0-3, b pairs 4-7
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a0 = a[2 * i], a1 = a[2 * i + 1], b0 = b[2 * i], b1 = b[2 * i + 1];
            a[2 * i] = a0 * cs[i] - a1 * sn[i];
            a[2 * i + 1] = a0 * sn[i] + a1 * cs[i];
            b[2 * i] = b0 * cs[4 + i] - b1 * sn[4 + i];
            b[2 * i + 1] = b0 * sn[4 + i] + b1 * cs[4 + i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float a0 = a[i], b0 = b[i];
            a[i] = a0 * cs[i] - b0 * sn[i];
            b[i] = a0 * sn[i] + b0 * cs[i];
          }
        }
      }
      if (here) {
        uint16_t* o = p.out[part] + t * p.out_stride[part] + hd;
        store8(o + 8 * ca, a);
        store8(o + 8 * cb, b);
      }
    }
  }
}

template <int kLanes>
cudaError_t launch_lanes(const RopeParams& p, bool f32, bool interleaved, int grid, cudaStream_t stream) {
  if (f32) {
    if (interleaved) qk_norm_rope_kernel<kLanes, true, true><<<grid, kThreads, 0, stream>>>(p);
    else qk_norm_rope_kernel<kLanes, true, false><<<grid, kThreads, 0, stream>>>(p);
  } else {
    if (interleaved) qk_norm_rope_kernel<kLanes, false, true><<<grid, kThreads, 0, stream>>>(p);
    else qk_norm_rope_kernel<kLanes, false, false><<<grid, kThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(const void* q, const void* k, int xtype, int64_t q_stride,
                                int64_t k_stride, const float* q_weight, const float* k_weight,
                                float eps, const int32_t* positions, const double* inv_freq,
                                int rot, bool interleaved, uint16_t* q_out, uint16_t* k_out,
                                int64_t q_out_stride, int64_t k_out_stride, int64_t T, int64_t H,
                                int64_t Hkv, int d, const DeviceInfo& dev, cudaStream_t stream) {
  if (T == 0 || H + Hkv == 0) return cudaSuccess;
  RopeParams p = {};
  p.x[0] = q;
  p.x[1] = k;
  p.x_stride[0] = q_stride;
  p.x_stride[1] = k_stride;
  p.w[0] = q_weight;
  p.w[1] = k_weight;
  p.out[0] = q_out;
  p.out[1] = k_out;
  p.out_stride[0] = q_out_stride;
  p.out_stride[1] = k_out_stride;
  p.heads[0] = static_cast<int>(H);
  p.heads[1] = static_cast<int>(Hkv);
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.eps = eps;
  p.inv_d = 1.0f / static_cast<float>(d);
  p.T = T;
  p.d = d;
  p.rot = rot;
  const int lanes = d <= 16 ? 1 : d <= 32 ? 2 : d <= 64 ? 4 : d <= 128 ? 8 : 16;
  const int64_t nh = H + Hkv, cap = static_cast<int64_t>(dev.sm_count) * 8;
  // one head a team until the GPU is full, then up to eight
  const int64_t full = cap * (kThreads / lanes);
  const int64_t per = std::min<int64_t>(8, std::max<int64_t>(1, T * nh / full));
  p.teams_per_token = static_cast<int>((nh + per - 1) / per);
  const int64_t blocks = (T * p.teams_per_token * lanes + kThreads - 1) / kThreads;
  const int grid = static_cast<int>(std::min(blocks, cap));
  const bool f32 = xtype == 0;
  switch (lanes) {
    case 1: return launch_lanes<1>(p, f32, interleaved, grid, stream);
    case 2: return launch_lanes<2>(p, f32, interleaved, grid, stream);
    case 4: return launch_lanes<4>(p, f32, interleaved, grid, stream);
    case 8: return launch_lanes<8>(p, f32, interleaved, grid, stream);
    default: return launch_lanes<16>(p, f32, interleaved, grid, stream);
  }
}

}  // namespace q8
