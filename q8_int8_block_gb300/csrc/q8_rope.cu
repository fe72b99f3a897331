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
//  - A block takes a few tokens with all their heads.  Its threads form the tokens' sines and
//    cosines once, in shared memory, while the first heads are on their way from memory; the
//    teams then walk the heads.  Small blocks of 64 registers, eight on an SM, hide both phases
//    of one another: 8192 tokens of 40 heads of 128 from binary32 take 47 us (5.3 TB/s, 0.79 of
//    the measured copy rate), 62 us with blocks of 256 threads that loaded further ahead, 49 and 51
//    with six and ten blocks an SM.
//  - Angles: the fraction of a turn that one position advances is formed as a 64-bit
//    fixed-point number; position * step modulo 2^64 is then the fraction of a turn at any
//    position (to 2^-31 turns for frequencies up to 1), and its top 32 bits become binary32,
//    which rounds off up to 2^-26 turns, about what sine and cosine are rounded to.  Binary64
//    arithmetic would cost more than the memory traffic on this GPU.
#include <cuda_bf16.h>

#include <algorithm>

#include "q8_internal.h"
#include "q8_quant_dev.cuh"
#include "q8_rope_dev.cuh"

namespace q8 {
namespace {

constexpr int kThreads = 128;

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
  int tokens;              // tokens of a block; its teams are dealt to them evenly
};

// A chunk of 8 channels as it is loaded.
template <bool kF32>
struct Chunk {
  uint4 v[kF32 ? 2 : 1];

  __device__ __forceinline__ void load(const void* x, int64_t at) {
    if constexpr (kF32) {
      const uint4* f = reinterpret_cast<const uint4*>(static_cast<const float*>(x) + at);
      v[0] = f[0];
      v[1] = f[1];
    } else {
      v[0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at);
    }
  }
  __device__ __forceinline__ void unpack(float (&f)[8]) const {
    if constexpr (kF32) {
      f[0] = __uint_as_float(v[0].x); f[1] = __uint_as_float(v[0].y);
      f[2] = __uint_as_float(v[0].z); f[3] = __uint_as_float(v[0].w);
      f[4] = __uint_as_float(v[1].x); f[5] = __uint_as_float(v[1].y);
      f[6] = __uint_as_float(v[1].z); f[7] = __uint_as_float(v[1].w);
    } else {
      bf16x8_to_f32(v[0], f);
    }
  }
};

__device__ __forceinline__ void store8(uint16_t* out, const float (&v)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(out) = make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ void read8(const float* s, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(s), b = *reinterpret_cast<const float4*>(s + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

constexpr int kMaxD = 256, kMaxTokens = 8;

template <int kLanes, bool kF32, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 8) qk_norm_rope_kernel(const RopeParams p) {
  constexpr int kTeams = kThreads / kLanes;
  constexpr int kAhead = kF32 ? 1 : 2;  // heads of a team in flight: 16 registers
  __shared__ __align__(16) float cos_s[kMaxTokens * kMaxD / 2], sin_s[kMaxTokens * kMaxD / 2];
  __shared__ __align__(16) float w_s[2][kMaxD];
  const int lane = threadIdx.x % kLanes, team = threadIdx.x / kLanes;
  const unsigned mask = ((1u << kLanes) - 1u) << (threadIdx.x & 31 & ~(kLanes - 1));
  const int per_token = kTeams / p.tokens, mine = team / per_token, first = team - mine * per_token;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.tokens, t = t0 + mine;
  const bool active = 16 * lane < p.d && t < p.T;
  const bool turns = 16 * lane < p.rot;  // this lane's pairs are rotated
  // chunks (of 8 channels) a and b
  const int ca = !kInterleaved && turns ? lane : 2 * lane;
  const int cb = !kInterleaved && turns ? lane + p.rot / 16 : 2 * lane + 1;
  const int nh = p.heads[0] + p.heads[1];

  Chunk<kF32> xa[kAhead], xb[kAhead];
  auto load = [&](int h0) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int h = h0 + u * per_token;
      if (active && h < nh) {
        const int part = h < p.heads[0] ? 0 : 1;
        const int64_t at = t * p.x_stride[part] + static_cast<int64_t>(part == 0 ? h : h - p.heads[0]) * p.d;
        xa[u].load(p.x[part], at + 8 * ca);
        xb[u].load(p.x[part], at + 8 * cb);
      }
    }
  };
  load(first);
  const int half = p.rot / 2;
  for (int i = threadIdx.x; i < p.tokens * half; i += kThreads) {
    const int tok = i / half, f = i - tok * half;
    if (t0 + tok < p.T) {
      const int64_t pos = p.positions[t0 + tok];
      bool ok;
      const uint64_t step = turn_step(p.inv_freq[f], &ok);
      const int32_t frac = static_cast<int32_t>((static_cast<uint64_t>(pos) * step) >> 32);
      const float half_turns = ok ? static_cast<float>(frac) * 4.656612873077392578125e-10f : NAN;  // 2^-31
      sincospif(half_turns, &sin_s[i], &cos_s[i]);
    }
  }
  for (int i = threadIdx.x; i < 2 * p.d; i += kThreads) {
    const int part = i < p.d ? 0 : 1, c = i - part * p.d;
    w_s[part][c] = p.w[part] != nullptr ? p.w[part][c] : 1.0f;  // 1 where heads are not normalised
  }
  __syncthreads();
  const bool norm_q = p.w[0] != nullptr, norm_k = p.w[1] != nullptr;
  for (int h0 = first; h0 < nh; h0 += kAhead * per_token) {
    if (h0 != first) load(h0);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int h = h0 + u * per_token;
      if (h >= nh) break;  // the same for the whole team
      const int part = h < p.heads[0] ? 0 : 1;
      float a[8] = {}, b[8] = {};
      if (active) {
        xa[u].unpack(a);
        xb[u].unpack(b);
      }
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(a[i], a[i], fmaf(b[i], b[i], ss));
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
      if (!active) continue;
      const float r = (part == 0 ? norm_q : norm_k) ? rsqrtf(fmaf(ss, p.inv_d, p.eps)) : 1.0f;
      float w[8];
      read8(w_s[part] + 8 * ca, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] *= r * w[i];
      read8(w_s[part] + 8 * cb, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] *= r * w[i];
      if (turns) {
        float cs[8], sn[8];  // read again for every head: held, they would spill the loads
        read8(cos_s + mine * half + 8 * lane, cs);
        read8(sin_s + mine * half + 8 * lane, sn);
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
      uint16_t* o = p.out[part] + t * p.out_stride[part] + static_cast<int64_t>(part == 0 ? h : h - p.heads[0]) * p.d;
      store8(o + 8 * ca, a);
      store8(o + 8 * cb, b);
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
  // Tokens of a block: the fewest that keep the teams of a token equally busy, as long as every
  // SM gets its blocks (8192 tokens of 40 heads of 128: 2 tokens, 5 heads a team)
  const int64_t nh = H + Hkv, teams = kThreads / lanes;
  p.tokens = 1;
  double best = 0.0;
  for (int n = 1; n <= kMaxTokens && n <= teams; n *= 2) {
    if (n > 1 && T < static_cast<int64_t>(n) * dev.sm_count * 8) break;
    const int64_t per = teams / n;
    const double even = static_cast<double>(nh) / static_cast<double>((nh + per - 1) / per * per);
    if (even > best) {
      best = even;
      p.tokens = n;
    }
  }
  const int64_t blocks = (T + p.tokens - 1) / p.tokens;
  const int grid = static_cast<int>(blocks);
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
