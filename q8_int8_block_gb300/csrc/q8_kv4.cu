// q8_kv4.cu -- what writes the 4-bit cache of keys and values and reads it back, and the table of
// a step's rotations.
//
// The hybrid models that "CUDA inference engine for running Qwen3.5/3.6 hybrid models on mining
// cards (CMP 100-210)" (news.hada.io topic 29953) runs keep long contexts in a compressed cache.
// Here: 4-bit codes with a bfloat16 scale for 32 channels of a token, 4.5 bits an element, in
// pages (q8_kv4.cuh has the format).
//
// Table: cosine and sine of positions[axis[i]][t] * inv_freq[i], once a step for all layers.  The
// fraction of a turn is a 64-bit fixed-point product (q8_rope_dev.cuh); the nearest quarter is
// taken off before it becomes binary32, so the rest, at most 1/8 turn, keeps 24 bits of its own
// and the results are good to about a rounding.
//
// Append: the heads' norm, the rotation and the quantiser in one pass.  Keys: z = x w; pairs turn,
// every product and sum rounded to binary32; blocks of 32: code = rint(z' * (7 / max |z'|)), scale
// = max |z'| r / 7 in bfloat16, r = 1 / sqrt(mean x^2 + eps): the norm's factor is one for the
// head, so it goes into the scales and the codes do not depend on how it was summed.
// Bound: bytes.  A lane owns 8 channels (one 16-byte load), d / 8 lanes a head; the rotation's
// partner comes from its lane by shuffle, a block's largest magnitude is a shuffle tree of four
// lanes.  A warp takes heads of one token, one kind (query, key, value) at a time, and loads the
// next ones ahead.
//
// Gather: rows of keys and values as bfloat16 or binary32.  Bound: the bytes written.
#include <cuda_bf16.h>

#include <algorithm>

#include "q8_internal.h"
#include "q8_kv4.cuh"
#include "q8_quant_dev.cuh"
#include "q8_rope_dev.cuh"

namespace q8 {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;

// ---- table -----------------------------------------------------------------------------------
struct TableParams {
  const int32_t* positions;  // [axes][T]
  const double* inv_freq;    // [half]
  const int32_t* axis;       // [half] or nullptr
  float* table;              // [T][2][half]
  int64_t T;
  int axes, half;
};

__global__ void __launch_bounds__(256) rope_table_kernel(const TableParams p) {
  const int64_t n = p.T * (p.half / 4), stride = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; at < n; at += stride) {
    const int64_t t = at / (p.half / 4);
    const int i0 = static_cast<int>(at - t * (p.half / 4)) * 4;
    float cs[4], sn[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int ax = p.axis != nullptr ? p.axis[i0 + e] : 0;
      bool ok;
      const uint64_t step = turn_step(p.inv_freq[i0 + e], &ok);
      ok = ok && ax >= 0 && ax < p.axes;
      const int64_t pos = ok ? p.positions[ax * p.T + t] : 0;
      const uint64_t frac = static_cast<uint64_t>(pos) * step;
      const uint32_t quarter = static_cast<uint32_t>((frac + (uint64_t{1} << 61)) >> 62);
      const int64_t rest = static_cast<int64_t>(frac - (static_cast<uint64_t>(quarter) << 62));
      float s, c;  // of rest / 2^64 turns; 2^30 of its units are 2^-33 half turns
      sincospif(static_cast<float>(static_cast<int32_t>(rest >> 30)) * 1.16415321826934814453125e-10f, &s, &c);
      const float a = (quarter & 1u) != 0 ? s : c, b = (quarter & 1u) != 0 ? c : s;
      cs[e] = !ok ? NAN : quarter == 1 || quarter == 2 ? -a : a;
      sn[e] = !ok ? NAN : quarter >= 2 ? -b : b;
    }
    float* out = p.table + t * 2 * p.half + i0;
    *reinterpret_cast<float4*>(out) = make_float4(cs[0], cs[1], cs[2], cs[3]);
    *reinterpret_cast<float4*>(out + p.half) = make_float4(sn[0], sn[1], sn[2], sn[3]);
  }
}

// ---- append ----------------------------------------------------------------------------------
constexpr int kAppendThreads = 128;

struct AppendParams {
  Kv4AppendArgs a;
  int nq, nk;         // warp rounds of query heads, of key (and of value) heads
  int parts, per;     // warps of a token, rounds of a warp
  float inv_d;
};

template <bool kF32>
struct Eight {  // 8 channels as they are loaded
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

__device__ __forceinline__ void load8(const float* s, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(s)), b = __ldg(reinterpret_cast<const float4*>(s) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

template <int D, bool kF32, bool kInterleaved>
__global__ void __launch_bounds__(kAppendThreads) kv4_append_kernel(const __grid_constant__ AppendParams p) {
  using Tile = Kv4Tile<D>;
  constexpr int L = D / 8, kTeams = 32 / L;  // lanes of a head, heads of a round
  const Kv4AppendArgs& a = p.a;
  const int lane = static_cast<int>(threadIdx.x & 31), c = lane % L, team = lane / L;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kAppendThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = unit / p.parts;
  if (t >= a.T) return;
  const int total = p.nq + 2 * p.nk;
  const int r0 = static_cast<int>(unit - t * p.parts) * p.per, r1 = r0 + p.per < total ? r0 + p.per : total;
  if (r0 >= r1) return;

  // round r: its kind (0 query, 1 key, 2 value) and this lane's head
  auto kind_of = [&](int r) { return r < p.nq ? 0 : r < p.nq + p.nk ? 1 : 2; };
  auto head_of = [&](int r, int kind) { return (kind == 0 ? r : kind == 1 ? r - p.nq : r - p.nq - p.nk) * kTeams + team; };
  Eight<kF32> x;
  auto load = [&](int r) {
    const int kind = kind_of(r), h = head_of(r, kind);
    if (h < (kind == 0 ? a.H : a.Hkv))
      x.load(kind == 0 ? a.q : kind == 1 ? a.k : a.v, t * a.st[kind] + static_cast<int64_t>(h) * D + 8 * c);
  };
  load(r0);

  // the lane's rotation: halves (the chunk's eight pairs) or neighbours (its four pairs)
  const bool turns = 8 * c < a.rot, upper = !kInterleaved && 16 * c >= a.rot;
  const int half = a.rot / 2, other = a.rot / 16;
  const int partner = !kInterleaved && turns ? lane + (upper ? -other : other) : lane;
  float cs[8] = {}, sn[8] = {};
  if (turns) {
    const float* row = a.table + t * 2 * half;
    if constexpr (kInterleaved) {
      const float4 u = __ldg(reinterpret_cast<const float4*>(row + 4 * c));
      const float4 w = __ldg(reinterpret_cast<const float4*>(row + half + 4 * c));
      cs[0] = u.x; cs[1] = u.y; cs[2] = u.z; cs[3] = u.w;
      sn[0] = w.x; sn[1] = w.y; sn[2] = w.z; sn[3] = w.w;
    } else {
      load8(row + 8 * (upper ? c - other : c), cs);
      load8(row + half + 8 * (upper ? c - other : c), sn);
    }
  }
  // the token's place: its tile of head 0
  const int64_t slot = a.slots[t];
  const int64_t page = slot / a.page;
  const int in_page = static_cast<int>(slot - page * a.page), tok = in_page & 31;
  const bool keep = slot >= 0 && page < a.pages;
  uint8_t* tile0 = a.cache + (keep ? page : 0) * a.page_stride + static_cast<int64_t>(in_page >> 5) * Tile::kBytes;
  const int64_t head_bytes = a.page / 32 * Tile::kBytes;
  if (slot >= 0 && !keep && lane == 0 && r0 == 0) atomicOr(a.err, kErrBadCache);

  for (int r = r0; r < r1; ++r) {
    const int kind = kind_of(r), h = head_of(r, kind);
    const bool on = h < (kind == 0 ? a.H : a.Hkv);
    float z[8] = {};
    if (on) x.unpack(z);
    if (r + 1 < r1) load(r + 1);
    float f = 1.0f;  // the norm's factor
    if (kind < 2) {
      const float* w = kind == 0 ? a.q_weight : a.k_weight;
      if (w != nullptr) {
        float ss = 0.0f, wv[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(z[i], z[i], ss);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
        f = rsqrtf(fmaf(ss, p.inv_d, a.eps));
        load8(w + 8 * c, wv);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = __fmul_rn(z[i], wv[i]);
      }
      // products and sums rounded one by one: the codes are then the same wherever they are formed
      if constexpr (kInterleaved) {
        if (turns) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float u = z[2 * i], v = z[2 * i + 1];
            z[2 * i] = __fsub_rn(__fmul_rn(u, cs[i]), __fmul_rn(v, sn[i]));
            z[2 * i + 1] = __fadd_rn(__fmul_rn(u, sn[i]), __fmul_rn(v, cs[i]));
          }
        }
      } else if (a.rot > 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float o = __shfl_sync(kFull, z[i], partner);
          if (turns) {
            const float u = __fmul_rn(z[i], cs[i]), v = __fmul_rn(o, sn[i]);
            z[i] = upper ? __fadd_rn(v, u) : __fsub_rn(u, v);
          }
        }
      }
    }
    if (kind == 0) {
      if (on) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(z[2 * i] * f, z[2 * i + 1] * f);
          u[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(a.q_out + t * a.st[3] + static_cast<int64_t>(h) * D + 8 * c) = make_uint4(u[0], u[1], u[2], u[3]);
      }
      continue;
    }
    // the quantiser: lanes 4 b .. 4 b + 3 of a head hold block b
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(z[i]));
    top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
    top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
    const bool zero = top < kKv4Zero;
    const float inv = zero ? 0.0f : __fdiv_rn(7.0f, top);
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // 1.5 2^23 + 8 is even, so adding it rounds as rint does, and the code + 8 is in the low bits
      const float m = __fadd_rn(__fmul_rn(z[i], inv), 12582920.0f);
      word |= (__float_as_uint(m) & 15u) << (4 * i);
    }
    const __nv_bfloat16 sc = __float2bfloat16_rn(zero ? 0.0f : __fmul_rn(__fmul_rn(top, f), 1.0f / 7.0f));
    uint8_t* tile = tile0 + static_cast<int64_t>(h) * head_bytes;
    const int b = c >> 2;
    if (kind == 1) {
      if (on && keep) {
        *reinterpret_cast<uint32_t*>(tile + Tile::key_word(tok, c)) = word;
        if ((c & 3) == 0) *reinterpret_cast<__nv_bfloat16*>(tile + Tile::kKeyScales + Tile::scale(tok, b)) = sc;
      }
    } else {
      // blocks 2 h and 2 h + 1 share words: of a lane's two halves the lane of the other block takes one
      const uint32_t give = (b & 1) == 0 ? word >> 16 : word & 0xFFFFu;
      const uint32_t got = __shfl_xor_sync(kFull, give, 4);
      const uint32_t both = (b & 1) == 0 ? (word & 0xFFFFu) | got << 16 : got | (word & 0xFFFF0000u);
      if (on && keep) {
        *reinterpret_cast<uint32_t*>(tile + Tile::value_word(tok, 2 * (c & 3) + (b & 1), b >> 1)) = both;
        if ((c & 3) == 0) *reinterpret_cast<__nv_bfloat16*>(tile + Tile::kValueScales + Tile::scale(tok, b)) = sc;
      }
    }
  }
}

// ---- gather ----------------------------------------------------------------------------------
constexpr int kGatherThreads = 256;

struct GatherParams {
  Kv4GatherArgs a;
  int heads;  // of a block
};

template <int D, bool kBf16>
__global__ void __launch_bounds__(kGatherThreads) kv4_gather_kernel(const __grid_constant__ GatherParams p) {
  using Tile = Kv4Tile<D>;
  constexpr int L = D / 8, kTeams = kGatherThreads / L;
  const Kv4GatherArgs& a = p.a;
  __shared__ const uint8_t* tile_s[32];  // of head 0; nullptr: no row
  __shared__ int tok_s[32];
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * 32;
  if (threadIdx.x < 32) {
    const int64_t row = row0 + threadIdx.x;
    const uint8_t* tile = nullptr;
    int tok = 0;
    if (row < a.T) {
      int64_t lo = 0, hi = a.B;  // the last sequence that begins at or in front of the row
      while (lo < hi) {
        const int64_t mid = (lo + hi + 1) >> 1;
        if (mid < a.B && a.cu[mid] <= row) lo = mid;
        else hi = mid - 1;
      }
      const int64_t begin = a.cu[lo];
      if (begin <= row && row < a.cu[lo + 1]) {
        const int64_t pos = (a.first != nullptr ? a.first[lo] : 0) + (row - begin);
        const int64_t at = pos >= 0 ? pos / a.page : a.width;
        const int64_t page = at < a.width ? a.block_table[lo * a.width + at] : -1;
        if (page >= 0 && page < a.pages) {
          const int in_page = static_cast<int>(pos - at * a.page);
          tok = in_page & 31;
          tile = a.cache + page * a.page_stride + static_cast<int64_t>(in_page >> 5) * Tile::kBytes;
        } else {
          atomicOr(a.err, kErrBadCache);
        }
      }
    }
    tile_s[threadIdx.x] = tile;
    tok_s[threadIdx.x] = tok;
  }
  __syncthreads();
  const int lane = static_cast<int>(threadIdx.x & 31), c = lane % L, b = c >> 2, u = c & 3;
  const int h0 = static_cast<int>(blockIdx.y) * p.heads, nh = a.Hkv - h0 < p.heads ? static_cast<int>(a.Hkv - h0) : p.heads;
  const int64_t head_bytes = a.page / 32 * Tile::kBytes;
  for (int i = static_cast<int>(threadIdx.x) / L; i < 32 * nh; i += kTeams) {  // 32 nh is a multiple of a warp's teams
    const int r = i & 31, h = h0 + (i >> 5), tok = tok_s[r];
    const uint8_t* tile = tile_s[r];
    const bool on = tile != nullptr;
    tile += on ? h * head_bytes : 0;
    uint32_t kw = 0, vw = 0, ks = 0, vs = 0;
    if (on) {
      kw = __ldg(reinterpret_cast<const uint32_t*>(tile + Tile::key_word(tok, c)));
      vw = __ldg(reinterpret_cast<const uint32_t*>(tile + Tile::value_word(tok, 2 * u + (b & 1), b >> 1)));
      ks = __ldg(reinterpret_cast<const uint16_t*>(tile + Tile::kKeyScales + Tile::scale(tok, b)));
      vs = __ldg(reinterpret_cast<const uint16_t*>(tile + Tile::kValueScales + Tile::scale(tok, b)));
    }
    const uint32_t got = __shfl_xor_sync(kFull, (b & 1) == 0 ? vw >> 16 : vw & 0xFFFFu, 4);
    vw = (b & 1) == 0 ? (vw & 0xFFFFu) | got << 16 : got | (vw & 0xFFFF0000u);
    if (!on) continue;
    const int64_t at = ((row0 + r) * a.Hkv + h) * D + 8 * c;
    auto put = [&](void* out, uint32_t w, uint32_t s16) {
      const float s = __uint_as_float(s16 << 16);
      float v[8];  // exact: 4 bits times 8
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = static_cast<float>(static_cast<int>((w >> (4 * e)) & 15u) - 8) * s;
      if constexpr (kBf16) {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __nv_bfloat162 x = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
          o[e] = *reinterpret_cast<const uint32_t*>(&x);
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) = make_uint4(o[0], o[1], o[2], o[3]);
      } else {
        float4* f = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
        f[0] = make_float4(v[0], v[1], v[2], v[3]);
        f[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
    };
    put(a.k, kw, ks);
    put(a.v, vw, vs);
  }
}

template <int D, bool kF32>
cudaError_t append_kernels(const AppendParams& p, bool interleaved, unsigned grid, cudaStream_t stream) {
  if (interleaved) kv4_append_kernel<D, kF32, true><<<grid, kAppendThreads, 0, stream>>>(p);
  else kv4_append_kernel<D, kF32, false><<<grid, kAppendThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t append(const Kv4AppendArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  AppendParams p = {};
  p.a = a;
  constexpr int kTeams = 32 / (D / 8);
  p.nq = static_cast<int>((a.H + kTeams - 1) / kTeams);
  p.nk = static_cast<int>((a.Hkv + kTeams - 1) / kTeams);
  p.inv_d = 1.0f / D;
  const int64_t rounds = p.nq + 2 * p.nk;
  const int64_t want = (static_cast<int64_t>(dev.sm_count) * 32 + a.T - 1) / a.T;
  p.parts = static_cast<int>(std::max<int64_t>(1, std::min(want, rounds)));
  p.per = static_cast<int>((rounds + p.parts - 1) / p.parts);
  p.parts = static_cast<int>((rounds + p.per - 1) / p.per);
  const int64_t blocks = (a.T * p.parts + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(blocks);
  return a.f32 ? append_kernels<D, true>(p, a.interleaved, grid, stream) : append_kernels<D, false>(p, a.interleaved, grid, stream);
}

template <int D>
cudaError_t gather(const Kv4GatherArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  GatherParams p = {};
  p.a = a;
  const int64_t chunks = (a.T + 31) / 32;
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(a.Hkv, (static_cast<int64_t>(dev.sm_count) * 8 + chunks - 1) / chunks));
  p.heads = static_cast<int>((a.Hkv + want - 1) / want);
  const dim3 grid(static_cast<unsigned>(chunks), static_cast<unsigned>((a.Hkv + p.heads - 1) / p.heads));
  if (a.bf16) kv4_gather_kernel<D, true><<<grid, kGatherThreads, 0, stream>>>(p);
  else kv4_gather_kernel<D, false><<<grid, kGatherThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_table(const int32_t* positions, int axes, const double* inv_freq, const int32_t* axis,
                              float* table, int64_t T, int half, const DeviceInfo& dev, cudaStream_t stream) {
  if (T == 0 || half == 0) return cudaSuccess;
  const TableParams p = {positions, inv_freq, axis, table, T, axes, half};
  const int64_t blocks = (T * (half / 4) + 255) / 256;
  rope_table_kernel<<<static_cast<unsigned>(std::min<int64_t>(blocks, dev.sm_count * 8)), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_kv4_append(Kv4AppendArgs a, const DeviceInfo& dev, cudaStream_t stream) {
  if (a.T == 0 || a.H + a.Hkv == 0) return cudaSuccess;
  a.err = dev.err_word;
  return a.d == 64 ? append<64>(a, dev, stream) : a.d == 128 ? append<128>(a, dev, stream) : append<256>(a, dev, stream);
}

cudaError_t launch_kv4_gather(Kv4GatherArgs a, const DeviceInfo& dev, cudaStream_t stream) {
  if (a.T == 0 || a.B == 0 || a.Hkv == 0) return cudaSuccess;
  a.err = dev.err_word;
  return a.d == 64 ? gather<64>(a, dev, stream) : a.d == 128 ? gather<128>(a, dev, stream) : gather<256>(a, dev, stream);
}

}  // namespace q8
