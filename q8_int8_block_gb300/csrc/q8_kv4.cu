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
// and the results are good to about a rounding.  8192 tokens of 64 pairs: 4.1 us.
//
// Append: the heads' norm, the rotation and the quantiser in one pass.  Keys: z = x w; pairs turn,
// every product and sum rounded to binary32; blocks of 32: code = rint(z' * (7 / max |z'|)), scale
// = max |z'| r / 7 in bfloat16, r = 1 / sqrt(mean x^2 + eps): the norm's factor is one for the
// head, so it goes into the scales and the codes do not depend on how it was summed.
// Bound: bytes (8192 tokens of 32 / 8 heads of 128: 34.2 us for a floor of 27; the queries alone are at
// 0.89 of the copy rate, keys and values, bound by their instructions, at 0.50).
// Queries: a lane owns the two chunks of 8 channels whose channels pair up, and norm weight and
// rotation are one matrix a pair.  Keys and values: a lane owns one chunk, the rotation's other
// channel comes by shuffle, a block's largest magnitude is a shuffle tree of four lanes.  Warps take
// one kind each, a few heads of a token, or (many tokens) go through tiles of 32 tokens.
//
// Gather: rows of keys and values as bfloat16 or binary32.  Bound: the bytes written (2 contexts of up to 16384
// tokens, 8 heads of 128: 13.5 us, 0.95 of the copy rate, into rows that the calls before have left in the
// L2; 14592 tokens 12.0 us into such rows and 15.7 into others).

#include <cuda_bf16.h>

#include <algorithm>

#include "q8_internal.h"
#include "q8_kv4.cuh"
#include "q8_launch_ptx.cuh"
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
  pdl_wait();
  pdl_launch_dependents();
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
constexpr int kTileHeads = 2;  // key/value heads of a block of kv4_append_tiles_kernel: four vectors, quantise_four's

struct AppendParams {
  Kv4AppendArgs a;
  int nq, nk;         // warp rounds of a token's query heads, of its key (and of its value) heads
  int pq, parts;      // warps of its query heads, of all
  int kv_blocks;      // (tiles) blocks of keys and values
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

__device__ __forceinline__ void store8(uint16_t* out, const float (&v)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(out) = make_uint4(u[0], u[1], u[2], u[3]);
}
// 16 neighbours (a, then b) <-> their even ones (a) and odd ones (b)
__device__ __forceinline__ void split_pairs(float (&a)[8], float (&b)[8]) {
  const float x[16] = {a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], b[0], b[1], b[2], b[3], b[4], b[5], b[6], b[7]};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a[i] = x[2 * i];
    b[i] = x[2 * i + 1];
  }
}
__device__ __forceinline__ void join_pairs(float (&a)[8], float (&b)[8]) {
  const float x[16] = {a[0], b[0], a[1], b[1], a[2], b[2], a[3], b[3], a[4], b[4], a[5], b[5], a[6], b[6], a[7], b[7]};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a[i] = x[i];
    b[i] = x[8 + i];
  }
}
// (Here and in the gather plain loads, not the read-only path: these kernels start while the one in
// front, which may be writing what they read, still runs, and a read-only load may move across the wait.)
__device__ __forceinline__ void load8(const float* s, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(s)[0], b = reinterpret_cast<const float4*>(s)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

constexpr uint32_t codes_offset() {
  uint32_t w = 0;
  for (int e = 0; e < 8; ++e) w = w * 16u + 0x4B400000u;
  return 0u - w;
}
constexpr uint32_t kCodes = codes_offset();

// The queries of a part: d / 16 lanes a head, each with two chunks of 8 channels whose channels pair
// up, so that pair i = (a, b) needs nothing from another lane.  Norm weight and rotation are one
// 2 x 2 matrix a pair, formed once for all heads.
template <int D, bool kF32, bool kInterleaved, int kRounds>
__device__ __forceinline__ void append_queries(const AppendParams& p, uint32_t t, int part, int lane) {
  constexpr int L = D / 16, kTeams = 32 / L;
  const Kv4AppendArgs& a = p.a;
  const int c = lane % L, team = lane / L;
  const bool turns = 16 * c < a.rot;
  const int ca = !kInterleaved && turns ? c : 2 * c, cb = !kInterleaved && turns ? c + a.rot / 16 : 2 * c + 1;
  const int heads = static_cast<int>(a.H), h0 = part * kRounds * kTeams + team;
  Eight<kF32> xa[kRounds], xb[kRounds];
  {
    const int64_t at = t * a.st[0];
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      const int h = h0 + i * kTeams;
      if (h < heads) {
        xa[i].load(a.q, at + static_cast<int64_t>(h) * D + 8 * ca);
        xb[i].load(a.q, at + static_cast<int64_t>(h) * D + 8 * cb);
      }
    }
  }
  // (a, b) -> (a aa + b ab, a ba + b bb)
  float aa[8], ab[8], ba[8], bb[8];
  {
    float wa[8], wb[8], cs[8], sn[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) wa[i] = wb[i] = cs[i] = 1.0f, sn[i] = 0.0f;
    if (a.q_weight != nullptr) {
      load8(a.q_weight + 8 * ca, wa);
      load8(a.q_weight + 8 * cb, wb);
      if constexpr (kInterleaved) split_pairs(wa, wb);
    }
    if (turns) {
      const float* row = a.table + static_cast<int64_t>(t) * a.rot + 8 * c;
      load8(row, cs);
      load8(row + a.rot / 2, sn);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      aa[i] = wa[i] * cs[i];
      ab[i] = -wb[i] * sn[i];
      ba[i] = wa[i] * sn[i];
      bb[i] = wb[i] * cs[i];
    }
  }
  uint16_t* out = a.q_out + t * a.st[3];
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    if (part * kRounds + i >= p.nq) break;
    const int h = h0 + i * kTeams;
    float za[8] = {}, zb[8] = {};
    if (h < heads) {
      xa[i].unpack(za);
      xb[i].unpack(zb);
    }
    if constexpr (kInterleaved) split_pairs(za, zb);
    float f = 1.0f;
    if (a.q_weight != nullptr) {
      float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float2 u = make_float2(za[e], za[e + 1]), v = make_float2(zb[e], zb[e + 1]);
        s2 = __ffma2_rn(u, u, __ffma2_rn(v, v, s2));
      }
      float ss = s2.x + s2.y;
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
      f = rsqrtf(fmaf(ss, p.inv_d, a.eps));
    }
    float oa[8], ob[8];
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float2 f2 = make_float2(f, f);
      const float2 u = __fmul2_rn(make_float2(za[e], za[e + 1]), f2), v = __fmul2_rn(make_float2(zb[e], zb[e + 1]), f2);
      // (0 times an infinity must not reach a channel that has no pair)
      const float2 ux = turns ? u : make_float2(0.0f, 0.0f), vx = turns ? v : make_float2(0.0f, 0.0f);
      const float2 x = __ffma2_rn(u, make_float2(aa[e], aa[e + 1]), __fmul2_rn(vx, make_float2(ab[e], ab[e + 1])));
      const float2 y = __ffma2_rn(ux, make_float2(ba[e], ba[e + 1]), __fmul2_rn(v, make_float2(bb[e], bb[e + 1])));
      oa[e] = x.x; oa[e + 1] = x.y;
      ob[e] = y.x; ob[e + 1] = y.y;
    }
    if constexpr (kInterleaved) join_pairs(oa, ob);
    if (h < heads) {
      store8(out + static_cast<int64_t>(h) * D + 8 * ca, oa);
      store8(out + static_cast<int64_t>(h) * D + 8 * cb, ob);
    }
  }
}

// Keys and values: d / 8 lanes a head, a chunk of 8 channels each.
//
// The lane's rotation of one token: halves (the chunk's eight pairs, whose other channel is lane
// `partner`'s) or neighbours (its four pairs).
template <bool kInterleaved>
struct Turn {
  float cs[8], sn[8];  // no rotation: 1 and 0
  int partner;
  bool turns;
  __device__ __forceinline__ void load(const AppendParams& p, int64_t t, int lane, int c) {
    const Kv4AppendArgs& a = p.a;
    const bool upper = !kInterleaved && 16 * c >= a.rot;
    const int half = a.rot / 2, other = a.rot / 16;
    turns = 8 * c < a.rot;
    partner = !kInterleaved && turns ? lane + (upper ? -other : other) : lane;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cs[i] = 1.0f;
      sn[i] = 0.0f;
    }
    if (!turns) return;
    const float* row = a.table + t * 2 * half;
    if constexpr (kInterleaved) {
      const float4 u = *reinterpret_cast<const float4*>(row + 4 * c);
      const float4 v = *reinterpret_cast<const float4*>(row + half + 4 * c);
      cs[0] = u.x; cs[1] = u.y; cs[2] = u.z; cs[3] = u.w;
      sn[0] = v.x; sn[1] = v.y; sn[2] = v.z; sn[3] = v.w;
    } else {
      load8(row + 8 * (upper ? c - other : c), cs);
      load8(row + half + 8 * (upper ? c - other : c), sn);
      if (!upper) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sn[i] = -sn[i];  // exact: a cos - b sin is a cos + b (-sin)
      }
    }
  }
};

// r, and z = x w turned in place.  Products and sums are rounded one by one: the codes are then the
// same wherever they are formed.
template <int D, bool kInterleaved>
__device__ __forceinline__ float norm_and_turn(const AppendParams& p, const Turn<kInterleaved>& rot, const float (&wv)[8],
                                               float (&z)[8]) {
  float f = 1.0f;
  if (p.a.k_weight != nullptr) {
    float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 u = make_float2(z[i], z[i + 1]), v = make_float2(__fmul_rn(u.x, wv[i]), __fmul_rn(u.y, wv[i + 1]));
      s2 = __ffma2_rn(u, u, s2);
      z[i] = v.x;
      z[i + 1] = v.y;
    }
    float ss = s2.x + s2.y;
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
    f = rsqrtf(fmaf(ss, p.inv_d, p.a.eps));
  }
  if constexpr (kInterleaved) {
    if (rot.turns) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float u = z[2 * i], v = z[2 * i + 1];
        z[2 * i] = __fsub_rn(__fmul_rn(u, rot.cs[i]), __fmul_rn(v, rot.sn[i]));
        z[2 * i + 1] = __fadd_rn(__fmul_rn(u, rot.sn[i]), __fmul_rn(v, rot.cs[i]));
      }
    }
  } else if (p.a.rot > 0) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 o = make_float2(__shfl_sync(kFull, z[i], rot.partner), __shfl_sync(kFull, z[i + 1], rot.partner));
      // scalar products: packed ones are fused into the sums even so
      const float2 v = __fadd2_rn(make_float2(__fmul_rn(z[i], rot.cs[i]), __fmul_rn(z[i + 1], rot.cs[i + 1])),
                                  make_float2(__fmul_rn(o.x, rot.sn[i]), __fmul_rn(o.y, rot.sn[i + 1])));
      z[i] = v.x;
      z[i + 1] = v.y;
    }
  }
  return f;
}

__device__ __forceinline__ float max_or_nan(float a, float b) {  // NaN if one of them is
  float c;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(c) : "f"(a), "f"(b));
  return c;
}

// Of a block: what its channels are multiplied by, its scale.
__device__ __forceinline__ float per_code(float top) { return top < kKv4Zero ? 0.0f : __fdiv_rn(7.0f, top); }
__device__ __forceinline__ __nv_bfloat16 block_scale(float top, float f) {
  return __float2bfloat16_rn(top < kKv4Zero ? 0.0f : __fmul_rn(__fmul_rn(top, f), 1.0f / 7.0f));
}
__device__ __forceinline__ uint32_t codes(const float (&z)[8], float per) {
  uint32_t word = 0;
#pragma unroll
  for (int e = 6; e >= 0; e -= 2) {
    // 1.5 2^23 + 8 is even, so adding it rounds as rint does; its bits are 0x4B400000 + code + 8,
    // and the first part of eight of them, each 16 times the next, is taken off at the end
    const float2 m = __fadd2_rn(make_float2(__fmul_rn(z[e], per), __fmul_rn(z[e + 1], per)), make_float2(12582920.0f, 12582920.0f));
    word = (word * 16u + __float_as_uint(m.y)) * 16u + __float_as_uint(m.x);
  }
  return word + kCodes;
}

// The quantiser: lanes 4 b .. 4 b + 3 of a head hold block b.  The lane's eight codes, and its block's
// scale.  A block with a NaN or an infinity has that for its scale, and any codes.
__device__ __forceinline__ uint32_t quantise(const float (&z)[8], float f, __nv_bfloat16* scale) {
  float top = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max_or_nan(top, fabsf(z[e]));
  top = max_or_nan(top, __shfl_xor_sync(kFull, top, 1));
  top = max_or_nan(top, __shfl_xor_sync(kFull, top, 2));
  *scale = block_scale(top, f);
  return codes(z, per_code(top));
}

// Four of them at once: each of a block's lanes (u = lane % 4) takes one's largest magnitude, and so
// its division and scale, and passes the quotient on.
__device__ __forceinline__ void quantise_four(const float (&z)[4][8], int u, float f, uint32_t (&word)[4], __nv_bfloat16* scale) {
  float top[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    top[v] = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) top[v] = max_or_nan(top[v], fabsf(z[v][e]));
  }
  const bool odd = (u & 1) != 0, high = (u & 2) != 0;
  const float lo = max_or_nan(odd ? top[1] : top[0], __shfl_xor_sync(kFull, odd ? top[0] : top[1], 1));
  const float hi = max_or_nan(odd ? top[3] : top[2], __shfl_xor_sync(kFull, odd ? top[2] : top[3], 1));
  const float mine = max_or_nan(high ? hi : lo, __shfl_xor_sync(kFull, high ? lo : hi, 2));
  *scale = block_scale(mine, f);
  const float per = per_code(mine);
#pragma unroll
  for (int v = 0; v < 4; ++v) word[v] = codes(z[v], __shfl_sync(kFull, per, v, 4));
}

// Blocks 2 h and 2 h + 1 of a value share words: of a lane's two halves the lane of the other block
// takes one.  The lane's word is that of channels 64 h + 4 g .. and + 32, g = 2 (c % 4) + b % 2.
__device__ __forceinline__ uint32_t pair_values(uint32_t word, int b) {
  const uint32_t got = __shfl_xor_sync(kFull, (b & 1) == 0 ? word >> 16 : word & 0xFFFFu, 4);
  return (b & 1) == 0 ? (word & 0xFFFFu) | got << 16 : got | (word & 0xFFFF0000u);
}

// A token's place from its slot; false: it is not kept.
__device__ __forceinline__ bool token_place(const Kv4AppendArgs& a, int slot, int tile_bytes, uint8_t** tile, int* tok) {
  const uint32_t page = static_cast<uint32_t>(slot) / static_cast<uint32_t>(a.page);
  const int in_page = static_cast<int>(static_cast<uint32_t>(slot) - page * static_cast<uint32_t>(a.page));
  *tok = in_page & 31;
  if (slot < 0 || page >= a.pages) return false;
  *tile = a.cache + page * a.page_stride + static_cast<int64_t>(in_page >> 5) * tile_bytes;
  return true;
}

// A warp takes kRounds rounds of one token's heads, of one kind, and loads them all before the first
// is worked on.
template <int D, bool kF32, bool kInterleaved, int kRounds>
__global__ void __launch_bounds__(kAppendThreads, kF32 ? 6 : 7) kv4_append_kernel(const __grid_constant__ AppendParams p) {
  using Tile = Kv4Tile<D>;
  constexpr int L = D / 8, kTeams = 32 / L;  // lanes of a head, heads of a round
  const Kv4AppendArgs& a = p.a;
  const int lane = static_cast<int>(threadIdx.x & 31), c = lane % L, team = lane / L;
  const uint32_t unit = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  const uint32_t t = unit / static_cast<uint32_t>(p.parts);
  pdl_wait();
  pdl_launch_dependents();
  if (t >= a.T) return;
  // the part's kind (0 query, 1 key, 2 value) and first round
  int part = static_cast<int>(unit - t * p.parts);
  const int pk = (p.parts - p.pq) / 2, kind = part < p.pq ? 0 : part < p.pq + pk ? 1 : 2;
  part -= kind == 0 ? 0 : kind == 1 ? p.pq : p.pq + pk;
  if (kind == 0) {
    append_queries<D, kF32, kInterleaved, kRounds>(p, t, part, lane);
    return;
  }
  const int r0 = part * kRounds, rounds = p.nk - r0, heads = static_cast<int>(a.Hkv);
  Eight<kF32> x[kRounds];
  {
    const void* from = kind == 1 ? a.k : a.v;
    const int64_t at = t * a.st[kind] + 8 * c;
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      const int h = (r0 + i) * kTeams + team;
      if (h < heads) x[i].load(from, at + static_cast<int64_t>(h) * D);
    }
  }
  Turn<kInterleaved> rot;
  float wv[8];
  if (kind == 1) {
    rot.load(p, t, lane, c);
    if (a.k_weight != nullptr) load8(a.k_weight + 8 * c, wv);
  }
  const int slot = a.slots[t];
  uint8_t* tile0 = nullptr;
  int tok;
  if (!token_place(a, slot, Tile::kBytes, &tile0, &tok)) {
    if (slot >= 0 && lane == 0 && r0 == 0) atomicOr(a.err, kErrBadCache);
    return;
  }
  const int64_t head_bytes = a.page / 32 * Tile::kBytes;
  const int b = c >> 2;
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    if (i >= rounds) break;
    const int h = (r0 + i) * kTeams + team;
    const bool on = h < heads;
    float z[8] = {}, f = 1.0f;
    if (on) x[i].unpack(z);
    if (kind == 1) f = norm_and_turn<D, kInterleaved>(p, rot, wv, z);
    __nv_bfloat16 sc;
    uint32_t word = quantise(z, f, &sc);
    if (kind == 2) word = pair_values(word, b);
    uint8_t* tile = tile0 + h * head_bytes;
    if (on) {
      *reinterpret_cast<uint32_t*>(tile + (kind == 1 ? Tile::key_word(tok, c) : Tile::value_word(tok, 2 * (c & 3) + (b & 1), b >> 1))) = word;
      if ((c & 3) == 0)
        *reinterpret_cast<__nv_bfloat16*>(tile + (kind == 1 ? Tile::kKeyScales : Tile::kValueScales) + Tile::scale(tok, b)) = sc;
    }
  }
}

// Many tokens: a block takes 32 neighbouring ones of one key/value head, or four parts of queries.
// What its warps have formed meets in shared memory and is written in the order of the tiles, so
// that sectors are written whole: the tokens one by one would write 18 sectors each, most of them 2
// or 8 bytes at a time (8192 tokens of 8 heads of 128: keys and values 14.2 us so, 21.5 one by one).
template <int D, bool kF32, bool kInterleaved>
__global__ void __launch_bounds__(kAppendThreads, kF32 ? 6 : 7) kv4_append_tiles_kernel(const __grid_constant__ AppendParams p) {
  using Tile = Kv4Tile<D>;
  constexpr int L = D / 8, kTeams = 32 / L, kRounds = 2;
  const Kv4AppendArgs& a = p.a;
  const int lane = static_cast<int>(threadIdx.x & 31), warp = static_cast<int>(threadIdx.x >> 5);
  if (blockIdx.x >= static_cast<uint32_t>(p.kv_blocks)) {
    const uint32_t unit = (blockIdx.x - static_cast<uint32_t>(p.kv_blocks)) * (kAppendThreads / 32) + warp;
    const uint32_t t = unit / static_cast<uint32_t>(p.pq);
    if (t < a.T) append_queries<D, kF32, kInterleaved, kRounds>(p, t, static_cast<int>(unit - t * p.pq), lane);
    return;
  }
  // a token's row: its words in the order of its tile (keys: pieces of kWords, values: of kHalves)
  constexpr int kStride = D / 8 + 4;
  __shared__ __align__(16) uint32_t words_s[kTileHeads][2][32][kStride];
  __shared__ __nv_bfloat16 scales_s[kTileHeads][2][Tile::kBlocks][32];
  const uint32_t groups = (static_cast<uint32_t>(a.Hkv) + kTileHeads - 1) / kTileHeads, chunk = blockIdx.x / groups;
  const int64_t h0 = static_cast<int64_t>(blockIdx.x - chunk * groups) * kTileHeads, t0 = static_cast<int64_t>(chunk) * 32;
  const int heads = a.Hkv - h0 < kTileHeads ? static_cast<int>(a.Hkv - h0) : kTileHeads;
  const int rows = a.T - t0 < 32 ? static_cast<int>(a.T - t0) : 32;
  const int c = lane % L, team = lane / L, b = c >> 2;
  const int slot = lane < rows ? a.slots[t0 + lane] : -1;
  // 8 rows a warp, kTeams at a time with all of the block's heads
  float wv[8];
  if (a.k_weight != nullptr) load8(a.k_weight + 8 * c, wv);
#pragma unroll 1
  for (int i = 0; i < 8 / kTeams; ++i) {
    const int row = 8 * warp + i * kTeams + team;
    const int64_t t = t0 + (row < rows ? row : rows - 1);  // behind the last row or head: that one again
    Eight<kF32> x[4];                                      // keys of both heads, values of both
#pragma unroll
    for (int hh = 0; hh < kTileHeads; ++hh) {
      const int64_t at = (h0 + (hh < heads ? hh : 0)) * D + 8 * c;
      x[hh].load(a.k, t * a.st[1] + at);
      x[2 + hh].load(a.v, t * a.st[2] + at);
    }
    Turn<kInterleaved> rot;
    rot.load(p, t, lane, c);
    float z[4][8], f[kTileHeads];
#pragma unroll
    for (int v = 0; v < 4; ++v) x[v].unpack(z[v]);
#pragma unroll
    for (int hh = 0; hh < kTileHeads; ++hh) f[hh] = norm_and_turn<D, kInterleaved>(p, rot, wv, z[hh]);
    const int u = c & 3;
    uint32_t word[4];
    __nv_bfloat16 sc;
    quantise_four(z, u, (u & 2) != 0 ? 1.0f : (u & 1) != 0 ? f[1] : f[0], word, &sc);
    scales_s[u & 1][u >> 1][b][row] = sc;
#pragma unroll
    for (int hh = 0; hh < kTileHeads; ++hh) {
      words_s[hh][0][row][((b >> 2) * 4 + u) * Tile::kWords + (b & 3)] = word[hh];
      words_s[hh][1][row][(2 * u + (b & 1)) * Tile::kHalves + (b >> 1)] = pair_values(word[2 + hh], b);
    }
  }
  __syncthreads();

  // neighbours in the cache: the end of one tile, then the beginning of another
  const int first = __shfl_sync(kFull, slot, 0), tok0 = first & 31, k = 32 - tok0, next = __shfl_sync(kFull, slot, k & 31);
  const bool follows = lane < k ? static_cast<uint32_t>(slot) == static_cast<uint32_t>(first) + lane
                                : static_cast<uint32_t>(slot) == static_cast<uint32_t>(next) + lane - k && (next & 31) == 0;
  uint8_t* tiles[2] = {nullptr, nullptr};
  int tok;
  bool ok = token_place(a, first, Tile::kBytes, &tiles[0], &tok);
  if (k < rows) ok = ok && token_place(a, next, Tile::kBytes, &tiles[1], &tok);
  const bool in_order = ok && __all_sync(kFull, lane >= rows || follows);
  for (int hh = 0; hh < heads; ++hh) {
    const int64_t head_at = (h0 + hh) * (a.page / 32) * Tile::kBytes;
    const auto& words = words_s[hh];
    const auto& scales = scales_s[hh];
    if (in_order) {
      const int id = static_cast<int>(threadIdx.x);
#pragma unroll 1
      for (int part = 0; part < 2; ++part) {
        if (part == 1 && k >= rows) break;
        uint8_t* tile = tiles[part] + head_at;
        // the row of a token of this tile, outside [0, rows): not one of them
        auto row_of = [&](int x) { return part == 0 ? x - tok0 : x + k < 32 ? x + k : -1; };
#pragma unroll
        for (int i = 0; i < D / kAppendThreads + (D < kAppendThreads ? 1 : 0); ++i) {  // keys: d pieces of 16 bytes
          const int at = id + i * kAppendThreads;
          if (at >= D) break;
          int x, piece;
          if constexpr (D == 64) {  // rows of two pieces
            x = at >> 1;
            piece = at & 1;
          } else {  // [j][b / 4][n][u]
            piece = at & 3;
            x = at >> 2;
          }
          int n, j;
          if constexpr (D == 256) {
            n = x & 7;
            piece += ((x >> 3) & 1) * 4;
            j = x >> 4;
          } else {
            n = x & 7;
            j = x >> 3;
          }
          const int row = row_of(8 * (n >> 1) + 2 * j + (n & 1));
          if (row >= 0 && row < rows)
            *reinterpret_cast<uint4*>(tile + at * 16) = *reinterpret_cast<const uint4*>(&words[0][row][piece * 4]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // values: 256 pieces of d / 64 words, [2 j + i][g][t]
          const int at = id + i * kAppendThreads, g = (at >> 2) & 7, row = row_of(8 * (at & 3) + (at >> 5));
          if (row >= 0 && row < rows) {
            uint8_t* dst = tile + Tile::kValues + at * 4 * Tile::kHalves;
            const uint32_t* src = &words[1][row][g * Tile::kHalves];
            if constexpr (D == 256) *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
            else if constexpr (D == 128) *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(src);
            else *reinterpret_cast<uint32_t*>(dst) = *src;
          }
        }
        const int row = row_of(lane);
        if (row >= 0 && row < rows)
          for (int e = warp; e < 2 * Tile::kBlocks; e += kAppendThreads / 32) {
            const int kv = e / Tile::kBlocks, blk = e % Tile::kBlocks;
            *reinterpret_cast<__nv_bfloat16*>(tile + (kv == 0 ? Tile::kKeyScales : Tile::kValueScales) + Tile::scale(lane, blk)) =
                scales[kv][blk][row];
          }
      }
      continue;
    }
    // tokens anywhere: each row by a team
#pragma unroll 1
    for (int i = 0; i < 8 / kTeams; ++i) {
      const int row = 8 * warp + i * kTeams + team;
      if (row >= rows) continue;
      uint8_t* tile = nullptr;
      const int s = a.slots[t0 + row];
      if (!token_place(a, s, Tile::kBytes, &tile, &tok)) {
        if (s >= 0 && c == 0 && h0 + hh == 0) atomicOr(a.err, kErrBadCache);
        continue;
      }
      tile += head_at;
      const int g = 2 * (c & 3) + (b & 1);
      *reinterpret_cast<uint32_t*>(tile + Tile::key_word(tok, c)) = words[0][row][((b >> 2) * 4 + (c & 3)) * Tile::kWords + (b & 3)];
      *reinterpret_cast<uint32_t*>(tile + Tile::value_word(tok, g, b >> 1)) = words[1][row][g * Tile::kHalves + (b >> 1)];
      if ((c & 3) == 0) {
        *reinterpret_cast<__nv_bfloat16*>(tile + Tile::kKeyScales + Tile::scale(tok, b)) = scales[0][b][row];
        *reinterpret_cast<__nv_bfloat16*>(tile + Tile::kValueScales + Tile::scale(tok, b)) = scales[1][b][row];
      }
    }
  }
}

// ---- gather ----------------------------------------------------------------------------------
constexpr int kGatherThreads = 128;

// A warp takes 32 rows of one head, or (kFew) as many as its teams of d / 8 lanes copy at once, four
// each.  Each lane finds one row's place in the cache.  Of 32 rows a team copies those at once that
// are 8 tokens apart, as they share the sectors that their values lie in.
template <int D, bool kBf16, bool kFew>
__global__ void __launch_bounds__(kGatherThreads) kv4_gather_kernel(const __grid_constant__ Kv4GatherArgs a) {
  using Tile = Kv4Tile<D>;
  constexpr int L = D / 8, kTeams = 32 / L, kAhead = 4, kRows = kFew ? kAhead * kTeams : 32;
  const int lane = static_cast<int>(threadIdx.x & 31);
  const uint32_t unit = blockIdx.x * (kGatherThreads / 32) + (threadIdx.x >> 5);
  const uint32_t chunk = unit / static_cast<uint32_t>(a.Hkv);
  const int h = static_cast<int>(unit - chunk * static_cast<uint32_t>(a.Hkv));
  const int64_t row0 = static_cast<int64_t>(chunk) * kRows;
  pdl_wait();
  if (row0 >= a.T) return;
  const uint8_t* mine = nullptr;  // the tile of row row0 + lane; nullptr: no row
  int mine_tok = 0;
  {
    // the last sequence that begins at or in front of the first row: of 32 at a time
    int64_t lo = 0, n = a.B;
    while (n > 1) {
      const int64_t step = (n + 31) / 32, at = static_cast<int64_t>(lane) * step;
      const int in = __popc(__ballot_sync(kFull, at < n && a.cu[lo + at] <= row0));
      if (in == 0) break;
      lo += (in - 1) * step;
      n = n - (in - 1) * step < step ? n - (in - 1) * step : step;
    }
    const int64_t row = row0 + lane;
    // the lane's own: among the 32 behind it, or further on
    const int64_t next = lo + 1 + lane < a.B ? a.cu[lo + 1 + lane] : a.T;
    int ahead = 0;
    if (__shfl_sync(kFull, next, 0) < row0 + kRows) {
#pragma unroll 4
      for (int i = 0; i < kRows; ++i) {
        const int passed = __popc(__ballot_sync(kFull, next <= row0 + i));
        ahead = lane == i ? passed : ahead;
      }
    }
    lo += ahead;
    if (ahead == 32) {
      int64_t hi = a.B - 1;
      while (lo < hi) {
        const int64_t mid = (lo + hi + 1) >> 1;
        if (a.cu[mid] <= row) lo = mid;
        else hi = mid - 1;
      }
    }
    if (lane < kRows && row < a.T) {
      const int64_t begin = a.cu[lo];
      if (begin <= row && row < a.cu[lo + 1]) {
        const int64_t pos = (a.first != nullptr ? a.first[lo] : 0) + (row - begin);
        int64_t page = -1;
        int in_page = 0;
        if (pos >= 0 && pos < a.width * a.page) {  // below 2^31
          const uint32_t at = static_cast<uint32_t>(pos) / static_cast<uint32_t>(a.page);
          in_page = static_cast<int>(static_cast<uint32_t>(pos) - at * static_cast<uint32_t>(a.page));
          page = a.block_table[lo * a.width + at];
        }
        if (page >= 0 && page < a.pages) {
          mine_tok = in_page & 31;
          mine = a.cache + page * a.page_stride +
                 (static_cast<int64_t>(h) * (a.page / 32) + (in_page >> 5)) * Tile::kBytes;
        } else if (h == 0) {
          atomicOr(a.err, kErrBadCache);
        }
      }
    }
  }
  __syncwarp();
  const int c = lane % L, team = lane / L, b = c >> 2, u = c & 3;
#pragma unroll
  for (int i = 0; i < kRows / (kAhead * kTeams); ++i) {
    uint32_t kw[kAhead], vw[kAhead], ks[kAhead], vs[kAhead];
    bool on[kAhead];
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      const int r = i * kTeams + team + (kFew ? kTeams : 8) * e;
      const uint8_t* tile = reinterpret_cast<const uint8_t*>(__shfl_sync(kFull, reinterpret_cast<unsigned long long>(mine), r));
      const int tok = __shfl_sync(kFull, mine_tok, r);
      on[e] = tile != nullptr;
      kw[e] = vw[e] = ks[e] = vs[e] = 0;
      if (on[e]) {
        kw[e] = *reinterpret_cast<const uint32_t*>(tile + Tile::key_word(tok, c));
        vw[e] = *reinterpret_cast<const uint32_t*>(tile + Tile::value_word(tok, 2 * u + (b & 1), b >> 1));
        ks[e] = *reinterpret_cast<const uint16_t*>(tile + Tile::kKeyScales + Tile::scale(tok, b));
        vs[e] = *reinterpret_cast<const uint16_t*>(tile + Tile::kValueScales + Tile::scale(tok, b));
      }
    }
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      const uint32_t got = __shfl_xor_sync(kFull, (b & 1) == 0 ? vw[e] >> 16 : vw[e] & 0xFFFFu, 4);
      const uint32_t both = (b & 1) == 0 ? (vw[e] & 0xFFFFu) | got << 16 : got | (vw[e] & 0xFFFF0000u);
      if (!on[e]) continue;
      const int64_t at = ((row0 + i * kTeams + team + (kFew ? kTeams : 8) * e) * a.Hkv + h) * D + 8 * c;
      auto put = [&](void* out, uint32_t w, uint32_t s16) {
        if constexpr (kBf16) {
          // pairs of nibbles (j, j + 4) as 128 + n, less 136 (exact), times the scale (rounded once)
          const uint32_t s2 = s16 | s16 << 16;
          uint32_t y[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t n = ((w >> (4 * j)) & 0x000F000Fu) | 0x43004300u, m = 0xC308C308u;  // -136
            const __nv_bfloat162 z = __hmul2(__hadd2(*reinterpret_cast<const __nv_bfloat162*>(&n), *reinterpret_cast<const __nv_bfloat162*>(&m)),
                                             *reinterpret_cast<const __nv_bfloat162*>(&s2));
            y[j] = *reinterpret_cast<const uint32_t*>(&z);
          }
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) =
              make_uint4(__byte_perm(y[0], y[1], 0x5410), __byte_perm(y[2], y[3], 0x5410), __byte_perm(y[0], y[1], 0x7632),
                         __byte_perm(y[2], y[3], 0x7632));
        } else {
          const float s = __uint_as_float(s16 << 16);
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)  // 2^23 + n, less 2^23 + 8, times the scale: exact, 4 bits times 8
            v[j] = (__uint_as_float(((w >> (4 * j)) & 15u) | 0x4B000000u) - 8388616.0f) * s;
          float4* f = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
          f[0] = make_float4(v[0], v[1], v[2], v[3]);
          f[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
      };
      put(a.k, kw[e], ks[e]);
      put(a.v, both, vs[e]);
    }
  }
}

// A step's kernels follow one another: each may start while the one before ends (it waits for it
// before it touches memory, and only then lets the next one start).  A decoded token's append and
// attention, 32 / 8 heads of 128 and 1000 tokens: 8.3 us a layer (8.2 and 8.7 without when it was brought in).
template <typename P>
cudaError_t launch_next(void (*kernel)(P), unsigned grid, unsigned threads, const P& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int D, bool kF32, int kRounds>
cudaError_t append_rounds(AppendParams p, cudaStream_t stream) {
  const Kv4AppendArgs& a = p.a;
  p.pq = (p.nq + kRounds - 1) / kRounds;
  p.parts = p.pq + 2 * ((p.nk + kRounds - 1) / kRounds);
  const int64_t blocks = (a.T * p.parts + kAppendThreads / 32 - 1) / (kAppendThreads / 32);  // a unit fits 32 bits: T (H + 2 Hkv) does
  const unsigned grid = static_cast<unsigned>(blocks);
  return launch_next(a.interleaved ? kv4_append_kernel<D, kF32, true, kRounds> : kv4_append_kernel<D, kF32, false, kRounds>, grid,
                     kAppendThreads, p, stream);
}

template <int D, bool kF32>
cudaError_t append(const Kv4AppendArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  AppendParams p = {};
  p.a = a;
  constexpr int kTeams = 32 / (D / 8), kMost = 2;
  p.nq = static_cast<int>((a.H + 2 * kTeams - 1) / (2 * kTeams));
  p.nk = static_cast<int>((a.Hkv + kTeams - 1) / kTeams);
  p.inv_d = 1.0f / D;
  // Tiles where their blocks are two an SM: fewer, each with 32 tokens to go through, end later than
  // tokens spread over all warps (bfloat16, 32 / 8 heads of 128: 372 blocks 14.4 us against 16.7, 256 blocks
  // 12.6 and 12.4, 128 blocks 9.1 and 6.8; 16 / 4 of 256: 256 blocks 21.8 both; 16 / 16 of 64 from
  // binary32: 512 blocks 9.4 and 10.0, 256 blocks 5.4 both)
  const int64_t kv_blocks = (a.T + 31) / 32 * ((a.Hkv + kTileHeads - 1) / kTileHeads);
  if (a.T >= 32 && kv_blocks >= 2 * static_cast<int64_t>(dev.sm_count)) {
    p.kv_blocks = static_cast<int>(kv_blocks);
    p.pq = (p.nq + kMost - 1) / kMost;
    const unsigned grid = static_cast<unsigned>(kv_blocks + (a.T * p.pq + kAppendThreads / 32 - 1) / (kAppendThreads / 32));
    // (not launched as the step's small kernels are: its blocks go through many waves, and waiting in
    // each took 8192 tokens of 32 / 8 heads and their gather from 45.5 us to 48.8 when it was tried)
    if (a.interleaved) kv4_append_tiles_kernel<D, kF32, true><<<grid, kAppendThreads, 0, stream>>>(p);
    else kv4_append_tiles_kernel<D, kF32, false><<<grid, kAppendThreads, 0, stream>>>(p);
    return cudaGetLastError();
  }
  // A second round a warp from 32 rounds of heads an SM on (bfloat16, 32 / 8 heads of 128, by one round and by two: 8 rounds
  // an SM 2.63 us and 2.76, 16 2.98 and 2.94, 24 3.55 and 3.03, 32 3.68 and 3.80, 40 4.34 and 4.00, 96 7.2 and 6.1; 16 / 16 of
  // 64 from binary32: 8 2.54 and 2.82, 16 2.86 and 3.04, 24 3.44 and 3.17, 32 3.58 and 3.83, 40 4.12 and 3.87; 16 / 4 of 256: 8
  // 2.61 and 2.79, 32 3.64 and 3.83, 40 4.34 and 4.07)
  const int64_t rounds = a.T * (p.nq + 2 * p.nk), warps = static_cast<int64_t>(dev.sm_count) * 16;
  return rounds >= warps * kMost ? append_rounds<D, kF32, kMost>(p, stream) : append_rounds<D, kF32, 1>(p, stream);
}

template <int D, bool kFew>
cudaError_t gather_rows(const Kv4GatherArgs& a, cudaStream_t stream) {
  constexpr int kRows = kFew ? 4 * 32 / (D / 8) : 32;
  const int64_t units = (a.T + kRows - 1) / kRows * a.Hkv;  // T Hkv fits 31 bits
  const unsigned grid = static_cast<unsigned>((units + kGatherThreads / 32 - 1) / (kGatherThreads / 32));
  return launch_next(a.bf16 ? kv4_gather_kernel<D, true, kFew> : kv4_gather_kernel<D, false, kFew>, grid, kGatherThreads, a, stream);
}

template <int D>
cudaError_t gather(const Kv4GatherArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  // Few rows a warp where 32 would not give every SM eight warps.  One context, by 32 rows and by few, into rows that
  // the call before has left in the L2: 8 heads of 128 in bfloat16, 2432 tokens (four warps an SM) 5.2 us and
  // 3.9, 4864 (eight) 5.9 and 5.4, 7296 6.9 both, 19456 16.1 and 17.5; 16 heads of 64 from 608 tokens (two) 3.6 and 2.9
  // to 2432 (eight) 4.1 and 3.9, 19456 16.7 and 18.0, in binary32 2432 7.2 and 7.4, 9728 18.0 and 20.3.  Rows in memory,
  // and heads of 256, keep few rows ahead: 19456 of 8 heads of 128 20.3 and 19.3, 9728 of 4 of 256 14.9 and 10.9.
  return (a.T + 31) / 32 * a.Hkv < 8 * static_cast<int64_t>(dev.sm_count) ? gather_rows<D, true>(a, stream) : gather_rows<D, false>(a, stream);
}

}  // namespace

cudaError_t launch_rope_table(const int32_t* positions, int axes, const double* inv_freq, const int32_t* axis,
                              float* table, int64_t T, int half, const DeviceInfo& dev, cudaStream_t stream) {
  if (T == 0 || half == 0) return cudaSuccess;
  const TableParams p = {positions, inv_freq, axis, table, T, axes, half};
  const int64_t blocks = (T * (half / 4) + 255) / 256;
  return launch_next(rope_table_kernel, static_cast<unsigned>(std::min<int64_t>(blocks, dev.sm_count * 8)), 256u, p, stream);
}

cudaError_t launch_kv4_append(Kv4AppendArgs a, const DeviceInfo& dev, cudaStream_t stream) {
  if (a.T == 0 || a.H + a.Hkv == 0) return cudaSuccess;
  a.err = dev.err_word;
  if (a.f32) return a.d == 64 ? append<64, true>(a, dev, stream) : a.d == 128 ? append<128, true>(a, dev, stream) : append<256, true>(a, dev, stream);
  return a.d == 64 ? append<64, false>(a, dev, stream) : a.d == 128 ? append<128, false>(a, dev, stream) : append<256, false>(a, dev, stream);
}

cudaError_t launch_kv4_gather(Kv4GatherArgs a, const DeviceInfo& dev, cudaStream_t stream) {
  if (a.T == 0 || a.B == 0 || a.Hkv == 0) return cudaSuccess;
  a.err = dev.err_word;
  return a.d == 64 ? gather<64>(a, dev, stream) : a.d == 128 ? gather<128>(a, dev, stream) : gather<256>(a, dev, stream);
}

}  // namespace q8
