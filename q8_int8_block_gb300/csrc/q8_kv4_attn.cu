// q8_kv4_attn.cu -- attention of the newest tokens of each request over its paged 4-bit cache.
//
// o = sum_j p_j v_j / sum_j p_j, p_j = exp(scale q . k_j), keys and values in the tiles of
// q8_kv4.cuh: k = s_b (n - 8), a nibble n and a scale s_b for 32 channels of a token.
//
// Mathematics.  Codes are multiplied as they lie: a nibble in the low bits of a bfloat16 is the
// subnormal n 2^-133, one four bits higher is 16 n 2^-133 (the encoding is linear up to 255), and
// the tensor pipe takes subnormals exactly, so one AND makes two operands and nothing is converted.
// The other factor carries 2^100 (queries, scaled by a power of two for each row) or 2^64
// (weights), which keeps every sum far inside binary32.  What is left is linear and comes last:
//   scores   s_b (sum q n - 8 sum q): the second sum belongs to the query, the block's scale is
//            applied to the binary32 sum of the block;
//   output   the value's scale multiplies the weight, w = bf16(bf16(p) s_b), and
//            sum w (n - 8) = sum w n - 8 sum w: the second sum is one more product, whose
//            constant operand has a row for each block of 32 channels.
// Weights and scales are rounded to bfloat16 twice where the other attention kernels round once
// (2^-9 of a weight on average, independent for each key); all sums are binary32.
//
// Bound: the cache's bytes, 9/8 d for a key and head.  At the copy rate an SM gets 41 elements a
// clock, so instructions are as scarce as bytes: about 200 warp instructions for 16 keys of 128
// channels against 400 issue slots.
//
// Split.  The work is the list of (request, head, rows, tile of 32 keys), and every warp takes an
// equal run of it, wherever that begins and ends: lengths do not matter.  A warp has a ring of
// tiles that one bulk copy each fills, so its loop has no barrier.  Where a run ends inside a
// request the partial results meet in the block's shared memory, and what crosses blocks goes to
// a second kernel.
#include <cuda_bf16.h>

#include <algorithm>

#include "q8_attn_ptx.cuh"
#include "q8_internal.h"
#include "q8_kv4.cuh"

namespace q8 {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;

__device__ __forceinline__ void pdl_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ uint32_t mul_bf16(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }

constexpr float kNone = -1e30f;     // reference of a row that has seen no key
constexpr float kLift = 64.0f;      // weights are carried as 2^64 p
constexpr float kSlack = 10.0f;     // a reference may lag behind the largest score by 2^10

struct Kv4Params {
  Kv4AttentionArgs a;
  int G;
  float scale_log2;
  int per_thread;    // requests whose counts a thread sums up
  float* part;       // [blocks][2], then [blocks][warps] partial results
  int4* meta;        // [blocks][2]: request, head, rows, flags
};
enum : int { kPartHeld = 1, kPartFromFront = 2, kPartGoesOn = 4 };  // flags of a partial result

template <int D, int NT>
struct Kv4Shape {
  using Tile = Kv4Tile<D>;
  static constexpr int kRows = 8 * NT;
  static constexpr int kWarps = D == 256 ? 8 : NT == 2 && D == 128 ? 12 : 16;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kStages = 221184 / (Tile::kBytes * kWarps);
  static constexpr int kRing = kStages * Tile::kBytes;       // of a warp
  static constexpr int kPad = D + 4;                         // floats of a row's partial result: o, reference, sum
  static constexpr int kPart = kRows * kPad;                 // floats of a partial result
  static constexpr int kOffBar = kWarps * kRing;
  static constexpr int kOffPre = kOffBar + kWarps * kStages * 8;
  static constexpr int kOffBad = kOffPre + (kThreads + 1) * 8;
  static constexpr int kOffMeta = (kOffBad + kWarps * kStages * 4 + 15) / 16 * 16;
  static constexpr int kSmem = kOffMeta + kWarps * 2 * 16;
  static_assert(kSmem <= 226 * 1024, "shared memory of a block");
  static_assert(kPart * 4 <= kRing, "a partial result in the ring's place");
  static_assert(kRing % 16 == 0, "alignment of bulk copies");
};

// What a request asks for.
struct Request {
  int64_t q0;        // its first query
  int lq, len;       // queries, keys
  uint32_t tiles;    // of keys (one at least: rows without a key are written too)
  uint32_t groups;   // of rows
};
template <int NT>
__device__ __forceinline__ Request request(const Kv4Params& p, int64_t b, bool* bad) {
  Request r;
  const Kv4AttentionArgs& a = p.a;
  r.q0 = b;
  int64_t lq = 1;
  if (a.cu_q != nullptr) {
    r.q0 = a.cu_q[b];
    lq = a.cu_q[b + 1] - r.q0;
    if (r.q0 < 0 || lq < 0 || r.q0 + lq > a.Tq) {
      *bad = true;
      lq = 0;
    }
  }
  int64_t len = a.kv_len[b];
  const int64_t most = a.width * a.page;
  if (len < 0 || len > most) {
    *bad = true;
    len = len < 0 ? 0 : most;
  }
  r.lq = static_cast<int>(lq);
  r.len = static_cast<int>(len);
  r.tiles = len > 0 ? static_cast<uint32_t>((len + 31) >> 5) : 1u;
  r.groups = static_cast<uint32_t>((lq * p.G + 8 * NT - 1) / (8 * NT));
  return r;
}
__device__ __forceinline__ uint64_t count(const Kv4Params& p, const Request& r) {
  return static_cast<uint64_t>(r.tiles) * r.groups * static_cast<uint32_t>(p.a.Hkv);
}

// Where a place of the work list is.
struct Place {
  int64_t b;
  uint32_t h, group, tile;
  Request r;
};
template <int D, int NT>
__device__ __forceinline__ Place place(const Kv4Params& p, const uint64_t* pre, uint64_t at) {
  int lo = 0, hi = Kv4Shape<D, NT>::kThreads - 1;  // the last thread whose requests begin at or in front of it
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= at) lo = mid;
    else hi = mid - 1;
  }
  Place w;
  bool bad;
  w.b = static_cast<int64_t>(lo) * p.per_thread;
  uint64_t rest = at - pre[lo];
  w.r = request<NT>(p, w.b, &bad);
  for (uint64_t n = count(p, w.r); rest >= n; n = count(p, w.r)) {
    rest -= n;
    ++w.b;
    w.r = request<NT>(p, w.b, &bad);
  }
  if (rest >> 32 == 0) {
    const uint32_t x = static_cast<uint32_t>(rest), y = x / w.r.tiles;
    w.tile = x - y * w.r.tiles;
    w.h = y / w.r.groups;
    w.group = y - w.h * w.r.groups;
  } else {
    const uint64_t y = rest / w.r.tiles;
    w.tile = static_cast<uint32_t>(rest - y * w.r.tiles);
    w.h = static_cast<uint32_t>(y / w.r.groups);
    w.group = static_cast<uint32_t>(y - static_cast<uint64_t>(w.h) * w.r.groups);
  }
  return w;
}

// Row `row` of a group of rows: its query token and head; false behind the request's last.
template <int NT>
__device__ __forceinline__ bool row_at(const Kv4Params& p, const Request& r, uint32_t h, uint32_t group, int row,
                                       int64_t* tok, int64_t* head) {
  const int64_t x = static_cast<int64_t>(group) * (8 * NT) + row, i = x / p.G;
  *tok = r.q0 + i;
  *head = static_cast<int64_t>(h) * p.G + (x - i * p.G);
  return i < r.lq;
}

template <int D, int NT>
__global__ void __launch_bounds__(Kv4Shape<D, NT>::kThreads, 1) kv4_attention_kernel(const __grid_constant__ Kv4Params p) {
  using Sh = Kv4Shape<D, NT>;
  using Tile = Kv4Tile<D>;
  constexpr int NB = Tile::kBlocks, S = Sh::kStages, kThreads = Sh::kThreads;
  pdl_launch_dependents();
  extern __shared__ __align__(1024) uint8_t sm[];
  __shared__ uint64_t warp_sum[Sh::kWarps];
  __shared__ int abort_flag;
  uint64_t* pre = reinterpret_cast<uint64_t*>(sm + Sh::kOffPre);
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int g = lane >> 2, t = lane & 3;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Sh::kOffBar) + warp * S;
  int* bad_s = reinterpret_cast<int*>(sm + Sh::kOffBad) + warp * S;
  uint8_t* ring = sm + warp * Sh::kRing;
  if (lane == 0) {
    for (int i = 0; i < S; ++i) mbar_init(&bars[i], 1);
    fence_barrier_init();
  }
  if (threadIdx.x == 0) abort_flag = 0;

  // the work of the requests in front of each thread's
  {
    uint64_t mine = 0;
    bool bad = false;
    const int64_t b0 = static_cast<int64_t>(threadIdx.x) * p.per_thread;
    for (int64_t b = b0; b < b0 + p.per_thread && b < p.a.B; ++b) mine += count(p, request<NT>(p, b, &bad));
    if (bad && blockIdx.x == 0) atomicOr(p.a.err, kErrBadCache);
    uint64_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t x = __shfl_up_sync(kFull, sum, o);
      if (lane >= o) sum += x;
    }
    if (lane == 31) warp_sum[warp] = sum;
    __syncthreads();
    uint64_t front = 0;
    for (int w = 0; w < warp; ++w) front += warp_sum[w];
    pre[threadIdx.x] = front + sum - mine;
    if (threadIdx.x == kThreads - 1) pre[kThreads] = front + sum;
    __syncthreads();
  }
  const uint64_t all = pre[kThreads];
  const uint64_t block0 = all * blockIdx.x / gridDim.x, block1 = all * (blockIdx.x + 1) / gridDim.x;
  const uint64_t per = (block1 - block0 + Sh::kWarps - 1) / Sh::kWarps;
  const uint64_t from = block0 + warp * per < block1 ? block0 + warp * per : block1;
  const int n = static_cast<int>((from + per < block1 ? from + per : block1) - from);

  // loads: lane l finds the source of every 32nd tile and starts its copy
  const uint8_t* src = nullptr;
  auto fill = [&](int i) {
    if (i >= n) return;
    if ((i & 31) == 0) {
      src = nullptr;
      if (i + lane < n) {
        const Place w = place<D, NT>(p, pre, from + i + lane);
        const uint32_t tpp = static_cast<uint32_t>(p.a.page / 32), page_at = w.tile / tpp;
        const int64_t page = w.r.len > 0 ? p.a.block_table[w.b * p.a.width + page_at] : -1;
        if (page >= 0 && page < p.a.pages)
          src = p.a.cache + page * p.a.page_stride + (static_cast<int64_t>(w.h) * tpp + (w.tile - page_at * tpp)) * Tile::kBytes;
        else if (w.r.len > 0)
          atomicOr(p.a.err, kErrBadCache);
      }
    }
    if (lane == (i & 31)) {
      const int st = i % S;
      bad_s[st] = src == nullptr;
      if (src != nullptr) {
        mbar_arrive_expect_tx(&bars[st], Tile::kBytes);
        bulk_load(ring + st * Tile::kBytes, src, Tile::kBytes, &bars[st]);
      } else {
        mbar_arrive(&bars[st]);
      }
    }
  };
  for (int i = 0; i < S; ++i) fill(i);

  Place w = {};
  uint32_t qa[NB][2][2 * NT];  // queries as A operands: block, product, (row g, row g + 8) x (nibbles 0 / 2, 1 / 3)
  float qsum[NT][NB];          // -8 2^-133 sum of a block's queries
  float f[NT];                 // scores in units of log2
  int lim[NT], lim0 = 0;       // keys that a lane's row sees; the first row
  float ref[NT], l[NT];
  float o[NT][NB][2][4], bias[NT][4];
  uint32_t one[NB];            // -8 2^-133 in the rows of a block
#pragma unroll
  for (int b = 0; b < NB; ++b) one[b] = g % NB == b ? 0x80088008u : 0u;

  auto begin = [&]() {  // a new group of rows: w
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      int64_t tok, head;
      const bool on = row_at<NT>(p, w.r, w.h, w.group, g + 8 * x, &tok, &head);
      const uint16_t* row = p.a.q + tok * p.a.st[0] + head * p.a.st[1] + 8 * t;
      uint4 v[NB];
      float top = 0.0f;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        v[b] = on ? *reinterpret_cast<const uint4*>(row + 32 * b) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t u[4] = {v[b].x, v[b].y, v[b].z, v[b].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(fabsf(bf16_lo(u[e])), fabsf(bf16_hi(u[e]))));
      }
      top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
      top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
      // 2^e at most the row's largest: times 2^(100 - e) (a row below 2^-27 keeps smaller values)
      const int e = max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -27);
      const float up = __uint_as_float(static_cast<uint32_t>(100 - e + 127) << 23);
      f[x] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(min(33 + e, 127) + 127) << 23);
      const int64_t seen = static_cast<int64_t>(w.r.len) - w.r.lq + (tok - w.r.q0) + 1;
      lim[x] = on ? static_cast<int>(seen < 0 ? 0 : seen) : w.r.len;
      if (x == 0) lim0 = __shfl_sync(kFull, lim[0], 0);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint32_t u[4] = {v[b].x, v[b].y, v[b].z, v[b].w};
        float c[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          c[2 * i] = bf16_lo(u[i]) * up;
          c[2 * i + 1] = bf16_hi(u[i]) * up;
        }
        float sum = ((c[0] + c[1]) + (c[2] + c[3])) + ((c[4] + c[5]) + (c[6] + c[7]));
        sum += __shfl_xor_sync(kFull, sum, 1);
        sum += __shfl_xor_sync(kFull, sum, 2);
        qsum[x][b] = sum * -1.1754943508222875e-38f * 0.0625f;  // -8 2^-133 = -2^-126 2^-4
        // nibbles 1, 3 (and 5, 7) of a word are taken four bits higher, times 16
        qa[b][0][x] = pack_bf16(c[0], c[4]);
        qa[b][0][NT + x] = pack_bf16(c[1] * 0.0625f, c[5] * 0.0625f);
        qa[b][1][x] = pack_bf16(c[2], c[6]);
        qa[b][1][NT + x] = pack_bf16(c[3] * 0.0625f, c[7] * 0.0625f);
      }
      ref[x] = kNone;
      l[x] = 0.0f;
#pragma unroll
      for (int e2 = 0; e2 < 4; ++e2) {
        bias[x][e2] = 0.0f;
#pragma unroll
        for (int b = 0; b < NB; ++b) o[x][b][0][e2] = o[x][b][1][e2] = 0.0f;
      }
    }
  };

  auto work = [&](const uint8_t* tile, int key0, bool bad) {  // 32 keys from key0 on
    float2 s[NT][4];  // scores of row g (+ 8 x) with keys 8 t + 2 j, + 1
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[x][j] = make_float2(0.0f, 0.0f);
    const uint8_t* keys = tile + lane * Tile::kWords * 4;
#pragma unroll
    for (int bq = 0; bq < Tile::kQuads; ++bq) {
      uint32_t sc[Tile::kWords][4];
#pragma unroll
      for (int bw = 0; bw < Tile::kWords; ++bw) {
        const uint4 v = *reinterpret_cast<const uint4*>(tile + Tile::kKeyScales + (4 * bq + bw) * 64 + 16 * t);
        sc[bw][0] = v.x; sc[bw][1] = v.y; sc[bw][2] = v.z; sc[bw][3] = v.w;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t kw[Tile::kWords];
        const uint8_t* at = keys + (j * Tile::kQuads + bq) * 128 * Tile::kWords;
        if constexpr (Tile::kWords == 4) {
          const uint4 v = *reinterpret_cast<const uint4*>(at);
          kw[0] = v.x; kw[1] = v.y; kw[2] = v.z; kw[3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(at);
          kw[0] = v.x; kw[1] = v.y;
        }
#pragma unroll
        for (int bw = 0; bw < Tile::kWords; ++bw) {
          const int b = 4 * bq + bw;
          const uint32_t lo = kw[bw], hi = kw[bw] >> 8;
          float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          mma_bf16(c, qa[b][0][0], NT == 2 ? qa[b][0][NT - 1] : 0u, qa[b][0][NT], NT == 2 ? qa[b][0][2 * NT - 1] : 0u,
                   lo & 0x000F000Fu, lo & 0x00F000F0u);
          mma_bf16(c, qa[b][1][0], NT == 2 ? qa[b][1][NT - 1] : 0u, qa[b][1][NT], NT == 2 ? qa[b][1][2 * NT - 1] : 0u,
                   hi & 0x000F000Fu, hi & 0x00F000F0u);
          const float2 sf = make_float2(bf16_lo(sc[bw][j]), bf16_hi(sc[bw][j]));
#pragma unroll
          for (int x = 0; x < NT; ++x) {
            const float2 d = __fadd2_rn(make_float2(c[2 * x], c[2 * x + 1]), make_float2(qsum[x][b], qsum[x][b]));
            s[x][j] = __ffma2_rn(d, sf, s[x][j]);
          }
        }
      }
    }
    // keys that a row does not see; values behind the last key may hold anything
    uint32_t keep[4] = {kFull, kFull, kFull, kFull};
    const bool edge = bad || key0 + 32 > lim0;
    if (edge) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = key0 + 8 * t + 2 * j;
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          if (bad || key >= lim[x]) s[x][j].x = -INFINITY;
          if (bad || key + 1 >= lim[x]) s[x][j].y = -INFINITY;
        }
        if (bad || key >= w.r.len) keep[j] &= 0xFFFF0000u;
        if (bad || key + 1 >= w.r.len) keep[j] &= 0x0000FFFFu;
      }
    }
    // the reference follows the largest score only when that has run ahead
    float top[NT];
    bool grow = false;
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      top[x] = fmaxf(fmaxf(fmaxf(s[x][0].x, s[x][0].y), fmaxf(s[x][1].x, s[x][1].y)),
                     fmaxf(fmaxf(s[x][2].x, s[x][2].y), fmaxf(s[x][3].x, s[x][3].y)));
      grow = grow || fmaf(top[x], f[x], -ref[x]) > kLift + kSlack;
    }
    if (__any_sync(kFull, grow)) {
#pragma unroll
      for (int x = 0; x < NT; ++x) {
        float m = fmaxf(top[x], __shfl_xor_sync(kFull, top[x], 1));
        m = fmaxf(m, __shfl_xor_sync(kFull, m, 2));
        m = fmaxf(ref[x], fmaf(m, f[x], -kLift));
        const float by = ex2(ref[x] - m);
        ref[x] = m;
        l[x] *= by;
        const float by0 = __shfl_sync(kFull, by, 8 * t), by1 = __shfl_sync(kFull, by, 8 * t + 4);  // rows 2 t, 2 t + 1
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float y = (e & 1) != 0 ? by1 : by0;
          bias[x][e] *= y;
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            o[x][b][0][e] *= y;
            o[x][b][1][e] *= y;
          }
        }
      }
    }
    uint32_t pw[NT][4];
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = ex2(fmaf(s[x][j].x, f[x], -ref[x])), b = ex2(fmaf(s[x][j].y, f[x], -ref[x]));
        sum += a + b;
        pw[x][j] = pack_bf16(a, b);
      }
      l[x] += sum;
    }
    const uint8_t* values = tile + Tile::kValues + lane * Tile::kHalves * 4;
#pragma unroll
    for (int k = 0; k < 2; ++k) {  // 16 keys: the lane's pairs j = 2 k and 2 k + 1
      uint32_t v[4][Tile::kHalves];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t* at = values + (4 * k + i) * 128 * Tile::kHalves;
        if constexpr (Tile::kHalves == 4) {
          const uint4 x = *reinterpret_cast<const uint4*>(at);
          v[i][0] = x.x; v[i][1] = x.y; v[i][2] = x.z; v[i][3] = x.w;
        } else if constexpr (Tile::kHalves == 2) {
          const uint2 x = *reinterpret_cast<const uint2*>(at);
          v[i][0] = x.x; v[i][1] = x.y;
        } else {
          v[i][0] = *reinterpret_cast<const uint32_t*>(at);
        }
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint2 sc = *reinterpret_cast<const uint2*>(tile + Tile::kValueScales + b * 64 + 16 * t + 8 * k);
        const int h = b >> 1;
        const unsigned pick = (b & 1) == 0 ? 0x5410u : 0x7632u;
        const uint32_t u0 = __byte_perm(v[0][h], v[1][h], pick), u1 = __byte_perm(v[2][h], v[3][h], pick);
        const uint32_t s0 = sc.x & keep[2 * k], s1 = sc.y & keep[2 * k + 1];
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          const uint32_t b0 = mul_bf16(pw[x][2 * k], s0), b1 = mul_bf16(pw[x][2 * k + 1], s1);
          mma_bf16(o[x][b][0], u0 & 0x000F000Fu, u0 & 0x00F000F0u, u1 & 0x000F000Fu, u1 & 0x00F000F0u, b0, b1);
          mma_bf16(o[x][b][1], (u0 >> 8) & 0x000F000Fu, (u0 >> 8) & 0x00F000F0u, (u1 >> 8) & 0x000F000Fu,
                   (u1 >> 8) & 0x00F000F0u, b0, b1);
          mma_bf16(bias[x], one[b], one[b], one[b], one[b], b0, b1);
        }
      }
    }
  };

  constexpr float k2p69 = 5.902958103587057e20f, k2m64 = 5.421010862427522e-20f;
  // The lane's share of a finished run: columns 2 t and 2 t + 1 of the rows, channels 32 b + 4 g .. + 3
  auto total = [&](int x, int b, int e, float (&v)[4]) {  // column 2 t + e; times 2^133
    const float c = __shfl_sync(kFull, bias[x][e], 4 * b + t);
    v[0] = o[x][b][0][e] + c;
    v[1] = fmaf(o[x][b][0][2 + e], 0.0625f, c);
    v[2] = o[x][b][1][e] + c;
    v[3] = fmaf(o[x][b][1][2 + e], 0.0625f, c);
  };
  int4* meta_s = reinterpret_cast<int4*>(sm + Sh::kOffMeta);  // [warp][2]: put aside, at the end
  // A run that is not a whole group of rows: to `part`, row by row o, reference and sum.
  auto put_part = [&](float* part) {
#pragma unroll
    for (int x = 0; x < NT; ++x) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v[4];
          total(x, b, e, v);
          *reinterpret_cast<float4*>(part + (8 * x + 2 * t + e) * Sh::kPad + 32 * b + 4 * g) =
              make_float4(v[0] * k2p69, v[1] * k2p69, v[2] * k2p69, v[3] * k2p69);
        }
      float sum = l[x] + __shfl_xor_sync(kFull, l[x], 1);
      sum += __shfl_xor_sync(kFull, sum, 2);
      if (t == 0)
        *reinterpret_cast<float2*>(part + (8 * x + g) * Sh::kPad + D) = make_float2(ref[x] + kLift, sum * k2m64);
    }
  };
  auto put_rows = [&]() {  // a whole group of rows: to o
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      float sum = l[x] + __shfl_xor_sync(kFull, l[x], 1);
      sum = (sum + __shfl_xor_sync(kFull, sum, 2)) * k2m64;
      const float inv = sum != 0.0f ? k2p69 / sum : 0.0f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float by = __shfl_sync(kFull, inv, 4 * (2 * t + e));
        int64_t tok, head;
        const bool on = row_at<NT>(p, w.r, w.h, w.group, 8 * x + 2 * t + e, &tok, &head);
        uint16_t* row = p.a.o + tok * p.a.st[2] + head * p.a.st[3] + 4 * g;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          float v[4];
          total(x, b, e, v);
          if (on) *reinterpret_cast<uint2*>(row + 32 * b) = make_uint2(pack_bf16(v[0] * by, v[1] * by), pack_bf16(v[2] * by, v[3] * by));
        }
      }
    }
  };
  // a run that ends inside the warp's: it waits in global memory, as the ring is still in use
  float* aside = p.part + (static_cast<int64_t>(gridDim.x) * 2 + static_cast<int64_t>(blockIdx.x) * Sh::kWarps) * Sh::kPart;

  if (lane < 2) meta_s[2 * warp + lane] = make_int4(0, 0, 0, 0);
  __syncwarp();
  bool ok = true, front = false;
  for (int i = 0; i < n; ++i) {
    if (i == 0 || w.tile == w.r.tiles) {
      w = place<D, NT>(p, pre, from + i);
      front = w.tile != 0;
      begin();
    }
    const int st = i % S;
    ok = warp_wait(&bars[st], static_cast<uint32_t>(i / S) & 1u, &abort_flag);
    if (!ok) {
      report_error(p.a.err, kErrWaitTimeout, &abort_flag);
      for (int k = i; k < n && k < i + S; ++k) mbar_wait(&bars[k % S], static_cast<uint32_t>(k / S) & 1u, nullptr);
      break;
    }
    work(ring + st * Tile::kBytes, static_cast<int>(w.tile) * 32, bad_s[st] != 0);
    __syncwarp();  // every lane has read the stage
    fill(i + S);
    ++w.tile;
    const bool whole = w.tile == w.r.tiles, last = i == n - 1;
    if (whole && !front) {
      put_rows();
    } else if (whole || last) {
      put_part(last ? reinterpret_cast<float*>(ring) : aside + static_cast<int64_t>(warp) * Sh::kPart);
      if (lane == 0)
        meta_s[2 * warp + (last ? 1 : 0)] =
            make_int4(static_cast<int>(w.b), static_cast<int>(w.h), static_cast<int>(w.group),
                      kPartHeld | (front ? kPartFromFront : 0) | (whole ? 0 : kPartGoesOn));
    }
  }
  __syncthreads();
  if (abort_flag != 0) return;

  // The block's chains: a run at a warp's end, those of the warps behind it while it goes on.
  int4 out0 = make_int4(0, 0, 0, 0), out1 = out0;
  auto join = [&](int w0, int n_end, bool tail) {  // the runs at the end of warps w0 .. w0 + n_end - 1, then one put aside
    const int4 head = n_end > 0 ? meta_s[2 * w0 + 1] : meta_s[2 * w0];
    const int v = w0 + n_end;
    const int4 end = tail ? meta_s[2 * v] : meta_s[2 * (v - 1) + 1];
    const bool from_front = (head.w & kPartFromFront) != 0, goes_on = (end.w & kPartGoesOn) != 0;
    const int4 who = make_int4(head.x, head.y, head.z, kPartHeld | (from_front ? kPartFromFront : 0) | (goes_on ? kPartGoesOn : 0));
    if (from_front) out0 = who;
    else if (goes_on) out1 = who;
    bool bad = false;
    Request r = {};
    if (!from_front && !goes_on) r = request<NT>(p, head.x, &bad);
    const int members = n_end + (tail ? 1 : 0);
    auto member = [&](int m) -> const float* {
      return m < n_end ? reinterpret_cast<const float*>(sm + (w0 + m) * Sh::kRing) : aside + static_cast<int64_t>(v) * Sh::kPart;
    };
    for (int at = static_cast<int>(threadIdx.x); at < Sh::kRows * (D / 2); at += kThreads) {
      const int row = at / (D / 2), c = 2 * (at - row * (D / 2));
      float top = kNone;
      for (int m = 0; m < members; ++m) top = fmaxf(top, member(m)[row * Sh::kPad + D]);
      float sum = 0.0f;
      float2 acc = make_float2(0.0f, 0.0f);
      for (int m = 0; m < members; ++m) {
        const float* src2 = member(m) + row * Sh::kPad;
        const float2 ml = *reinterpret_cast<const float2*>(src2 + D), v2 = *reinterpret_cast<const float2*>(src2 + c);
        const float by = ex2(ml.x - top);
        sum = fmaf(ml.y, by, sum);
        acc.x = fmaf(v2.x, by, acc.x);
        acc.y = fmaf(v2.y, by, acc.y);
      }
      if (from_front || goes_on) {
        float* dst = p.part + (static_cast<int64_t>(blockIdx.x) * 2 + (from_front ? 0 : 1)) * Sh::kPart + row * Sh::kPad;
        *reinterpret_cast<float2*>(dst + c) = acc;
        if (c == 0) *reinterpret_cast<float2*>(dst + D) = make_float2(top, sum);
      } else {
        int64_t tok, hd;
        if (row_at<NT>(p, r, static_cast<uint32_t>(head.y), static_cast<uint32_t>(head.z), row, &tok, &hd)) {
          const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
          *reinterpret_cast<uint32_t*>(p.a.o + tok * p.a.st[2] + hd * p.a.st[3] + c) = pack_bf16(acc.x * inv, acc.y * inv);
        }
      }
    }
  };
  if (meta_s[0].w != 0) join(0, 0, true);
  for (int w0 = 0; w0 < Sh::kWarps; ++w0) {
    const int fl = meta_s[2 * w0 + 1].w;
    if (fl == 0 || (w0 > 0 && (fl & kPartFromFront) != 0)) continue;
    int n_end = 1;
    bool tail = false, on = (fl & kPartGoesOn) != 0;
    while (on && w0 + n_end < Sh::kWarps) {
      if (meta_s[2 * (w0 + n_end)].w != 0) {
        tail = true;
        break;
      }
      const int nx = meta_s[2 * (w0 + n_end) + 1].w;
      if (nx == 0) break;  // the block's last warps have no work: the run goes on in the next block
      ++n_end;
      on = (nx & kPartGoesOn) != 0;
    }
    join(w0, n_end, tail);
  }
  if (threadIdx.x == 0) {
    p.meta[2 * blockIdx.x] = out0;
    p.meta[2 * blockIdx.x + 1] = out1;
  }
}

// Runs that cross blocks: block x joins the one that begins in block x of the attention kernel, row y.
template <int D, int NT>
__global__ void __launch_bounds__(D / 2) kv4_join_kernel(const __grid_constant__ Kv4Params p) {
  using Sh = Kv4Shape<D, NT>;
  pdl_wait();
  const int4 who = p.meta[2 * blockIdx.x + 1];
  if ((who.w & kPartHeld) == 0) return;
  bool bad;
  const Request r = request<NT>(p, who.x, &bad);
  const int row = static_cast<int>(blockIdx.y), c = 2 * static_cast<int>(threadIdx.x);
  int64_t tok, head;
  if (!row_at<NT>(p, r, static_cast<uint32_t>(who.y), static_cast<uint32_t>(who.z), row, &tok, &head)) return;
  const int nb = static_cast<int>(gridDim.x);
  float top = kNone, sum = 0.0f;
  float2 acc = make_float2(0.0f, 0.0f);
  auto add = [&](int slot) {
    const float* src = p.part + static_cast<int64_t>(slot) * Sh::kPart + row * Sh::kPad;
    const float2 ml = *reinterpret_cast<const float2*>(src + D), v = *reinterpret_cast<const float2*>(src + c);
    const float m = fmaxf(top, ml.x), old = ex2(top - m), by = ex2(ml.x - m);
    top = m;
    sum = fmaf(sum, old, ml.y * by);
    acc.x = fmaf(acc.x, old, v.x * by);
    acc.y = fmaf(acc.y, old, v.y * by);
  };
  add(2 * static_cast<int>(blockIdx.x) + 1);
  for (int x = static_cast<int>(blockIdx.x) + 1; x < nb; ++x) {
    const int flags = p.meta[2 * x].w;
    if (flags == 0) continue;  // a block without work
    add(2 * x);
    if ((flags & kPartGoesOn) == 0) break;
  }
  const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
  *reinterpret_cast<uint32_t*>(p.a.o + tok * p.a.st[2] + head * p.a.st[3] + c) = pack_bf16(acc.x * inv, acc.y * inv);
}

// ---- host ------------------------------------------------------------------------------------
// Rows of a group: 8, or 16 where a request's rows may be more (256 channels: 8, sixteen would
// not fit the registers).
int row_tiles(int64_t G, bool one_query, int64_t d) { return d == 256 || (one_query && G <= 8) ? 1 : 2; }

template <int D, int NT>
size_t ws_bytes(const DeviceInfo& dev) {
  using Sh = Kv4Shape<D, NT>;
  const size_t blocks = static_cast<size_t>(dev.sm_count);
  return blocks * (2 + Sh::kWarps) * Sh::kPart * 4 + blocks * 2 * sizeof(int4);
}

template <int D, int NT>
cudaError_t attention(const Kv4AttentionArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  using Sh = Kv4Shape<D, NT>;
  Kv4Params p = {};
  p.a = a;
  p.G = static_cast<int>(a.H / a.Hkv);
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.per_thread = static_cast<int>((a.B + Sh::kThreads - 1) / Sh::kThreads);
  const unsigned blocks = static_cast<unsigned>(dev.sm_count);
  p.part = static_cast<float*>(a.part);
  p.meta = reinterpret_cast<int4*>(p.part + static_cast<size_t>(blocks) * (2 + Sh::kWarps) * Sh::kPart);
  const auto kernel = kv4_attention_kernel<D, NT>;
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kernel), Sh::kSmem, dev.device);
  if (e != cudaSuccess) return e;
  kernel<<<blocks, Sh::kThreads, Sh::kSmem, stream>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, Sh::kRows);
  cfg.blockDim = dim3(D / 2);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_join_kernel<D, NT>, p);
}

}  // namespace

size_t kv4_attention_ws_bytes(int64_t H, int64_t Hkv, int64_t d, bool one_query, const DeviceInfo& dev) {
  const int nt = row_tiles(H / Hkv, one_query, d);
  if (d == 256) return ws_bytes<256, 1>(dev);
  if (d == 128) return nt == 1 ? ws_bytes<128, 1>(dev) : ws_bytes<128, 2>(dev);
  return nt == 1 ? ws_bytes<64, 1>(dev) : ws_bytes<64, 2>(dev);
}

cudaError_t launch_kv4_attention(Kv4AttentionArgs a, const DeviceInfo& dev, cudaStream_t stream) {
  if (a.B == 0 || a.Tq == 0 || a.H == 0) return cudaSuccess;
  a.err = dev.err_word;
  const int nt = row_tiles(a.H / a.Hkv, a.cu_q == nullptr, a.d);
  if (a.d == 256) return attention<256, 1>(a, dev, stream);
  if (a.d == 128) return nt == 1 ? attention<128, 1>(a, dev, stream) : attention<128, 2>(a, dev, stream);
  return nt == 1 ? attention<64, 1>(a, dev, stream) : attention<64, 2>(a, dev, stream);
}

}  // namespace q8
