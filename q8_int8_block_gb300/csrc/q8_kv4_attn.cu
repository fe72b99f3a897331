// q8_kv4_attn.cu -- attention of the newest tokens of each request over its paged 4-bit cache.
//
// o = sum_j p_j v_j / sum_j p_j, p_j = exp(scale q . k_j), keys and values in the tiles of
// q8_kv4.cuh: k = s_b (n - 8), a nibble n and a scale s_b for 32 channels of a token.
//
// Mathematics.  Codes are multiplied as they lie: a nibble in the low bits of a bfloat16 is the
// subnormal n 2^-133, one four bits higher is 16 n 2^-133 (the encoding is linear up to 255), and
// the tensor pipe takes subnormals exactly, so an AND makes two operands and nothing is converted.
// The other factor carries 2^100 (queries, scaled by a power of two for each row) or 2^64
// (weights), which keeps every sum far inside binary32.  What is left is linear and comes last:
//   scores   s_b (sum q n - 8 sum q): the second sum belongs to the query, the block's scale is
//            applied to the binary32 sum of the block;
//   output   the value's scale multiplies the weight, w = bf16(p s_b), and
//            sum w (n - 8) = sum w n - 8 sum w: the second sum is one more product, whose
//            constant operand has a row for each block of 32 channels.
// Weights change lanes between the two products as bfloat16: the leading 8 bits and the rest apart, so
// that w is rounded once, as in the other attention kernels (rounding p as well took 3 % off the
// time: 64 x 16384 tokens 190 us against 198).  All sums are binary32.  Over the measured cases the error
// against binary64 is 0.0017 to 0.0019 of the output's norm, of which the bfloat16 output's own
// rounding is 0.0016.
//
// Bound: the cache's bytes, 9/8 d for a key and head.  At the copy rate (6694.8 GB/s over 152 SMs at 2070 MHz)
// an SM gets 21.3 bytes, 38 elements, a clock, a tile of 32 keys of 128 channels in 217: 866 issue slots,
// for 535 warp instructions with everything around the loop (16 x 16384 tokens; many of them on the
// integer pipe, whose rate is half: 51 % busy).
//
// Split.  The work is the list of (request, head, rows, tile of 32 keys), and every warp takes an
// equal run of it, wherever that begins and ends: lengths do not matter.  A warp has a ring of
// tiles that one bulk copy each fills, so its loop has no barrier.  Where a run ends inside a
// request the partial results meet in the block's shared memory, and what crosses blocks goes to
// a second kernel.  Small calls are one launch of clusters instead (alone_blocks).
//
// Measured (device time, 32 / 8 heads of 128): 64 requests of 16384 tokens 198 us (6.1 TB/s, 0.91 of the
// measured copy rate), 256 of 2048 111 us (0.82), 2 of up to 131072 34.2 us (0.66: 4 us to the first
// tile, 6 from the last to the end of the second launch), one of 1000 6.2 us by a cluster, 3.4 more by the list.
#include <cuda_bf16.h>

#include <algorithm>

#include "q8_attn_ptx.cuh"
#include "q8_internal.h"
#include "q8_kv4.cuh"
#include "q8_kv4_ring.h"
#include "q8_launch_ptx.cuh"

namespace q8 {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t mul_bf16(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t fma_bf16(uint32_t a, uint32_t b, uint32_t c) {  // a b + c, rounded once
  const __nv_bfloat162 r = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b),
                                   *reinterpret_cast<const __nv_bfloat162*>(&c));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// bulk_load of what leaves the L2 first: a cache is read once a step, and what the kernels need again
// (their code among it) should not have to make room for it
__device__ __forceinline__ uint64_t read_once() {
  uint64_t policy;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  return policy;
}
__device__ __forceinline__ void bulk_load_once(void* smem_dst, const void* gmem_src, uint32_t bytes, uint64_t* bar,
                                               uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::
          "r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(gmem_src)), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}
// an 8 x 8 matrix of 16-bit elements, two of a row to a lane, transposed
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }

// What a group of rows costs a warp beside its tiles (queries, results), in tiles: the work list counts
// it in, so that short requests do not hold up the warp that gets many (64 requests of up to 8192 keys,
// with one, two, three, four, six: 32.0, 29.5, 28.8, 29.0, 30.6 us; 2 of up to 131072 37.9, 34.6, 34.7, 35.4,
// 35.7; 64 of 2048 36.9, 36.6, 36.3, 37.5, 37.6).
constexpr int kExtra = 3;
// Weights are 2^((s - ref) f) of the sums s before their factor f (in units of log2): s - ref is exact
// where it is small, however large the scores are (a reference in units of log2 is itself rounded, for
// scores of 2^31 by more than the weights' range).
constexpr float kNone = -3.402823466e38f;  // reference of a row that has seen no key: below every finite sum
constexpr float kLift = 64.0f;             // weights are carried as 2^64 p
constexpr float kSlack = 10.0f;            // a reference may lag behind the largest score by 2^10
constexpr float kNoPart = -1.0f;           // sum of a partial result that is none
constexpr float kMostFactor = 3.402823466e38f;

struct Kv4Params {
  Kv4AttentionArgs a;
  int G;
  float scale_log2;
  int per_lane;      // requests whose counts a lane sums up
  uint64_t by_G, by_tpp;  // 2^64 / n + 1 of the heads of a group and the tiles of a page: the high half
                          // of x times it is x / n (x n < 2^64; not used for n = 1)
  uint32_t by_grid;       // 2^32 / blocks
  int cluster;       // (alone) blocks of a cluster
  float* part;       // [blocks][2] partial results
  struct Record* meta;  // [blocks]: the run that begins in the block and goes on in others
};
constexpr int kMaxBlocks = 256;     // of the attention kernel
enum : int { kPartHeld = 1, kPartFromFront = 2, kPartGoesOn = 4 };  // flags of a partial result
struct __align__(16) Record {  // whose partial result it is
  int h, group, lq, flags;
  int64_t q0;
  int64_t end;       // where its item ends in the work list; in memory: the last block that has some of it
};

// A group of rows of a request: the unit whose keys are walked.
struct Item {
  int64_t b, q0;     // request, its first query
  int lq, len;       // its queries, keys
  int tiles;         // of keys (one at least: rows without a key are written too)
  int groups;        // of rows of a head
  int h, group;      // key/value head, group
  int start;         // its place in the work list, from the warp's first on
};

template <int D, int NT>
struct Kv4Shape {
  using Tile = Kv4Tile<D>;
  static constexpr int kRows = 8 * NT;
  // as many as the registers of a lane allow (128 channels: 12 warps of 168 registers; 16 of 128 spill)
  static constexpr int kWarps = D == 64 ? (NT == 1 ? 16 : 12) : D == 128 && NT == 1 ? 12 : 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kPad = D + 4;                         // floats of a row's partial result: o, reference, sum, f
  static constexpr int kPart = kRows * kPad;                 // floats of a partial result
  static constexpr int kStages = (225 * 1024 / kWarps - kPart * 4) / Tile::kBytes;
  static constexpr int kRing = kStages * Tile::kBytes;       // of a warp
  static constexpr int kOffAside = kWarps * kRing;           // a warp's partial result while the ring is in use
  static constexpr int kOffRec = kOffAside + kWarps * kPart * 4;
  static constexpr int kOffItem = kOffRec + kWarps * 2 * static_cast<int>(sizeof(Record));
  static constexpr int kOffBar = kOffItem + kWarps * static_cast<int>(sizeof(Item));
  static constexpr int kOffHeld = kOffBar + kWarps * kStages * 8;
  static constexpr int kSmem = kOffHeld + kWarps * kStages * 4;
  static_assert(kSmem <= 227 * 1024 - 64, "shared memory of a block");
  static_assert(kPart * 4 <= kRing, "a partial result in the ring's place");
  static_assert(kRing % 16 == 0, "alignment of bulk copies");
  static_assert(kStages < 32 && kWarps < 32, "a lane for each");
};

template <int NT>
__device__ __forceinline__ void request(const Kv4Params& p, Item& it, bool* bad) {  // what request it.b asks for
  const Kv4AttentionArgs& a = p.a;
  it.q0 = it.b;
  int64_t lq = 1;
  if (a.cu_q != nullptr) {
    it.q0 = a.cu_q[it.b];
    lq = a.cu_q[it.b + 1] - it.q0;
    if (it.q0 < 0 || lq < 0 || it.q0 + lq > a.Tq) {
      *bad = true;
      lq = 0;
    }
  }
  int64_t len = a.kv_len[it.b];
  const int64_t most = a.width * a.page;
  if (len < 0 || len > most) {
    *bad = true;
    len = len < 0 ? 0 : most;
  }
  it.lq = static_cast<int>(lq);
  it.len = static_cast<int>(len);
  it.tiles = len > 0 ? static_cast<int>((len + 31) >> 5) : 1;
  it.groups = static_cast<int>((static_cast<uint32_t>(it.lq) * static_cast<uint32_t>(p.G) + 8 * NT - 1) / (8 * NT));
}
__device__ __forceinline__ uint64_t count(const Kv4Params& p, const Item& it) {
  return static_cast<uint64_t>(it.tiles + kExtra) * static_cast<uint32_t>(it.groups) * static_cast<uint32_t>(p.a.Hkv);
}
// the group of rows behind it (there is one)
template <int NT>
__device__ __forceinline__ void next_item(const Kv4Params& p, Item& it) {
  it.start += it.tiles + kExtra;
  if (++it.group < it.groups) return;
  it.group = 0;
  if (++it.h < p.a.Hkv) return;
  it.h = 0;
  bool bad;
  do {
    ++it.b;
    request<NT>(p, it, &bad);
  } while (it.groups == 0 && it.b + 1 < p.a.B);
}

// x / y, quicker for x below 2^22 (the quotient in binary32 is then off by one at most)
__device__ __forceinline__ uint32_t divide(uint32_t x, uint32_t y) {
  if (x >> 22 != 0) return x / y;
  const uint32_t z = static_cast<uint32_t>(__fdividef(static_cast<float>(x), static_cast<float>(y)));
  const int rest = static_cast<int>(x - z * y);
  return rest < 0 ? z - 1 : rest >= static_cast<int>(y) ? z + 1 : z;
}

// Place `at` of the work list, `before` the work in front of each lane's requests; returns the first
// tile at or behind it.
template <int NT>
__device__ __forceinline__ int place(const Kv4Params& p, uint64_t before, uint64_t at, Item& it) {
  const int c = __popc(__ballot_sync(kFull, before <= at)) - 1;  // the last lane that begins at or in front of it
  uint64_t rest = at - __shfl_sync(kFull, before, c);
  bool bad;
  it.b = static_cast<int64_t>(c) * p.per_lane;
  request<NT>(p, it, &bad);
  for (uint64_t m = count(p, it); rest >= m; m = count(p, it)) {
    rest -= m;
    ++it.b;
    request<NT>(p, it, &bad);
  }
  const uint32_t size = static_cast<uint32_t>(it.tiles + kExtra);
  uint64_t y;
  if (rest >> 32 == 0) y = divide(static_cast<uint32_t>(rest), size);
  else y = rest / size;
  const uint32_t y32 = static_cast<uint32_t>(y);  // groups of a request: below 2^31
  it.h = it.groups == 1 ? static_cast<int>(y32) : static_cast<int>(divide(y32, static_cast<uint32_t>(it.groups)));
  it.group = static_cast<int>(y32 - static_cast<uint32_t>(it.h) * static_cast<uint32_t>(it.groups));
  it.start = -static_cast<int>(rest - y * size);
  return it.start < -kExtra ? -it.start - kExtra : 0;
}

// Row `row` of a group of rows: its query token (of the request) and head; false behind the last.
template <int NT>
__device__ __forceinline__ bool row_at(const Kv4Params& p, int lq, int h, int group, int row, int* query, int64_t* head) {
  const uint32_t x = static_cast<uint32_t>(group) * (8 * NT) + row;
  const uint32_t i = p.G == 1 ? x : static_cast<uint32_t>(__umul64hi(x, p.by_G));
  *query = static_cast<int>(i);
  *head = static_cast<int64_t>(h) * p.G + (x - i * static_cast<uint32_t>(p.G));
  return i < static_cast<uint32_t>(lq);
}

// Rows of a group that are a query's.
template <int NT>
__device__ __forceinline__ int rows_used(const Kv4Params& p, int lq, int group) {
  const int64_t left = static_cast<int64_t>(lq) * p.G - static_cast<int64_t>(group) * (8 * NT);
  return left < 8 * NT ? static_cast<int>(left) : 8 * NT;
}

// A row of `members` partial results, member(m) the m-th's: reference, sum, f (the same in all), the lane's
// channels.
template <int D, typename F>
__device__ __forceinline__ void add_up(int lane, int members, const F& member, float& top, float& sum, float& f,
                                       float (&acc)[D / 32]) {
  constexpr int E = D / 32;
  const float4 ml = lane < members ? *reinterpret_cast<const float4*>(member(lane) + D) : make_float4(kNone, 0.0f, 0.0f, 0.0f);
  top = ml.x;
  f = __shfl_sync(kFull, ml.z, 0);
#pragma unroll
  for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, i));
  const float by = ex2((ml.x - top) * f);
  sum = ml.y * by;
#pragma unroll
  for (int i = 16; i > 0; i >>= 1) sum += __shfl_xor_sync(kFull, sum, i);
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.0f;
#pragma unroll 4
  for (int m = 0; m < members; ++m) {
    const float* part = member(m) + E * lane;
    const float by_m = __shfl_sync(kFull, by, m);
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float2 x = *reinterpret_cast<const float2*>(part + e);
      acc[e] = fmaf(x.x, by_m, acc[e]);
      acc[e + 1] = fmaf(x.y, by_m, acc[e + 1]);
    }
  }
}

// kAlone: each group of rows is one cluster's, whose blocks share its keys and join through one
// another's shared memory: one launch and no workspace.
template <int D, int NT, bool kAlone>
__global__ void __launch_bounds__(Kv4Shape<D, NT>::kThreads, 1) kv4_attention_kernel(const __grid_constant__ Kv4Params p) {
  using Sh = Kv4Shape<D, NT>;
  using Tile = Kv4Tile<D>;
  constexpr int NB = Tile::kBlocks, S = Sh::kStages;
  extern __shared__ __align__(16) uint8_t sm[];
  __shared__ int abort_flag;
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int g = lane >> 2, t = lane & 3;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Sh::kOffBar) + warp * S;
  int* held_s = reinterpret_cast<int*>(sm + Sh::kOffHeld) + warp * S;
  uint8_t* ring = sm + warp * Sh::kRing;
  if (threadIdx.x == 0) abort_flag = 0;

  Item* item = reinterpret_cast<Item*>(sm + Sh::kOffItem) + warp;  // the current one
  int tile = 0, tiles = 0, len = 0;
  int n = 0;                            // places of the work list that are this warp's
  uint64_t from = 0, q = 0, run = 0;    // the first of them; a block's places, this block's
  uint32_t r = 0;
  const uint32_t nb = gridDim.x;
  auto share = [&](uint32_t block) { return __umulhi(r * block, p.by_grid + 1); };  // r block / blocks: 2^16 at most
  int users = 0;                        // (alone) warps of this block that have keys
  if (lane == 0) {
    for (int i = 0; i < S; ++i) mbar_init(&bars[i], 1);
    fence_barrier_init();
  }
  // what the kernels in front have written is there for the whole grid once one warp has waited (waited
  // for by every thread the work list's loop is compiled 1 % slower: 64 x 16384 tokens 201 us against 198)
  if (kAlone || warp == 0) pdl_wait();
  __syncthreads();  // nor does a wait look at the flag before it is cleared
  if constexpr (!kAlone) pdl_launch_dependents();
  if constexpr (kAlone) {
    // equal runs of the group's tiles: a block's, and of that a warp's
    const uint32_t c = static_cast<uint32_t>(p.cluster), x = blockIdx.x / c, rank = blockIdx.x - x * c;
    Item it;
    bool bad = false;
    it.b = x / static_cast<uint32_t>(p.a.Hkv);
    it.h = static_cast<int>(x - static_cast<uint32_t>(it.b) * static_cast<uint32_t>(p.a.Hkv));
    it.group = 0;
    request<NT>(p, it, &bad);
    if (bad && threadIdx.x == 0) atomicOr(p.a.err, kErrBadCache);
    const int per_block = (it.tiles + static_cast<int>(c) - 1) / static_cast<int>(c), block0 = static_cast<int>(rank) * per_block;
    const int mine = it.tiles - block0 < per_block ? it.tiles - block0 : per_block;
    const int per = mine > 0 ? (mine + Sh::kWarps - 1) / Sh::kWarps : 1;
    users = mine > 0 ? (mine + per - 1) / per : 0;
    if (warp < users) {
      tile = block0 + warp * per;
      n = mine - warp * per < per ? mine - warp * per : per;
    }
    it.start = -tile - kExtra;
    if (lane == 0) *item = it;
    __syncwarp();
  } else {
    // the work in front of each lane's requests: every warp for itself
    uint64_t before = 0, all;
    {
      uint64_t mine = 0;
      bool bad = false;
      Item it;
      it.b = static_cast<int64_t>(lane) * p.per_lane;
      const int64_t b1 = it.b + p.per_lane < p.a.B ? it.b + p.per_lane : p.a.B;
      for (; it.b < b1; ++it.b) {
        request<NT>(p, it, &bad);
        mine += count(p, it);
      }
      if (bad && blockIdx.x == 0 && warp == 0) atomicOr(p.a.err, kErrBadCache);
      before = mine;
      if (!__any_sync(kFull, mine >> 26 != 0)) {
        uint32_t sum = static_cast<uint32_t>(mine);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t x = __shfl_up_sync(kFull, sum, o);
          if (lane >= o) sum += x;
        }
        before = sum;
      } else {
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
          const uint64_t x = __shfl_up_sync(kFull, before, o);
          if (lane >= o) before += x;
        }
      }
      all = __shfl_sync(kFull, before, 31);
      before -= mine;
    }
    // equal runs: a block's, and of that a warp's; the longer ones are spread over the blocks
    if (all >> 32 == 0) {
      const uint32_t x = static_cast<uint32_t>(all), y = __umulhi(x, p.by_grid);  // one too few at most
      r = x - y * nb;
      q = r >= nb ? y + 1 : y;
      r = r >= nb ? r - nb : r;
    } else {
      q = all / nb;
      r = static_cast<uint32_t>(all - q * nb);
    }
    const uint32_t r0 = share(blockIdx.x), r1 = share(blockIdx.x + 1);
    const uint64_t block0 = q * blockIdx.x + r0;
    run = q + r1 - r0;
    const uint64_t per = (run + Sh::kWarps - 1) / Sh::kWarps, skip = static_cast<uint64_t>(warp) * per;
    from = block0 + skip;
    n = skip >= run ? 0 : static_cast<int>(run - skip < per ? run - skip : per);
    if (n > 0) {
      Item it;
      tile = place<NT>(p, before, from, it);
      if (lane == 0) *item = it;
      __syncwarp();
    }
  }
  // queries as they are loaded: row g (+ 8 x), channels 32 b + 8 t ..
  auto load_queries = [&](const Item& it, uint4 (&qv)[NT][NB]) {
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      int query;
      int64_t head;
      const bool on = row_at<NT>(p, it.lq, it.h, it.group, g + 8 * x, &query, &head);
      const uint16_t* row = p.a.q + (it.q0 + query) * p.a.st[0] + head * p.a.st[1] + 8 * t;
#pragma unroll
      for (int b = 0; b < NB; ++b)
        qv[x][b] = on ? *reinterpret_cast<const uint4*>(row + 32 * b) : make_uint4(0u, 0u, 0u, 0u);
    }
  };

  // loads: lane l finds the source of every 32nd tile, from the current item on, and starts its copy
  const uint64_t once = read_once();
  const uint8_t* src = nullptr;
  int held = kStageNone;  // what its stage will hold
  auto fill = [&](int i, int ahead) {  // ahead: tiles between the current one and the i-th
    if ((i & 31) == 0) {
      Item it = *item;
      int x = tile + ahead + lane;
      while (x >= it.tiles && it.start + it.tiles + 2 * kExtra < n) {
        x -= it.tiles;
        next_item<NT>(p, it);
      }
      src = nullptr;
      const bool in_run = x < it.tiles && it.start + kExtra + x < n;
      if (in_run && it.len > 0) {
        const uint32_t tpp = static_cast<uint32_t>(p.a.page) / 32;
        const uint32_t page_at = tpp == 1 ? static_cast<uint32_t>(x) : static_cast<uint32_t>(__umul64hi(static_cast<uint32_t>(x), p.by_tpp));
        const int64_t page = p.a.block_table[it.b * p.a.width + page_at];
        if (page >= 0 && page < p.a.pages)
          src = p.a.cache + page * p.a.page_stride +
                (static_cast<int64_t>(it.h) * tpp + (static_cast<uint32_t>(x) - page_at * tpp)) * Tile::kBytes;
        else
          atomicOr(p.a.err, kErrBadCache);
      }
      held = stage_state(in_run, src != nullptr);
      __syncwarp();
    }
    if (lane == (i & 31)) {
      const int st = i % S;
      held_s[st] = held;
      if (held == kStageTile) {
        mbar_arrive_expect_tx(&bars[st], Tile::kBytes);
        bulk_load_once(ring + st * Tile::kBytes, src, Tile::kBytes, &bars[st], once);
      } else if (held == kStageNoPage) {
        mbar_arrive(&bars[st]);
      }
    }
  };

  uint32_t qb[NT][NB][2][2];   // queries as B operands: block, product, (nibbles 0 / 2, 1 / 3) with (4 / 6, 5 / 7)
  float2 qsum[NT][NB];         // -8 2^-133 sum of a block's queries, rows 2 t and 2 t + 1
  float f[NT][2];              // what makes these rows' sums scores in units of log2
  int lim[NT][2], lim0 = 0;    // keys that they see; that the first row sees
  float ref[NT][2], l[NT][2];
  float o[NT][NB][2][4], bias[NT][4];
  uint32_t one[NB];            // -8 2^-133 in the rows of a block
#pragma unroll
  for (int b = 0; b < NB; ++b) one[b] = g % NB == b ? 0x80088008u : 0u;

  auto begin = [&](const Item& it, const uint4 (&qv)[NT][NB]) {  // a new group of rows
    tiles = it.tiles;
    len = it.len;
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      float top = 0.0f;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint32_t u[4] = {qv[x][b].x, qv[x][b].y, qv[x][b].z, qv[x][b].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(fabsf(bf16_lo(u[e])), fabsf(bf16_hi(u[e]))));
      }
      top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
      top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
      // 2^e at most the row's largest: times 2^(100 - e) (a row below 2^-27 keeps smaller values)
      const int e = max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -27);
      const float up = __uint_as_float(static_cast<uint32_t>(100 - e + 127) << 23);
      const float fg = fminf(p.scale_log2 * __uint_as_float(static_cast<uint32_t>(min(33 + e, 127) + 127) << 23), kMostFactor);
      int query;
      int64_t head;
      const bool on = row_at<NT>(p, it.lq, it.h, it.group, g + 8 * x, &query, &head);
      const int64_t seen = static_cast<int64_t>(it.len) - it.lq + query + 1;
      const int lg = on ? static_cast<int>(seen < 0 ? 0 : seen) : it.len;
      if (x == 0) lim0 = __shfl_sync(kFull, lg, 0);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        f[x][r] = __shfl_sync(kFull, fg, 8 * t + 4 * r);
        lim[x][r] = __shfl_sync(kFull, lg, 8 * t + 4 * r);
        ref[x][r] = kNone;
        l[x][r] = 0.0f;
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint32_t u[4] = {qv[x][b].x, qv[x][b].y, qv[x][b].z, qv[x][b].w};
        float c[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          c[2 * i] = bf16_lo(u[i]) * up;
          c[2 * i + 1] = bf16_hi(u[i]) * up;
        }
        float sum = ((c[0] + c[1]) + (c[2] + c[3])) + ((c[4] + c[5]) + (c[6] + c[7]));
        sum += __shfl_xor_sync(kFull, sum, 1);
        sum += __shfl_xor_sync(kFull, sum, 2);
        sum *= -1.1754943508222875e-38f * 0.0625f;  // -8 2^-133 = -2^-126 2^-4
        qsum[x][b] = make_float2(__shfl_sync(kFull, sum, 8 * t), __shfl_sync(kFull, sum, 8 * t + 4));
        // nibbles 1, 3 (and 5, 7) of a word are taken four bits higher, times 16
        qb[x][b][0][0] = pack_bf16(c[0], c[4]);
        qb[x][b][0][1] = pack_bf16(c[1] * 0.0625f, c[5] * 0.0625f);
        qb[x][b][1][0] = pack_bf16(c[2], c[6]);
        qb[x][b][1][1] = pack_bf16(c[3] * 0.0625f, c[7] * 0.0625f);
      }
#pragma unroll
      for (int e2 = 0; e2 < 4; ++e2) {
        bias[x][e2] = 0.0f;
#pragma unroll
        for (int b = 0; b < NB; ++b) o[x][b][0][e2] = o[x][b][1][e2] = 0.0f;
      }
    }
  };

  const unsigned pick = (g & 1) != 0 ? 0x3244u : 0x1044u;  // the lane's token of a pair, as binary32
  auto work = [&](uint8_t* at0, int key0, bool bad) {  // 32 keys from key0 on
    // scores: rows of a product are the keys 8 (g / 2) + 2 j + g % 2 of j = 2 jp (elements 0, 1) and
    // 2 jp + 1 (2, 3), columns the rows 2 t, 2 t + 1 (+ 8 x)
    float2 s[NT][2][2];
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int jp = 0; jp < 2; ++jp) s[x][jp][0] = s[x][jp][1] = make_float2(0.0f, 0.0f);
    const uint8_t* keys = at0 + lane * Tile::kWords * 4;
#pragma unroll
    for (int bq = 0; bq < Tile::kQuads; ++bq) {
#pragma unroll
      for (int jp = 0; jp < 2; ++jp) {
        uint32_t kw[2][Tile::kWords];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint8_t* at = keys + ((2 * jp + i) * Tile::kQuads + bq) * 128 * Tile::kWords;
          if constexpr (Tile::kWords == 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(at);
            kw[i][0] = v.x; kw[i][1] = v.y; kw[i][2] = v.z; kw[i][3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(at);
            kw[i][0] = v.x; kw[i][1] = v.y;
          }
        }
#pragma unroll
        for (int bw = 0; bw < Tile::kWords; ++bw) {
          const int b = 4 * bq + bw;
          const uint2 sc = *reinterpret_cast<const uint2*>(at0 + Tile::kKeyScales + b * 64 + 16 * (g >> 1) + 8 * jp);
          const float s0 = __uint_as_float(__byte_perm(sc.x, 0u, pick)), s1 = __uint_as_float(__byte_perm(sc.y, 0u, pick));
          const uint32_t k0 = kw[0][bw], k1 = kw[1][bw], h0 = k0 >> 8, h1 = k1 >> 8;
#pragma unroll
          for (int x = 0; x < NT; ++x) {
            float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            mma_bf16(c, k0 & 0x000F000Fu, k1 & 0x000F000Fu, k0 & 0x00F000F0u, k1 & 0x00F000F0u, qb[x][b][0][0], qb[x][b][0][1]);
            mma_bf16(c, h0 & 0x000F000Fu, h1 & 0x000F000Fu, h0 & 0x00F000F0u, h1 & 0x00F000F0u, qb[x][b][1][0], qb[x][b][1][1]);
            s[x][jp][0] = __ffma2_rn(__fadd2_rn(make_float2(c[0], c[1]), qsum[x][b]), make_float2(s0, s0), s[x][jp][0]);
            s[x][jp][1] = __ffma2_rn(__fadd2_rn(make_float2(c[2], c[3]), qsum[x][b]), make_float2(s1, s1), s[x][jp][1]);
          }
        }
      }
    }
    // keys that a row does not see; values behind the last key may hold anything: their scales become 0
    if (bad || key0 + 32 > lim0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = key0 + 8 * (g >> 1) + 2 * j + (g & 1);
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          if (bad || key >= lim[x][0]) s[x][j >> 1][j & 1].x = -INFINITY;
          if (bad || key >= lim[x][1]) s[x][j >> 1][j & 1].y = -INFINITY;
        }
      }
      uint16_t* scales = reinterpret_cast<uint16_t*>(at0 + Tile::kValueScales + Tile::scale(lane, 0));
      bool drop = bad || key0 + lane >= len;
      if constexpr (NT == 2 || D == 256) {
        // a value that is not finite, of a token that not every row sees: 0 times its scale would reach
        // them all.  The rows that see the token become NaN here.
        bool odd = false;
#pragma unroll
        for (int b = 0; b < NB; ++b) odd = odd || (scales[32 * b] & 0x7F80u) == 0x7F80u;
        odd = odd && !drop && key0 + lane >= lim0;
        drop = drop || odd;
        const unsigned at = __ballot_sync(kFull, odd);
        if (at != 0) {
          const int first = key0 + __ffs(at) - 1;
#pragma unroll
          for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int r = 0; r < 2; ++r)
              if (lim[x][r] > first) bias[x][r] = bias[x][2 + r] = NAN;
        }
      }
      if (drop) {
#pragma unroll
        for (int b = 0; b < NB; ++b) scales[32 * b] = 0;
      }
      fence_proxy_async_smem();  // before the next copy into the stage
      __syncwarp();
    }
    // the reference follows the largest score only when that has run ahead
    float top[NT][2];
    bool grow = false;
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      top[x][0] = fmaxf(fmaxf(s[x][0][0].x, s[x][0][1].x), fmaxf(s[x][1][0].x, s[x][1][1].x));
      top[x][1] = fmaxf(fmaxf(s[x][0][0].y, s[x][0][1].y), fmaxf(s[x][1][0].y, s[x][1][1].y));
#pragma unroll
      for (int r = 0; r < 2; ++r) grow = grow || (top[x][r] - ref[x][r]) * f[x][r] > kSlack;
    }
    if (__any_sync(kFull, grow)) {
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float m = top[x][r];
#pragma unroll
          for (int i = 4; i < 32; i <<= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, i));
          m = fmaxf(ref[x][r], m);
          const float by = ex2((ref[x][r] - m) * f[x][r]);
          ref[x][r] = m;
          l[x][r] *= by;
          bias[x][r] *= by;
          bias[x][2 + r] *= by;
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int m2 = 0; m2 < 2; ++m2) {
              o[x][b][m2][r] *= by;
              o[x][b][m2][2 + r] *= by;
            }
        }
    }
    // weights as B operands: row g (+ 8 x), keys 8 t + 2 j, + 1; their leading 8 bits, and the rest
    uint32_t pw[NT][4], pr[NT][4];
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 v = __fadd2_rn(s[x][j >> 1][j & 1], make_float2(-ref[x][0], -ref[x][1]));
        const float2 e = __ffma2_rn(v, make_float2(f[x][0], f[x][1]), make_float2(kLift, kLift));
        const float a = ex2(e.x), b = ex2(e.y);
        l[x][0] += a;
        l[x][1] += b;
        pw[x][j] = transpose_8x8(__byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632));
        pr[x][j] = transpose_8x8(pack_bf16(a - bf16_hi(__float_as_uint(a)), b - bf16_hi(__float_as_uint(b))));
      }
    const uint8_t* values = at0 + Tile::kValues + lane * Tile::kHalves * 4;
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
        const uint2 sc = *reinterpret_cast<const uint2*>(at0 + Tile::kValueScales + b * 64 + 16 * t + 8 * k);
        const int h = b >> 1;
        const unsigned half = (b & 1) == 0 ? 0x5410u : 0x7632u;
        const uint32_t u0 = __byte_perm(v[0][h], v[1][h], half), u1 = __byte_perm(v[2][h], v[3][h], half);
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          const uint32_t b0 = fma_bf16(pw[x][2 * k], sc.x, mul_bf16(pr[x][2 * k], sc.x));
          const uint32_t b1 = fma_bf16(pw[x][2 * k + 1], sc.y, mul_bf16(pr[x][2 * k + 1], sc.y));
          // rows g: a nibble n; rows g + 8: the byte n + 16 n' that it is in, parted in the sums
          mma_bf16(o[x][b][0], u0 & 0x000F000Fu, u0 & 0x00FF00FFu, u1 & 0x000F000Fu, u1 & 0x00FF00FFu, b0, b1);
          const uint32_t y0 = __byte_perm(u0, 0u, 0x4341), y1 = __byte_perm(u1, 0u, 0x4341);
          mma_bf16(o[x][b][1], y0 & 0x000F000Fu, y0, y1 & 0x000F000Fu, y1, b0, b1);
          mma_bf16(bias[x], one[b], one[b], one[b], one[b], b0, b1);
        }
      }
    }
  };

  // The lane's share of a finished run: columns 2 t and 2 t + 1 of the rows, channels 32 b + 4 g .. + 3
  constexpr float k2p69 = 5.902958103587057e20f, k2m64 = 5.421010862427522e-20f;
  auto total = [&](int x, int b, int e, float (&v)[4]) {  // column 2 t + e; times 2^133
    const float c = __shfl_sync(kFull, bias[x][e], 4 * b + t);
    v[0] = o[x][b][0][e] + c;
    v[1] = fmaf(o[x][b][0][2 + e] - o[x][b][0][e], 0.0625f, c);
    v[2] = o[x][b][1][e] + c;
    v[3] = fmaf(o[x][b][1][2 + e] - o[x][b][1][e], 0.0625f, c);
  };
  auto row_sum = [&](int x, int e) {
    float sum = l[x][e];
#pragma unroll
    for (int i = 4; i < 32; i <<= 1) sum += __shfl_xor_sync(kFull, sum, i);
    return sum * k2m64;
  };
  Record* rec = reinterpret_cast<Record*>(sm + Sh::kOffRec);  // [warp][2]: put aside, at the end
  // The end of a run: a whole group of rows goes to o, others to `part`, row by row o, reference, sum and f.
  auto put = [&](float* part, bool rows) {
    const Item it = *item;
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * x + 2 * t + e;
        const float sum = row_sum(x, e);
        float by = k2p69;
        if (rows) by = sum != 0.0f ? k2p69 / sum : 0.0f;
        int query;
        int64_t head;
        const bool on = row_at<NT>(p, it.lq, it.h, it.group, r, &query, &head);
        uint16_t* dst = p.a.o + (it.q0 + query) * p.a.st[2] + head * p.a.st[3] + 4 * g;
        float* row = part + r * Sh::kPad;
        if (!rows && g == 0) *reinterpret_cast<float4*>(row + D) = make_float4(ref[x][e], sum, f[x][e], 0.0f);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          float v[4];
          total(x, b, e, v);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] *= by;
          if (!rows) *reinterpret_cast<float4*>(row + 32 * b + 4 * g) = make_float4(v[0], v[1], v[2], v[3]);
          else if (on) *reinterpret_cast<uint2*>(dst + 32 * b) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
        }
      }
  };
  // a run that ends inside the warp's waits beside the ring, which is still in use
  float* aside = reinterpret_cast<float*>(sm + Sh::kOffAside);

  if (lane < 2) rec[2 * warp + lane].flags = 0;
  __syncwarp();
  bool front = tile != 0, ok = true;  // the current run begins inside its item
  bool more = n > 0 && item->start + kExtra + tile < n;
  for (int i = 0, st = 0, ph = 0; more;) {
    int end;
    {
      uint4 qv[NT][NB];
      const Item it = *item;
      load_queries(it, qv);
      if (i == 0) {  // behind the queries, which would wait for them
        for (int k = 0; k < S; ++k) fill(k, k);
      }
      begin(it, qv);
      end = n - kExtra - it.start < tiles ? n - kExtra - it.start : tiles;
    }
    for (; tile < end; ++i) {
      ok = warp_wait(&bars[st], static_cast<uint32_t>(ph), &abort_flag);
      if (!ok) break;
      work(ring + st * Tile::kBytes, tile * 32, held_s[st] != kStageTile);
      __syncwarp();  // every lane has read the stage
      fill(i + S, S);
      if (++st == S) {
        st = 0;
        ph ^= 1;
      }
      ++tile;
    }
    if (!ok) {  // a copy did not come: report it, and wait for those still under way
      report_error(p.a.err, kErrWaitTimeout, &abort_flag);
      for (int k = i; k < i + S; ++k)
        if (stage_completes(held_s[k % S])) mbar_wait(&bars[k % S], static_cast<uint32_t>(k / S) & 1u, nullptr);
      break;
    }
    Item it = *item;
    const bool whole = tile == tiles, rows = !kAlone && whole && !front;
    more = !kAlone && whole && it.start + tiles + 2 * kExtra < n;
    put(more ? aside + warp * Sh::kPart : reinterpret_cast<float*>(ring), rows);
    if (!kAlone && !rows && lane == 0)
      rec[2 * warp + (more ? 0 : 1)] = {it.h, it.group, it.lq,
                                        kPartHeld | (front ? kPartFromFront : 0) | (whole ? 0 : kPartGoesOn), it.q0,
                                        static_cast<int64_t>(from) + it.start + it.tiles + kExtra};
    if (more) {
      next_item<NT>(p, it);
      __syncwarp();  // every lane has read the old one
      if (lane == 0) *item = it;
      __syncwarp();
      tile = 0;
      front = false;
    }
  }
  __syncthreads();
  constexpr int E = D / 32;
  auto write_row = [&](int lq, int h, int group, int64_t q0, int row, float sum, const float (&acc)[E]) {
    int query;
    int64_t head;
    if (row_at<NT>(p, lq, h, group, row, &query, &head)) {
      const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
      uint32_t* dst = reinterpret_cast<uint32_t*>(p.a.o + (q0 + query) * p.a.st[2] + head * p.a.st[3] + E * lane);
#pragma unroll
      for (int e = 0; e < E; e += 2) dst[e / 2] = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
    }
  };
  if constexpr (kAlone) {
    // the block's warps, then the cluster's blocks, which share the rows.  (After a wait that gave up
    // the rows hold anything, but no block may leave the others waiting.)
    const Item it = *reinterpret_cast<const Item*>(sm + Sh::kOffItem);
    const int used = rows_used<NT>(p, it.lq, it.group);
    for (int row = warp; row < used; row += Sh::kWarps) {
      float top, sum, fr, acc[E];
      auto member = [&](int m) { return reinterpret_cast<const float*>(sm + m * Sh::kRing) + row * Sh::kPad; };
      add_up<D>(lane, users, member, top, sum, fr, acc);
#pragma unroll
      for (int e = 0; e < E; e += 2) *reinterpret_cast<float2*>(aside + row * Sh::kPad + E * lane + e) = make_float2(acc[e], acc[e + 1]);
      if (lane == 0) *reinterpret_cast<float4*>(aside + row * Sh::kPad + D) = make_float4(top, sum, fr, 0.0f);
    }
    cluster_sync();
    const int c = p.cluster, rank = static_cast<int>(blockIdx.x) % c;
    for (int row = rank + c * warp; row < used; row += c * Sh::kWarps) {
      const float* mine = aside + row * Sh::kPad;
      float top = kNone, sum = 0.0f, acc[E] = {};
      const float fr = peer_load(mine + D + 2, 0);  // the first block has a tile
      for (int x = 0; x < c; ++x) top = fmaxf(top, peer_load(mine + D, x));
#pragma unroll 4
      for (int x = 0; x < c; ++x) {
        const float by = ex2((peer_load(mine + D, x) - top) * fr);
        sum = fmaf(peer_load(mine + D + 1, x), by, sum);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(peer_load(mine + E * lane + e, x), by, acc[e]);
      }
      write_row(it.lq, it.h, it.group, it.q0, row, sum, acc);
    }
    cluster_sync();  // no block leaves while another reads its shared memory
    return;
  }
  if (abort_flag != 0) {  // the join must not take what an earlier call has left for a record
    if (threadIdx.x == 0) p.meta[blockIdx.x].flags = 0;
    return;
  }

  // The block's chains: a run at a warp's end and those of the warps behind it while it goes on, in the
  // end one put aside.  A warp takes one row of a chain at a time.
  Record out;
  out.flags = 0;
  const int fa = lane < Sh::kWarps ? rec[2 * lane].flags : 0, fe = lane < Sh::kWarps ? rec[2 * lane + 1].flags : 0;
  const unsigned asides = __ballot_sync(kFull, fa != 0), ends = __ballot_sync(kFull, fe != 0);
  const unsigned fronts = __ballot_sync(kFull, (fe & kPartFromFront) != 0), onward = __ballot_sync(kFull, (fe & kPartGoesOn) != 0);
  const unsigned stops = ~onward | asides >> 1 | ~((asides | ends) >> 1);  // the chain's last run at a warp's end
  int task = 0;
#pragma unroll 1
  for (unsigned todo = (ends & (~fronts | 1u)) << 1 | (asides & 1u); todo != 0; todo &= todo - 1) {
    const int w1 = __ffs(todo) - 1, w0 = w1 > 0 ? w1 - 1 : 0;  // 0: the run that warp 0 put aside, alone
    const int n_end = w1 > 0 ? __ffs(stops >> w0) : 0;         // warps whose runs at the end belong to it
    const bool tail = w1 == 0 || ((onward >> (w0 + n_end - 1) & 1u) != 0 && (asides >> (w0 + n_end) & 1u) != 0);
    Record who = rec[w1 > 0 ? 2 * w0 + 1 : 0];
    const int end = tail ? 0 : rec[2 * (w0 + n_end - 1) + 1].flags;  // what is put aside does not go on
    const int v = w0 + n_end, members = n_end + (tail ? 1 : 0);
    const bool from_front = (who.flags & kPartFromFront) != 0, goes_on = (end & kPartGoesOn) != 0;
    if (goes_on && !from_front) out = who;
    const int used = rows_used<NT>(p, who.lq, who.group);
#pragma unroll 1
    for (int row = (warp + Sh::kWarps - task % Sh::kWarps) % Sh::kWarps; row < used; row += Sh::kWarps) {
      auto member = [&](int m) {
        return reinterpret_cast<const float*>(m < n_end ? sm + (w0 + m) * Sh::kRing : sm + Sh::kOffAside + v * Sh::kPart * 4) + row * Sh::kPad;
      };
      float top, sum, fr, acc[E];
      add_up<D>(lane, members, member, top, sum, fr, acc);
      if (from_front || goes_on) {
        float* dst = p.part + (static_cast<int64_t>(blockIdx.x) * 2 + (from_front ? 0 : 1)) * Sh::kPart + row * Sh::kPad;
#pragma unroll
        for (int e = 0; e < E; e += 2) *reinterpret_cast<float2*>(dst + E * lane + e) = make_float2(acc[e], acc[e + 1]);
        if (lane == 0) *reinterpret_cast<float4*>(dst + D) = make_float4(top, sum, fr, 0.0f);
      } else {
        write_row(who.lq, who.h, who.group, who.q0, row, sum, acc);
      }
    }
    task += used;
  }
  if (warp != 0) return;
  if (out.flags != 0) {  // the last block whose run begins in front of the item's end
    int last = static_cast<int>(blockIdx.x);
    for (uint32_t k0 = blockIdx.x + 1; k0 < nb; k0 += 32) {
      const uint32_t k = k0 + lane;
      const unsigned in = __ballot_sync(kFull, k < nb && static_cast<int64_t>(q * k + share(k)) < out.end);
      last += __popc(in);
      if (in != kFull) break;
    }
    out.end = last;
  }
  if (lane == 0) p.meta[blockIdx.x] = out;
  // a block without work adds nothing to a run that passes it
  if (run == 0 && lane < Sh::kRows)
    *reinterpret_cast<float2*>(p.part + static_cast<int64_t>(blockIdx.x) * 2 * Sh::kPart + lane * Sh::kPad + D) = make_float2(kNone, kNoPart);
}

// Runs that cross blocks: block x joins the one that begins in block x of the attention kernel.  The
// parts of all its blocks are loaded at once, a few warps to a row (a trip to another SM's results
// takes about a microsecond: two of them, the record and the parts, are all there is).
template <int D, int NT>
__global__ void __launch_bounds__(1024) kv4_join_kernel(const __grid_constant__ Kv4Params p) {
  using Sh = Kv4Shape<D, NT>;
  constexpr int E = D / 32, kW = 32 / Sh::kRows, kAhead = 16 / E;  // warps of a row, parts in flight
  __shared__ float acc_s[32][D];
  __shared__ float2 ml_s[32];
  pdl_wait();
  const int x = static_cast<int>(blockIdx.x);
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const Record who = p.meta[x];
  if (who.flags == 0) return;
  const int row = warp / kW, w0 = row * kW, n = min(static_cast<int>(who.end), static_cast<int>(gridDim.x) - 1) - x + 1;
  float top = kNone, sum = 0.0f, acc[E] = {};
  const float f = p.part[static_cast<int64_t>(2 * x + 1) * Sh::kPart + row * Sh::kPad + D + 2];  // the same in all parts
  for (int m0 = warp - w0; m0 < n; m0 += kW * kAhead) {
    float2 ml[kAhead];
    float v[kAhead][E];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int m = m0 + i * kW;
      const float* src = p.part + static_cast<int64_t>(2 * (x + m) + (m == 0 ? 1 : 0)) * Sh::kPart + row * Sh::kPad;
      ml[i] = make_float2(kNone, kNoPart);
      if (m < n) {
        ml[i] = *reinterpret_cast<const float2*>(src + D);
#pragma unroll
        for (int e = 0; e < E; e += 2) *reinterpret_cast<float2*>(&v[i][e]) = *reinterpret_cast<const float2*>(src + E * lane + e);
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (ml[i].y == kNoPart) continue;  // its place holds anything
      const float to = fmaxf(top, ml[i].x), old = ex2((top - to) * f), by = ex2((ml[i].x - to) * f);
      top = to;
      sum = fmaf(sum, old, ml[i].y * by);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(acc[e], old, v[i][e] * by);
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) acc_s[warp][E * lane + e] = acc[e];
  if (lane == 0) ml_s[warp] = make_float2(top, sum);
  __syncthreads();
  top = kNone;
#pragma unroll
  for (int w = 0; w < kW; ++w) top = fmaxf(top, ml_s[w0 + w].x);
  int query;
  int64_t head;
  if (!row_at<NT>(p, who.lq, who.h, who.group, row, &query, &head)) return;
  const int c = 2 * (static_cast<int>(threadIdx.x) - 32 * w0);
  for (int k = c; k < D; k += 64 * kW) {
    float t = 0.0f, u = 0.0f, v = 0.0f;
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      const float by = ex2((ml_s[w0 + w].x - top) * f);
      t = fmaf(ml_s[w0 + w].y, by, t);
      u = fmaf(acc_s[w0 + w][k], by, u);
      v = fmaf(acc_s[w0 + w][k + 1], by, v);
    }
    const float inv = t != 0.0f ? 1.0f / t : 0.0f;
    *reinterpret_cast<uint32_t*>(p.a.o + (who.q0 + query) * p.a.st[2] + head * p.a.st[3] + k) = pack_bf16(u * inv, v * inv);
  }
}

// ---- host ------------------------------------------------------------------------------------
// Rows of a group: 8, or 16 where a request's rows may be more (256 channels: 8, sixteen would
// not fit the registers).  64 requests of 4096 tokens, 16 rows against two groups of 8: 4 heads of 128 a group and 4 new
// tokens 92.9 us and 109.3, 16 heads a group 92.5 and 109.3, of 64 channels 59.2 and 70.8.  How many queries a request
// has is not known here: with cu_q, 8 rows or fewer pay for 16 (one new token of 4 heads of 128 89.5 us, 60.1 by 8).
int row_tiles(int64_t G, bool one_query, int64_t d) { return d == 256 || (one_query && G <= 8) ? 1 : 2; }

int grid_blocks(const DeviceInfo& dev) { return std::min(dev.sm_count, kMaxBlocks); }

// Blocks of a cluster that takes a group of rows alone, 0 where the work list is better: one group a
// request and head, all of them at once on the GPU, and few keys for a block even if one request
// has all that its row of the block table can name.  Device time alone and with the list, lengths
// spread over the logarithm up to the table's: 1 request of 8192 tokens, 32 / 8 heads of 128, 8 blocks a
// cluster 10.1 and 11.0 us, of 16384 14.2 and 13.4; 4 requests of up to 4096, 4 blocks 10.1 both; 16 of
// 1536, one block 10.3 and 9.8; the second launch and the workspace take the host about 5 us more.  (The
// lengths themselves are not known here: one request of 1000 behind a table of 16384 or more gets the list.)
int alone_blocks(const Kv4AttentionArgs& a, int nt, const DeviceInfo& dev) {
  const int64_t items = a.B * a.Hkv, keys = a.width * a.page, sms = dev.sm_count;
  if (a.cu_q != nullptr || a.H / a.Hkv > 8 * nt || items > sms) return 0;
  int64_t c = 8;
  // clusters do not fill the GPU's parts: 16 of 8 blocks take a second wave
  while (c > 1 && 8 * items * c > (c == 8 ? 6 : 7) * sms) c /= 2;
  while (c > 1 && c * 64 > keys) c /= 2;  // two tiles a block at least
  return keys <= c * 1536 ? static_cast<int>(c) : 0;
}

template <int D, int NT>
size_t ws_bytes(const DeviceInfo& dev) {
  using Sh = Kv4Shape<D, NT>;
  const size_t blocks = static_cast<size_t>(grid_blocks(dev));
  return blocks * (2 * Sh::kPart * 4 + sizeof(Record));
}

template <typename K>
cudaError_t launch_one(K kernel, int blocks, int threads, size_t smem, int cluster, const Kv4Params& p,
                       cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int D, int NT>
cudaError_t attention(const Kv4AttentionArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  using Sh = Kv4Shape<D, NT>;
  Kv4Params p = {};
  p.a = a;
  p.G = static_cast<int>(a.H / a.Hkv);
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.per_lane = static_cast<int>((a.B + 31) / 32);
  p.by_G = ~uint64_t{0} / static_cast<uint64_t>(p.G) + 1;
  p.by_tpp = ~uint64_t{0} / static_cast<uint64_t>(a.page / 32) + 1;
  p.cluster = alone_blocks(a, NT, dev);
  if (p.cluster > 0) {
    const auto kernel = kv4_attention_kernel<D, NT, true>;
    const cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kernel), Sh::kSmem, dev.device);
    if (e != cudaSuccess) return e;
    return launch_one(kernel, static_cast<int>(a.B * a.Hkv) * p.cluster, Sh::kThreads, Sh::kSmem, p.cluster, p, stream);
  }
  const int blocks = grid_blocks(dev);
  p.by_grid = static_cast<uint32_t>((uint64_t{1} << 32) / static_cast<uint64_t>(blocks));
  p.part = static_cast<float*>(a.part);
  p.meta = reinterpret_cast<Record*>(p.part + static_cast<size_t>(blocks) * 2 * Sh::kPart);
  const auto kernel = kv4_attention_kernel<D, NT, false>;
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kernel), Sh::kSmem, dev.device);
  if (e != cudaSuccess) return e;
  if ((e = launch_one(kernel, blocks, Sh::kThreads, Sh::kSmem, 1, p, stream)) != cudaSuccess) return e;
  return launch_one(kv4_join_kernel<D, NT>, blocks, 1024, 0, 1, p, stream);
}

}  // namespace

size_t kv4_attention_ws_bytes(const Kv4AttentionArgs& a, const DeviceInfo& dev) {
  const int nt = row_tiles(a.H / a.Hkv, a.cu_q == nullptr, a.d);
  if (alone_blocks(a, nt, dev) > 0) return 0;
  if (a.d == 256) return ws_bytes<256, 1>(dev);
  if (a.d == 128) return nt == 1 ? ws_bytes<128, 1>(dev) : ws_bytes<128, 2>(dev);
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
