// q8_attn.cu -- attention over packed prompts and over a shared prefix.
//
// The attention layers of the hybrid models that "CUDA inference engine for running
// Qwen3.5/3.6 hybrid models on mining cards (CMP 100-210)" (news.hada.io topic 29953) runs:
// o = softmax(scale q . k) v over the keys a query sees, H query heads over Hkv key/value
// heads of 64 or 128 channels (two S and two O of 256 would not fit the 512 columns of TMEM).
//
// Both entry points walk the keys once with a running reference m and sum l per row (online
// softmax; Milakov and Gimelshein, 2018): for a block of scores s, w = 2^(s' - m) with
// s' = s scale log2(e);  l += sum w;  O += w V;  where a row's maximum has left m behind, l and
// O are first scaled by 2^(m - m').  Parts of a row that different blocks walked are joined by
// o = sum_p 2^(m_p - M) O_p / sum_p 2^(m_p - M) l_p, M = max m_p, in a fixed order.
// Scores, m, l and O are binary32; w is rounded to bfloat16 for the product with V only (l sums
// the unrounded weights), o once at the end.  The MMAs take A and B of one type, and V is
// bfloat16: w in more bits would be a second product for its rest, half as many tensor cycles
// again.  It moves o by less than its own rounding does (with both, 1.2 to 1.5 times the error
// of the rounded o alone over the measured cases).
//
//  attn_tile_kernel    whole prompts, and a batch's queries over its shared prefix: tensor work
//  attn_own_kernel     a request's own keys, which no other reads: the bytes of its cache
//  *_join_kernel       the splits of a row
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "q8_internal.h"
#include "q8_attn_ptx.cuh"
#include "q8_launch_ptx.cuh"

namespace q8 {
namespace {

constexpr uint32_t kErrBadLength = 1u << 9;  // a sequence or cache length outside its array

__device__ __forceinline__ bool bounds_ok(const PromptArgs& a, int64_t q0, int64_t q1, int64_t k0, int64_t k1) {
  return 0 <= q0 && q0 <= q1 && q1 <= a.Tq && 0 <= k0 && k0 <= k1 && k1 <= a.Tk;
}

// whether sequence s lies inside the arrays
__device__ __forceinline__ bool sequence_ok(const PromptArgs& a, int64_t s) {
  return bounds_ok(a, a.cu_q[s], a.cu_q[s + 1], a.cu_k[s], a.cu_k[s + 1]);
}

// ---- the tile kernel ---------------------------------------------------------------------
// The rows of a tile are the G heads of 128 / G neighbouring tokens: the heads that share a
// key/value head are rows of the same products, so K and V are read once for all of them and
// a causal tile of few tokens wastes little of its diagonal block.
//
// Bound: the tensor pipe.  A block of 128 keys takes d / 16 + 8 MMAs of 64 cycles (S = Q K^T, and
// O += P V): 1024 cycles at d = 128.  Its softmax takes about 1100, 1500 from the S committed to
// the P handed over, so one stream of blocks would leave the pipe idle most of the time.  Hence
// two streams, A and B, each with its S (128 columns of TMEM) and O (d columns): while one is in its
// softmax the pipe works on the other.
//  - kTwo: the streams are two tiles behind one another in the sequence that walk the same
//    blocks of K and V (each is loaded once for 256 rows).
//  - else: one tile, whose even and odd blocks are the streams; their O are joined at the end.
// P takes the place of S in TMEM, as the A operand of P V; with d = 64 there is room for it beside
// S, and the stream's next S is computed during the softmax (8192 tokens of 32 heads of 64: 246 us,
// 259 with P over S).  Softmax: sixteen warps, eight a
// stream, two for 32 rows, each thread half a row (64 scores in registers, no shuffles); with
// four warps a stream, a row a thread, 8192 tokens took 480 us instead of 372.  One warp finds the items and
// loads (TMA, a ring of 5 to 8 K or V blocks that runs over from item to item), one elected
// thread issues the MMAs.
// The reference moves only when a row's maximum gains more than 2^8 (weights stay below 2^8, far
// from the ends of binary32 and of bfloat16's equal range): rescaling O is rare.
// The blocks are persistent: the next item (tile, head, split) is asked for while the current
// one is in work, the last ones of a sequence, which see the most keys, first.
//
// 32 query heads, 8 key/value heads of 128: 8192 tokens in 344 us (1.60 PFLOP/s counted over the
// causal half, 0.84 of the measured dense rate; 1762 MHz under the power cap), 16384 tokens in
// 1320 (1.67 PFLOP/s, 1717 MHz).  What is left there is the clock under load, and the ends: the
// first S and the last O of a block's items.
constexpr int kRows = 128;     // query rows of a tile: 128 / G tokens x G heads
constexpr int kKeys = 128;     // keys of a block
constexpr int kSoftWarps = 16;  // softmax: 8 warps a stream, two (a half of the keys each) for 32 rows
constexpr int kTileThreads = 32 * (kSoftWarps + 2);  // and one warp for the loads, one for the MMAs
// Barrier 0 is the one at the kernel's end.  The softmax warps use 1 to 8 (two warps of 32 rows)
// and 9, 10 (a stream).  The start has a number of its own: the load warp only arrives there, and
// a barrier counts arrivals, not warps, so its arrival at the end must not be able to stand in
// for a warp that is still on its way to the start.
constexpr int kStartBar = 11;

constexpr float kRescaleLog2 = 8.0f;  // move the exponent reference when a row's maximum gains > 2^8

template <int D, bool kTwo>
struct TileShape {
  static constexpr uint32_t kTile = kRows * D * 2;           // a Q tile
  static constexpr uint32_t kStage = kKeys * D * 2;          // a K or V block
  static constexpr uint32_t kHalf = kKeys * 128;             // 64 channels of 128 rows
  // P beside S in TMEM (128 channels leave no room for it)
  static constexpr bool kApart = D == 64;
  static constexpr int kLead = (kTwo ? 1 : 2) + (kApart ? 1 : 0);  // K blocks in front of the first V block
  static constexpr int kStages = D == 128 ? (kTwo ? 5 : 6) : 8;
  static constexpr uint32_t kOffRing = (kTwo ? 2 : 1) * kTile;
  static constexpr uint32_t kOffMax = kOffRing + kStages * kStage;  // float [2 streams][2 halves][rows]
  static constexpr uint32_t kOffBar = kOffMax + 4 * kRows * 4;
  static constexpr int kBars = 24 + 2 * kStages;
  static constexpr uint32_t kOffWork = kOffBar + kBars * 8;
  static constexpr uint32_t kSmem = kOffWork + 2 * 64 + 16 + 16;  // two items, the next grid index, TMEM address and flag
  static_assert(kOffWork % 16 == 0, "alignment");
  static_assert(kSmem <= 227 * 1024, "shared memory of a block");
};

// What the load warp tells the others about an item.
struct Work {
  int tok, tok_end, lk;  // Item
  int hk, split, b0;     // key/value head, split, its first block
  int cnt, nA, nB;       // blocks (-1: no more items), and each stream's
  int tail;              // rows of the last block that are the sequence's (kKeys: all)
};
static_assert(sizeof(Work) <= 64, "an item's place");

struct TileParams {
  PromptArgs a;            // strides of q, k, v, o; for the prefix B, Tq are the requests and Tk is P
  int G, nt;               // heads of a group, tokens of a tile
  int64_t nslots;
  int splits;              // blocks of keys are dealt to this many CTAs
  int to_parts;            // 0: o is written here (one split), 1: partial results
  int k_head, v_head;      // 0: all key / value heads are one (stride 0)
  float scale_log2;
  float* part_o;           // [splits][Tq * H][D]
  float2* part_ml;         // [splits][Tq * H]
};

// 3-D tile load
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int32_t x, int32_t y,
                                            int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// true on one lane of the (converged) warp
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(p));
  return p != 0;
}

// D[tmem] (+)= A[tmem] * B[smem], kind::f16: A's rows are TMEM lanes, two values a column
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// A value that is the same on all lanes, told to the compiler as such (loop counts and branches
// on it then need no reconvergence; 5 % of a long prompt).
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

// A test of a barrier's phase that does not suspend: polling with it sees a phase complete about
// 100 cycles sooner than try_wait does.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// One thread's wait that polls (bounded as mbar_wait).
__device__ __forceinline__ bool mbar_poll(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (mbar_test(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_test(bar, parity))
    if (*abort_flag != 0 || clock64() - t0 > kWaitBudgetCycles) return false;
  return true;
}

// Work stealing: a block asks for the index of one that has not been launched yet, which then
// never is.  The answer (16 bytes) lands in shared memory and completes on the barrier.
__device__ __forceinline__ void ask_next(void* answer, uint64_t* bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(answer)),
               "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ bool read_next(const void* answer, uint32_t* x, uint32_t* y) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 h;\n\t"
      "ld.shared.b128 h, [%3];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "mov.u32 %2, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, %2, _, _}, h;\n\t}"
      : "=r"(ok), "=r"(*x), "=r"(*y)
      : "r"(smem_u32(answer))
      : "memory");
  return ok != 0;
}

// Transposes 16-byte pieces among groups of kN neighbouring lanes: lane b of a group gives its
// pieces 0 .. kN - 1 and gets piece b of each of the group's lanes.
template <int kN>
__device__ __forceinline__ void transpose_pieces(uint4 (&v)[kN], int lane) {
#pragma unroll
  for (int m = 1; m < kN; m <<= 1) {
    const bool up = (lane & m) != 0;
#pragma unroll
    for (int q = 0; q < kN; ++q)
      if ((q & m) == 0) {
        uint4 x = up ? v[q] : v[q | m];
        x.x = __shfl_xor_sync(0xFFFFFFFFu, x.x, m);
        x.y = __shfl_xor_sync(0xFFFFFFFFu, x.y, m);
        x.z = __shfl_xor_sync(0xFFFFFFFFu, x.z, m);
        x.w = __shfl_xor_sync(0xFFFFFFFFu, x.w, m);
        if (up) v[q] = x;
        else v[q | m] = x;
      }
  }
}

// Which queries and keys a CTA works on (all counts fit 32 bits: see the entry points' limits).
struct Item {
  int tok;      // first query token of stream A's tile
  int tok_end;  // behind the last query token of the sequence
  int key0;     // row of the sequence's first key
  int lk;       // its keys
};

// Keys that query token t (below tok_end) sees: the last one all lk, each one before one less;
// behind a prefix all of them.
template <bool kPrefix>
__device__ __forceinline__ int visible(const Item& it, int t) {
  if (kPrefix) return it.lk;
  const int n = it.lk - (it.tok_end - 1 - t);
  return n < 0 ? 0 : n;
}

// Slots: sequence s owns the slots from cu_q[s] / n + s on, at least as many as it has groups
// of n tokens (there are Tq / n + B in all), so a slot finds its sequence by a search over cu_q
// alone: no plan is made in front of the launch.  All
// lanes of a warp search together: 32 probes a round until 32 sequences are left, whose four
// bounds are then read at once, so up to 32 sequences cost one memory latency.
__device__ __forceinline__ bool prompt_item(const PromptArgs& a, int slot, int n, int lane, Item* it) {
  auto first = [&](int s, int q) { return static_cast<int>(static_cast<unsigned>(q / n) + static_cast<unsigned>(s)); };
  int lo = 0, hi = static_cast<int>(a.B);
  while (hi - lo > 32) {
    const int step = (hi - lo + 31) / 32, s = lo + lane * step;
    const unsigned ok = __ballot_sync(0xFFFFFFFFu, s < hi && first(s, a.cu_q[s]) <= slot);
    if (ok == 0) return false;
    lo += (31 - __clz(ok)) * step;
    if (lo + step < hi) hi = lo + step;
  }
  const int mine = lo + lane;
  int q0 = 0, q1 = 0, k0 = 0, k1 = 0;
  if (mine < hi) {
    q0 = a.cu_q[mine];
    q1 = a.cu_q[mine + 1];
    k0 = a.cu_k[mine];
    k1 = a.cu_k[mine + 1];
  }
  const int begin = first(mine, q0);
  const unsigned ok = __ballot_sync(0xFFFFFFFFu, mine < hi && begin <= slot);
  if (ok == 0) return false;
  const int from = 31 - __clz(ok);
  q0 = __shfl_sync(0xFFFFFFFFu, q0, from);
  q1 = __shfl_sync(0xFFFFFFFFu, q1, from);
  k0 = __shfl_sync(0xFFFFFFFFu, k0, from);
  k1 = __shfl_sync(0xFFFFFFFFu, k1, from);
  const int tile = slot - __shfl_sync(0xFFFFFFFFu, begin, from);
  const int64_t tok = q0 + static_cast<int64_t>(tile) * n;  // 64 bits: the bounds may be malformed
  if (!bounds_ok(a, q0, q1, k0, k1) || tile < 0 || tok >= q1) return false;
  it->tok = static_cast<int>(tok);
  it->tok_end = q1;
  it->key0 = k0;
  it->lk = k1 - k0;
  return true;
}

template <bool kPrefix>
__device__ __forceinline__ bool find_item(const TileParams& p, int slot, int n, int lane, Item* it) {
  if constexpr (kPrefix) {  // the requests are the tokens, all of them see all keys
    it->tok = slot * n;
    it->tok_end = static_cast<int>(p.a.Tq);
    it->key0 = 0;
    it->lk = static_cast<int>(p.a.Tk);
    return it->tok < it->tok_end;
  } else {
    return prompt_item(p.a, slot, n, lane, it);
  }
}

// Key blocks that the tile of n tokens from tok on needs, and the ones of a split.
template <bool kPrefix>
__device__ __forceinline__ int tile_blocks(const Item& it, int tok, int n) {
  if (tok >= it.tok_end) return 0;
  return (visible<kPrefix>(it, min(tok + n, it.tok_end) - 1) + kKeys - 1) / kKeys;
}
__device__ __forceinline__ int blocks_per_split(int blocks, int splits) {
  return splits == 1 ? blocks : (blocks + splits - 1) / splits;
}

template <int D, bool kTwo, bool kPrefix>
__global__ void __launch_bounds__(kTileThreads, 1)
    attn_tile_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ TileParams p) {
  using Sh = TileShape<D, kTwo>;
  constexpr int NS = Sh::kStages;
  constexpr bool kSteal = !kPrefix, kApart = Sh::kApart;
  constexpr int kLead = Sh::kLead;
  // the requests' own keys, or the join, may start (2 us of one token behind 2000 keys)
  if (kPrefix || p.to_parts != 0) pdl_launch_dependents();
  extern __shared__ __align__(1024) uint8_t sm[];
  const int warp = uniform(static_cast<int>(threadIdx.x >> 5)), lane = static_cast<int>(threadIdx.x & 31);
  if ((smem_u32(sm) & 1023u) != 0) {  // the whole CTA leaves before touching anything
    if (threadIdx.x == 0) atomicOr(p.a.err, kErrBadLaunch);
    return;
  }
  constexpr int kTiles = kTwo ? 2 : 1;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Sh::kOffBar);
  uint64_t* q_full = bars;           // [1] an item's Q landed
  uint64_t* q_empty = bars + 1;      // [1] its last S is done
  uint64_t* tail_done = bars + 2;    // [2] (by item) the last V block's rows behind the keys are zero
  uint64_t* s_full = bars + 4;       // [2] S of a stream computed (and its earlier P V done)
  uint64_t* p_full = bars + 6;       // [2] P written, O rescaled: an arrival of each warp
  uint64_t* o_full = bars + 8;       // [2] a stream's last P V of an item done (kApart: each P V)
  uint64_t* o_empty = bars + 10;     // [2] an item's O has been read
  uint64_t* work_full = bars + 12;   // [2] an item's place written
  uint64_t* work_empty = bars + 14;  // [2] the softmax and MMA warps are done with the item
  uint64_t* next_bar = bars + 16;    // [1] the next grid index
  uint64_t* end_bar = bars + 17;     // [1]
  uint64_t* s_read = bars + 18;      // [2] kApart: S is in the softmax warps' registers
  uint64_t* full = bars + 20;        // [NS]
  uint64_t* empty = full + NS;       // [NS]
  auto work_at = [&](int w) { return reinterpret_cast<Work*>(sm + Sh::kOffWork + 64 * w); };
  void* next_index = sm + Sh::kOffWork + 128;
  uint32_t& tmem_slot = *reinterpret_cast<uint32_t*>(sm + Sh::kOffWork + 144);
  int& abort_flag = *reinterpret_cast<int*>(sm + Sh::kOffWork + 148);
  if (warp == kSoftWarps && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tail_done[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], kSoftWarps / 2);
      mbar_init(&o_full[i], 1);
      mbar_init(&s_read[i], kSoftWarps / 2);
      mbar_init(&o_empty[i], kSoftWarps / 2);
      mbar_init(&work_full[i], 1);
      mbar_init(&work_empty[i], kSoftWarps + 1);
    }
    mbar_init(next_bar, 1);
    mbar_init(end_bar, 1);
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kSoftWarps + 1) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  if (warp == kSoftWarps) {  // made the barriers, and needs nothing of the others: its loads may start
    __syncwarp();
    asm volatile("bar.arrive %0, %1;" ::"n"(kStartBar), "n"(kTileThreads) : "memory");
  } else {
    tc_fence_before();
    asm volatile("bar.sync %0, %1;" ::"n"(kStartBar), "n"(kTileThreads) : "memory");
    tc_fence_after();
  }
  const uint32_t tbase = warp == kSoftWarps ? 0u : static_cast<uint32_t>(uniform(static_cast<int>(tmem_slot)));
  // columns: S of the streams, then O, then P where it does not take the place of S
  constexpr uint32_t kColO = 256, kColP = kApart ? kColO + 2 * D : 0, kStepP = kApart ? 64 : kKeys;
  // where the second 64 keys' P begins: over S behind it, so that half a row's warp overwrites
  // what it has read itself
  constexpr uint32_t kHalfP = kApart ? 32 : 64;
  // The ring holds the K and V blocks in the order of their use, item behind item.  Two tiles:
  // K0 V0 K1 V1 ...; one tile with two streams: K0 K1 V0 K2 V1 K3 V2 ...; one K block more in front
  // where the next S does not wait for P V.  Loads and MMAs walk it with a cursor each.
  struct Cursor {
    int st = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void step() {
      ph = st + 1 == NS ? ph ^ 1 : ph;
      st = st + 1 == NS ? 0 : st + 1;
    }
  };

  if (warp == kSoftWarps) {
    // ---------------- items and loads ----------------
    bool ok = true;
    int items = 0, loaded = 0;       // items handed over; those with blocks
    unsigned issued = 0;             // copies under way or done
    Cursor at, last;                 // the next one's place, the last one's
    uint32_t x = blockIdx.x, y = blockIdx.y, asked = 0;
    while (true) {
      const int hk = static_cast<int>(x % static_cast<unsigned>(p.a.Hkv)), split = static_cast<int>(y);
      const int slot = static_cast<int>(p.nslots) - 1 - static_cast<int>(x / static_cast<unsigned>(p.a.Hkv));
      Item it = {};
      const bool found = find_item<kPrefix>(p, slot, kTiles * p.nt, lane, &it);
      const int nbA = found ? tile_blocks<kPrefix>(it, it.tok, p.nt) : 0;
      const int nbB = kTwo ? (found ? tile_blocks<kPrefix>(it, it.tok + p.nt, p.nt) : 0) : nbA;
      const int nb = nbA > nbB ? nbA : nbB;
      const int per = blocks_per_split(nb, p.splits);
      const int b0 = split * per;
      const int cnt = nb - b0 < per ? nb - b0 : per;  // blocks of this split (<= 0: none)
      if (found && (split == 0 || cnt > 0)) {
        const int w = items & 1;
        // rows of the last block that are the sequence's
        const int tail = cnt > 0 && (b0 + cnt) * kKeys > it.lk ? it.lk - (b0 + cnt - 1) * kKeys : kKeys;
        if (lane == 0) {
          if (items >= 2) ok = mbar_wait_sleep(&work_empty[w], static_cast<uint32_t>((items >> 1) - 1) & 1, &abort_flag);
          if (ok) {
            // blocks of each stream: both tiles walk the same blocks, or one tile's are dealt in turn
            auto clampn = [](int v, int hi) { return v < 0 ? 0 : v < hi ? v : hi; };
            Work o;
            o.tok = it.tok;
            o.tok_end = it.tok_end;
            o.lk = it.lk;
            o.hk = hk;
            o.split = split;
            o.b0 = b0;
            o.cnt = cnt;
            o.nA = kTwo ? clampn(nbA - b0, cnt) : (cnt + 1) / 2;
            o.nB = kTwo ? clampn(nbB - b0, cnt) : cnt / 2;
            o.tail = tail;
            *work_at(w) = o;
            mbar_arrive(&work_full[w]);
          }
          if (ok && cnt > 0) {
            auto load = [&](bool isK, int j) {
              // the place's last copy but this one has been read (the phase before the copy's own)
              if (ok && issued >= NS) ok = mbar_wait_sleep(&empty[at.st], at.ph ^ 1, &abort_flag);
              if (!ok) return;
              mbar_arrive_expect_tx(&full[at.st], Sh::kStage);
              const int32_t row = it.key0 + (b0 + j) * kKeys;
              for (int c = 0; c < D / 64; ++c)
                tma_load_3d(sm + Sh::kOffRing + at.st * Sh::kStage + c * Sh::kHalf, isK ? &tmK : &tmV, &full[at.st],
                            64 * c, isK ? (p.k_head ? hk : 0) : (p.v_head ? hk : 0), row);
              last = at;
              at.step();
              ++issued;
            };
            load(true, 0);
            if (ok && loaded > 0) ok = mbar_wait_sleep(q_empty, static_cast<uint32_t>(loaded - 1) & 1, &abort_flag);
            if (ok) {
              mbar_arrive_expect_tx(q_full, kTiles * (D / 64) * 128u * static_cast<uint32_t>(p.G * p.nt));
              for (int t = 0; t < kTiles; ++t)
                for (int c = 0; c < D / 64; ++c)
                  tma_load_3d(sm + t * Sh::kTile + c * Sh::kHalf, &tmQ, q_full, 64 * c, hk * p.G, it.tok + t * p.nt);
              ++loaded;
            }
#pragma unroll
            for (int j = 1; j < kLead; ++j)
              if (cnt > j) load(true, j);
            for (int j = 0; j < cnt; ++j) {
              load(false, j);
              if (j + kLead < cnt) load(true, j + kLead);
            }
          }
        }
        ok = __shfl_sync(0xFFFFFFFFu, ok ? 1 : 0, 0) != 0;
        if (ok && tail < kKeys) {
          // a weight of 0 does not silence a NaN behind the sequence: those rows of V become 0
          const int st = __shfl_sync(0xFFFFFFFFu, last.st, 0);  // the item's last copy
          ok = warp_wait(&full[st], __shfl_sync(0xFFFFFFFFu, last.ph, 0), &abort_flag);
          uint8_t* v = sm + Sh::kOffRing + st * Sh::kStage;
          if (ok) {
            for (int c = 0; c < D / 64; ++c)
              for (int i = tail * 8 + lane; i < kKeys * 8; i += 32)
                reinterpret_cast<uint4*>(v + c * Sh::kHalf)[i] = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tail_done[w]);
          }
        }
        ++items;
      }
      if (!kSteal) break;
      // asked for as late as the ring's lead allows: what others may take is not held back here
      if (lane == 0) {
        mbar_arrive_expect_tx(next_bar, 16);
        ask_next(next_index, next_bar);
      }
      __syncwarp();
      ok = warp_wait(next_bar, asked & 1, nullptr) && ok;  // the answer lands in any case
      if (!ok) break;
      ++asked;
      const bool more = read_next(next_index, &x, &y);
      fence_proxy_async_smem();  // the answer has been read before the next one may land
      __syncwarp();
      if (!more) break;
    }
    if (lane == 0) {
      if (ok) {  // no more items
        const int w = items & 1;
        if (items >= 2) ok = mbar_wait_sleep(&work_empty[w], static_cast<uint32_t>((items >> 1) - 1) & 1, &abort_flag);
        if (ok) {
          work_at(w)->cnt = -1;
          mbar_arrive(&work_full[w]);
        }
      }
      if (!ok) report_error(p.a.err, kErrWaitTimeout, &abort_flag);
      // no copy may still be landing in shared memory when the CTA ends
      if (loaded > 0) mbar_wait(q_full, static_cast<uint32_t>(loaded - 1) & 1, nullptr);
      for (int i = 0; i < NS && issued >= static_cast<unsigned>(NS); ++i, at.step()) mbar_wait(&full[at.st], at.ph ^ 1, nullptr);
      for (int i = 0; i < at.st && issued < static_cast<unsigned>(NS); ++i) mbar_wait(&full[i], 0, nullptr);
    }
  } else if (warp == kSoftWarps + 1) {
    // ---------------- MMAs ----------------
    // One elected thread walks the loop.  elect.sync tells the compiler that it is alone: behind a
    // plain lane == 0 every MMA is issued by a loop over the lanes that might be active (250
    // cycles an MMA next to the softmax warps, against the pipe's 64).
    if (elect_one()) {
    constexpr uint32_t idS = idesc_bf16(kRows, kKeys, 0, 0), idO = idesc_bf16(kRows, D, 0, 1);
    const uint64_t dQ = sdesc_k_sw128(smem_u32(sm)), dK = sdesc_k_sw128(smem_u32(sm + Sh::kOffRing));
    const uint64_t dV = sdesc_mn_sw128(smem_u32(sm + Sh::kOffRing), Sh::kHalf, 1024);
    bool ok = true;
    int loaded = 0, tails = 0;   // items with blocks; bit w: parity of the tails of place w
    Cursor at;
    int doneA = 0, doneB = 0;    // blocks of each stream in earlier items
    for (int items = 0; ok; ++items) {
      const int w = items & 1;
      ok = mbar_poll(&work_full[w], static_cast<uint32_t>(items >> 1) & 1, &abort_flag);
      if (!ok) break;
      const Work* o = work_at(w);
      const int cnt = o->cnt, nA = o->nA, nB = o->nB, tail = o->tail;
      if (cnt < 0) break;
      if (cnt > 0) {
        auto landed = [&](const Cursor& c) { ok = ok && mbar_poll(&full[c.st], c.ph, &abort_flag); };
        int left = nA + nB;  // S still to come
        auto issue_s = [&](int s, const Cursor& c) {  // stream s with a block of K, which has landed
          const uint64_t a = dQ + static_cast<uint64_t>(((kTwo ? s : 0) * Sh::kTile) >> 4);
          const uint64_t b = dK + static_cast<uint64_t>((c.st * Sh::kStage) >> 4);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint64_t off = static_cast<uint64_t>(((k >> 2) * Sh::kHalf + (k & 3) * 32) >> 4);
            mma_f16_ss(tbase + s * kKeys, a + off, b + off, idS, k > 0 ? 1u : 0u);
          }
          mma_commit(&s_full[s]);
        };
        auto issue_pv = [&](int s, const Cursor& c, bool first) {  // 16 keys a step: 8 columns of P, 16 rows of V
          const uint64_t b = dV + static_cast<uint64_t>((c.st * Sh::kStage) >> 4);
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k)
            mma_f16_ts(tbase + kColO + s * D, tbase + kColP + s * kStepP + 8 * k + (k >= 4 ? kHalfP - 32 : 0),
                       b + static_cast<uint64_t>(k * (2048 >> 4)), idO, k > 0 || !first ? 1u : 0u);
        };
        // P V of the stream's i-th block and, in the same go, S of its next one
        auto turn = [&](int s, int i, const Cursor& v, const Cursor& k, bool more, bool release_v, bool release_k) {
          const uint32_t ph = static_cast<uint32_t>((s == 0 ? doneA : doneB) + i) & 1;
          // several at once: one latency where all are there, which is the rule for loads
          const bool there = mbar_test(&full[v.st], v.ph) & (!more || mbar_test(&full[k.st], k.ph)) & mbar_test(&p_full[s], ph);
          if (!there) {
            landed(v);
            if (more) landed(k);
            ok = ok && mbar_poll(&p_full[s], ph, &abort_flag);
          }
          // the item before has to be out of the accumulator
          if (i == 0 && items > 0) ok = ok && mbar_poll(&o_empty[s], static_cast<uint32_t>(items - 1) & 1, &abort_flag);
          if (!ok) return;
          tc_fence_after();
          if (more) --left;
          issue_pv(s, v, i == 0);
          if (!more) mma_commit(&o_full[s]);
          if (release_v) mma_commit(&empty[v.st]);
          if (more) {
            issue_s(s, k);
            if (release_k) mma_commit(&empty[k.st]);
            if (left == 0) mma_commit(q_empty);
          }
        };
        // kApart: S of the stream's block behind the i-th one, once that one's S has been read
        auto next_s = [&](int s, int i, const Cursor& k, bool release) {
          landed(k);
          ok = ok && mbar_poll(&s_read[s], static_cast<uint32_t>((s == 0 ? doneA : doneB) + i) & 1, &abort_flag);
          if (!ok) return;
          tc_fence_after();
          issue_s(s, k);
          if (release) mma_commit(&empty[k.st]);
          if (--left == 0) mma_commit(q_empty);
        };
        auto pv = [&](int s, int i, const Cursor& v, bool release) {
          landed(v);
          ok = ok && mbar_poll(&p_full[s], static_cast<uint32_t>((s == 0 ? doneA : doneB) + i) & 1, &abort_flag);
          // the item before has to be out of the accumulator
          if (i == 0 && items > 0) ok = ok && mbar_poll(&o_empty[s], static_cast<uint32_t>(items - 1) & 1, &abort_flag);
          if (!ok) return;
          tc_fence_after();
          issue_pv(s, v, i == 0);
          mma_commit(&o_full[s]);
          if (release) mma_commit(&empty[v.st]);
        };
        ok = mbar_poll(q_full, static_cast<uint32_t>(loaded) & 1, &abort_flag);
        ++loaded;
        const Cursor k0 = at;
        at.step();
        const Cursor k1 = at;
        landed(k0);
        if (kLead > 1 && cnt > 1) {
          at.step();
          if (!kTwo) landed(k1);
        }
        Cursor kn = kTwo ? k1 : at;  // kApart: the block of K for the next S
        if (kLead > 2 && cnt > 2) at.step();
        tc_fence_after();
        left -= kTwo ? (nA > 0) + (nB > 0) : (cnt > 1 ? 2 : 1);
        if (ok) {
          if constexpr (kTwo) {
            if (nA > 0) issue_s(0, k0);
            if (nB > 0) issue_s(1, k0);
            mma_commit(&empty[k0.st]);
          } else {
            issue_s(0, k0);
            mma_commit(&empty[k0.st]);
            if (cnt > 1) {
              issue_s(1, k1);
              mma_commit(&empty[k1.st]);
            }
          }
          if (left == 0) mma_commit(q_empty);
        }
        for (int j = 0; ok && j < cnt; ++j) {
          if (j == cnt - 1 && tail < kKeys) {
            ok = mbar_poll(&tail_done[w], static_cast<uint32_t>(tails >> w) & 1, &abort_flag);
            tails ^= 1 << w;
          }
          const Cursor v = at;
          at.step();
          const Cursor k = at;
          if (j + kLead < cnt) at.step();
          if constexpr (kApart) {
            constexpr int kStep = kTwo ? 1 : 2;
            if (ok && j + kStep < cnt) {
              if constexpr (kTwo) {
                if (j + 1 < nA) next_s(0, j, kn, j + 1 >= nB);
                if (ok && j + 1 < nB) next_s(1, j, kn, true);
              } else {
                next_s(j & 1, j >> 1, kn, true);
              }
              kn = k;
            }
            if constexpr (kTwo) {
              if (ok && j < nA) pv(0, j, v, j >= nB);
              if (ok && j < nB) pv(1, j, v, true);
            } else {
              if (ok) pv(j & 1, j >> 1, v, true);
            }
          } else if constexpr (kTwo) {  // the last stream that walks a block releases it
            if (ok && j < nA) turn(0, j, v, k, j + 1 < nA, j >= nB, j + 1 >= nB);
            if (ok && j < nB) turn(1, j, v, k, j + 1 < nB, true, true);
          } else {
            if (ok) turn(j & 1, j >> 1, v, k, j + 2 < cnt, true, true);
          }
        }
        doneA += nA;
        doneB += nB;
      }
      mbar_arrive(&work_empty[w]);
    }
    if (!ok) report_error(p.a.err, kErrWaitTimeout, &abort_flag);
    // every MMA issued has finished before the CTA frees TMEM and shared memory
    mma_commit(end_bar);
    mbar_wait(end_bar, 0, nullptr);
    }
  } else {
    // ---------------- softmax, half a row a thread ----------------
    const int s = warp >> 3, qd = warp & 3, hf = (warp >> 2) & 1;
    const int r = 32 * qd + lane;
    const uint32_t tl = tbase + (static_cast<uint32_t>(32 * qd) << 16);
    const uint32_t tS = tl + s * kKeys + 64 * hf, tP = tl + kColP + s * kStepP + kHalfP * hf, tO = tl + kColO + s * D + (D / 2) * hf;
    const int pair_bar = 1 + 4 * s + qd;  // named barrier of the two warps of these rows
    float* mx_own = reinterpret_cast<float*>(sm + Sh::kOffMax) + (2 * s + hf) * kRows + r;
    float* mx_other = reinterpret_cast<float*>(sm + Sh::kOffMax) + (2 * s + (hf ^ 1)) * kRows + r;
    const int rt = r / p.G;
    const float sl2 = p.scale_log2;
    if constexpr (!kPrefix) {
      if (blockIdx.x == 0 && blockIdx.y == 0) {  // one block looks every sequence over, while its first loads run
        bool bad = false;
#pragma unroll 4
        for (int64_t i = threadIdx.x; i < p.a.B; i += 32 * kSoftWarps) bad |= !sequence_ok(p.a, i);
        if (bad) atomicOr(p.a.err, kErrBadLength);
      }
    }
    bool ok = true;
    int done = 0, outs = 0;  // blocks of earlier items; earlier items with blocks
    for (int items = 0;; ++items) {
      const int w = items & 1;
      ok = ok && warp_wait(&work_full[w], static_cast<uint32_t>(items >> 1) & 1, &abort_flag);
      // the warps that meet at barriers below go on together or leave together
      if (kTwo ? wg_barrier_any<256>(9 + s, !ok) : wg_barrier_any<512>(9, !ok)) {
        ok = false;
        break;
      }
      const Work* o = work_at(w);
      const int cnt = o->cnt, n = s == 0 ? o->nA : o->nB;
      if (cnt < 0) break;
      int lim, whole;
      {
        Item it;
        it.tok_end = o->tok_end;
        it.lk = o->lk;
        const int tok = o->tok + (kTwo ? s * p.nt : 0) + rt;
        const bool valid = rt < p.nt && tok < it.tok_end;
        // keys this row sees, counted from the split's first block
        lim = max(0, (valid ? visible<kPrefix>(it, tok) : 0) - o->b0 * kKeys);
        whole = __reduce_min_sync(0xFFFFFFFFu, valid ? lim : 0x7FFFFFFF);  // the warp's rows see all keys below
      }
      float ref = -INFINITY, l = 0.0f;
      for (int i = 0; i < n; ++i) {
        const int j = kTwo ? i : 2 * i + s;  // block, counted from b0
        // a wait that gave up is met by all warps of a stream: each goes on to the pair's barrier
        ok = ok && warp_wait(&s_full[s], static_cast<uint32_t>(done + i) & 1, &abort_flag);
        tc_fence_after();
        uint32_t x[2][32];
#pragma unroll
        for (int c = 0; c < 2; ++c) tmem_ld_32x32b_x32(tS + 32 * c, x[c]);
        tmem_ld_wait();
        if constexpr (kApart) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_read[s]);
        }
        if ((j + 1) * kKeys > whole) {
          const int rem = lim - j * kKeys - 64 * hf;
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (32 * c + e >= rem) x[c][e] = 0xFF800000u;  // -inf
        }
        float m4[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          m4[c] = __uint_as_float(x[c >> 1][16 * (c & 1)]);
#pragma unroll
          for (int e = 1; e < 16; ++e) m4[c] = fmaxf(m4[c], __uint_as_float(x[c >> 1][16 * (c & 1) + e]));
        }
        const float mine = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        // Nearly always the reference of the earlier blocks serves: no row of either half is more
        // than 2^8 above it.  Only where one is do the halves exchange their maxima.  (The next
        // block's may overwrite them: both warps have met at its barrier then, and so have read these.)
        float alpha = 1.0f;
        const bool any = wg_barrier_any<64>(pair_bar, mine * sl2 > ref + kRescaleLog2);
        if (any) {
          *mx_own = mine;
          asm volatile("bar.sync %0, 64;" ::"r"(pair_bar) : "memory");
          const float mn = fmaxf(mine, *mx_other) * sl2;
          if (mn > ref + kRescaleLog2) {  // the first block with a visible key always
            alpha = ex2(ref - mn);        // 0 on the first
            ref = mn;
          }
        }
        const float base = ref == -INFINITY ? 0.0f : ref;  // no key seen so far: every weight is 2^-inf = 0
        const float2 sc2 = make_float2(sl2, sl2), nb2 = make_float2(-base, -base);
        float2 sum2 = make_float2(0.0f, 0.0f);
        uint32_t pk2[kApart ? 2 : 1][16];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t (&pk)[16] = pk2[kApart ? c : 0];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float2 t = __ffma2_rn(make_float2(__uint_as_float(x[c][2 * e]), __uint_as_float(x[c][2 * e + 1])), sc2, nb2);
            t.x = ex2(t.x);
            t.y = ex2(t.y);
            sum2 = __fadd2_rn(sum2, t);
            pk[e] = pack_bf16(t.x, t.y);
          }
          if (!kApart) tmem_st_32x32b_x16(tP + 16 * c, pk);
        }
        if constexpr (kApart) {  // the P V before has read its P, and O holds it
          if (i > 0) {
            ok = ok && warp_wait(&o_full[s], static_cast<uint32_t>(done + i - 1) & 1, &abort_flag);
            tc_fence_after();
          }
          tmem_st_32x32b_x16(tP, pk2[0]);
          tmem_st_32x32b_x16(tP + 16, pk2[kApart ? 1 : 0]);
        }
        l = fmaf(l, alpha, sum2.x + sum2.y);
        if (any && i > 0) {
          // a row's reference moved: scale its O (half of it in each warp), which holds all
          // earlier P V (they were done before this S was)
#pragma unroll 1
          for (int c = 0; c < D / 2; c += 32) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(tO + c, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st_32x32b_x32(tO + c, o);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[s]);
      }
      done += n;
      if (ok && n > 0) {  // the stream's products are done
        ok = warp_wait(&o_full[s], static_cast<uint32_t>(kApart ? done - 1 : outs) & 1, &abort_flag);
        tc_fence_after();
      }
      outs += n > 0 ? 1 : 0;
      // the row's sum: both halves'
      *mx_own = l;
      asm volatile("bar.sync %0, 64;" ::"r"(pair_bar) : "memory");
      l += *mx_other;
      asm volatile("bar.sync %0, 64;" ::"r"(pair_bar) : "memory");
      float scale = 1.0f, other_scale = 0.0f;
      const bool both = !kTwo && o->nB > 0;  // the other stream has an O of these rows too
      if constexpr (!kTwo) {
        // the two streams' references and sums; stream A then reads both accumulators
        float2* ml = reinterpret_cast<float2*>(sm + Sh::kOffMax);
        asm volatile("bar.sync 9, 512;" ::: "memory");  // the sums' places are free now
        if (hf == 0) ml[s * kRows + r] = make_float2(n > 0 ? ref : -INFINITY, n > 0 ? l : 0.0f);
        asm volatile("bar.sync 9, 512;" ::: "memory");
        const float2 other = ml[(s ^ 1) * kRows + r];
        const float top = fmaxf(ref, other.x);
        scale = ref == -INFINITY ? 0.0f : ex2(ref - top);
        other_scale = other.x == -INFINITY ? 0.0f : ex2(other.x - top);
        l = l * scale + other.y * other_scale;
        ref = top;
        asm volatile("bar.sync 9, 512;" ::: "memory");  // read before the next item's maxima come
      }
      if (kTwo || s == 0) {
        const int tok = o->tok + (kTwo ? s * p.nt : 0) + rt;
        const bool valid = rt < p.nt && tok < o->tok_end;
        const int head = o->hk * p.G + (r - rt * p.G);
        const bool final_out = p.to_parts == 0;
        const bool saw = l > 0.0f || l != l;
        // A row without a key is 0, whatever is in the V that its tile's other rows see (its
        // accumulator has 0 V, NaN where V is not finite); looked at a warp at a time
        const bool all_saw = __all_sync(0xFFFFFFFFu, saw);
        const float over = final_out && saw ? 1.0f / l : 1.0f;
        const float inv = scale * over, inv_other = other_scale * over;
        const int64_t row = static_cast<int64_t>(o->split) * p.a.Tq * p.a.H + static_cast<int64_t>(tok) * p.a.H + head;
        if (!final_out && valid && cnt > 0 && hf == 0) p.part_ml[row] = make_float2(ref, l);
        // where this lane's half row goes
        const uint64_t at = final_out ? reinterpret_cast<uint64_t>(p.a.o + tok * p.a.st[6] + head * p.a.st[7] + (D / 2) * hf)
                                      : reinterpret_cast<uint64_t>(p.part_o + row * D + (D / 2) * hf);
        const unsigned rows = __ballot_sync(0xFFFFFFFFu, valid && (final_out || cnt > 0));
        // kN pieces of 16 bytes of every row, from byte `from` on: transposed among kN lanes, so
        // that a store covers whole lines (one row a lane would take a store 32 lines)
        auto put = [&](auto& v, int from) {
          constexpr int kN = sizeof(v) / 16;
          transpose_pieces<kN>(v, lane);
#pragma unroll
          for (int e = 0; e < kN; ++e) {
            const int from_lane = (lane & ~(kN - 1)) + e;  // whose row this piece belongs to
            const uint64_t to = __shfl_sync(0xFFFFFFFFu, at, from_lane) + static_cast<uint64_t>(from + 16 * (lane & (kN - 1)));
            if ((rows >> from_lane) & 1u) *reinterpret_cast<uint4*>(to) = v[e];
          }
        };
        auto channels = [&](int c, float (&f)[32]) {  // 32 of this lane's, from c on
          if (ok && n > 0) {
            uint32_t t[32];
            tmem_ld_32x32b_x32(tO + c, t);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(t[e]) * inv;
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) f[e] = 0.0f;  // no key: 0
          }
          if (both && ok) {
            uint32_t t[32];
            tmem_ld_32x32b_x32(tO + D + c, t);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) f[e] = fmaf(__uint_as_float(t[e]), inv_other, f[e]);
          }
          if (!all_saw) {
#pragma unroll
            for (int e = 0; e < 32; ++e) f[e] = saw ? f[e] : 0.0f;
          }
        };
        if (final_out) {
          uint4 v[D / 16];
#pragma unroll
          for (int c = 0; c < D / 2; c += 32) {
            float f[32];
            channels(c, f);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              v[c / 8 + e] = make_uint4(pack_bf16(f[8 * e], f[8 * e + 1]), pack_bf16(f[8 * e + 2], f[8 * e + 3]),
                                        pack_bf16(f[8 * e + 4], f[8 * e + 5]), pack_bf16(f[8 * e + 6], f[8 * e + 7]));
          }
          put(v, 0);
        } else if (cnt > 0) {
#pragma unroll 1
          for (int c = 0; c < D / 2; c += 32) {
            float f[32];
            channels(c, f);
            uint4 v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              v[e] = make_uint4(__float_as_uint(f[4 * e]), __float_as_uint(f[4 * e + 1]), __float_as_uint(f[4 * e + 2]),
                                __float_as_uint(f[4 * e + 3]));
            put(v, 4 * c);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&o_empty[s]);
          if (!kTwo) mbar_arrive(&o_empty[1]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&work_empty[w]);
    }
    if (!ok) report_error(p.a.err, kErrWaitTimeout, &abort_flag);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kSoftWarps + 1) tmem_dealloc(tbase, 512);
}

// ---- joining the splits of a row -----------------------------------------------------------
// o = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s, one warp a row.
// `place` gives the row of a split.  A warp takes the splits from, from + step, ...: their
// references and sums are read by the lanes, their rows four at a time.
template <int D, typename F>
__device__ __forceinline__ void join_parts(int used, int from, int step, int lane, const float2* ml, const float* o,
                                           F place, float& l, float (&acc)[D / 32]) {
  constexpr int E = D / 32;
  float top = -INFINITY;  // of all splits
  for (int s = lane; s < used; s += 32) top = fmaxf(top, ml[place(s)].x);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
  l = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.0f;
  for (int s0 = from; s0 < used; s0 += 32 * step) {
    float w = 0.0f, sum = 0.0f;  // this lane's split
    if (s0 + lane * step < used) {
      const float2 v = ml[place(s0 + lane * step)];
      w = v.x == -INFINITY && v.y == 0.0f ? 0.0f : ex2(v.x - top);
      sum = v.y * w;
    }
    const int n = min(32, (used - s0 + step - 1) / step);
#pragma unroll 4
    for (int s = 0; s < n; ++s) {
      const float ws = __shfl_sync(0xFFFFFFFFu, w, s);
      const float* src = o + place(s0 + s * step) * D + E * lane;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(src[e], ws, acc[e]);
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, x);
    l += sum;
  }
}

// The splits of a prompt's rows (one tile a block: two are only taken where nothing is split).
template <int D>
__global__ void __launch_bounds__(256) prompt_join_kernel(const __grid_constant__ TileParams p) {
  constexpr int E = D / 32;
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int hk = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.a.Hkv));
  const int slot = static_cast<int>(p.nslots) - 1 - static_cast<int>(blockIdx.x / static_cast<unsigned>(p.a.Hkv));
  Item it;
  const bool found = prompt_item(p.a, slot, p.nt, lane, &it);
  pdl_wait();  // in every block: what follows on the stream has to find the tiles done
  if (!found) return;
  const int nb = tile_blocks<false>(it, it.tok, p.nt);
  const int per = blocks_per_split(nb, p.splits), used = per > 0 ? (nb + per - 1) / per : 0;
  const int64_t rows = p.a.Tq * p.a.H;
  const int r = static_cast<int>(blockIdx.y) * 8 + warp;
  const int64_t tok = it.tok + r / p.G;
  if (r < p.nt * p.G && tok < it.tok_end) {
    const int64_t head = hk * p.G + r % p.G, row = tok * p.a.H + head;
    float l, acc[E];
    join_parts<D>(used, 0, 1, lane, p.part_ml, p.part_o, [&](int s) { return s * rows + row; }, l, acc);
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.a.o + tok * p.a.st[6] + head * p.a.st[7] + E * lane);
#pragma unroll
    for (int e = 0; e < E; e += 2) dst[e / 2] = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
  }
}

// ---- the requests' own keys ---------------------------------------------------------------
// Few rows (the G heads of one request) over keys that no other request reads: bound by the
// bytes of the cache.  One CTA for a request, a key/value head, 16 of its query heads and a
// range of keys; each of its four warps walks 16-key pieces of that range by itself (pieces w,
// w + 4, ...) with a ring of asynchronous copies of its own, so the loop has no barrier, and
// three CTAs on an SM keep 192 KB in flight.  The products run on mma.sync: 16 rows are all
// there is, and the tensor pipe is not what bounds this.  Rows behind the request's keys are
// not read (zeros are filled in).
// Long caches are read at the copy rate (32/8 heads of 128: 64 requests with 4096 keys 161
// us, 6.7 TB/s; 8 with 65536 309 us, 6.9 TB/s), short ones below it (64 with 512: 28 us, 4.8
// TB/s); with two warps a block and six blocks an SM, 64 requests with up to 512 keys took 24.6 us
// instead of 16.2.
// kAlone: no other kernel works on this call.  The prefix, short or of one request only, is
// walked here in front of the own keys, and the CTAs that share a row's keys are a cluster
// that joins them through its shared memory: one launch and no workspace.
constexpr int kOwnWarps = 4, kOwnKeys = 16, kOwnStages = 2, kOwnRows = 16;

struct OwnParams {
  PrefixArgs a;
  int G, chunks;   // heads of a group; 16-head chunks of it
  int splits;      // at most so many CTAs share a request's keys (alone: a cluster of exactly so many)
  int prefix_splits;  // partial results of the prefix
  float scale_log2;
  float* part_o;    // [prefix_splits + splits][B * H][D]
  float2* part_ml;
};

template <int D>
struct OwnShape {
  static constexpr int kPiece = kOwnKeys * D * 2;                 // K or V of a piece
  static constexpr int kWarp = kOwnStages * 2 * kPiece;           // a warp's ring
  static constexpr int kSmem = kOwnWarps * kWarp;
  static constexpr int kPad = D + 4;                              // floats of an exchanged row
  static_assert(kWarp >= kOwnRows * kPad * 4, "exchange buffer");
};

// Keys of a split of a request with n keys (whole pieces for every warp).
__device__ __forceinline__ int64_t own_per_split(int64_t n, int splits) {
  constexpr int64_t kUnit = kOwnWarps * kOwnKeys;
  const int64_t per = (n + splits - 1) / splits;
  return (per + kUnit - 1) / kUnit * kUnit;
}

__device__ __forceinline__ int64_t own_length(const PrefixArgs& a, int64_t b) {
  const int64_t n = a.own_len[b];
  return n < 0 ? 0 : n < a.cap ? n : a.cap;
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <int D, bool kAlone>
__global__ void __launch_bounds__(32 * kOwnWarps, 3) attn_own_kernel(const __grid_constant__ OwnParams p) {
  using Sh = OwnShape<D>;
  constexpr int KS = D / 16, C16 = D / 8;  // k steps of a score; 16-byte chunks of a row
  if constexpr (!kAlone) pdl_launch_dependents();
  extern __shared__ __align__(1024) uint8_t sm[];
  __shared__ float2 ml_s[kOwnWarps][kOwnRows];
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int g = lane >> 2, t = lane & 3;
  const PrefixArgs& a = p.a;
  const unsigned per_b = static_cast<unsigned>(a.Hkv) * static_cast<unsigned>(p.chunks);
  const int64_t b = blockIdx.x / per_b;
  const int rem = static_cast<int>(blockIdx.x - static_cast<unsigned>(b) * per_b);
  const int hk = rem / p.chunks, chunk = rem - hk * p.chunks, split = static_cast<int>(blockIdx.y);
  const int64_t shared = kAlone ? a.P : 0;  // keys of the prefix, in front
  const int64_t own = own_length(a, b), n = shared + own, per = own_per_split(n, p.splits);
  if (threadIdx.x == 0 && rem == 0 && split == 0 && own != a.own_len[b]) atomicOr(a.err, kErrBadLength);
  const int64_t k0 = split * per, k1 = k0 + per < n ? k0 + per : n;
  if (!kAlone && k0 >= k1) {
    pdl_wait();
    return;
  }
  const int nrows = p.G - chunk * kOwnRows < kOwnRows ? p.G - chunk * kOwnRows : kOwnRows;
  const int64_t head0 = static_cast<int64_t>(hk) * p.G + chunk * kOwnRows;
  const int npieces = k1 > k0 ? static_cast<int>((k1 - k0 + kOwnKeys - 1) / kOwnKeys) : 0;
  const int mine = npieces > warp ? (npieces - warp + kOwnWarps - 1) / kOwnWarps : 0;
  uint8_t* ring = sm + warp * Sh::kWarp;
  const uint16_t* kbase = a.ko + b * a.st[6] + hk * a.st[8];
  const uint16_t* vbase = a.vo + b * a.st[9] + hk * a.st[11];
  const uint16_t* kshared = a.kp + hk * a.st[3];
  const uint16_t* vshared = a.vp + hk * a.st[5];
  auto load = [&](int i) {  // the warp's i-th piece
    if (i < mine) {
      uint8_t* dst = ring + (i % kOwnStages) * 2 * Sh::kPiece;
      const int64_t key = k0 + static_cast<int64_t>(warp + i * kOwnWarps) * kOwnKeys;
#pragma unroll
      for (int c = lane; c < kOwnKeys * C16; c += 32) {
        const int row = c / C16, col = c % C16;
        const bool on = key + row < k1;
        const int64_t at = on ? key + row : k0;  // a key of this range stands in where none is read
        const int off = row * D * 2 + ((col ^ (row & 7)) << 4);
        const uint16_t *ks, *vs;
        if (kAlone && at < shared) {
          ks = kshared + at * a.st[2];
          vs = vshared + at * a.st[4];
        } else {
          ks = kbase + (at - shared) * a.st[7];
          vs = vbase + (at - shared) * a.st[10];
        }
        cp_async16(dst + off, ks + 8 * col, on);
        cp_async16(dst + Sh::kPiece + off, vs + 8 * col, on);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kOwnStages; ++i) load(i);
  // Q: rows g and g + 8 of the 16, zeros behind the group
  uint32_t q[KS][4];
  {
    const uint16_t* q0 = a.q + b * a.st[0] + (head0 + g) * a.st[1] + 2 * t;
    const uint16_t* q8 = q0 + 8 * a.st[1];
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      q[k][0] = g < nrows ? *reinterpret_cast<const uint32_t*>(q0 + 16 * k) : 0u;
      q[k][1] = g + 8 < nrows ? *reinterpret_cast<const uint32_t*>(q8 + 16 * k) : 0u;
      q[k][2] = g < nrows ? *reinterpret_cast<const uint32_t*>(q0 + 16 * k + 8) : 0u;
      q[k][3] = g + 8 < nrows ? *reinterpret_cast<const uint32_t*>(q8 + 16 * k + 8) : 0u;
    }
  }
  float o[D / 8][4] = {};
  float ref[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
  const float sl2 = p.scale_log2;
  // a lane's row in an ldmatrix of four 8 x 8 matrices: keys (lane & 7) + 8 [bit], chunk [bit]
  const int krow = (lane & 7) + ((lane >> 4) << 3), kbit = (lane >> 3) & 1;   // K: matrices (k lo, k hi) x keys
  const int vrow = (lane & 7) + (((lane >> 3) & 1) << 3), vbit = lane >> 4;   // V: matrices (keys lo, hi) x channels
  for (int i = 0; i < mine; ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kOwnStages - 1) : "memory");
    __syncwarp();
    const uint32_t ks = smem_u32(ring + (i % kOwnStages) * 2 * Sh::kPiece), vs = ks + Sh::kPiece;
    float s[2][4] = {};
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      uint32_t r[4];
      ldmatrix_x4(r, ks + krow * D * 2 + (((2 * k + kbit) ^ (krow & 7)) << 4));
      mma_16816(s[0], q[k], r[0], r[1]);
      mma_16816(s[1], q[k], r[2], r[3]);
    }
    const int64_t left = k1 - (k0 + static_cast<int64_t>(warp + i * kOwnWarps) * kOwnKeys);
    if (left < kOwnKeys) {
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (8 * x + 2 * t + (e & 1) >= left) s[x][e] = -INFINITY;
    }
    float alpha[2], base[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float m = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
      m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2)) * sl2;
      alpha[h] = 1.0f;
      if (m > ref[h]) {
        alpha[h] = ex2(ref[h] - m);
        ref[h] = m;
      }
      base[h] = ref[h] == -INFINITY ? 0.0f : ref[h];  // scores of -inf only: every weight is 0
    }
    uint32_t pa[4];
    float w[2][4];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) w[x][e] = ex2(fmaf(s[x][e], sl2, -base[e >> 1]));
#pragma unroll
    for (int h = 0; h < 2; ++h)
      l[h] = fmaf(l[h], alpha[h], (w[0][2 * h] + w[0][2 * h + 1]) + (w[1][2 * h] + w[1][2 * h + 1]));
    pa[0] = pack_bf16(w[0][0], w[0][1]);
    pa[1] = pack_bf16(w[0][2], w[0][3]);
    pa[2] = pack_bf16(w[1][0], w[1][1]);
    pa[3] = pack_bf16(w[1][2], w[1][3]);
    if (__any_sync(0xFFFFFFFFu, alpha[0] != 1.0f || alpha[1] != 1.0f)) {
#pragma unroll
      for (int c = 0; c < D / 8; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[c][e] *= alpha[e >> 1];
    }
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      uint32_t r[4];
      ldmatrix_x4_trans(r, vs + vrow * D * 2 + (((2 * c + vbit) ^ (vrow & 7)) << 4));
      mma_16816(o[2 * c], pa, r[0], r[1]);
      mma_16816(o[2 * c + 1], pa, r[2], r[3]);
    }
    __syncwarp();  // every lane has read the stage
    load(i + kOwnStages);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
  // the warps' results meet in shared memory, each in its own ring
  float* mineo = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 1);
    l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 2);
    if (t == 0) ml_s[warp][g + 8 * h] = make_float2(ref[h], l[h]);
    if (g + 8 * h < nrows) {
#pragma unroll
      for (int c = 0; c < D / 8; ++c)
        *reinterpret_cast<float2*>(mineo + (g + 8 * h) * Sh::kPad + 8 * c + 2 * t) = make_float2(o[c][2 * h], o[c][2 * h + 1]);
    }
  }
  constexpr int E = D / 32;
  // (reference, sum, the lane's channels) of a row from the four warps of a CTA
  auto join_warps = [&](int r, float& top, float& sum, float (&acc)[E]) {
    top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kOwnWarps; ++w) top = fmaxf(top, ml_s[w][r].x);
    sum = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
#pragma unroll
    for (int w = 0; w < kOwnWarps; ++w) {
      const float2 ml = ml_s[w][r];
      if (ml.x == -INFINITY && ml.y == 0.0f) continue;  // a warp without a piece
      const float f = ex2(ml.x - top);
      sum = fmaf(ml.y, f, sum);
      const float* src = reinterpret_cast<const float*>(sm + w * Sh::kWarp) + r * Sh::kPad + E * lane;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(src[e], f, acc[e]);
    }
  };
  __syncthreads();
  if constexpr (kAlone) {
    // each CTA joins its warps into warp 0's place, then the cluster's CTAs share the rows
    for (int r = warp; r < nrows; r += kOwnWarps) {
      float top, sum, acc[E];
      join_warps(r, top, sum, acc);
      __syncwarp();  // every lane has read the row before it is overwritten
      float* dst = reinterpret_cast<float*>(sm) + r * Sh::kPad + E * lane;
#pragma unroll
      for (int e = 0; e < E; ++e) dst[e] = acc[e];
      if (lane == 0) ml_s[0][r] = make_float2(top, sum);
    }
    cluster_sync();
    for (int r = split * kOwnWarps + warp; r < nrows; r += p.splits * kOwnWarps) {
      float top = -INFINITY, sum = 0.0f, acc[E] = {};
      for (int x = 0; x < p.splits; ++x) top = fmaxf(top, peer_load(&ml_s[0][r].x, x));
      for (int x = 0; x < p.splits; ++x) {
        const float m = peer_load(&ml_s[0][r].x, x), l1 = peer_load(&ml_s[0][r].y, x);
        if (m == -INFINITY && l1 == 0.0f) continue;  // a CTA without keys
        const float f = ex2(m - top);
        sum = fmaf(l1, f, sum);
        const float* src = reinterpret_cast<const float*>(sm) + r * Sh::kPad + E * lane;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(peer_load(src + e, x), f, acc[e]);
      }
      const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
      uint32_t* dst = reinterpret_cast<uint32_t*>(a.o + b * a.st[12] + (head0 + r) * a.st[13] + E * lane);
#pragma unroll
      for (int e = 0; e < E; e += 2) dst[e / 2] = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
    }
    cluster_sync();  // no CTA leaves while another reads its shared memory
  } else {
    for (int r = warp; r < nrows; r += kOwnWarps) {
      float top, sum, acc[E];
      join_warps(r, top, sum, acc);
      const int64_t at = static_cast<int64_t>(p.prefix_splits + split) * a.B * a.H + b * a.H + head0 + r;
      if (lane == 0) p.part_ml[at] = make_float2(top, sum);
#pragma unroll
      for (int e = 0; e < E; e += 2)
        *reinterpret_cast<float2*>(p.part_o + at * D + E * lane + e) = make_float2(acc[e], acc[e + 1]);
    }
    pdl_wait();  // the join waits for this kernel only: it has to end after the prefix's
  }
}

// A row's partial results: the splits of the prefix, then those of the request's own keys.  kW warps
// a row, each with every kW-th split.
template <int kW>
constexpr int kJoinWarps = kW < 4 ? 4 : kW;  // of a block
template <int D, int kW>
__global__ void __launch_bounds__(32 * kJoinWarps<kW>) prefix_join_kernel(const __grid_constant__ OwnParams p) {
  constexpr int E = D / 32, kWarps = kJoinWarps<kW>;
  __shared__ float acc_s[kWarps][D];
  __shared__ float l_s[kWarps];
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int w = warp % kW, w0 = warp - w;  // of the row's warps; the first one
  const PrefixArgs& a = p.a;
  const int64_t rows = a.B * a.H, row = static_cast<int64_t>(blockIdx.x) * (kWarps / kW) + warp / kW;
  const int64_t b = row / a.H, head = row - b * a.H;
  int used = 0;
  if (row < rows) {
    const int64_t n = own_length(a, b), per = own_per_split(n, p.splits);
    used = p.prefix_splits + (per > 0 ? static_cast<int>((n + per - 1) / per) : 0);
  }
  pdl_wait();
  float l, acc[E];
  join_parts<D>(used, w, kW, lane, p.part_ml, p.part_o, [&](int s) { return s * rows + row; }, l, acc);
#pragma unroll
  for (int e = 0; e < E; ++e) acc_s[warp][E * lane + e] = acc[e];
  if (lane == 0) l_s[warp] = l;
  if (kW > 1) __syncthreads();
  else __syncwarp();
  for (int c = 2 * (32 * w + lane); row < rows && c < D; c += 64 * kW) {
    float sum = 0.0f, x = 0.0f, y = 0.0f;
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      sum += l_s[w0 + i];
      x += acc_s[w0 + i][c];
      y += acc_s[w0 + i][c + 1];
    }
    const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
    *reinterpret_cast<uint32_t*>(a.o + b * a.st[12] + head * a.st[13] + c) = pack_bf16(x * inv, y * inv);
  }
}

// ---- host ----------------------------------------------------------------------------------
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn attn_encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

// [tokens][heads][d] bfloat16 with the given strides, loaded as 64 channels x bh heads x bt
// tokens with 128-byte swizzle.  A dimension of one item gets a stride that any array has.
bool encode_rows(CUtensorMap* map, const void* ptr, int64_t d, int64_t heads, int64_t tokens, int64_t head_stride,
                 int64_t tok_stride, int bh, int bt) {
  EncodeTiledFn enc = attn_encode_fn();
  if (enc == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(heads > 1 ? head_stride : d) * 2,
                                 static_cast<cuuint64_t>(tokens > 1 ? tok_stride : d) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(bh), static_cast<cuuint32_t>(bt)}, estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A launch that may begin before the kernel in front of it has ended (dependent), or whose
// `cluster` blocks of the same grid column form a cluster.
template <typename K, typename... A>
cudaError_t launch_with(K kernel, dim3 grid, unsigned threads, size_t smem, bool dependent, int cluster,
                        cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  if (dependent) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = 1;
    attr[cfg.numAttrs].val.clusterDim.y = static_cast<unsigned>(cluster);
    attr[cfg.numAttrs++].val.clusterDim.z = 1;
  }
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int D, bool kTwo, bool kPrefix>
cudaError_t launch_tiles(TileParams& p, const DeviceInfo& dev, cudaStream_t stream) {
  const PromptArgs& a = p.a;
  CUtensorMap mq, mk, mv;
  p.k_head = a.Hkv > 1 && a.st[3] > 0;
  p.v_head = a.Hkv > 1 && a.st[5] > 0;
  const bool keys = a.Tk > 0;  // without any key nothing is loaded: the maps only have to be valid
  if (!encode_rows(&mq, a.q, D, a.H, a.Tq, a.st[1], a.st[0], p.G, p.nt) ||
      !encode_rows(&mk, keys ? a.k : a.q, D, p.k_head ? a.Hkv : 1, keys ? a.Tk : 1, a.st[3], a.st[2], 1, kKeys) ||
      !encode_rows(&mv, keys ? a.v : a.q, D, p.v_head ? a.Hkv : 1, keys ? a.Tk : 1, a.st[5], a.st[4], 1, kKeys))
    return cudaErrorInvalidValue;
  const auto kernel = attn_tile_kernel<D, kTwo, kPrefix>;
  constexpr uint32_t smem = TileShape<D, kTwo>::kSmem;
  const cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kernel), smem, dev.device);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(p.nslots * a.Hkv), static_cast<unsigned>(p.splits));
  kernel<<<grid, kTileThreads, smem, stream>>>(mq, mk, mv, p);
  return cudaGetLastError();
}

// How a prompt call is cut up.
struct PromptPlan {
  bool two;
  int64_t nslots;
  int splits;
};
PromptPlan prompt_plan(int64_t B, int64_t Tq, int64_t Tk, int64_t H, int64_t Hkv, const DeviceInfo& dev) {
  const int64_t nt = kRows / (H / Hkv);
  PromptPlan pl;
  // Two tiles a block where that still gives every SM one: K and V are then loaded once for 256
  // rows, and no O is joined (4 prompts of up to 1531 tokens, 16 heads of 64: 26 us, 28.7 with one
  // tile; 2 x 512 tokens behind 16384 cached ones, which make too few: 107 us with one tile, 114
  // with two and split keys)
  pl.two = (Tq / (2 * nt) + 1) * Hkv >= dev.sm_count;
  const int64_t n = pl.two ? 2 * nt : nt;
  pl.nslots = Tq / n + B;
  // Keys are split where the blocks in work leave SMs without any (a sequence counts as one block at
  // least: 64 single tokens of 2048 keys take 86 us so, 114 in two splits): four key blocks a split
  // at least (one token behind 2000 keys: 11.9 us, 14.2 with eight), sixteen splits at most (behind
  // 16384: 18.0, 19.5 with nineteen), and none of so few keys that two would do (128 tokens behind
  // 1000: 11.8 us, 13.7 in two)
  const int64_t busy = (Tq / n + std::min(B, Tq)) * Hkv, blocks = (Tk + kKeys - 1) / kKeys;
  pl.splits = blocks < 12 ? 1 : static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({dev.sm_count / busy, 16, blocks / 4})));
  return pl;
}

template <int D>
cudaError_t prompt_attention(const PromptArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  TileParams p = {};
  p.a = a;
  const PromptPlan pl = prompt_plan(a.B, a.Tq, a.Tk, a.H, a.Hkv, dev);
  p.G = static_cast<int>(a.H / a.Hkv);
  p.nt = kRows / p.G;
  p.nslots = pl.nslots;
  p.splits = pl.splits;
  p.to_parts = pl.splits > 1;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.part_o = static_cast<float*>(a.part);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + static_cast<int64_t>(pl.splits) * a.Tq * a.H * D);
  cudaError_t e = pl.two ? launch_tiles<D, true, false>(p, dev, stream) : launch_tiles<D, false, false>(p, dev, stream);
  if (e != cudaSuccess || pl.splits == 1) return e;
  // a warp a row (128 tokens behind 16384: 40.1 us, 45.4 with four rows a warp)
  const dim3 grid(static_cast<unsigned>(pl.nslots * a.Hkv), kRows / 8);
  return launch_with(prompt_join_kernel<D>, grid, 256, 0, true, 1, stream, p);
}

// How a prefix call is cut up.
struct PrefixPlan {
  bool two;                   // two tiles of requests a block
  int64_t nslots;
  int prefix_splits, own_splits, chunks;
  bool alone;                 // the own kernel walks the prefix too
  size_t partials() const { return alone ? 0 : static_cast<size_t>(prefix_splits + own_splits); }
};
PrefixPlan prefix_plan(int64_t B, int64_t P, int64_t cap, int64_t H, int64_t Hkv, const DeviceInfo& dev) {
  const int64_t G = H / Hkv, nt = kRows / G;
  PrefixPlan pl;
  // Two tiles a block only where one already fills the GPU twice: fewer blocks would have to split
  // the keys, and each split writes partial results (64 requests behind 8192 keys: 31 us a call
  // with one tile, 33 with two).  Beyond that K and V are loaded half as often (device time with two
  // tiles and one, 32/8 heads of 128: 1216 requests behind 1000 keys 111 and 117 us, 2432 behind
  // 8192 333 and 351; the other way round by 2 to 3 % for 2432 requests of 64-wide heads behind 8192,
  // 282 and 278, and 1000 of 40 heads behind 4000, 314 and 304)
  pl.two = (B + nt - 1) / nt * Hkv >= 2 * dev.sm_count;
  const int64_t n = pl.two ? 2 * nt : nt, blocks = (P + kKeys - 1) / kKeys;
  pl.nslots = (B + n - 1) / n;
  pl.chunks = static_cast<int>((G + kOwnRows - 1) / kOwnRows);
  const int64_t busy = B * Hkv * pl.chunks;
  // Alone: few shared keys are read again for every request, which costs less than a second and a
  // third launch where a block has few keys (device time: 1 request behind 1000 keys 8.0 us, 9.6 with
  // three launches; 16 with up to 100 own ones behind 256: 8.7 against 9.6).  Not where the cluster's
  // blocks or the SMs are too few for that (8 requests with up to 2000 keys: 13.1 us alone, 10.3 with
  // more blocks and a join), and with one block a row while it ends soon (256 requests with up to 300
  // keys: 25.3 us against 28.2; 64 with up to 512: 16.5 against 12.9)
  const int64_t keys = P + cap;
  const int64_t one = std::max<int64_t>(1, std::min<int64_t>({8, 3 * dev.sm_count / busy, (keys + 127) / 128}));
  pl.alone = B * P <= 4096 && keys <= one * (one > 1 ? 160 : 384);
  if (pl.alone) {
    pl.prefix_splits = 0;
    pl.own_splits = static_cast<int>(one);
    return pl;
  }
  const int64_t s = std::max<int64_t>(1, std::min(dev.sm_count / (pl.nslots * Hkv), blocks / 2));
  const int64_t per = (blocks + s - 1) / s;
  pl.prefix_splits = P > 0 ? static_cast<int>((blocks + per - 1) / per) : 0;
  // One wave of three blocks an SM; with more than a few requests, whose lengths differ, more and
  // smaller ones (256 keys of the longest each, 32 an SM, 64 results to join at most): those of
  // shorter requests end at once (64 requests with up to 4000 keys behind 8192: 51 us against 59
  // with one wave; 512 keys: 30 us with two a request, 31 with four; 1 request with 131072 keys:
  // 92 us with one wave, 109 with 64 splits)
  const int64_t few = 3 * dev.sm_count / busy;
  const int64_t many = std::min<int64_t>({cap / 256, 32 * dev.sm_count / busy, 64});
  pl.own_splits = static_cast<int>(std::max<int64_t>(1, std::min(few < 16 ? std::max(few, many) : few, cap / 128)));
  return pl;
}

template <int D>
cudaError_t prefix_attention(const PrefixArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  const PrefixPlan pl = prefix_plan(a.B, a.P, a.cap, a.H, a.Hkv, dev);
  float* part_o = static_cast<float*>(a.part);
  float2* part_ml = reinterpret_cast<float2*>(part_o + pl.partials() * a.B * a.H * D);
  const float scale_log2 = a.scale * 1.4426950408889634f;
  const int G = static_cast<int>(a.H / a.Hkv);
  cudaError_t e;
  const bool tiles = pl.prefix_splits > 0;
  if (tiles) {
    TileParams t = {};
    t.a.q = a.q;
    t.a.k = a.kp;
    t.a.v = a.vp;
    t.a.B = 1;
    t.a.Tq = a.B;
    t.a.Tk = a.P;
    t.a.H = a.H;
    t.a.Hkv = a.Hkv;
    t.a.d = D;
    std::copy(a.st, a.st + 6, t.a.st);
    t.a.err = a.err;
    t.G = G;
    t.nt = kRows / G;
    t.nslots = pl.nslots;
    t.splits = pl.prefix_splits;
    t.to_parts = 1;
    t.scale_log2 = scale_log2;
    t.part_o = part_o;
    t.part_ml = part_ml;
    e = pl.two ? launch_tiles<D, true, true>(t, dev, stream) : launch_tiles<D, false, true>(t, dev, stream);
    if (e != cudaSuccess) return e;
  }
  OwnParams p = {};
  p.a = a;
  p.G = G;
  p.chunks = pl.chunks;
  p.splits = pl.own_splits;
  p.prefix_splits = pl.prefix_splits;
  p.scale_log2 = scale_log2;
  p.part_o = part_o;
  p.part_ml = part_ml;
  constexpr int smem = OwnShape<D>::kSmem;
  const dim3 grid(static_cast<unsigned>(a.B * a.Hkv * pl.chunks), static_cast<unsigned>(pl.own_splits));
  if (pl.alone) {
    const auto kernel = attn_own_kernel<D, true>;
    if ((e = ensure_smem(reinterpret_cast<const void*>(kernel), smem, dev.device)) != cudaSuccess) return e;
    return launch_with(kernel, grid, 32 * kOwnWarps, smem, false, pl.own_splits, stream, p);
  }
  const auto kernel = attn_own_kernel<D, false>;
  if ((e = ensure_smem(reinterpret_cast<const void*>(kernel), smem, dev.device)) != cudaSuccess) return e;
  if ((e = launch_with(kernel, grid, 32 * kOwnWarps, smem, tiles, 1, stream, p)) != cudaSuccess) return e;
  // Warps of a row: no more than its results (four at least), and one wave of warps in all (device
  // time, 8 requests with up to 16000 keys: 34.5 us with sixteen, 36.9 with four, 49.8 with one; 300
  // with up to 1000 behind 1000: 58.1 with one, 63.0 with four, 92.4 with sixteen)
  const int64_t rows = a.B * a.H;
  const int64_t most = std::min<int64_t>(64 * dev.sm_count / rows, std::max<int64_t>(4, static_cast<int64_t>(pl.partials())));
  auto join = [&](auto w) {
    constexpr int kW = decltype(w)::value, kWarps = kJoinWarps<kW>;
    return launch_with(prefix_join_kernel<D, kW>, dim3(static_cast<unsigned>((rows * kW + kWarps - 1) / kWarps)),
                       32 * kWarps, 0, true, 1, stream, p);
  };
  if (most >= 16) return join(std::integral_constant<int, 16>{});
  if (most >= 8) return join(std::integral_constant<int, 8>{});
  if (most >= 4) return join(std::integral_constant<int, 4>{});
  return join(std::integral_constant<int, 1>{});
}

}  // namespace

size_t prompt_ws_bytes(int64_t B, int64_t Tq, int64_t Tk, int64_t H, int64_t Hkv, int64_t d, const DeviceInfo& dev) {
  const int64_t splits = prompt_plan(B, Tq, Tk, H, Hkv, dev).splits;
  return splits == 1 ? 0 : static_cast<size_t>(splits * Tq * H * (d + 2)) * 4;
}
size_t prefix_ws_bytes(int64_t B, int64_t P, int64_t cap, int64_t H, int64_t Hkv, int64_t d, const DeviceInfo& dev) {
  return prefix_plan(B, P, cap, H, Hkv, dev).partials() * static_cast<size_t>(B * H * (d + 2)) * 4;
}

cudaError_t launch_prompt_attention(PromptArgs a, const DeviceInfo& dev, cudaStream_t stream) {
  if (a.Tq == 0 || a.H == 0 || a.B == 0) return cudaSuccess;
  a.err = dev.err_word;
  return a.d == 64 ? prompt_attention<64>(a, dev, stream) : prompt_attention<128>(a, dev, stream);
}

cudaError_t launch_prefix_attention(PrefixArgs a, const DeviceInfo& dev, cudaStream_t stream) {
  if (a.B == 0 || a.H == 0) return cudaSuccess;
  a.err = dev.err_word;
  return a.d == 64 ? prefix_attention<64>(a, dev, stream) : prefix_attention<128>(a, dev, stream);
}

}  // namespace q8
