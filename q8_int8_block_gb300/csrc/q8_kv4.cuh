// q8_kv4.cuh -- the tile format of the 4-bit cache of keys and values, shared by the kernels that
// write, read back and attend to it.
//
// A page holds, for every key/value head, page / 32 tiles of 32 neighbouring tokens.  A tile of d
// channels is 36 d bytes: the keys' codes (16 d bytes), their scales (bfloat16 [d / 32][32
// tokens], 2 d bytes), the values' codes (16 d) and their scales (2 d).  A code is a nibble, 8 + q
// with q in -7 .. 7; eight share a 32-bit word, the first in its lowest bits.  The words lie in the
// order in which the lanes of a warp (g = lane / 4, t = lane % 4) read the operands of
// mma.sync.m16n8k16 from them, so that every load of the attention kernel is one contiguous piece
// of the tile and no word is exchanged:
//   - a token of a tile is 8 t + 2 j + i (t, j in 0 .. 3, i in 0, 1): a lane's eight keys are
//     neighbours, and column 2 t + i of the j-th product of scores is token 8 t + 2 j + i;
//   - keys: word (j, b / 4, n = 2 t + i, u, b % 4) holds channels 32 b + 8 u .. + 7 of token
//     8 t + 2 j + i: lane (g = n, t = u) reads the words of up to four blocks b in one piece;
//   - values: word (2 j + i, g, t, h) holds channels 64 h + 4 g .. + 3 in its low half and 64 h +
//     32 + 4 g .. + 3 in its high half.
#pragma once
#include <cstdint>

namespace q8 {

enum : uint32_t { kErrBadCache = 1u << 10 };  // a slot, page, sequence or length outside the cache

template <int D>
struct Kv4Tile {
  static_assert(D == 64 || D == 128 || D == 256, "head size");
  static constexpr int kTokens = 32;
  static constexpr int kBlocks = D / 32;                     // scales of a token
  static constexpr int kBytes = 36 * D;
  static constexpr int kKeyScales = 16 * D, kValues = 18 * D, kValueScales = 34 * D;
  static constexpr int kQuads = D > 128 ? D / 128 : 1;       // pieces of a key that a lane reads
  static constexpr int kWords = D > 128 ? 4 : D / 32;        // 32-bit words of a piece
  static constexpr int kHalves = D / 64;                     // words of a lane's value

  // byte of the word that holds channels 8 c .. 8 c + 7 of a key
  __device__ __forceinline__ static int key_word(int tok, int c) {
    const int b = c >> 2, u = c & 3;
    return ((((((tok >> 1) & 3) * kQuads + (b >> 2)) * 32 + ((tok >> 3) * 2 + (tok & 1)) * 4 + u) * kWords) + (b & 3)) * 4;
  }
  // byte of the word of channels 64 h + 4 g .. + 3 and 64 h + 32 + 4 g .. + 3 of a value
  __device__ __forceinline__ static int value_word(int tok, int g, int h) {
    return kValues + (((tok & 7) * 32 + 4 * g + (tok >> 3)) * kHalves + h) * 4;
  }
  // byte of a block's scale (keys; values: kValueScales)
  __device__ __forceinline__ static int scale(int tok, int b) { return (b * 32 + tok) * 2; }
};

// Largest magnitude below which a block counts as zero: 7 over it stays finite.
constexpr float kKv4Zero = 7.52316384526264e-37f;  // 2^-120

}  // namespace q8
