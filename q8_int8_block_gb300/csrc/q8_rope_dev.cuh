// q8_rope_dev.cuh -- angles of the rotation by position, shared by its kernels.
#pragma once
#include <cstdint>

namespace q8 {

// inv_freq / (2 pi) as a fraction of a turn in units of 2^-64, modulo whole turns, from the
// bits of the binary64 value m 2^e: m 2^11 times the leading 64 bits of 2 / pi, shifted.
// Of frequencies from 2^32 on, infinities and NaN the 64 bits say too little: *ok is false.
__device__ __forceinline__ uint64_t turn_step(double f, bool* ok) {
  const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(f));
  const int ex = static_cast<int>((bits >> 52) & 0x7FF);
  *ok = ex < 1023 + 32;
  if (ex == 0) return 0;  // zero; a subnormal frequency turns by less than 2^-64
  const uint64_t m = (bits & 0xFFFFFFFFFFFFFull) | 0x10000000000000ull;
  const uint64_t x = __umul64hi(m << 11, 0xA2F9836E4E441529ull);  // floor(m (2 / pi) 2^11)
  const int sh = ex - 1075 + 51;  // f / (2 pi) 2^64 = x 2^(ex - 1075 + 51)
  const uint64_t s = sh <= -64 ? 0 : sh < 0 ? x >> -sh : x << (sh & 63);
  return (bits >> 63) != 0 ? 0 - s : s;
}

}  // namespace q8
