// q8_attn.cu -- attention over packed prompts and over a shared prefix.
//
// The attention layers of the hybrid models that "CUDA inference engine for running
// Qwen3.5/3.6 hybrid models on mining cards (CMP 100-210)" (news.hada.io topic 29953) runs:
// o = softmax(scale q . k) v over the keys a query sees, H query heads over Hkv key/value
// heads.
//
// One warp per query row (token and head) walks the row's keys with the running maximum and
// sum of the softmax: the dot product is split over the lanes, each of which holds d / 32
// channels of q and o.
#include <cuda_bf16.h>

#include "q8_internal.h"

namespace q8 {
namespace {

constexpr uint32_t kErrBadLength = 1u << 9;  // a sequence or cache length outside its array

__device__ __forceinline__ float bf16_f32(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

// whether sequence s lies inside the arrays
__device__ __forceinline__ bool sequence_ok(const PromptArgs& a, int64_t s) {
  const int64_t q0 = a.cu_q[s], q1 = a.cu_q[s + 1], k0 = a.cu_k[s], k1 = a.cu_k[s + 1];
  return 0 <= q0 && q0 <= q1 && q1 <= a.Tq && 0 <= k0 && k0 <= k1 && k1 <= a.Tk;
}

template <int D>
struct Row {
  static constexpr int E = D / 32;
  float q[E], o[E], m, l;

  __device__ void begin(const uint16_t* src, float scale, int lane) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      q[i] = bf16_f32(src[E * lane + i]) * scale;
      o[i] = 0.0f;
    }
    m = -INFINITY;
    l = 0.0f;
  }

  __device__ void attend(const uint16_t* k, const uint16_t* v, int64_t k_stride, int64_t v_stride, int64_t n,
                         int lane) {
    for (int64_t j = 0; j < n; ++j) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < E; ++i) s = fmaf(q[i], bf16_f32(k[j * k_stride + E * lane + i]), s);
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, x);
      const float mn = fmaxf(m, s), a = __expf(m - mn), p = __expf(s - mn);
      l = fmaf(l, a, p);
#pragma unroll
      for (int i = 0; i < E; ++i) o[i] = fmaf(o[i], a, p * bf16_f32(v[j * v_stride + E * lane + i]));
      m = mn;
    }
  }

  __device__ void end(uint16_t* dst, int lane) {
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) dst[E * lane + i] = __bfloat16_as_ushort(__float2bfloat16_rn(o[i] * inv));
  }
};

template <int D>
__global__ void __launch_bounds__(128) prompt_rows_kernel(const PromptArgs a) {
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x) / 32;
  const int lane = threadIdx.x & 31;
  if (row >= a.Tq * a.H) return;
  if (row == 0)  // one warp looks every sequence over
    for (int64_t s = lane; s < a.B; s += 32)
      if (!sequence_ok(a, s)) atomicOr(a.err, kErrBadLength);
  const int64_t t = row / a.H, h = row - t * a.H, hk = h / (a.H / a.Hkv);
  // the last sequence that begins at or before t and holds it
  int64_t lo = 0, hi = a.B;  // cu_q[lo] <= t < cu_q[hi]
  if (a.cu_q[0] > t || a.cu_q[a.B] <= t) return;
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) / 2;
    if (a.cu_q[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int64_t q0 = a.cu_q[lo], q1 = a.cu_q[lo + 1], k0 = a.cu_k[lo], k1 = a.cu_k[lo + 1];
  if (!sequence_ok(a, lo) || t < q0 || t >= q1) return;
  const int64_t seen = (t - q0) + (k1 - k0) - (q1 - q0) + 1;
  Row<D> r;
  r.begin(a.q + t * a.st[0] + h * a.st[1], a.scale, lane);
  r.attend(a.k + k0 * a.st[2] + hk * a.st[3], a.v + k0 * a.st[4] + hk * a.st[5], a.st[2], a.st[4], seen, lane);
  r.end(a.o + t * a.st[6] + h * a.st[7], lane);
}

template <int D>
__global__ void __launch_bounds__(128) prefix_rows_kernel(const PrefixArgs a) {
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x) / 32;
  const int lane = threadIdx.x & 31;
  if (row >= a.B * a.H) return;
  const int64_t b = row / a.H, h = row - b * a.H, hk = h / (a.H / a.Hkv);
  int64_t n = a.own_len[b];
  if (n < 0 || n > a.cap) {
    if (lane == 0) atomicOr(a.err, kErrBadLength);
    n = n < 0 ? 0 : a.cap;
  }
  Row<D> r;
  r.begin(a.q + b * a.st[0] + h * a.st[1], a.scale, lane);
  r.attend(a.kp + hk * a.st[3], a.vp + hk * a.st[5], a.st[2], a.st[4], a.P, lane);
  r.attend(a.ko + b * a.st[6] + hk * a.st[8], a.vo + b * a.st[9] + hk * a.st[11], a.st[7], a.st[10], n, lane);
  r.end(a.o + b * a.st[12] + h * a.st[13], lane);
}

}  // namespace

size_t prompt_ws_bytes(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, const DeviceInfo&) { return 0; }
size_t prefix_ws_bytes(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, const DeviceInfo&) { return 0; }

cudaError_t launch_prompt_attention(PromptArgs a, const DeviceInfo& dev, cudaStream_t stream) {
  if (a.Tq == 0 || a.H == 0 || a.B == 0) return cudaSuccess;
  a.err = dev.err_word;
  const unsigned grid = static_cast<unsigned>((a.Tq * a.H + 3) / 4);
  if (a.d == 64) prompt_rows_kernel<64><<<grid, 128, 0, stream>>>(a);
  else prompt_rows_kernel<128><<<grid, 128, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_prefix_attention(PrefixArgs a, const DeviceInfo& dev, cudaStream_t stream) {
  if (a.B == 0 || a.H == 0) return cudaSuccess;
  a.err = dev.err_word;
  const unsigned grid = static_cast<unsigned>((a.B * a.H + 3) / 4);
  if (a.d == 64) prefix_rows_kernel<64><<<grid, 128, 0, stream>>>(a);
  else prefix_rows_kernel<128><<<grid, 128, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace q8
