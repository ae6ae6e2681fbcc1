// 8-bit cache codes: conversions and the scale of a block.
//
// A code c of a slot stands for c * scale[slot].  The library's own writes use powers of two as
// scales: multiplying and dividing by them is exact, so a code's only rounding is its own, a
// block whose scale grows keeps every code that stays in the normal range as it was, and the
// dequantised values are bf16 numbers.  For a floating-point code a power of two costs no
// precision (a finer scale moves the values within a binade, not the number of their bits).
#pragma once

#include "common.cuh"

namespace scout {

template <int F>
struct Fp8;

template <>
struct Fp8<SCOUT_FP8_E4M3> {
  static constexpr int kTop = 8;  // largest finite value: 1.75 * 2^8 = 448
  static __device__ __forceinline__ uint32_t unpack(uint16_t c) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
    return r;
  }
  static __device__ __forceinline__ uint16_t pack(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
  }
};

template <>
struct Fp8<SCOUT_FP8_E5M2> {
  static constexpr int kTop = 15;  // 1.75 * 2^15 = 57344
  static __device__ __forceinline__ uint32_t unpack(uint16_t c) {
    uint32_t r;
    asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(r) : "h"(c));
    return r;
  }
  static __device__ __forceinline__ uint16_t pack(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
  }
};

// Codes 0, 1 (lo) and 2, 3 (hi) of a word as f16 pairs: exact, both formats lie inside f16.
template <int F>
__device__ __forceinline__ void unpack4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  lo = Fp8<F>::unpack((uint16_t)(w & 0xffffu));
  hi = Fp8<F>::unpack((uint16_t)(w >> 16));
}

__device__ __forceinline__ float2 half2_floats(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Biased exponent of the smallest power of two s >= 2^-126 with amax <= 1.75 * 2^kTop * s
// (amax finite and >= 0): both largest codes have the significand 1.75.
template <int F>
__device__ __forceinline__ uint32_t scale_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - Fp8<F>::kTop + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(e, 1);
}
__device__ __forceinline__ float pow2_biased(uint32_t e) { return __uint_as_float(e << 23); }

inline bool valid_fp8(int fmt) { return fmt == SCOUT_FP8_E4M3 || fmt == SCOUT_FP8_E5M2; }

// ---------------------------------------------------------------------------
// Request lengths.  prev (NULL: 0) and seq are clamped to 0 <= prev <= seq <= capacity.
// ---------------------------------------------------------------------------
constexpr int kMaxBatch = 4096;  // sequences of a batch whose prefixes a CTA keeps in shared memory

struct SeqSpan {
  int prev, seq;
};
__device__ __forceinline__ SeqSpan seq_span(const int32_t* prev_len, const int32_t* seq_len, int b, int cap_tokens) {
  const int n = min(max(seq_len[b], 0), cap_tokens);
  const int p = prev_len != nullptr ? min(max(prev_len[b], 0), n) : 0;
  return SeqSpan{p, n};
}

// What the clamping changed, in the status word.
__device__ __forceinline__ void report_span(int32_t* status, const int32_t* prev_len, const int32_t* seq_len, int b,
                                            int cap_tokens) {
  const int n = seq_len[b], p = prev_len != nullptr ? prev_len[b] : 0;
  if (n > cap_tokens) report(status, SCOUT_DEV_OVERFLOW);
  if (n < 0 || p < 0 || p > max(n, 0)) report(status, SCOUT_DEV_BAD_INDEX);
}

// K exclusive prefixes over b < B at once: f(b, x) gives the K values of b, out[k][b] the sum of those
// before it and out[k][B] the total.  By all threads of a CTA (a multiple of 32, at most 1024), a run
// of b a thread; f is called twice, so that a thread's first reads are all in flight together and
// the second ones hit L1.  partial: K * 32 ints.  Ends with a barrier.
template <int K, class F>
__device__ __forceinline__ void cta_prefixes(int B, int* const (&out)[K], int* partial, F f) {
  const int tid = threadIdx.x, n = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int per = (B + n - 1) / n, lo = min(B, tid * per), hi = min(B, lo + per);
  int sum[K], run[K], x[K];
#pragma unroll
  for (int k = 0; k < K; ++k) sum[k] = 0;
#pragma unroll 4
  for (int b = lo; b < hi; ++b) {
    f(b, x);
#pragma unroll
    for (int k = 0; k < K; ++k) sum[k] += x[k];
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    run[k] = sum[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, run[k], o);
      if (lane >= o) run[k] += y;
    }
    if (lane == 31) partial[k * 32 + warp] = run[k];
    run[k] -= sum[k];
  }
  __syncthreads();
  for (int w = 0; w < warp; ++w)
#pragma unroll
    for (int k = 0; k < K; ++k) run[k] += partial[k * 32 + w];
  for (int b = lo; b < hi; ++b) {
    f(b, x);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      out[k][b] = run[k];
      run[k] += x[k];
    }
  }
  if (tid == n - 1)
#pragma unroll
    for (int k = 0; k < K; ++k) out[k][B] = run[k];
  __syncthreads();
}

// The last b in [0, B) with v[b] <= x < v[B]: the sequence (or unit) that item x belongs to.
__device__ __forceinline__ int owner_of(const int* v, int B, int x) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (v[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

}  // namespace scout
