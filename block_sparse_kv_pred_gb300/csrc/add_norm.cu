// scout_add_norm: a block's output added to the residual stream, and the stream normalised, in one pass.
//
// A row is T threads', in registers from its reads to its writes: the output (normalised first where a norm
// follows the block), the sum, its mean square (and mean), the normalised row for one or two sets of weights.  Two
// chunks of eight a thread where rows are up to 8,192 long: more CTAs of fewer registers overlap better than four a thread
// (GB300, 16,384 x 5,120, bf16 stream, two norms: 127 us against 136; 40 rows 2.7 against 3.7).  Sums go through
// shuffles and one barrier each, in one order whatever the timing; the variance of SCOUT_NORM_LAYER is a second sum
// over the differences from the mean.
//
// Bound by DRAM: GB300, 131,072 x 4,096, fp32 stream, norms before and after, a gate: 925 us for 6.44 GB (7.0 TB/s, above the
// measured copy rate); 40 x 5,120 2.8 us, the launch and one read.  Rows past 16,384 are one a SM at a time, whose reads and
// writes do not overlap (8,192 x 32,768: 5.1 TB/s).
// A row of 128 leaves half of its warp's lanes without a chunk (1,048,576 rows, bf16 stream, two norms: 280 us, 4.8 TB/s; 524,288
// rows of 256: 193 us, 7.0 TB/s).  SCOUT_NORM_LAYER waits for a sum more between a row's reads and writes, and reads biases:
// 154 us for 16,384 x 5,120 (125), 895 for 131,072 x 4,096 (770), 392 and 222 for the two above, 3.1 for 40 x 5,120 (2.7).
#include "common.cuh"

namespace scout {
namespace {

struct NormArgs {
  const __nv_bfloat16 *Y, *w_post, *b_post, *gate;
  int64_t ld_y, ld_gate;
  float alpha;
  const void* H;
  void* H_out;
  int64_t ld_h, ld_h_out;
  const __nv_bfloat16 *w, *b, *w_ahead, *b_ahead;
  __nv_bfloat16 *X, *X_ahead;
  int M, N;
  float eps;
};

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
__device__ __forceinline__ uint4 ldg_weights(const __nv_bfloat16* p) {
  return __ldg(reinterpret_cast<const uint4*>(p));
}

// The sum of v over the row's threads, for all of them: in one order whatever the timing.
template <bool ONE>
__device__ __forceinline__ float row_sum(float v, float* part, int& buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (ONE) return v;
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  float* p = part + buf * 32;
  buf ^= 1;  // the next sum's slots: a thread that is a sum ahead does not overwrite this one's
  if (lane == 0) p[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < warps ? p[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// (mean, factor) of a row's norm.
template <int KIND, int V, bool ONE>
__device__ __forceinline__ float2 row_norm(const float (&x)[V][8], int n, const NormArgs& a, float* part, int& buf) {
  float mean = 0.f, s = 0.f;
  if (KIND == SCOUT_NORM_LAYER) {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += x[i][e];  // chunks past the row hold zeros
    mean = row_sum<ONE>(s, part, buf) / (float)a.N;
    s = 0.f;
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (i < n)
#pragma unroll
      for (int e = 0; e < 8; ++e) s = fmaf(x[i][e] - mean, x[i][e] - mean, s);
  return make_float2(mean, rsqrtf(row_sum<ONE>(s, part, buf) / (float)a.N + a.eps));
}

template <int KIND>
__device__ __forceinline__ void apply_norm(float (&x)[8], const float2& m, const __nv_bfloat16* w,
                                           const __nv_bfloat16* b, int c) {
  float v[8];
  unpack8(ldg_weights(w + c), v);
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = (KIND == SCOUT_NORM_LAYER ? x[e] - m.x : x[e]) * m.y * v[e];
  if (KIND == SCOUT_NORM_LAYER && b != nullptr) {
    unpack8(ldg_weights(b + c), v);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] += v[e];
  }
}

// V chunks of eight a thread; ONE: a row is one warp's, blockDim.x / 32 rows a CTA.
template <int KIND, bool WIDE, int V, bool ONE>
__global__ void __launch_bounds__(512) add_norm_kernel(const NormArgs a) {
  __shared__ float part[64];
  int buf = 0;
  start_dependent();
  const int T = ONE ? 32 : blockDim.x, t = ONE ? threadIdx.x & 31 : threadIdx.x;
  const int64_t row = ONE ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  if (row >= a.M) return;
  const int chunks = a.N / 8;
  int n = 0;  // the thread's chunks t, t + T, ...
#pragma unroll
  for (int i = 0; i < V; ++i) n += t + i * T < chunks;
  float h[V][8];
  uint4 y[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (t + i * T) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) h[i][e] = 0.f;
    y[i] = make_uint4(0u, 0u, 0u, 0u);
    if (i >= n) continue;
    if (a.Y != nullptr) y[i] = ld_stream(a.Y + row * a.ld_y + c);
    if (WIDE) {
      const float* p = static_cast<const float*>(a.H) + row * a.ld_h + c;
      const uint4 lo = ld_stream(p), hi = ld_stream(p + 4);
      const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) h[i][e] = __uint_as_float(w[e]);
    } else {
      unpack8(ld_stream(static_cast<const __nv_bfloat16*>(a.H) + row * a.ld_h + c), h[i]);
    }
  }
  if (a.Y != nullptr) {
    float2 m = make_float2(0.f, 1.f);
    if (a.w_post != nullptr) {
      float x[V][8];
#pragma unroll
      for (int i = 0; i < V; ++i) unpack8(y[i], x[i]);
      m = row_norm<KIND, V, ONE>(x, n, a, part, buf);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (i >= n) continue;
      const int c = (t + i * T) * 8;
      float x[8], g[8];
      unpack8(y[i], x);
      if (a.w_post != nullptr) apply_norm<KIND>(x, m, a.w_post, a.b_post, c);
      if (a.gate != nullptr) {
        unpack8(ldg_weights(a.gate + row * a.ld_gate + c), g);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= g[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) h[i][e] = fmaf(a.alpha, x[e], h[i][e]);
      if (WIDE) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(a.H_out) + row * a.ld_h_out + c);
        p[0] = make_float4(h[i][0], h[i][1], h[i][2], h[i][3]);
        p[1] = make_float4(h[i][4], h[i][5], h[i][6], h[i][7]);
      } else {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.H_out) + row * a.ld_h_out + c) = pack8(h[i]);
      }
    }
  }
  const float2 m = row_norm<KIND, V, ONE>(h, n, a, part, buf);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (i >= n) continue;
    const int c = (t + i * T) * 8;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = h[i][e];
    apply_norm<KIND>(x, m, a.w, a.b, c);
    *reinterpret_cast<uint4*>(a.X + row * a.N + c) = pack8(x);
    if (a.X_ahead != nullptr) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = h[i][e];
      apply_norm<KIND>(x, m, a.w_ahead, a.b_ahead, c);
      *reinterpret_cast<uint4*>(a.X_ahead + row * a.N + c) = pack8(x);
    }
  }
}

template <int KIND, bool WIDE, int V>
int launch_norm(const NormArgs& a, int threads, cudaStream_t st) {
  if constexpr (V == 2) {  // (only the shortest rows are a warp's)
    if (threads == 32) {
      constexpr int kRows = 4;  // rows of a CTA
      return launch_dependent(add_norm_kernel<KIND, WIDE, V, true>, a.M / kRows + (a.M % kRows != 0), kRows * 32, 0, st, a);
    }
  }
  return launch_dependent(add_norm_kernel<KIND, WIDE, V, false>, a.M, threads, 0, st, a);
}

template <int KIND, bool WIDE>
int dispatch_norm(const NormArgs& a, cudaStream_t st) {
  const int chunks = a.N / 8;
  const int V = chunks <= 512 * 2 ? 2 : chunks <= 512 * 4 ? 4 : 8;
  const int threads = ((chunks + V - 1) / V + 31) / 32 * 32;
  return V == 2   ? launch_norm<KIND, WIDE, 2>(a, threads, st)
         : V == 4 ? launch_norm<KIND, WIDE, 4>(a, threads, st)
                  : launch_norm<KIND, WIDE, 8>(a, threads, st);
}

}  // namespace
}  // namespace scout

extern "C" int scout_add_norm(int kind, const void* Y, int64_t ld_y, const void* w_post, const void* b_post,
                              const void* gate, int64_t ld_gate, float alpha, int h_type, const void* H, int64_t ld_h,
                              void* H_out, int64_t ld_h_out, const void* w, const void* b, void* X, const void* w_ahead,
                              const void* b_ahead, void* X_ahead, int M, int N, float eps, cudaStream_t stream) {
  using namespace scout;
  const bool rms = kind == SCOUT_NORM_RMS;
  if ((!rms && kind != SCOUT_NORM_LAYER) || (h_type != SCOUT_BF16 && h_type != SCOUT_FP32) || H == nullptr ||
      w == nullptr || X == nullptr || M < 0 || N <= 0 || ld_h < N || !(eps >= 0.f) || eps - eps != 0.f ||
      alpha - alpha != 0.f)
    return SCOUT_ERR_INVALID_ARG;
  if (Y != nullptr ? H_out == nullptr || ld_y < N || ld_h_out < N : H_out != nullptr || gate != nullptr || w_post != nullptr)
    return SCOUT_ERR_INVALID_ARG;
  if ((gate != nullptr && ld_gate != 0 && ld_gate < N) || (w_ahead == nullptr) != (X_ahead == nullptr) ||
      (b_post != nullptr && (rms || w_post == nullptr)) || (b != nullptr && rms) ||
      (b_ahead != nullptr && (rms || w_ahead == nullptr)))
    return SCOUT_ERR_INVALID_ARG;
  if (N % 8 != 0 || N > 32768 || ld_h % 8 != 0 || (Y != nullptr && (ld_y % 8 != 0 || ld_h_out % 8 != 0)) || (gate != nullptr && ld_gate % 8 != 0))
    return SCOUT_ERR_UNSUPPORTED;
  for (const void* p : {Y, w_post, b_post, gate, H, static_cast<const void*>(H_out), w, b, static_cast<const void*>(X),
                        w_ahead, b_ahead, static_cast<const void*>(X_ahead)})
    if (!aligned16(p)) return SCOUT_ERR_UNSUPPORTED;
  if (M == 0) return SCOUT_OK;
  auto bf = [](const void* p) { return static_cast<const __nv_bfloat16*>(p); };
  NormArgs a;
  a.Y = bf(Y);
  a.w_post = bf(w_post);
  a.b_post = bf(b_post);
  a.gate = bf(gate);
  a.ld_y = ld_y;
  a.ld_gate = ld_gate;
  a.alpha = alpha;
  a.H = H;
  a.H_out = H_out;
  a.ld_h = ld_h;
  a.ld_h_out = ld_h_out;
  a.w = bf(w);
  a.b = bf(b);
  a.w_ahead = bf(w_ahead);
  a.b_ahead = bf(b_ahead);
  a.X = static_cast<__nv_bfloat16*>(X);
  a.X_ahead = static_cast<__nv_bfloat16*>(X_ahead);
  a.M = M;
  a.N = N;
  a.eps = eps;
  if (h_type == SCOUT_FP32) return rms ? dispatch_norm<SCOUT_NORM_RMS, true>(a, stream) : dispatch_norm<SCOUT_NORM_LAYER, true>(a, stream);
  return rms ? dispatch_norm<SCOUT_NORM_RMS, false>(a, stream) : dispatch_norm<SCOUT_NORM_LAYER, false>(a, stream);
}
