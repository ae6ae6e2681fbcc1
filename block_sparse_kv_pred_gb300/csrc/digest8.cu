// scout_build_digest8: per-block key digests over an 8-bit paged cache.
// ScoutAttention (arXiv HTML), section 2.2: Quest min/max pooling, MoBA mean pooling.
//
// One warp per (unit, block).  Eight lanes hold a token's 128 codes (16 bytes each), so a warp
// instruction reads four rows and the block is read once, coalesced.  Minima and maxima are taken
// over the codes (as f16 pairs, exact) and scaled once at the end, rounded down and up: a digest
// still bounds every score of its block.  The sum of the mean is compensated fp32.
#include "fp8.cuh"

namespace scout {
namespace {

constexpr int kD8Warps = 8;

__device__ __forceinline__ uint32_t h2min(uint32_t a, uint32_t b) {
  const __half2 r = __hmin2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t h2max(uint32_t a, uint32_t b) {
  const __half2 r = __hmax2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Neumaier's compensated summation step
__device__ __forceinline__ void sum_add(float& s, float& c, float x) {
  const float t = s + x;
  c += fabsf(s) >= fabsf(x) ? (s - t) + x : (x - t) + s;
  s = t;
}

// code * scale rounded down (up) to bf16: the product is first rounded the same way to fp32, so
// the two roundings together never cross the exact value
__device__ __forceinline__ uint32_t down2(uint32_t h, float s) {
  const float2 f = half2_floats(h);
  const __nv_bfloat16 x = __float2bfloat16_rd(__fmul_rd(f.x, s)), y = __float2bfloat16_rd(__fmul_rd(f.y, s));
  return (uint32_t)__bfloat16_as_ushort(x) | ((uint32_t)__bfloat16_as_ushort(y) << 16);
}
__device__ __forceinline__ uint32_t up2(uint32_t h, float s) {
  const float2 f = half2_floats(h);
  const __nv_bfloat16 x = __float2bfloat16_ru(__fmul_ru(f.x, s)), y = __float2bfloat16_ru(__fmul_ru(f.y, s));
  return (uint32_t)__bfloat16_as_ushort(x) | ((uint32_t)__bfloat16_as_ushort(y) << 16);
}

template <int P, int KIND, int F>
__global__ void __launch_bounds__(kD8Warps * 32) digest8_kernel(const uint8_t* __restrict__ K_pool,
                                                                const float* __restrict__ K_scale, int64_t n_slots,
                                                                const int32_t* __restrict__ page_table,
                                                                const int32_t* __restrict__ seq_len, int Hkv,
                                                                int64_t units, int nblk_cap, int64_t n_items,
                                                                const int32_t* __restrict__ block_list, void* digest,
                                                                int32_t* status) {
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * kD8Warps + (threadIdx.x >> 5);
  if (item >= n_items) return;
  int64_t u, j;
  if (block_list != nullptr) {
    u = block_list[2 * item];
    j = block_list[2 * item + 1];
    if (u == -1 && j == -1) return;  // padding
  } else {
    u = item / nblk_cap;
    j = item - u * nblk_cap;
  }
  if (u < 0 || j < 0 || j >= nblk_cap || u >= units) {
    if (lane == 0) report(status, SCOUT_DEV_BAD_INDEX);
    return;
  }
  const int valid = min(P, seq_len[u / Hkv] - (int)(j * P));
  if (valid <= 0) return;  // block holds no tokens: left untouched
  const int32_t slot = page_table[u * nblk_cap + j];
  if (slot < 0 || slot >= n_slots) {
    if (lane == 0) report(status, SCOUT_DEV_BAD_INDEX);
    return;
  }
  const int sub = lane >> 3, chunk = lane & 7;
  const uint8_t* base = K_pool + (int64_t)slot * (P * kD) + chunk * 16;
  const float scale = K_scale[slot];
  constexpr int kRows = P / 4;  // rows a lane reads
  uint4 v[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int t = 4 * i + sub;
    v[i] = t < valid ? ldg_stream(base + t * kD) : make_uint4(0u, 0u, 0u, 0u);
  }
  const int64_t blk = u * nblk_cap + j;
  if (KIND == SCOUT_DIGEST_MINMAX) {
    uint32_t lo[8], hi[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      lo[e] = 0x7c007c00u;  // +inf, -inf
      hi[e] = 0xfc00fc00u;
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (4 * i + sub >= valid) continue;
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t a, b;
        unpack4<F>(w[q], a, b);
        lo[2 * q] = h2min(lo[2 * q], a);
        lo[2 * q + 1] = h2min(lo[2 * q + 1], b);
        hi[2 * q] = h2max(hi[2 * q], a);
        hi[2 * q + 1] = h2max(hi[2 * q + 1], b);
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
      for (int o = 8; o < 32; o <<= 1) {
        lo[e] = h2min(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], o));
        hi[e] = h2max(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], o));
      }
    }
    // lanes 0-7 and 8-15 write the min row, 16-23 and 24-31 the max row: 16 bytes each
    const bool top = lane >= 16, second = (sub & 1) != 0;
    uint32_t src[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t mn = second ? lo[4 + e] : lo[e], mx = second ? hi[4 + e] : hi[e];
      src[e] = top ? up2(mx, scale) : down2(mn, scale);
    }
    reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(digest) + blk * 2 * kD + (top ? kD : 0) + chunk * 16 +
                             (second ? 8 : 0))[0] = make_uint4(src[0], src[1], src[2], src[3]);
  } else {
    float s[16], c[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) s[e] = c[e] = 0.f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (4 * i + sub >= valid) continue;
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t a, b;
        unpack4<F>(w[q], a, b);
        const float2 f = half2_floats(a), g = half2_floats(b);
        sum_add(s[4 * q], c[4 * q], f.x);
        sum_add(s[4 * q + 1], c[4 * q + 1], f.y);
        sum_add(s[4 * q + 2], c[4 * q + 2], g.x);
        sum_add(s[4 * q + 3], c[4 * q + 3], g.y);
      }
    }
    const float f = scale / (float)valid;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
#pragma unroll
      for (int o = 8; o < 32; o <<= 1) {
        const float ps = __shfl_xor_sync(0xffffffffu, s[e], o), pc = __shfl_xor_sync(0xffffffffu, c[e], o);
        c[e] += pc;
        sum_add(s[e], c[e], ps);
      }
      s[e] = (s[e] + c[e]) * f;
    }
    // each group of eight lanes writes a quarter of its 16 channels
    float4 o4 = make_float4(s[0], s[1], s[2], s[3]);
    if (sub == 1) o4 = make_float4(s[4], s[5], s[6], s[7]);
    if (sub == 2) o4 = make_float4(s[8], s[9], s[10], s[11]);
    if (sub == 3) o4 = make_float4(s[12], s[13], s[14], s[15]);
    *reinterpret_cast<float4*>(static_cast<float*>(digest) + blk * kD + chunk * 16 + sub * 4) = o4;
  }
}

struct Dig8Args {
  const uint8_t* K_pool;
  const float* K_scale;
  int64_t n_slots;
  const int32_t* page_table;
  const int32_t* seq_len;
  int Hkv;
  int64_t units;
  int nblk_cap;
  int64_t n_items;
  const int32_t* block_list;
  void* digest;
  int32_t* status;
};

template <int P, int KIND, int F>
int launch_digest8(const Dig8Args& a, cudaStream_t st) {
  const unsigned grid = (unsigned)((a.n_items + kD8Warps - 1) / kD8Warps);
  digest8_kernel<P, KIND, F><<<grid, kD8Warps * 32, 0, st>>>(a.K_pool, a.K_scale, a.n_slots, a.page_table, a.seq_len,
                                                             a.Hkv, a.units, a.nblk_cap, a.n_items, a.block_list,
                                                             a.digest, a.status);
  return launch_status();
}
template <int KIND, int F>
int digest8_by_P(int P, const Dig8Args& a, cudaStream_t st) {
  switch (P) {
    case 16: return launch_digest8<16, KIND, F>(a, st);
    case 32: return launch_digest8<32, KIND, F>(a, st);
    default: return launch_digest8<64, KIND, F>(a, st);
  }
}
template <int F>
int digest8_by_kind(int kind, int P, const Dig8Args& a, cudaStream_t st) {
  return kind == SCOUT_DIGEST_MINMAX ? digest8_by_P<SCOUT_DIGEST_MINMAX, F>(P, a, st)
                                     : digest8_by_P<SCOUT_DIGEST_MEAN, F>(P, a, st);
}

}  // namespace
}  // namespace scout

extern "C" int scout_build_digest8(int kind, int fmt, const void* K_pool, const float* K_scale, int64_t n_slots,
                                   const int32_t* page_table, const int32_t* seq_len, int B, int Hkv, int D, int P,
                                   int nblk_cap, const int32_t* block_list, int n_list, void* digest,
                                   int32_t* dev_status, cudaStream_t stream) {
  using namespace scout;
  if (K_pool == nullptr || K_scale == nullptr || page_table == nullptr || seq_len == nullptr || digest == nullptr)
    return SCOUT_ERR_INVALID_ARG;
  if (B <= 0 || Hkv <= 0 || nblk_cap <= 0 || n_slots <= 0 || n_list < 0 || !valid_fp8(fmt) ||
      (kind != SCOUT_DIGEST_MINMAX && kind != SCOUT_DIGEST_MEAN))
    return SCOUT_ERR_INVALID_ARG;
  if (D != kD || !valid_P(P) || !aligned16(K_pool) || !aligned16(digest)) return SCOUT_ERR_UNSUPPORTED;
  const int64_t n_items = block_list != nullptr ? (int64_t)n_list : (int64_t)B * Hkv * nblk_cap;
  if (n_items == 0) return SCOUT_OK;
  if ((n_items + kD8Warps - 1) / kD8Warps > 0x7fffffffLL) return SCOUT_ERR_UNSUPPORTED;
  const Dig8Args a{static_cast<const uint8_t*>(K_pool), K_scale, n_slots, page_table, seq_len, Hkv,
                   (int64_t)B * Hkv, nblk_cap, n_items, block_list, digest, dev_status};
  return fmt == SCOUT_FP8_E4M3 ? digest8_by_kind<SCOUT_FP8_E4M3>(kind, P, a, stream)
                               : digest8_by_kind<SCOUT_FP8_E5M2>(kind, P, a, stream);
}
