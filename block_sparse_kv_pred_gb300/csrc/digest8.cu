// scout_build_digest8: per-block key digests over an 8-bit paged cache.
// ScoutAttention (arXiv HTML), section 2.2: Quest min/max pooling, MoBA mean pooling.
//
// A warp takes a (unit, block) at a time and reads where the next one lies while it works.  Eight
// lanes hold a token's 128 codes (16 bytes each), so a warp instruction reads four rows and the
// block is read once, coalesced.  Minima and maxima are taken over the codes (as f16 pairs, exact)
// and scaled once at the end, rounded down and up: a digest still bounds every score of its
// block.  The mean sums codes in fp32.
//
// Bound by DRAM and its start: GB300, 8 x 16K tokens, 8 KV heads, blocks of 32, min/max: 27.3 us
// for 151 MB (5.5 TB/s, 0.82 of the measured copy bandwidth, launch and first reads included); mean
// digests of 2,800 blocks of 64: 5.3 us.
#include "fp8.cuh"

namespace scout {
namespace {

constexpr int kD8Warps = 8;
// CTAs an SM (three are resident, the others follow).  Minima and maxima of 32,768 blocks of 32 tokens,
// GB300: 27.2 us with three, 29.8 with four, 27.0 with six, 27.5 with twelve, 29.2 with 24.
constexpr int kD8PerSm = 6;

__device__ __forceinline__ uint32_t h2min(uint32_t a, uint32_t b) {
  const __half2 r = __hmin2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t h2max(uint32_t a, uint32_t b) {
  const __half2 r = __hmax2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
constexpr uint32_t kNeg2 = 0x80008000u;  // the signs of a pair

// code * scale rounded down to bf16: the product is first rounded the same way to fp32, so the two
// roundings together never cross the exact value.  Down is truncation for positive numbers, and one
// magnitude more for negative ones unless the dropped bits are zero.
__device__ __forceinline__ uint32_t down_bits(float x, float s) {
  const uint32_t b = __float_as_uint(__fmul_rd(x, s));
  return b + ((uint32_t)((int32_t)b >> 31) >> 16);
}
__device__ __forceinline__ uint32_t down2(uint32_t h, float s) {
  const float2 f = half2_floats(h);
  return __byte_perm(down_bits(f.x, s), down_bits(f.y, s), 0x7632);
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

// Where an item's block lies: valid = 0 where there is nothing to do.
struct Block8 {
  int64_t blk;
  int slot, valid;
};
template <int P>
__device__ __forceinline__ Block8 block_of(const Dig8Args& a, int64_t item) {
  Block8 k{0, 0, 0};
  if (item >= a.n_items) return k;
  int u, j;
  if (a.block_list != nullptr) {
    u = a.block_list[2 * item];
    j = a.block_list[2 * item + 1];
  } else {
    u = (int)((unsigned)item / (unsigned)a.nblk_cap);
    j = (int)item - u * a.nblk_cap;
  }
  if (u == -1 && j == -1) return k;  // padding
  k.slot = -1;
  k.valid = -1;
  if (u < 0 || j < 0 || j >= a.nblk_cap || u >= a.units) return k;
  k.blk = (int64_t)u * a.nblk_cap + j;
  k.valid = (int)max((int64_t)0, min((int64_t)P, a.seq_len[u / a.Hkv] - (int64_t)j * P));  // no tokens: left untouched
  k.slot = a.page_table[k.blk];
  return k;
}

// A warp goes from block to block; where the next one lies is read while this one is worked on.
template <int P, int KIND, int F>
__global__ void __launch_bounds__(kD8Warps * 32) digest8_kernel(const Dig8Args a) {
  const int lane = threadIdx.x & 31, sub = lane >> 3, chunk = lane & 7;
  const int64_t step = (int64_t)gridDim.x * kD8Warps;
  constexpr int kRows = P / 4 < 8 ? P / 4 : 8;  // rows a lane holds at a time
  int64_t item = (int64_t)blockIdx.x * kD8Warps + (threadIdx.x >> 5);
  Block8 next = block_of<P>(a, item);
  for (; item < a.n_items; item += step) {
    const Block8 k = next;
    const bool bad = k.valid < 0 || (k.valid > 0 && (k.slot < 0 || k.slot >= a.n_slots));
    if (bad || k.valid == 0) {
      if (bad && lane == 0) report(a.status, SCOUT_DEV_BAD_INDEX);
      next = block_of<P>(a, item + step);
      continue;
    }
    const uint8_t* base = a.K_pool + (int64_t)k.slot * (P * kD) + chunk * 16;
    const int64_t blk = k.blk;
    uint4 v[kRows];
    auto load = [&](int c) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int t = 4 * (c * kRows + i) + sub;
        v[i] = t < k.valid ? ldg_stream(base + t * kD) : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    load(0);
    const float scale = a.K_scale[k.slot];
    next = block_of<P>(a, item + step);
    if (KIND == SCOUT_DIGEST_MINMAX) {
      uint32_t lo[8], hi[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        lo[e] = 0x7c007c00u;  // +inf, -inf
        hi[e] = 0xfc00fc00u;
      }
#pragma unroll
      for (int c = 0; c < P / 4 / kRows; ++c) {
        if (c > 0) load(c);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          if (4 * (c * kRows + i) + sub >= k.valid) continue;
          const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t x, y;
            unpack4<F>(w[q], x, y);
            lo[2 * q] = h2min(lo[2 * q], x);
            lo[2 * q + 1] = h2min(lo[2 * q + 1], y);
            hi[2 * q] = h2max(hi[2 * q], x);
            hi[2 * q + 1] = h2max(hi[2 * q + 1], y);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) hi[e] ^= kNeg2;  // from here on minima of the negatives
      // Four lanes hold parts of the same 16 channels.  They halve what they keep with each exchange:
      // the upper two go on with the maxima, the odd ones with the second half of the channels, so
      // that each ends with the 16 bytes of output it writes.
      const bool top = lane >= 16, second = (sub & 1) != 0;
      uint32_t keep[8], out[4];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, top ? lo[e] : hi[e], 16);
        keep[e] = h2min(top ? hi[e] : lo[e], got);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, second ? keep[e] : keep[4 + e], 8);
        out[e] = h2min(second ? keep[4 + e] : keep[e], got);
      }
      const uint32_t flip = top ? kNeg2 : 0u;
#pragma unroll
      for (int e = 0; e < 4; ++e) out[e] = down2(out[e], scale) ^ flip;
      reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.digest) + blk * 2 * kD + (top ? kD : 0) + chunk * 16 +
                               (second ? 8 : 0))[0] = make_uint4(out[0], out[1], out[2], out[3]);
    } else {
      // Rows past the block's tokens are zero codes.  Four rows at a time, then the fours, then the
      // lanes: every e4m3 sum is exact (multiples of 2^-9 below 2^15), an e5m2 value passes
      // through at most 2 + 3 + 2 roundings.
      float s[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) s[e] = 0.f;
#pragma unroll
      for (int c = 0; c < P / 4 / kRows; ++c) {
        if (c > 0) load(c);
#pragma unroll
        for (int i = 0; i < kRows; i += 4) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float2 f[4][2];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              uint32_t x, y;
              unpack4<F>(q == 0 ? v[i + r].x : q == 1 ? v[i + r].y : q == 2 ? v[i + r].z : v[i + r].w, x, y);
              f[r][0] = half2_floats(x);
              f[r][1] = half2_floats(y);
            }
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              s[4 * q + 2 * z] += (f[0][z].x + f[1][z].x) + (f[2][z].x + f[3][z].x);
              s[4 * q + 2 * z + 1] += (f[0][z].y + f[1][z].y) + (f[2][z].y + f[3][z].y);
            }
          }
        }
      }
      // the same halving: each lane ends with the sums of the four channels it writes
      const bool top = lane >= 16, second = (sub & 1) != 0;
      float keep[8], out[4];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        keep[e] = (top ? s[8 + e] : s[e]) + __shfl_xor_sync(0xffffffffu, top ? s[e] : s[8 + e], 16);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        out[e] = (second ? keep[4 + e] : keep[e]) + __shfl_xor_sync(0xffffffffu, second ? keep[e] : keep[4 + e], 8);
      const float f = scale / (float)k.valid;
      *reinterpret_cast<float4*>(static_cast<float*>(a.digest) + blk * kD + chunk * 16 + (top ? 8 : 0) + (second ? 4 : 0)) =
          make_float4(out[0] * f, out[1] * f, out[2] * f, out[3] * f);
    }
  }
}

template <int P, int KIND, int F>
int launch_digest8(const Dig8Args& a, cudaStream_t st) {
  const int64_t want = (a.n_items + kD8Warps - 1) / kD8Warps, most = (int64_t)sm_count() * kD8PerSm;
  digest8_kernel<P, KIND, F><<<(unsigned)(want < most ? want : most), kD8Warps * 32, 0, st>>>(a);
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
  if (D != kD || !valid_P(P) || !aligned16(K_pool) || !aligned16(digest) || (int64_t)B * Hkv > 0x7fffffffLL ||
      (int64_t)B * Hkv * nblk_cap > 0x7fffffffLL || n_slots > 0x7fffffffLL)
    return SCOUT_ERR_UNSUPPORTED;
  const int64_t n_items = block_list != nullptr ? (int64_t)n_list : (int64_t)B * Hkv * nblk_cap;
  if (n_items == 0) return SCOUT_OK;
  const Dig8Args a{static_cast<const uint8_t*>(K_pool), K_scale, n_slots, page_table, seq_len, Hkv,
                   (int64_t)B * Hkv, nblk_cap, n_items, block_list, digest, dev_status};
  return fmt == SCOUT_FP8_E4M3 ? digest8_by_kind<SCOUT_FP8_E4M3>(kind, P, a, stream)
                               : digest8_by_kind<SCOUT_FP8_E5M2>(kind, P, a, stream);
}
