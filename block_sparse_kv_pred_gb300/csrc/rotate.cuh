// A head's norm and its turn by a position, shared by the kernels that make queries and keys.
//
// Eight lanes hold a head: lane `sub` two chunks of eight channels, placed so that both channels of
// each of its pairs are its own, and its pairs are 8 sub .. 8 sub + 7 in either layout.  No shuffle is
// needed to turn, three to sum the squares, and a warp moves four heads of consecutive tokens with
// 16-byte accesses.  A lane's cosines and sines depend on the token alone: they are made once and serve
// every head of the token.
//
// The angle is an integer product modulo 2^64 (turns as fractions of 2^64), so a far position costs no
// precision and no reduction.  Every rounding is
// written out (no contraction is left to the compiler), so that each kernel that turns a head gets the same bits.
#pragma once

#include "common.cuh"

namespace scout {

struct Rope {
  const uint64_t* turns;
  float amplitude;
  int n;  // lanes of the eight that turn: rot_dim / 16
};

inline bool valid_rope(const scout_rope* r) {
  return r != nullptr && r->turns != nullptr && (r->layout == SCOUT_ROPE_HALF || r->layout == SCOUT_ROPE_INTERLEAVED) &&
         r->amplitude - r->amplitude == 0.f;  // finite
}
// the part of it that a caller's shape decides (SCOUT_ERR_UNSUPPORTED)
inline bool supported_rope(const scout_rope* r) {
  return r->rot_dim >= 16 && r->rot_dim <= kD && r->rot_dim % 16 == 0 && aligned16(r->turns);
}
inline Rope rope_of(const scout_rope* r) { return Rope{r->turns, r->amplitude, r->rot_dim / 16}; }
inline bool valid_eps(float eps) { return eps >= 0.f && eps - eps == 0.f; }

// First channels of a lane's two chunks.
template <int LAYOUT>
__device__ __forceinline__ int2 lane_chunks(int sub, int n) {
  if (LAYOUT == SCOUT_ROPE_HALF && sub < n) return make_int2(sub * 8, (sub + n) * 8);
  return make_int2(sub * 16, sub * 16 + 8);
}

// sin and cos of a turn given as a fraction of 2^32: the nearest quarter turn by integers, and polynomials
// in the square of the rest, |rest| <= 1/8 turn (minimax, fitted by exchange: the sine's quotient by the rest to
// 2^-28, the cosine to 2^-34).  Off by at most 1.7 and 1.2 roundings of fp32 over 2 million angles, with a
// third of the instructions of sincospi, whose code a short launch has to fetch.
__device__ __forceinline__ void sincos_turn(uint32_t turn, float& s, float& c) {
  const uint32_t quarter = (turn + 0x20000000u) & 0xc0000000u;
  const float x = __fmul_rn((float)(int32_t)(turn - quarter), 0x1p-32f), z = __fmul_rn(x, x);
  float p = __fmaf_rn(-75.40206909179688f, z, 81.5925521850586f);
  p = __fmaf_rn(p, z, -41.3416633605957f);
  p = __fmul_rn(__fmaf_rn(p, z, 6.2831854820251465f), x);
  float q = __fmaf_rn(59.22040557861328f, z, -85.44285583496094f);
  q = __fmaf_rn(q, z, 64.93931579589844f);
  q = __fmaf_rn(q, z, -19.739208221435547f);
  q = __fmaf_rn(q, z, 1.f);
  const bool odd = quarter & 0x40000000u;  // a quarter turn further: (s, c) -> (c, -s)
  s = __uint_as_float(__float_as_uint(odd ? q : p) ^ (quarter & 0x80000000u));
  c = __uint_as_float(__float_as_uint(odd ? p : q) ^ ((quarter + 0x40000000u) & 0x80000000u));
}

// cos and sin (times the amplitude) of a lane's eight pairs at a position; lanes past n get none.
struct Turn {
  float c[8], s[8];
};
__device__ __forceinline__ Turn lane_turn(const Rope& r, int sub, uint32_t pos) {
  Turn t;
  if (sub < r.n) {
    const ulonglong2* f = reinterpret_cast<const ulonglong2*>(r.turns + sub * 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const ulonglong2 v = __ldg(f + i);
      const uint64_t w[2] = {v.x, v.y};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float s, c;
        sincos_turn((uint32_t)(((uint64_t)pos * w[j] + 0x80000000ull) >> 32), s, c);
        t.s[2 * i + j] = __fmul_rn(s, r.amplitude);
        t.c[2 * i + j] = __fmul_rn(c, r.amplitude);
      }
    }
  }
  return t;
}

// A lane's 16 channels: the first chunk's eight, then the second's.
__device__ __forceinline__ void unpack16(const uint4& a, const uint4& b, float (&x)[16]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ void pack16(const float (&x)[16], uint4& a, uint4& b) {
  a = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  b = make_uint4(pack_bf16(x[8], x[9]), pack_bf16(x[10], x[11]), pack_bf16(x[12], x[13]), pack_bf16(x[14], x[15]));
}

// A lane's 16 weights of a norm, packed.
struct Weights {
  uint4 a, b;
};
__device__ __forceinline__ Weights lane_weights(const __nv_bfloat16* norm, const int2& at) {
  return Weights{__ldg(reinterpret_cast<const uint4*>(norm + at.x)), __ldg(reinterpret_cast<const uint4*>(norm + at.y))};
}

// The head's norm: by the eight lanes that hold it, all of them.
__device__ __forceinline__ void norm_head(float (&x)[16], const Weights& weights, float eps) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) ss = __fmaf_rn(x[i], x[i], ss);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const float r = rsqrtf(__fmaf_rn(ss, 1.f / kD, eps));
  float w[16];
  unpack16(weights.a, weights.b, w);
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = __fmul_rn(__fmul_rn(x[i], r), w[i]);
}

template <int LAYOUT>
__device__ __forceinline__ void turn_head(float (&x)[16], const Turn& t, bool turns) {
  if (!turns) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int ia = LAYOUT == SCOUT_ROPE_HALF ? i : 2 * i, ib = LAYOUT == SCOUT_ROPE_HALF ? 8 + i : 2 * i + 1;
    const float a = x[ia], b = x[ib];
    x[ia] = __fmaf_rn(a, t.c[i], -__fmul_rn(b, t.s[i]));
    x[ib] = __fmaf_rn(b, t.c[i], __fmul_rn(a, t.s[i]));
  }
}

}  // namespace scout
