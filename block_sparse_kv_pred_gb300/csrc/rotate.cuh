// A head's norm and its turn by a position, shared by the kernels that make queries and keys.
//
// Eight lanes hold a head: lane `sub` two chunks of eight channels, placed so that both channels of
// each of its pairs are its own, and its pairs are 8 sub .. 8 sub + 7 in either layout.  No shuffle is
// needed to turn, three to sum the squares, and a warp moves four heads of consecutive tokens with
// 16-byte accesses.  A lane's cosines and sines depend on the token alone: they are made once and serve
// every head of the token.
//
// The angle is an integer product modulo 2^64 (turns as fractions of 2^64), so a far position costs no
// precision beside the table's own, and no reduction.  Every rounding is
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
// 2^-28, the cosine to 2^-34).  Off by at most 1.7 and 1.2 times 2^-24, and by 2.9 and 1.7 times 2^-24 of themselves,
// over 2 million angles (bounds by arithmetic: 4 and 3 of themselves), with a third of the instructions of sincospi, whose code a short launch has to fetch.
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
  float p[4];  // four sums side by side: a chain of sixteen would be waited for
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = __fmul_rn(x[i], x[i]);
#pragma unroll
  for (int i = 4; i < 16; ++i) p[i & 3] = __fmaf_rn(x[i], x[i], p[i & 3]);
  float ss = __fadd_rn(__fadd_rn(p[0], p[1]), __fadd_rn(p[2], p[3]));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, o));
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

// The same with two values an instruction (fma.rn.f32x2), bit for bit: fewer instructions, but more registers that have to lie
// in pairs.  GB300: the keys and values of the 8-bit write's prompts take 94 us without and 90 us with it; the
// queries, and everything in the bf16 write, are slower with it (266 -> 338 us: their loads no longer go out together).
using f2 = unsigned long long;
__device__ __forceinline__ f2 pair2(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 split2(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// A lane's 16 channels: the first and the second of its pairs (the channels of its two chunks, in a lane that does not turn).
struct Pairs {
  f2 a[4], b[4];
};
template <int LAYOUT>
__device__ __forceinline__ Pairs unpack_pairs(const uint4& lo, const uint4& hi) {
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  Pairs x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (LAYOUT == SCOUT_ROPE_HALF) {
      x.a[i] = pair2(bf16_lo(w[i]), bf16_hi(w[i]));
      x.b[i] = pair2(bf16_lo(w[4 + i]), bf16_hi(w[4 + i]));
    } else {
      x.a[i] = pair2(bf16_lo(w[2 * i]), bf16_lo(w[2 * i + 1]));
      x.b[i] = pair2(bf16_hi(w[2 * i]), bf16_hi(w[2 * i + 1]));
    }
  }
  return x;
}
template <int LAYOUT>
__device__ __forceinline__ void pack_pairs(const Pairs& x, uint4& lo, uint4& hi) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = split2(x.a[i]), b = split2(x.b[i]);
    w[LAYOUT == SCOUT_ROPE_HALF ? i : 2 * i] = LAYOUT == SCOUT_ROPE_HALF ? pack_bf16(a.x, a.y) : pack_bf16(a.x, b.x);
    w[LAYOUT == SCOUT_ROPE_HALF ? 4 + i : 2 * i + 1] = LAYOUT == SCOUT_ROPE_HALF ? pack_bf16(b.x, b.y) : pack_bf16(a.y, b.y);
  }
  lo = make_uint4(w[0], w[1], w[2], w[3]);
  hi = make_uint4(w[4], w[5], w[6], w[7]);
}
template <int LAYOUT>
__device__ __forceinline__ void norm_pairs(Pairs& x, const Weights& weights, float eps) {
  // the four sums of norm_head, two in each of these, in its order
  f2 s0 = mul2(x.a[0], x.a[0]), s1 = LAYOUT == SCOUT_ROPE_HALF ? mul2(x.a[1], x.a[1]) : mul2(x.b[0], x.b[0]);
  float ss;
  if (LAYOUT == SCOUT_ROPE_HALF) {
    s0 = fma2(x.b[2], x.b[2], fma2(x.b[0], x.b[0], fma2(x.a[2], x.a[2], s0)));
    s1 = fma2(x.b[3], x.b[3], fma2(x.b[1], x.b[1], fma2(x.a[3], x.a[3], s1)));
    const float2 p = split2(s0), q = split2(s1);
    ss = __fadd_rn(__fadd_rn(p.x, p.y), __fadd_rn(q.x, q.y));
  } else {
#pragma unroll
    for (int i = 1; i < 4; ++i) {
      s0 = fma2(x.a[i], x.a[i], s0);
      s1 = fma2(x.b[i], x.b[i], s1);
    }
    const float2 p = split2(s0), q = split2(s1);
    ss = __fadd_rn(__fadd_rn(p.x, q.x), __fadd_rn(p.y, q.y));
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, o));
  const float r = rsqrtf(__fmaf_rn(ss, 1.f / kD, eps));
  const f2 r2 = pair2(r, r);
  const Pairs w = unpack_pairs<LAYOUT>(weights.a, weights.b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x.a[i] = mul2(mul2(x.a[i], r2), w.a[i]);
    x.b[i] = mul2(mul2(x.b[i], r2), w.b[i]);
  }
}
// c, s: cosines and sines of the lane's pairs, in order
__device__ __forceinline__ void turn_pairs(Pairs& x, const f2 (&c)[4], const f2 (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f2 a = x.a[i], b = x.b[i];
    x.a[i] = fma2(a, c[i], mul2(b, s[i]) ^ 0x8000000080000000ull);
    x.b[i] = fma2(b, c[i], mul2(a, s[i]));
  }
}

}  // namespace scout
