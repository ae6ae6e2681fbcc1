// scout_sparse_attn8(_merge): paged GQA decode attention over the listed blocks of an 8-bit cache
// with one scale per slot.  ScoutAttention (arXiv HTML), section 3.2 and Algorithm 1 (A_gpu).
//
//   s_t = scale * ks[slot] * q . k8_t,   p = softmax(s),   O = sum_t p_t vs[slot] v8_t
//
// Arithmetic.  Codes become f16 exactly, and so do the queries: each query head is multiplied by
// the power of two that brings its largest element to [2^14, 2^15), which keeps every bf16 bit of
// elements down to 2^-31 of it.  The products run on the tensor cores (mma.sync m16n8k16, f16 in,
// fp32 accumulate).  A block's K scale multiplies its scores in fp32.  Its V scale goes into the
// weights: with vs = f 2^e, 1 <= f < 2, the weight of a token is f 2^(s + e - M), M the running
// maximum of s + e + 1 over the tokens seen, so it lies in [0, 1] whatever the scales, and a block
// of small values whose tokens take all the probability loses nothing.  The softmax's own sum has
// the plain running maximum.  Weights are split into an f16 high and low part (22 bits), as one
// f16 would be worse than the fp32 partial that is handed on.
//
// Tiles.  With at most eight query heads a product's free sides are tokens (scores) and channels
// (output), so both are computed transposed: S^T = K Q^T (16 tokens x 8 heads), O^T += V^T W^T (16
// channels x 8 heads).  The contraction order of the first and the row order of the second are
// free, so a lane takes 16-byte pieces of rows and uses every byte where it lies: no shared memory
// transposes.  A step is 32 tokens: two 16-token tiles, each inside one page.
//
// Split.  The steps of all units are dealt as contiguous ranges to CTAs; a range's steps go round
// its warps.  Whole units are finished by their CTA, cut ones by the last CTA to arrive.
#include "fp8.cuh"

namespace scout {
namespace {

constexpr int kNW = 8;                 // warps of a CTA
constexpr int kThreads8 = kNW * 32;
constexpr int kCtasPerSm = 2;
constexpr int kMaxUnits8 = 4096;
constexpr int kMaxGrid8 = 1024;
constexpr int64_t kMaxSteps = (int64_t)1 << 29;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kWBoost = 14;            // weights are kept as 2^14 w, so that their low parts stay normal f16
// A warp's output state in shared memory: channel 16 g + x of head h at h * kHS + 18 g + x, which
// spreads the eight-byte stores of a half-warp over all banks.
constexpr int kHS = 148;

struct Attn8Args {
  const __nv_bfloat16* q;
  const uint8_t* K_pool;
  const uint8_t* V_pool;
  const float* K_scale;
  const float* V_scale;
  const int32_t* page_table;
  const int32_t* seq_len;
  const int32_t* res_list;
  const int32_t* res_count;
  int Hkv, G, nblk_cap, k, units;
  int64_t n_slots;
  float scale_log2;  // scale * log2(e)
  float* O_part;
  float* lse_part;
  // merge mode (O_out != nullptr)
  const float* O_cpu;
  const float* lse_cpu;
  __nv_bfloat16* O_out;
  float* lse_out;
  int32_t* counters;  // [units]
  float* slot_lse;    // [kMaxGrid8][2][kMaxG]
  float* slot_O;      // [kMaxGrid8][2][kMaxG][kD]
  int32_t* status;
};

// Steps (32 tokens) of a unit with n listed blocks.
template <int P>
__device__ __forceinline__ int steps_of(int n) {
  return P == 16 ? (n + 1) / 2 : P == 32 ? n : 2 * n;
}

// D = A(16x16, row) * B(16x8, col) + D, f16 inputs, fp32 accumulators.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Where a 16-token tile lies: its first pool row (0 tokens: nothing there), and its scales.
struct Tile {
  int row, nt;
  float ks, vs;
};

struct State {
  float m[2], l[2];  // of heads 2t, 2t+1: running max of s, this lane's running sum of 2^(s - m)
  float M[2];        // running max of s + e + 1 (the weights' reference)
  float o[8][4];     // O^T: channels 16g + 2md (+1) x heads 2t, 2t+1
};

// Q^T fragments of unit u: head g, channels 64 i + 16 t + 4 w .. +3 for k-step 4 i + w, scaled by
// a power of two of the head; qf: that factor undone and the softmax scale, for heads 2t, 2t+1.
__device__ __forceinline__ void load_q8(const Attn8Args& a, int u, int lane, uint32_t (&qb)[8][2], float (&qf)[2]) {
  const int g = lane >> 2, t = lane & 3;
  const __nv_bfloat16* row = a.q + ((int64_t)u * a.G + g) * kD + 16 * t;
  uint32_t w[16];
#pragma unroll
  for (int ks = 0; ks < 8; ++ks) {
    const uint2 v = g < a.G ? *reinterpret_cast<const uint2*>(row + 64 * (ks >> 2) + 4 * (ks & 3)) : make_uint2(0u, 0u);
    w[2 * ks] = v.x;
    w[2 * ks + 1] = v.y;
  }
  uint32_t mx = 0u;
#pragma unroll
  for (int i = 0; i < 16; ++i) mx = max(mx, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
  mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
  const int e = (int)(mx >> 7);                    // biased exponent of the largest magnitude
  const int sh = min(max(14 + 127 - e, -126), 126);  // 2^sh brings it to [2^14, 2^15)
  const float up = __uint_as_float((uint32_t)(sh + 127) << 23);
  const float down = __uint_as_float((uint32_t)(127 - sh) << 23) * a.scale_log2;
#pragma unroll
  for (int ks = 0; ks < 8; ++ks) {
    qb[ks][0] = pack_half(bf16_lo(w[2 * ks]) * up, bf16_hi(w[2 * ks]) * up);
    qb[ks][1] = pack_half(bf16_lo(w[2 * ks + 1]) * up, bf16_hi(w[2 * ks + 1]) * up);
  }
  qf[0] = __shfl_sync(0xffffffffu, down, 8 * t);
  qf[1] = __shfl_sync(0xffffffffu, down, 8 * t + 4);
}

// K of one tile: lane (g, t) holds bytes 16 t .. +15 and 64 + 16 t .. +15 of rows g and g + 8.
// V of one tile: bytes 16 g .. +15 of rows 2t, 2t+1, 2t+8, 2t+9.  Rows past the tile's tokens read
// as zero (a stale V code could be NaN; its weight of zero would not hide it).
__device__ __forceinline__ void load_k(const uint8_t* pool, const Tile& tl, int lane, uint4 (&k)[4]) {
  const int g = lane >> 2, t = lane & 3;
  const uint8_t* p = pool + (int64_t)(tl.row + g) * kD + 16 * t;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    k[i] = g + 8 * (i >> 1) < tl.nt ? ldg_stream(p + 8 * (i >> 1) * kD + 64 * (i & 1)) : make_uint4(0u, 0u, 0u, 0u);
}
__device__ __forceinline__ void load_v(const uint8_t* pool, const Tile& tl, int lane, uint4 (&v)[4]) {
  const int g = lane >> 2, t = lane & 3;
  const uint8_t* p = pool + (int64_t)(tl.row + 2 * t) * kD + 16 * g;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = (i & 1) + 8 * (i >> 1);
    v[i] = 2 * t + r < tl.nt ? ldg_stream(p + r * kD) : make_uint4(0u, 0u, 0u, 0u);
  }
}

// Scores of one tile: s[0], s[1] = token g, heads 2t, 2t+1; s[2], s[3] = token g + 8.
template <int F>
__device__ __forceinline__ void tile_scores(const uint4 (&k)[4], const uint32_t (&qb)[8][2], float (&s)[4]) {
  const uint32_t* lo = reinterpret_cast<const uint32_t*>(&k[0]);  // row g: words 0..7
  const uint32_t* hi = reinterpret_cast<const uint32_t*>(&k[2]);  // row g + 8
  float s2[4] = {0.f, 0.f, 0.f, 0.f};
  s[0] = s[1] = s[2] = s[3] = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    uint32_t a0, a1, a2, a3;
    unpack4<F>(lo[w], a0, a2);
    unpack4<F>(hi[w], a1, a3);
    mma_f16(w & 1 ? s2 : s, a0, a1, a2, a3, qb[w][0], qb[w][1]);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) s[e] += s2[e];
}

// O^T += V^T W^T of one tile; w[]: the weights in the layout of the scores.
template <int F>
__device__ __forceinline__ void tile_output(const uint4 (&v)[4], const float (&w)[4], State& st) {
  const uint32_t ht = pack_half(w[0], w[1]), hb = pack_half(w[2], w[3]);
  const float2 ft = half2_floats(ht), fb = half2_floats(hb);
  const uint32_t lt = pack_half(w[0] - ft.x, w[1] - ft.y), lb = pack_half(w[2] - fb.x, w[3] - fb.y);
  const uint32_t bh0 = transpose8x8(ht), bh1 = transpose8x8(hb);
  const uint32_t bl0 = transpose8x8(lt), bl1 = transpose8x8(lb);
  const uint32_t* r0 = reinterpret_cast<const uint32_t*>(&v[0]);  // token 2t
  const uint32_t* r1 = reinterpret_cast<const uint32_t*>(&v[1]);  // 2t + 1
  const uint32_t* r2 = reinterpret_cast<const uint32_t*>(&v[2]);  // 2t + 8
  const uint32_t* r3 = reinterpret_cast<const uint32_t*>(&v[3]);  // 2t + 9
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // pairs (token 2t, token 2t + 1) of channels 4 i, 4 i + 1 | 4 i + 2, 4 i + 3, and of tokens + 8
    uint32_t a[2][2], c[2][2];
    unpack4<F>(__byte_perm(r0[i], r1[i], 0x5140), a[0][0], a[0][1]);
    unpack4<F>(__byte_perm(r0[i], r1[i], 0x7362), a[1][0], a[1][1]);
    unpack4<F>(__byte_perm(r2[i], r3[i], 0x5140), c[0][0], c[0][1]);
    unpack4<F>(__byte_perm(r2[i], r3[i], 0x7362), c[1][0], c[1][1]);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      mma_f16(st.o[2 * i + x], a[x][0], a[x][1], c[x][0], c[x][1], bh0, bh1);
      mma_f16(st.o[2 * i + x], a[x][0], a[x][1], c[x][0], c[x][1], bl0, bl1);
    }
  }
}

// vs = f 2^e: e (at least -126, so that zero has f = 0), f through the result.
__device__ __forceinline__ float split_scale(float vs, float& e) {
  const int be = max((int)((__float_as_uint(vs) >> 23) & 0xffu), 1);
  e = (float)(be - 127);
  return be <= 1 ? vs * 0x1p126f : __uint_as_float((__float_as_uint(vs) & 0x807fffffu) | 0x3f800000u);
}

// Softmax update of one step (two tiles) and its output.
template <int F>
__device__ __forceinline__ void step_output(float (&s)[2][4], const Tile (&tl)[2], const uint4 (&v)[2][4], State& st) {
  float e[2], f[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) f[x] = split_scale(tl[x].vs, e[x]);
  float al[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    float b0 = fmaxf(s[0][c], s[0][2 + c]), b1 = fmaxf(s[1][c], s[1][2 + c]);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      b0 = fmaxf(b0, __shfl_xor_sync(0xffffffffu, b0, o));
      b1 = fmaxf(b1, __shfl_xor_sync(0xffffffffu, b1, o));
    }
    const float n = fmaxf(st.m[c], fmaxf(b0, b1));
    const float N = fmaxf(st.M[c], fmaxf(b0 + (e[0] + 1.f), b1 + (e[1] + 1.f)));
    const float base = n == -INFINITY ? 0.f : n, Base = N == -INFINITY ? 0.f : N;  // no finite score yet
    st.l[c] *= exp2f(st.m[c] - base);
    al[c] = exp2f(st.M[c] - Base);
    st.m[c] = n;
    st.M[c] = N;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const float ew = (e[x] + (float)kWBoost) - Base;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float sc = s[x][2 * r + c];
        st.l[c] += exp2f(sc - base);
        s[x][2 * r + c] = exp2f(sc + ew) * f[x];
      }
    }
  }
  // the sums move only when some head's reference rose (rarely, after the first steps)
  if (!__all_sync(0xffffffffu, al[0] == 1.f && al[1] == 1.f)) {
#pragma unroll
    for (int md = 0; md < 8; ++md) {
      st.o[md][0] *= al[0];
      st.o[md][1] *= al[1];
      st.o[md][2] *= al[0];
      st.o[md][3] *= al[1];
    }
  }
#pragma unroll
  for (int x = 0; x < 2; ++x)
    if (tl[x].nt > 0) tile_output<F>(v[x], s[x], st);
}

__device__ __forceinline__ int64_t first_of(int c, int64_t N, int Gp) { return (int64_t)c * N / Gp; }
// the CTA whose range holds step x
__device__ __forceinline__ int holder_of(int64_t x, int64_t N, int Gp) { return (int)(((x + 1) * Gp + N - 1) / N) - 1; }

// Final rows of unit u from (fin lse, normalised output): thread d2 of 64 holds channels 2 d2, +1.
__device__ __forceinline__ void write_unit(const Attn8Args& a, int u, int h, int d2, float lse, float2 o) {
  const int64_t row = (int64_t)u * a.G + h;
  if (a.O_out == nullptr) {
    reinterpret_cast<float2*>(a.O_part + row * kD)[d2] = o;
    if (d2 == 0) a.lse_part[row] = lse;
    return;
  }
  const float lc = a.lse_cpu[row];
  const float2 oc = reinterpret_cast<const float2*>(a.O_cpu + row * kD)[d2];
  const float m = fmaxf(lse, lc);
  float wg = 0.f, wc = 0.f, out = -INFINITY;
  if (m != -INFINITY) {
    wg = expf(lse - m);
    wc = expf(lc - m);
    const float sum = wg + wc;
    out = m + logf(sum);
    wg /= sum;
    wc /= sum;
  }
  reinterpret_cast<uint32_t*>(a.O_out + row * kD)[d2] = pack_bf16(wg * o.x + wc * oc.x, wg * o.y + wc * oc.y);
  if (d2 == 0 && a.lse_out != nullptr) a.lse_out[row] = out;
}

template <int P, int F>
__global__ void __launch_bounds__(kThreads8, kCtasPerSm) attn8_kernel(const Attn8Args a) {
  extern __shared__ __align__(16) float sm8[];
  __shared__ int partial[32];
  __shared__ float wm[kMaxG][kNW], wl[kMaxG][kNW], wM[kMaxG][kNW], ww[kMaxG][kNW], own_lse[kMaxG], unit_pow[kMaxG];
  __shared__ int last_piece;
  float* wo = sm8;                                                   // [kNW][G][kHS]
  int* prefix = reinterpret_cast<int*>(sm8 + kNW * a.G * kHS);       // [units + 1] steps before a unit
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  wait_prerequisites();
  for (int u = tid; u < a.units; u += kThreads8) prefix[u] = steps_of<P>(min(max(a.res_count[u], 0), a.k));
  __syncthreads();
  cta_exclusive_prefix(prefix, a.units, partial);
  const int64_t N = prefix[a.units];
  // units with no listed block: O = 0, lse = -inf
  for (int u = blockIdx.x; u < a.units; u += gridDim.x) {
    if (prefix[u + 1] != prefix[u]) continue;
    for (int i = tid; i < a.G * (kD / 2); i += kThreads8)
      write_unit(a, u, i >> 6, i & 63, -INFINITY, make_float2(0.f, 0.f));
  }
  const int Gp = (int)min((int64_t)gridDim.x, (N + kNW - 1) / kNW);
  const int c = blockIdx.x;
  if (c >= Gp) return;
  const int64_t start = first_of(c, N, Gp), end = first_of(c + 1, N, Gp);
  int u = owner_of(prefix, a.units, (int)start);
  for (int64_t pos = start; pos < end;) {
    while (prefix[u + 1] <= pos) ++u;  // the next unit with steps
    const int64_t hi = min(end, (int64_t)prefix[u + 1]);
    const int b = u / a.Hkv, len = a.seq_len[b], n = min(max(a.res_count[u], 0), a.k);
    uint32_t qb[8][2];
    float qf[2];
    load_q8(a, u, lane, qb, qf);
    State st;
    st.m[0] = st.m[1] = st.M[0] = st.M[1] = -INFINITY;
    st.l[0] = st.l[1] = 0.f;
#pragma unroll
    for (int md = 0; md < 8; ++md) st.o[md][0] = st.o[md][1] = st.o[md][2] = st.o[md][3] = 0.f;
    for (int64_t x = pos + warp; x < hi; x += kNW) {
      const int step = (int)(x - prefix[u]);
      Tile tl[2];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int entry = P == 16 ? 2 * step + y : P == 32 ? step : step >> 1;
        const int off = P == 16 ? 0 : P == 32 ? 16 * y : 32 * (step & 1) + 16 * y;  // first token in the page
        tl[y] = Tile{0, 0, 0.f, 0.f};
        if (entry < n) {
          const int j = a.res_list[(int64_t)u * a.k + entry];
          const int nv = j >= 0 && j < a.nblk_cap ? min(P, len - j * P) : 0;
          const int slot = nv > 0 ? a.page_table[(int64_t)u * a.nblk_cap + j] : -1;
          if (slot < 0 || slot >= a.n_slots) {
            if (lane == 0) report(a.status, SCOUT_DEV_BAD_INDEX);
          } else {
            tl[y].row = slot * P + off;
            tl[y].nt = min(max(nv - off, 0), 16);
            tl[y].ks = a.K_scale[slot];
            tl[y].vs = a.V_scale[slot];
          }
        }
      }
      if (tl[0].nt + tl[1].nt == 0) continue;
      uint4 kk[4], vv[2][4];
      float s[2][4];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        load_k(a.K_pool, tl[y], lane, kk);
        tile_scores<F>(kk, qb, s[y]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          s[y][e] = g + 8 * (e >> 1) < tl[y].nt ? s[y][e] * (tl[y].ks * qf[e & 1]) : -INFINITY;
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) load_v(a.V_pool, tl[y], lane, vv[y]);
      step_output<F>(s, tl, vv, st);
    }
    // the warps' states of this segment, through shared memory
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      st.l[0] += __shfl_xor_sync(0xffffffffu, st.l[0], o);
      st.l[1] += __shfl_xor_sync(0xffffffffu, st.l[1], o);
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int h = 2 * t + x;
      if (h >= a.G) continue;
      if (g == 0) {
        wm[h][warp] = st.m[x];
        wl[h][warp] = st.l[x];
        wM[h][warp] = st.M[x];
      }
      float2* dst = reinterpret_cast<float2*>(wo + (warp * a.G + h) * kHS + 18 * g);
#pragma unroll
      for (int md = 0; md < 8; ++md) dst[md] = make_float2(st.o[md][x], st.o[md][2 + x]);
    }
    __syncthreads();
    if (tid < a.G) {
      float m = -INFINITY, L = 0.f;
      for (int w = 0; w < kNW; ++w) m = fmaxf(m, wm[tid][w]);
      const float base = m == -INFINITY ? 0.f : m;
      for (int w = 0; w < kNW; ++w) L += wl[tid][w] * exp2f(wm[tid][w] - base);
      // a NaN anywhere makes L NaN: it is passed on, not taken for an empty set
      const bool none = L == 0.f;
      // the power of two of the result's size is kept apart, so that no factor leaves the normal
      // range while the result lies in it
      float top = -INFINITY;
      for (int w = 0; w < kNW; ++w) top = fmaxf(top, wM[tid][w]);
      const float E = top == -INFINITY ? 0.f : fminf(fmaxf(rintf(top - base), -100.f), 100.f);
      for (int w = 0; w < kNW; ++w) ww[tid][w] = none ? 0.f : exp2f(wM[tid][w] - base - E) / L;
      unit_pow[tid] = exp2f(E - (float)kWBoost);
      own_lse[tid] = none ? -INFINITY : (m + log2f(L)) * kLn2;
    }
    __syncthreads();
    const bool whole = pos == prefix[u] && hi == prefix[u + 1];
    const int64_t piece = (int64_t)c * 2 + (prefix[u] <= start ? 0 : 1);
    for (int i = tid; i < a.G * (kD / 2); i += kThreads8) {
      const int h = i >> 6, d2 = i & 63;
      float2 o = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kNW; ++w) {
        const float2 v = reinterpret_cast<const float2*>(wo + (w * a.G + h) * kHS + 18 * (d2 >> 3))[d2 & 7];
        o.x += ww[h][w] * v.x;
        o.y += ww[h][w] * v.y;
      }
      o.x *= unit_pow[h];
      o.y *= unit_pow[h];
      if (whole) {
        write_unit(a, u, h, d2, own_lse[h], o);
      } else {
        reinterpret_cast<float2*>(a.slot_O + (piece * kMaxG + h) * kD)[d2] = o;
        if (d2 == 0) a.slot_lse[piece * kMaxG + h] = own_lse[h];
      }
    }
    if (!whole) {
      // the last CTA to count itself merges the pieces, in the order of the ranges
      const int c0 = holder_of(prefix[u], N, Gp), c1 = holder_of(prefix[u + 1] - 1, N, Gp);
      __threadfence();
      __syncthreads();
      if (tid == 0) last_piece = atomicAdd(&a.counters[u], 1) == c1 - c0;
      __syncthreads();
      if (last_piece) {
        __threadfence();
        for (int i = tid; i < a.G * (kD / 2); i += kThreads8) {
          const int h = i >> 6, d2 = i & 63;
          float m = -INFINITY, L = 0.f;
          float2 o = make_float2(0.f, 0.f);
          for (int cc = c0; cc <= c1; ++cc) {
            const int64_t pc = (int64_t)cc * 2 + (prefix[u] <= first_of(cc, N, Gp) ? 0 : 1);
            const float lse = __ldcg(a.slot_lse + pc * kMaxG + h);
            const float2 v = __ldcg(reinterpret_cast<const float2*>(a.slot_O + (pc * kMaxG + h) * kD) + d2);
            if (lse == -INFINITY) continue;  // a piece without tokens weighs nothing
            const float n = fmaxf(m, lse), keep = expf(m - n), w = expf(lse - n);
            o.x = o.x * keep + w * v.x;
            o.y = o.y * keep + w * v.y;
            L = L * keep + w;
            m = n;
          }
          const float r = L == 0.f ? 0.f : 1.f / L;
          write_unit(a, u, h, d2, L == 0.f ? -INFINITY : m + logf(L), make_float2(o.x * r, o.y * r));
        }
        if (tid == 0) a.counters[u] = 0;  // ready for the next call
      }
    }
    __syncthreads();  // the shared state may be written again
    pos = hi;
  }
  release_dependents();
}

inline size_t counters8_bytes(int64_t units) { return (size_t)((units * 4 + 255) / 256 * 256); }
constexpr size_t kSlotLse8 = (size_t)kMaxGrid8 * 2 * kMaxG * sizeof(float);
constexpr size_t kSlotO8 = (size_t)kMaxGrid8 * 2 * kMaxG * kD * sizeof(float);

template <int P, int F>
int launch_attn8(const Attn8Args& a, const scout_launch* launch, cudaStream_t stream) {
  auto kern = attn8_kernel<P, F>;
  const size_t smem = (size_t)kNW * a.G * kHS * sizeof(float) + (size_t)(a.units + 1) * 4;
  if (smem > 32 * 1024 &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return SCOUT_ERR_CUDA;
  const int max_ctas = launch != nullptr ? launch->max_ctas : 0;
  const int grid = min(kMaxGrid8, max_ctas > 0 ? max_ctas : sm_count() * kCtasPerSm);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads8);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  cfg.numAttrs = early_start_attrs(launch, attr, 0);
  if (cudaLaunchKernelEx(&cfg, kern, a) != cudaSuccess) {
    cudaGetLastError();
    return SCOUT_ERR_CUDA;
  }
  return launch_status();
}
template <int F>
int attn8_by_P(int P, const Attn8Args& a, const scout_launch* launch, cudaStream_t stream) {
  switch (P) {
    case 16: return launch_attn8<16, F>(a, launch, stream);
    case 32: return launch_attn8<32, F>(a, launch, stream);
    default: return launch_attn8<64, F>(a, launch, stream);
  }
}

int attn8_entry(int fmt, const void* q, const void* K_pool, const void* V_pool, const float* K_scale,
                const float* V_scale, int64_t n_slots, const int32_t* page_table, const int32_t* seq_len,
                const int32_t* res_list, const int32_t* res_count, int B, int Hq, int Hkv, int D, int P, int nblk_cap,
                int k, float scale, float* O_part, float* lse_part, const float* O_cpu, const float* lse_cpu,
                __nv_bfloat16* O_out, float* lse_out, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                const scout_launch* launch, cudaStream_t stream) {
  const bool merge = O_out != nullptr;
  if (q == nullptr || K_pool == nullptr || V_pool == nullptr || K_scale == nullptr || V_scale == nullptr ||
      page_table == nullptr || seq_len == nullptr || res_list == nullptr || res_count == nullptr)
    return SCOUT_ERR_INVALID_ARG;
  if (merge ? (O_cpu == nullptr || lse_cpu == nullptr) : (O_part == nullptr || lse_part == nullptr))
    return SCOUT_ERR_INVALID_ARG;
  if (!valid_fp8(fmt) || B <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || n_slots <= 0 || nblk_cap <= 0 || k <= 0 ||
      !(scale > 0.f))
    return SCOUT_ERR_INVALID_ARG;
  if (launch != nullptr && launch->max_ctas < 0) return SCOUT_ERR_INVALID_ARG;
  const int64_t units = (int64_t)B * Hkv;
  const int G = Hq / Hkv;
  if (D != kD || !valid_P(P) || G > kMaxG || units > kMaxUnits8 || !aligned16(K_pool) || !aligned16(V_pool) ||
      (reinterpret_cast<uintptr_t>(q) & 7u) || n_slots * P > 0x7fffffffLL || units * k > kMaxSteps / 2)
    return SCOUT_ERR_UNSUPPORTED;
  if (merge ? (reinterpret_cast<uintptr_t>(O_cpu) & 7u) || (reinterpret_cast<uintptr_t>(O_out) & 3u)
            : (reinterpret_cast<uintptr_t>(O_part) & 7u))
    return SCOUT_ERR_UNSUPPORTED;
  if (workspace == nullptr || workspace_bytes < scout_sparse_attn8_workspace_bytes(B, Hq, Hkv, D, P))
    return SCOUT_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) & 15u) return SCOUT_ERR_UNSUPPORTED;
  Attn8Args a;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.K_pool = static_cast<const uint8_t*>(K_pool);
  a.V_pool = static_cast<const uint8_t*>(V_pool);
  a.K_scale = K_scale;
  a.V_scale = V_scale;
  a.page_table = page_table;
  a.seq_len = seq_len;
  a.res_list = res_list;
  a.res_count = res_count;
  a.Hkv = Hkv;
  a.G = G;
  a.nblk_cap = nblk_cap;
  a.k = k;
  a.units = (int)units;
  a.n_slots = n_slots;
  a.scale_log2 = scale * kLog2e;
  a.O_part = O_part;
  a.lse_part = lse_part;
  a.O_cpu = O_cpu;
  a.lse_cpu = lse_cpu;
  a.O_out = O_out;
  a.lse_out = lse_out;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.counters = reinterpret_cast<int32_t*>(ws);
  a.slot_lse = reinterpret_cast<float*>(ws + counters8_bytes(units));
  a.slot_O = reinterpret_cast<float*>(ws + counters8_bytes(units) + kSlotLse8);
  a.status = dev_status;
  return fmt == SCOUT_FP8_E4M3 ? attn8_by_P<SCOUT_FP8_E4M3>(P, a, launch, stream)
                               : attn8_by_P<SCOUT_FP8_E5M2>(P, a, launch, stream);
}

}  // namespace
}  // namespace scout

extern "C" size_t scout_sparse_attn8_workspace_bytes(int B, int Hq, int Hkv, int D, int P) {
  (void)Hq;
  (void)D;
  (void)P;
  if (B <= 0 || Hkv <= 0) return 0;
  return scout::counters8_bytes((int64_t)B * Hkv) + scout::kSlotLse8 + scout::kSlotO8;
}

extern "C" int scout_sparse_attn8(int fmt, const void* q, const void* K_pool, const void* V_pool,
                                  const float* K_scale, const float* V_scale, int64_t n_slots,
                                  const int32_t* page_table, const int32_t* seq_len, const int32_t* res_list,
                                  const int32_t* res_count, int B, int Hq, int Hkv, int D, int P, int nblk_cap, int k,
                                  float scale, float* O_part, float* lse_part, void* workspace, size_t workspace_bytes,
                                  int32_t* dev_status, const scout_launch* launch, cudaStream_t stream) {
  if (O_part == nullptr || lse_part == nullptr) return SCOUT_ERR_INVALID_ARG;
  return scout::attn8_entry(fmt, q, K_pool, V_pool, K_scale, V_scale, n_slots, page_table, seq_len, res_list,
                            res_count, B, Hq, Hkv, D, P, nblk_cap, k, scale, O_part, lse_part, nullptr, nullptr,
                            nullptr, nullptr, workspace, workspace_bytes, dev_status, launch, stream);
}

extern "C" int scout_sparse_attn8_merge(int fmt, const void* q, const void* K_pool, const void* V_pool,
                                        const float* K_scale, const float* V_scale, int64_t n_slots,
                                        const int32_t* page_table, const int32_t* seq_len, const int32_t* res_list,
                                        const int32_t* res_count, int B, int Hq, int Hkv, int D, int P, int nblk_cap,
                                        int k, float scale, const float* O_cpu, const float* lse_cpu, void* O_out,
                                        float* lse_out, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                        const scout_launch* launch, cudaStream_t stream) {
  if (O_out == nullptr) return SCOUT_ERR_INVALID_ARG;
  return scout::attn8_entry(fmt, q, K_pool, V_pool, K_scale, V_scale, n_slots, page_table, seq_len, res_list,
                            res_count, B, Hq, Hkv, D, P, nblk_cap, k, scale, nullptr, nullptr, O_cpu, lse_cpu,
                            static_cast<__nv_bfloat16*>(O_out), lse_out, workspace, workspace_bytes, dev_status,
                            launch, stream);
}
