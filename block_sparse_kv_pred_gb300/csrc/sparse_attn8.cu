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
// Streaming.  Each warp keeps a ring of two halves (K or V of a step, 4 KB, one TMA box) and
// reloads a half as soon as it has read it.  The places of its steps are resolved 16 steps at a time, a
// tile a lane, one batch ahead.
//
// Tiles.  With at most eight query heads a product's free sides are tokens (scores) and channels
// (output), so both are computed transposed: S^T = K Q^T (16 tokens x 8 heads), O^T += V^T W^T (16
// channels x 8 heads).  The contraction order of the first and the row order of the second are
// free, so a lane takes 16-byte pieces of rows and uses every byte where it lies: no shared memory
// transposes.  A step is 32 tokens: two 16-token tiles, each inside one page.
//
// Split.  A warp gets a contiguous part of the steps of all units, and while it streams it waits for
// nothing but its own copies.  It finishes the units inside its part alone; units that a boundary
// between warps cuts are joined when the warps are done: in shared memory within a CTA, in
// distributed shared memory within a cluster, and across CTAs through the workspace, by the last CTA
// to count itself.  Which of these occurs is a matter of the split:
//   few units, short lists    the CTAs of a cluster take equal parts of one unit;
//   many units                a cluster takes whole units, its steps dealt to its 64 warps;
//   units nearly as many as CTAs, or a long one among many: whole units, or the even split, by CTA.
//
// What bounds it.  mma.sync rather than tcgen05: five to eight query heads fill an eighth of a tcgen05
// tile, and its operands would need q and the weights in 8 bits or K and V widened in shared
// memory.  The products take 52 ns of an SM's time a step (48 at 1.08 ns), the conversions about
// as much; a step's 8 KB take 182 ns of the SM's share of DRAM, so a long launch is bound by DRAM:
// GB300, 4 x 128K tokens dense, 172 us for 1.08 GB (6.2 TB/s, 0.92 of the measured copy bandwidth;
// the SMs' shares of it differ, and the first are done at 0.75 of the time).  40 sequences of 58
// blocks of 32 tokens, 8 x 5 heads: 38.4 us for 152 MB, of which the first 4 go by before the copies start
// (counts, list, page table), 24 stream at 6.3 TB/s, and the rest is the slowest warp and the end
// phase (barrier, join, barrier).  One 4K sequence: 6.7 us, all latency.
#include <atomic>

#include "fp8.cuh"

namespace scout {
namespace {

constexpr int kNW = 8;                 // warps of a CTA
constexpr int kThreads8 = kNW * 32;
constexpr int kCtasPerSm = 2;
// A CTA takes whole units when its warps then have at most this many steps more than with an even
// split, which pays for the even split's joins.  Measured on GB300, whole | even, lists of 58 blocks of
// 32 tokens, 8 KV heads: 1 sequence (7 steps more) 18.3 | 11.3 us, 16 (4 more) 25.7 | 22.2 us, 32 (1
// more) 29.3 | 31.6 us.
constexpr int kWholeSteps = 2;
constexpr int kPieces = 8;             // of a cut unit, merged at a time
// Clusters.  With few units and lists that give each warp at most kClusterSteps steps (as long as they may
// be: the host does not know the counts), the CTAs of a cluster share one unit.  Measured on GB300,
// even split | cluster, lists of 58 blocks of 32 tokens, 8 KV heads x 4: 1 sequence 11.9 | 7.2 us, 8
// 17.2 | 11.4, 16 23.3 | 18.4; 4 of 512 blocks (8 steps a warp) 32.3 | 27.8, 1 of 1,024 (16 steps)
// 27.1 | 33.4.
constexpr int kMaxCluster = 8;
constexpr int kClusterSteps = 8;
// With at least kSnapUnits units for each cluster of kSnap CTAs that the device holds, a cluster takes
// whole units.  Even split | clusters: 40 sequences of 8 x 5 heads, 58 blocks, 41.4 | 38.6 us; with
// ragged lists 47.1 | 39.6; 24 sequences 31.3 | 29.5; 64 of 29 blocks 34.5 | 34.0.
constexpr int kSnap = 8;
constexpr int kSnapUnits = 4;
constexpr int kMaxUnits8 = 4096;
constexpr int kMaxGrid8 = 512;
constexpr int64_t kMaxEntries8 = (int64_t)1 << 28;  // list entries of a launch: at most two steps each, so steps fit an int
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kWBoost = 14;            // weights are kept as 2^14 w, so that their low parts stay normal f16
constexpr int kHalf = 4096;            // K or V of a step: 32 tokens x 128 bytes
// Halves of a warp's ring.  Two, so that an SM has at most 128 KB in flight: with three it had 192
// KB, which bought no bandwidth but longer queues for every other access (40 sequences of 58
// blocks of 32 tokens, 8 KV heads: 42.8 us with two, 46.5 with three; 4 x 128K tokens: 176 and 189 us).
constexpr int kHalves = 2;
constexpr int kBatch = 16;             // steps whose tiles are resolved together (32 tiles, one a lane)
constexpr int kRingBytes8 = kNW * kHalves * kHalf;
constexpr int kTileBytes = kNW * 2 * 2 * kBatch * 16;

// A warp's output state in one half of its ring: channel pair md of group g (channels 16 g + 2 md,
// + 1) of head h, in units of float2; the XOR spreads the stores of a half-warp over all banks.
__device__ __forceinline__ int state_at(int h, int g, int md) {
  return h * 64 + 8 * g + (md ^ ((h >> 1) + 4 * ((g >> 1) & 1)));
}

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
  int32_t* counters;  // [units][kMaxG]
  float* slot_lse;    // [kMaxGrid8][2][kMaxG]
  float* slot_O;      // [kMaxGrid8][2][kMaxG][kD] a CTA's pieces of units it shares with others
  float* piece_O;     // [kMaxGrid8][kNW][kMaxG][kD] a warp's first piece, while it goes on
  int32_t* status;
  int inject;         // SCOUT_INJECT_* (tests)
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
// The same without an addend: no accumulator has to be cleared.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
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

// Where a 16-token tile lies: its first pool row and its tokens (0: nothing there), and its scales.
struct Tile {
  int row, nt;
  float ks, vs;
};
static_assert(sizeof(Tile) == 16, "a tile is one 16-byte shared-memory access");

struct State {
  float m[2], l[2];  // of heads 2t, 2t+1: running max of s, this lane's running sum of 2^(s - m)
  float M[2];        // running max of s + e + 1 (the weights' reference)
  float o[8][4];     // O^T: channels 16g + 2md (+1) x heads 2t, 2t+1
};

// Q^T fragments of unit u: head g, channels 32 t + 4 w .. +3 for k-step w, scaled by a power of two of the head; qf: that factor undone and the softmax scale, for heads 2t, 2t+1.
__device__ __forceinline__ void load_q8(const Attn8Args& a, int u, int lane, uint32_t (&qb)[8][2], float (&qf)[2]) {
  const int g = lane >> 2, t = lane & 3;
  const __nv_bfloat16* row = a.q + ((int64_t)u * a.G + g) * kD + 32 * t;
  uint32_t w[16];
#pragma unroll
  for (int ks = 0; ks < 8; ++ks) {
    const uint2 v = g < a.G ? *reinterpret_cast<const uint2*>(row + 4 * ks) : make_uint2(0u, 0u);
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

// A half stage holds 32 rows of 128 bytes as TMA writes them with its 128-byte swizzle: 16-byte
// piece c of row r lies at piece c ^ (r & 7).  A lane reads whole pieces, and the pieces that eight
// neighbouring lanes read lie in eight different bank groups, for K and for V.
// K of one tile: lane (g, t) takes pieces 2t, 2t + 1 of rows g and g + 8: k[2 x + i] = row g + 8 x.
// V of one tile: piece g of rows 2t, 2t+1, 2t+8, 2t+9.
struct LaneOffsets {
  uint32_t k[2], v[2];  // bytes from the tile's start; row + 8 lies 1024 bytes on
};
__device__ __forceinline__ LaneOffsets lane_offsets(int lane) {
  const int g = lane >> 2, t = lane & 3;
  LaneOffsets o;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    o.k[i] = (uint32_t)(g * 128 + (((2 * t + i) ^ g) << 4));
    o.v[i] = (uint32_t)((2 * t + i) * 128 + ((g ^ (2 * t + i)) << 4));
  }
  return o;
}
__device__ __forceinline__ void read_pieces(const uint8_t* tile, const uint32_t (&off)[2], uint4 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const uint4*>(tile + off[i & 1] + 1024 * (i >> 1));
}
// Rows past the tile's tokens: a stale V code could be NaN, which its weight of zero would not hide.
__device__ __forceinline__ void clear_past(uint4 (&v)[4], int nt, int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (2 * (lane & 3) + (i & 1) + 8 * (i >> 1) >= nt) v[i] = make_uint4(0u, 0u, 0u, 0u);
}

// Scores of a step's two tiles: s[y][0], s[y][1] = token g of tile y, heads 2t, 2t+1; s[y][2], s[y][3] =
// token g + 8.  Both tiles advance together, two chains of products each.
template <int F>
__device__ __forceinline__ void step_scores(const uint8_t* half, const uint32_t (&off)[2], const uint32_t (&qb)[8][2],
                                            float (&s)[2][4]) {
  float s2[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {  // pieces 2t + i: k-steps 4 i .. 4 i + 3
    uint4 lo[2], hi[2];          // rows g and g + 8
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      lo[y] = *reinterpret_cast<const uint4*>(half + y * 2048 + off[i]);
      hi[y] = *reinterpret_cast<const uint4*>(half + y * 2048 + off[i] + 1024);
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        uint32_t a0, a1, a2, a3;
        unpack4<F>(w == 0 ? lo[y].x : w == 1 ? lo[y].y : w == 2 ? lo[y].z : lo[y].w, a0, a2);
        unpack4<F>(w == 0 ? hi[y].x : w == 1 ? hi[y].y : w == 2 ? hi[y].z : hi[y].w, a1, a3);
        if (i == 0 && w < 2) mma_f16_first(w & 1 ? s2[y] : s[y], a0, a1, a2, a3, qb[4 * i + w][0], qb[4 * i + w][1]);
        else mma_f16(w & 1 ? s2[y] : s[y], a0, a1, a2, a3, qb[4 * i + w][0], qb[4 * i + w][1]);
      }
    }
  }
#pragma unroll
  for (int y = 0; y < 2; ++y)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[y][e] += s2[y][e];
}

// O^T += V^T W^T of one tile; w[]: the weights in the layout of the scores.  A tile's products start
// from zero and are added to the sums by an ordinary fp32 addition: the tensor cores drop the low
// bits of what they add to an accumulator, and over a long list those losses add up (128K tokens:
// 1.2e-6 of the output, relative, accumulated in place; 0.65e-6 like this, 2% more time).
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
      float d[4];
      mma_f16_first(d, a[x][0], a[x][1], c[x][0], c[x][1], bl0, bl1);
      mma_f16(d, a[x][0], a[x][1], c[x][0], c[x][1], bh0, bh1);
#pragma unroll
      for (int e = 0; e < 4; ++e) st.o[2 * i + x][e] += d[e];
    }
  }
}

// vs = f 2^e: e (at least -126, so that zero has f = 0), f through the result.  Infinities and NaN are
// their own f, so that they are passed on.
__device__ __forceinline__ float split_scale(float vs, float& e) {
  const int be = max((int)((__float_as_uint(vs) >> 23) & 0xffu), 1);
  e = (float)(be - 127);
  const float f = __uint_as_float((__float_as_uint(vs) & 0x807fffffu) | 0x3f800000u);
  return be <= 1 ? vs * 0x1p126f : be == 255 ? vs : f;
}

// 2^x, results below the normal range as zero (weights and probabilities are relative to 1)
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The sums move only when some head's reference rose (rarely, after the first steps).
__device__ __forceinline__ void rescale(State& st, const float (&al)[2]) {
  if (__all_sync(0xffffffffu, al[0] == 1.f && al[1] == 1.f)) return;
#pragma unroll
  for (int md = 0; md < 8; ++md) {
    st.o[md][0] *= al[0];
    st.o[md][1] *= al[1];
    st.o[md][2] *= al[0];
    st.o[md][3] *= al[1];
  }
}

// Softmax update of one step: the products s become weights, the sums move to the new references.
// Which path is taken is the same for the whole warp.
//
// The usual step: 32 tokens of one page, scales of ordinary size.  One exponential a score gives
// its weight f 2^(s + e + boost - M); the softmax's sum takes the weights' sum times one factor.
__device__ __forceinline__ bool step_weights_page(float (&s)[2][4], const float (&kf)[2], float vs, State& st) {
  float e;
  const float f = split_scale(vs, e);
  float N[2], n[2], shift[2];
  bool near = f != 0.f;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    float b = fmaxf(fmaxf(s[0][c], s[0][2 + c]), fmaxf(s[1][c], s[1][2 + c]));
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, o));
    b *= kf[c];
    n[c] = fmaxf(st.m[c], b);
    N[c] = fmaxf(st.M[c], b + (e + 1.f));
    shift[c] = (e + (float)kWBoost) - N[c];       // weight = f 2^(s + shift)
    near = near && fabsf(n[c] + shift[c]) < 64.f;  // false for NaN and infinities too
  }
  if (!__all_sync(0xffffffffu, near)) return false;
  float al[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    al[c] = fast_exp2(st.M[c] - N[c]);
    float sum = 0.f;
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float w = fast_exp2(fmaf(s[x][2 * r + c], kf[c], shift[c]));
        sum += w;
        s[x][2 * r + c] = w * f;
      }
    // p = 2^(s - n) = 2^(s + shift) 2^-(n + shift)
    st.l[c] = st.l[c] * fast_exp2(st.m[c] - n[c]) + sum * fast_exp2(-(n[c] + shift[c]));
    st.m[c] = n[c];
    st.M[c] = N[c];
  }
  rescale(st, al);
  return true;
}

// Any step: two tiles of different pages and scales, tokens g, g + 8 of tile x past nt[x] masked.
__device__ __forceinline__ void step_weights_any(float (&s)[2][4], const float (&kf)[2][2], int nt0, int nt1, float vs0,
                                              float vs1, int g, State& st) {
  const int nt[2] = {nt0, nt1};
  float e[2], f[2], al[2];
  f[0] = split_scale(vs0, e[0]);
  f[1] = split_scale(vs1, e[1]);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    float b[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
#pragma unroll
      for (int r = 0; r < 2; ++r) s[x][2 * r + c] = g + 8 * r < nt[x] ? s[x][2 * r + c] * kf[x][c] : -INFINITY;
      b[x] = fmaxf(s[x][c], s[x][2 + c]);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) b[x] = fmaxf(b[x], __shfl_xor_sync(0xffffffffu, b[x], o));
    }
    const float n = fmaxf(st.m[c], fmaxf(b[0], b[1]));
    const float N = fmaxf(st.M[c], fmaxf(b[0] + (e[0] + 1.f), b[1] + (e[1] + 1.f)));
    const float base = n == -INFINITY ? 0.f : n, Base = N == -INFINITY ? 0.f : N;  // no finite score yet
    st.l[c] *= fast_exp2(st.m[c] - base);
    al[c] = fast_exp2(st.M[c] - Base);
    st.m[c] = n;
    st.M[c] = N;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const float shift = (e[x] + (float)kWBoost) - Base;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float sc = s[x][2 * r + c];
        st.l[c] += fast_exp2(sc - base);
        s[x][2 * r + c] = fast_exp2(sc + shift) * f[x];
      }
    }
  }
  rescale(st, al);
}

// N steps dealt to Gp CTAs: CTA c takes [first(c), first(c + 1)), first(c) = floor(c N / Gp), written
// with 32-bit arithmetic (c < 2^9, so c (N mod Gp) < 2^18).
struct Ranges {
  int Gp, each, rest;
  float inv;
  __device__ __forceinline__ Ranges(int N, int grid) : Gp(grid) {
    each = N / grid;
    rest = N - each * grid;
    inv = (float)grid / (float)N;
  }
  __device__ __forceinline__ int first(int c) const { return c * each + (int)((unsigned)(c * rest) / (unsigned)Gp); }
  // the CTA whose range holds step x: the estimate is off by one at most
  __device__ __forceinline__ int holder(int x) const {
    int c = min((int)((float)x * inv), Gp - 1);
    if (first(c) > x) --c;
    else if (first(c + 1) <= x) ++c;
    return c;
  }
};

// One head's result, two channel pairs a lane: d2 = lane and lane + 32.  The CPU partial it is merged
// with (merge mode) is loaded ahead of its use.
struct CpuPart8 {
  float2 o[2];
  float lse;
};
__device__ __forceinline__ CpuPart8 load_cpu8(const Attn8Args& a, int u, int h, int lane) {
  CpuPart8 c;
  c.lse = -INFINITY;
  c.o[0] = c.o[1] = make_float2(0.f, 0.f);
  if (a.O_out != nullptr) {
    const int64_t row = (int64_t)u * a.G + h;
    c.lse = a.lse_cpu[row];
    c.o[0] = reinterpret_cast<const float2*>(a.O_cpu + row * kD)[lane];
    c.o[1] = reinterpret_cast<const float2*>(a.O_cpu + row * kD)[lane + 32];
  }
  return c;
}
__device__ __forceinline__ void write_head(const Attn8Args& a, int u, int h, int lane, float lse, const float2 (&o)[2],
                                           const CpuPart8& c) {
  const int64_t row = (int64_t)u * a.G + h;
  if (a.O_out == nullptr) {
    reinterpret_cast<float2*>(a.O_part + row * kD)[lane] = o[0];
    reinterpret_cast<float2*>(a.O_part + row * kD)[lane + 32] = o[1];
    if (lane == 0) a.lse_part[row] = lse;
    return;
  }
  const float m = fmaxf(lse, c.lse);
  float wg = 0.f, wc = 0.f, out = -INFINITY;
  if (lse != -INFINITY || c.lse != -INFINITY) {  // (a NaN on one side is not two empty sides)
    wg = expf(lse - m);
    wc = expf(c.lse - m);
    const float sum = wg + wc;
    out = m + logf(sum);
    wg /= sum;
    wc /= sum;
  }
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    // an empty CPU partial's output is not read: it may never have been written
    const float2 oc = c.lse == -INFINITY ? make_float2(0.f, 0.f) : make_float2(wc * c.o[x].x, wc * c.o[x].y);
    reinterpret_cast<uint32_t*>(a.O_out + row * kD)[lane + 32 * x] = pack_bf16(wg * o[x].x + oc.x, wg * o[x].y + oc.y);
  }
  if (lane == 0 && a.lse_out != nullptr) a.lse_out[row] = out;
}

// The weight f of a lane's piece (m, l, M) in the join of all lanes' pieces: output = pow * sum f o.
// The power of two of the result's size is kept apart, so that no factor leaves the normal range
// while the result lies in it.  A NaN in any piece makes every weight NaN: it is passed on, not
// taken for an empty set.
struct Joined {
  float f, pow, lse;
};
__device__ __forceinline__ Joined join_at(bool has, float m, float l, float M, float top_m, float top_M, float L,
                                          float base) {
  const float E = top_M == -INFINITY ? 0.f : fminf(fmaxf(rintf(top_M - base), -100.f), 100.f);
  const bool none = L == 0.f;
  Joined j;
  j.f = none || !has ? 0.f : __fdividef(fast_exp2(M - base - E), L);
  j.pow = fast_exp2(E - (float)kWBoost);
  j.lse = none ? -INFINITY : (top_m + __log2f(L)) * kLn2;
  return j;
}
// lanes LANES i + w, w < LANES: piece w
template <int LANES = kNW>
__device__ __forceinline__ Joined join(bool has, float m, float l, float M) {
  float top_m = m, top_M = M;
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) {
    top_m = fmaxf(top_m, __shfl_xor_sync(0xffffffffu, top_m, o));
    top_M = fmaxf(top_M, __shfl_xor_sync(0xffffffffu, top_M, o));
  }
  const float base = top_m == -INFINITY ? 0.f : top_m;
  float L = has ? l * fast_exp2(m - base) : 0.f;
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  return join_at(has, m, l, M, top_m, top_M, L, base);
}
__device__ __forceinline__ Joined join_one(float m, float l, float M) {
  const float base = m == -INFINITY ? 0.f : m;
  return join_at(true, m, l, M, m, M, l * fast_exp2(m - base), base);
}

// distributed shared memory of a cluster
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t in_rank(uint32_t smem, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem), "r"(rank));
  return r;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
// the same place as p (shared memory of this CTA) in another CTA of the cluster, as a generic address
template <class T>
__device__ __forceinline__ const T* in_rank_generic(const T* p, uint32_t rank) {
  uint64_t r;
  asm volatile("mapa.u64 %0, %1, %2;" : "=l"(r) : "l"(reinterpret_cast<uint64_t>(p)), "r"(rank));
  return reinterpret_cast<const T*>(r);
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// One warp's steps, streamed through its ring.  MAP: map(x, unit, step) gives the unit of step x of
// the CTA's numbering, and its number in the unit.
template <int P, int F, class MAP>
struct WarpStream {
  const Attn8Args& a;
  const CUtensorMap *tmK, *tmV;
  uint8_t* ring;     // this warp's halves
  Tile* tiles;       // two batches
  uint64_t* full;    // a half has landed
  const MAP& map;
  int lane, wlo, n_mine;  // its steps: wlo + i, i < n_mine
  LaneOffsets off;
  int i, at;         // the next step, and the ring half of its K
  uint32_t phase;    // of that half's barrier
  int n_issue;       // n_mine; 0 once a bounded wait ran out: nothing more is issued or computed
  int lost;          // the half whose wait ran out, -1
  int trigger;       // the step at which the next batch's resolution goes on
  // a tile on its way through the three dependent reads: list entry, page-table slot, scales
  int ru, rj, rlen, rslot, rrow, rnt;
  float rks, rvs;

  __device__ __forceinline__ WarpStream(const Attn8Args& args, const CUtensorMap* k, const CUtensorMap* v, uint8_t* sm,
                                        uint64_t* bars, const MAP& mp, int warp, int ln, int lo, int n)
      : a(args), tmK(k), tmV(v), ring(sm + warp * (kHalves * kHalf)),
        tiles(reinterpret_cast<Tile*>(sm + kRingBytes8) + warp * (4 * kBatch)), full(bars + warp * kHalves), map(mp),
        lane(ln), wlo(lo), n_mine(n), off(lane_offsets(ln)), i(0), at(0), phase(0), n_issue(n), lost(-1),
        trigger(args.inject == SCOUT_INJECT_ABANDON ? min(1, n - 1) : n > kBatch ? 0 : 0x7fffffff), ru(0), rj(-1), rlen(0), rslot(-1), rrow(0), rnt(0), rks(0.f), rvs(0.f) {}

  // Tile 2 kBatch b + lane of this warp.
  __device__ __forceinline__ void resolve_entry(int batch) {
    const int k = batch * kBatch + (lane >> 1), y = lane & 1;
    rj = -1;
    rlen = 0;
    rrow = P == 16 ? 0 : 16 * y;  // first token of the tile in its page
    if (k < n_mine) {
      int step;
      map(wlo + k, ru, step);
      const int entry = P == 16 ? 2 * step + y : P == 32 ? step : step >> 1;
      if (P == 64) rrow += 32 * (step & 1);
      if (P != 16 || entry < min(max(a.res_count[ru], 0), a.k)) {
        rj = a.res_list[(int64_t)ru * a.k + entry];
        rlen = a.seq_len[ru / a.Hkv];
        if (rj < 0 || rj >= a.nblk_cap) rj = -2;
      }
    }
  }
  __device__ __forceinline__ void resolve_slot() {
    rslot = rj >= 0 ? a.page_table[(int64_t)ru * a.nblk_cap + rj] : -1;
  }
  __device__ __forceinline__ void resolve_tile() {
    // in 64 bits: the table's columns may number more tokens than 32 bits do
    const int nv = rj >= 0 ? (int)max((int64_t)0, min((int64_t)P, rlen - (int64_t)rj * P)) : 0;
    const bool fine = nv > 0 && rslot >= 0 && rslot < a.n_slots;
    if (!fine && rj != -1) report(a.status, SCOUT_DEV_BAD_INDEX);
    rnt = fine ? min(max(nv - rrow, 0), 16) : 0;
    rrow = fine ? rslot * P + rrow : 0;
    rks = fine ? __ldg(a.K_scale + rslot) : 0.f;
    rvs = fine ? __ldg(a.V_scale + rslot) : 0.f;
  }
  __device__ __forceinline__ Tile* tile_of(int k, int y) {
    return tiles + ((2 * k) & (4 * kBatch - 1)) + y;
  }

  // Half h: K (even) or V (odd) of step h / 2, into ring half `to` = h % kHalves.  One lane; every
  // lane has read what was there.  The box starts at a whole row (x = 0).
  __device__ __forceinline__ void issue(int h, int to) {
    const int k = h >> 1;
    if (lane != 0 || k >= n_issue) return;
    uint64_t* bar = full + to;
    uint8_t* dst = ring + to * kHalf;
    const CUtensorMap* m = h & 1 ? tmV : tmK;
    const int2 w0 = *reinterpret_cast<const int2*>(tile_of(k, 0));
    if (P != 16) {
      if (w0.y > 0) {
        mbar_arrive_tx(bar, kHalf);
        tma_load_2d(dst, m, 0, w0.x, bar);
      } else {
        mbar_arrive(bar);
      }
      return;
    }
    const int2 w1 = *reinterpret_cast<const int2*>(tile_of(k, 1));
    const uint32_t bytes = (w0.y > 0 ? 2048u : 0u) + (w1.y > 0 ? 2048u : 0u);
    if (bytes == 0u) {
      mbar_arrive(bar);
      return;
    }
    mbar_arrive_tx(bar, bytes);
    if (w0.y > 0) tma_load_2d(dst, m, 0, w0.x, bar);
    if (w1.y > 0) tma_load_2d(dst + 2048, m, 0, w1.x, bar);
  }
  // Waits for half h; false (for the whole warp) once a wait has run out.
  __device__ __forceinline__ bool landed(int h) {
    if (n_issue == 0) return false;
    if (__all_sync(0xffffffffu, mbar_wait(full + at, phase))) return true;
    give_up(h);
    return false;
  }
  // The wait for half h has run out: nothing more is issued or computed.
  __device__ __forceinline__ void give_up(int h) {
    if (lane == 0) report(a.status, SCOUT_DEV_TIMEOUT);
    lost = h;
    n_issue = 0;
  }
  // The next batch's resolution, in four parts while this batch runs.  (Under SCOUT_INJECT_ABANDON: what
  // happens when the wait for this step's K runs out.)
  __device__ __forceinline__ void go_on() {
    if (a.inject == SCOUT_INJECT_ABANDON) {
      trigger = 0x7fffffff;
      give_up(2 * i);
      return;
    }
    const int ib = i % kBatch, next = i / kBatch + 1;
    if (ib == 0) resolve_entry(next);
    if (ib == 4) resolve_slot();
    if (ib == 8) resolve_tile();
    if (ib == 12) {
      tiles[(next & 1) * (2 * kBatch) + lane] = Tile{rrow, rnt, rks, rvs};
      __syncwarp();
    }
    trigger = ib < 12 ? i + 4 : (next + 1) * kBatch < n_mine ? next * kBatch : 0x7fffffff;
  }
  __device__ __forceinline__ void next_half() {
    if (++at == kHalves) {
      at = 0;
      phase ^= 1u;
    }
  }

  __device__ __forceinline__ void begin() {
    resolve_entry(0);
    resolve_slot();
    resolve_tile();
    *reinterpret_cast<int2*>(&tiles[lane].row) = make_int2(rrow, rnt);
    __syncwarp();
    for (int h = 0; h < kHalves; ++h) issue(h, h);
    *reinterpret_cast<float2*>(&tiles[lane].ks) = make_float2(rks, rvs);
    __syncwarp();
  }

  // Steps i .. i_end - 1 (at least one), all of one unit, into its state; leaves the state in the
  // ring half that the last V left, which is not reloaded before release().
  __device__ __forceinline__ float2* run(int i_end, const uint32_t (&qb)[8][2], const float (&qf)[2], State& st) {
    const int g = lane >> 2, t = lane & 3;
    st.m[0] = st.m[1] = st.M[0] = st.M[1] = -INFINITY;
    st.l[0] = st.l[1] = 0.f;
#pragma unroll
    for (int md = 0; md < 8; ++md) st.o[md][0] = st.o[md][1] = st.o[md][2] = st.o[md][3] = 0.f;
    int was;
    while (true) {
      if (i == trigger) go_on();
      const Tile t0 = *tile_of(i, 0), t1 = *tile_of(i, 1);
      const float kf[2][2] = {{t0.ks * qf[0], t0.ks * qf[1]}, {t1.ks * qf[0], t1.ks * qf[1]}};
      float s[2][4];
      bool any = landed(2 * i) && t0.nt + t1.nt > 0;
      if (any) step_scores<F>(ring + at * kHalf, off.k, qb, s);
      // the reads above have returned: the products that use them have been issued
      __syncwarp();
      issue(2 * i + kHalves, at);
      next_half();
      if (any) {
        if (!(P != 16 && t1.nt == 16 && step_weights_page(s, kf[0], t0.vs, st)))
          step_weights_any(s, kf, t0.nt, t1.nt, t0.vs, t1.vs, g, st);
      }
      any = landed(2 * i + 1) && any;
      if (any) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          uint4 v[4];
          const int nt = y ? t1.nt : t0.nt;
          read_pieces(ring + at * kHalf + y * 2048, off.v, v);
          if (nt < 16) clear_past(v, nt, lane);
          tile_output<F>(v, s[y], st);
        }
      }
      __syncwarp();  // every lane has read its V
      was = at;
      next_half();
      if (++i == i_end) break;
      issue(2 * i - 1 + kHalves, was);
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      st.l[0] += __shfl_xor_sync(0xffffffffu, st.l[0], o);
      st.l[1] += __shfl_xor_sync(0xffffffffu, st.l[1], o);
    }
    // steps are missing from this state: as NaN it spoils its heads' results rather than pass for a sum
    if (n_issue == 0) st.l[0] = st.l[1] = __uint_as_float(0x7fffffffu);
    float2* own = reinterpret_cast<float2*>(ring + was * kHalf);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int h = 2 * t + x;
#pragma unroll
      for (int md = 0; md < 8; ++md)
        if (h < a.G) own[state_at(h, g, md)] = make_float2(st.o[md][x], st.o[md][2 + x]);
    }
    return own;
  }
  // The state has been read: the half that held it goes on.
  __device__ __forceinline__ void release(const float2* own) {
    __syncwarp();
    fence_proxy_async();  // the state was written and read by ordinary accesses, the next copy is not one
    issue(2 * i - 1 + kHalves, (int)((reinterpret_cast<const uint8_t*>(own) - ring) / kHalf));
  }
  // Given up: let the copies that were started land (again for a bounded time) before leaving.
  __device__ __forceinline__ void drain() {
    // at most kHalves are on their way: the one that was waited for and what follows it
    for (int h = lost; lost >= 0 && h < min(lost + kHalves, 2 * n_mine); ++h)
      mbar_wait(full + h % kHalves, (uint32_t)(h / kHalves) & 1u);
  }
};

// A head's join of the pieces of a CTA's warps w0 .. w1 (those that have steps), for the whole warp that
// calls it: weights in every lane group of kNW, output in o (channel pairs lane and lane + 32).  lo: where
// warp w's part begins; from: where the unit's begins.
struct Pieces {
  const float2* at[kNW][2];  // a warp's first piece, and its other one: in its ring or the workspace
  float m[kNW][2][kMaxG], l[kNW][2][kMaxG], M[kNW][2][kMaxG];
  __device__ __forceinline__ void put(int warp, int slot, int lane, const float2* where, const State& st) {
    if (lane < 4) {  // row g = 0 of the layout: heads 2t, 2t + 1
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        m[warp][slot][2 * lane + x] = st.m[x];
        l[warp][slot][2 * lane + x] = st.l[x];
        M[warp][slot][2 * lane + x] = st.M[x];
      }
    }
    if (lane == 0) at[warp][slot] = where;
  }
  // has, slot: of warp lane % kNW; slot_of(w): the same slot, for any w
  template <class SLOT>
  __device__ __forceinline__ float join_head(int h, int lane, bool has, SLOT slot_of, float2 (&o)[2]) const {
    const int wl = lane & (kNW - 1), slot = slot_of(wl);
    const Joined j = join(has, has ? m[wl][slot][h] : -INFINITY, has ? l[wl][slot][h] : 0.f,
                          has ? M[wl][slot][h] : -INFINITY);
    float2 p[kNW][2];
    float f[kNW];
#pragma unroll
    for (int w = 0; w < kNW; ++w) {
      f[w] = __shfl_sync(0xffffffffu, j.f, w);
      p[w][0] = p[w][1] = make_float2(0.f, 0.f);
      if (f[w] != 0.f) {
        const float2* src = at[w][slot_of(w)];
        p[w][0] = src[state_at(h, lane >> 3, lane & 7)];
        p[w][1] = src[state_at(h, (lane + 32) >> 3, lane & 7)];
      }
    }
    o[0] = o[1] = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kNW; ++w)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        o[x].x += f[w] * p[w][x].x;
        o[x].y += f[w] * p[w][x].y;
      }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      o[x].x *= j.pow;
      o[x].y *= j.pow;
    }
    return j.lse;
  }
};

// Weighted sum of np <= kPieces finished parts (their own lse, normalised output): lane e % kPieces
// holds lse of part e; read(e, x) loads channel pair lane + 32 x of part e.  Added to (m, L, o).
template <class READ>
__device__ __forceinline__ void add_parts(float lse, int np, int lane, READ read, float& m, float& L, float2 (&o)[2]) {
  float2 p[kPieces][2];
#pragma unroll
  for (int e = 0; e < kPieces; ++e)
#pragma unroll
    for (int x = 0; x < 2; ++x) p[e][x] = e < np ? read(e, x) : make_float2(0.f, 0.f);
  float n = fmaxf(m, lse);
#pragma unroll
  for (int x = kPieces / 2; x > 0; x >>= 1) n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, x));
  const float base = n == -INFINITY ? 0.f : n;
  const float keep = expf(m - base), wt = expf(lse - base);
  float sum = wt;
#pragma unroll
  for (int x = kPieces / 2; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
  L = L * keep + sum;
  m = n;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    o[x].x *= keep;
    o[x].y *= keep;
  }
#pragma unroll
  for (int e = 0; e < kPieces; ++e) {
    const float w = __shfl_sync(0xffffffffu, wt, e);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      o[x].x += w * p[e][x].x;
      o[x].y += w * p[e][x].y;
    }
  }
}
__device__ __forceinline__ void write_parts(const Attn8Args& a, int u, int h, int lane, float m, float L, float2 (&o)[2],
                                            const CpuPart8& cpu) {
  const float r = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    o[x].x *= r;
    o[x].y *= r;
  }
  write_head(a, u, h, lane, L == 0.f ? -INFINITY : m + logf(L), o, cpu);
}

// The end of a cluster that has taken the units of steps [lo, lo + len), dealt to its 64 warps: the
// (unit, head) pairs that boundaries between warps cut are dealt to all of them again, whose steps
// they ever were.  The pieces lie in the warps' rings, or in the workspace.
__device__ __forceinline__ void join_in_cluster(const Attn8Args& a, const int* prefix, const Pieces& pieces, int lo,
                                                int len, int c, int rank, int warp, int lane) {
  auto part = [&](int w) { return lo + (int)(((int64_t)len * w) >> 6); };  // of the cluster's warp w
  auto last_part = [&](int x) {  // the last warp whose part begins at or before step x
    return __popc(__ballot_sync(0xffffffffu, part(lane) <= x)) + __popc(__ballot_sync(0xffffffffu, part(lane + 32) <= x)) - 1;
  };
  // lane, and 32 + lane: the unit at the boundary before warp w + 1, if it is cut there for the first time
  int unit[2];
  uint32_t cut[2];
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const int w = lane + 32 * y + 1, x = part(w);
    unit[y] = owner_of(prefix, a.units, min(x, lo + len - 1));
    cut[y] = __ballot_sync(0xffffffffu, w < 64 && x < lo + len && prefix[unit[y]] < x && part(w - 1) <= prefix[unit[y]]);
  }
  cluster_barrier();
  const int n0 = __popc(cut[0]), tasks = (n0 + __popc(cut[1])) * a.G;
#pragma unroll 1
  for (int task = warp * kSnap + rank; task < tasks; task += kSnap * kNW) {
    const int k = task / a.G, h = task - k * a.G;  // the k-th cut unit
    const bool low = k < n0;
    const uint32_t in = low ? cut[0] : cut[1];
    const int nth = low ? k : k - n0;
    const int from = __ffs(__ballot_sync(0xffffffffu, ((in >> lane) & 1u) != 0u && __popc(in & ((1u << lane) - 1u)) == nth)) - 1;
    const int v = __shfl_sync(0xffffffffu, low ? unit[0] : unit[1], from);
    const CpuPart8 cpu = load_cpu8(a, v, h, lane);
    // the cluster's warps that have steps of it; lane p: piece p, of warp g0 + p
    const int g0 = last_part(prefix[v]), np = last_part(prefix[v + 1] - 1) - g0 + 1;
    const int gw = g0 + min(lane, np - 1), lo_w = part(gw), hi_w = part(gw + 1), w = gw % kNW;
    const bool has = lane < np && lo_w < hi_w;
    const int slot = lo_w >= prefix[v] ? 0 : 1;
    const Pieces* there = in_rank_generic(&pieces, (uint32_t)(gw / kNW));
    float m = -INFINITY, l = 0.f, M = -INFINITY;
    const float2* at = nullptr;
    if (has) {
      m = there->m[w][slot][h];
      l = there->l[w][slot][h];
      M = there->M[w][slot][h];
      if (min(prefix[v + 1], hi_w) == hi_w)  // the warp's last piece: in its ring
        at = in_rank_generic(there->at[w][slot], (uint32_t)(gw / kNW));
      else
        at = reinterpret_cast<const float2*>(a.piece_O + ((int64_t)(c - rank) * kNW + gw) * (kMaxG * kD));
    }
    const Joined j = join<32>(has, m, l, M);
    float2 o[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
    for (int e0 = 0; e0 < np; e0 += kPieces) {
      float2 p[kPieces][2];
      float f[kPieces];
#pragma unroll
      for (int e = 0; e < kPieces; ++e) {
        f[e] = __shfl_sync(0xffffffffu, j.f, (e0 + e) & 31);
        const float2* src = reinterpret_cast<const float2*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(at), (e0 + e) & 31));
        p[e][0] = p[e][1] = make_float2(0.f, 0.f);
        if (e0 + e >= np) f[e] = 0.f;
        if (f[e] != 0.f) {
          p[e][0] = src[state_at(h, lane >> 3, lane & 7)];
          p[e][1] = src[state_at(h, (lane + 32) >> 3, lane & 7)];
        }
      }
#pragma unroll
      for (int e = 0; e < kPieces; ++e)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          o[x].x += f[e] * p[e][x].x;
          o[x].y += f[e] * p[e][x].y;
        }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      o[x].x *= j.pow;
      o[x].y *= j.pow;
    }
    write_head(a, v, h, lane, j.lse, o, cpu);
  }
  cluster_barrier();  // no CTA leaves while another reads its pieces
}

struct FlatMap {  // steps of all units in a row
  const int* prefix;
  int units;
  __device__ __forceinline__ void operator()(int x, int& u, int& step) const {
    u = owner_of(prefix, units, x);
    step = x - prefix[u];
  }
};
struct UnitMap {  // steps of one unit
  int unit;
  __device__ __forceinline__ void operator()(int x, int& u, int& step) const {
    u = unit;
    step = x;
  }
};

// CL: launched in clusters of kSnap CTAs.  As long as no unit is long against a cluster's share, a
// cluster then takes whole units (its share's ends moved to the nearest unit's), deals their steps to
// its warps, and joins them through distributed shared memory; nothing is left to be merged
// through the workspace.
template <int P, int F, bool CL>
__global__ void __launch_bounds__(kThreads8, kCtasPerSm) attn8_kernel(const __grid_constant__ CUtensorMap tmK,
                                                                          const __grid_constant__ CUtensorMap tmV,
                                                                          const Attn8Args a) {
  extern __shared__ uint8_t smem_raw8[];
  // [ring, 1024-byte aligned for the swizzle][tiles][prefix]
  uint8_t* sm8 = smem_raw8 + ((1024u - (smem_u32(smem_raw8) & 1023u)) & 1023u);
  __shared__ uint64_t full[kNW][kHalves];  // a half has landed
  __shared__ int partial[kNW], longest[kNW];
  __shared__ Pieces pieces;
  int* prefix = reinterpret_cast<int*>(sm8 + kRingBytes8 + kTileBytes);  // [units + 1] steps before a unit
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < kNW * kHalves) mbar_init(&full[0][0] + tid, 1);
  if (tid < kNW * kHalves) fence_mbar_init();
  if (tid == 64) {
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  wait_prerequisites();
  // exclusive prefix of the units' steps, a run of units a thread: the counts are read twice, the
  // second time from L1, so that all of a thread's first reads are in flight together
  int most = 0;
  {
    const int per = (a.units + kThreads8 - 1) / kThreads8, u0 = tid * per, u1 = min(a.units, u0 + per);
    int sum = 0;
#pragma unroll 4
    for (int u = u0; u < u1; ++u) {
      const int n = steps_of<P>(min(max(a.res_count[u], 0), a.k));
      sum += n;
      most = max(most, n);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    int run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += x;
    }
    if (lane == 31) {
      partial[warp] = run;
      longest[warp] = most;
    }
    __syncthreads();
    run -= sum;
#pragma unroll
    for (int w = 0; w < kNW; ++w) {
      run += w < warp ? partial[w] : 0;
      most = max(most, longest[w]);
    }
    for (int u = u0; u < u1; ++u) {
      prefix[u] = run;
      run += steps_of<P>(min(max(a.res_count[u], 0), a.k));
    }
    if (tid == kThreads8 - 1) prefix[a.units] = run;
    __syncthreads();
  }
  const int N = prefix[a.units];
  // units with no listed block: O = 0, lse = -inf
  for (int u = blockIdx.x; u < a.units; u += gridDim.x) {
    if (prefix[u + 1] != prefix[u]) continue;
    const float2 none[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    if (warp < a.G) write_head(a, u, warp, lane, -INFINITY, none, load_cpu8(a, u, warp, lane));
  }
  // CTA c takes steps [c N / Gp, (c + 1) N / Gp) of all units, or unit c whole: nothing is cut then,
  // and no merge of pieces (three more round trips) ends the launch.
  const int even = min((int)gridDim.x, (N + kNW - 1) / kNW);
  const bool by_unit = a.units <= (int)gridDim.x &&
                       (most + kNW - 1) / kNW <= (N + even * kNW - 1) / max(even * kNW, 1) + kWholeSteps;
  const int clusters = (int)gridDim.x / kSnap;
  // a unit then lies in at most 32 of the cluster's warps
  const bool snap = CL && !by_unit && most <= N / clusters / kSnapUnits;
  const int Gp = by_unit ? a.units : snap ? clusters : even;
  const int c = blockIdx.x;
  if (!snap && c >= Gp) return;
  const Ranges ranges(max(N, 1), Gp);
  const int rank = CL ? (int)cluster_rank() : 0;
  int lo, len;
  if (snap) {  // lanes 0 and 1: where this cluster's units begin, and the next one's
    const int k = c / kSnap + (lane & 1), x = min(ranges.first(k), N - 1), v = owner_of(prefix, a.units, x);
    int at = k >= Gp ? N : x - prefix[v] <= prefix[v + 1] - x ? prefix[v] : prefix[v + 1];
    if (k == 0) at = 0;
    lo = __shfl_sync(0xffffffffu, at, 0);
    len = __shfl_sync(0xffffffffu, at, 1) - lo;
  } else {
    lo = by_unit ? prefix[c] : ranges.first(c);
    len = (by_unit ? prefix[c + 1] : ranges.first(c + 1)) - lo;
  }
  if (len == 0) return;  // (all CTAs of the cluster alike)
  // steps lo .. lo + len - 1 are dealt evenly to 2^parts_log warps, of which this CTA's first is number w_first
  const int parts_log = snap ? 6 : 3, w_first = snap ? rank * kNW : 0;
  static_assert(kNW == 8 && kSnap * kNW == 64, "parts are eighths or 64ths");
  // A warp's steps are a contiguous part: units that lie inside it are finished by the warp alone,
  // and what a boundary cuts is joined once, when all warps are done.
  auto part = [&](int w) { return lo + (int)(((int64_t)len * (w_first + w)) >> parts_log); };
  const int start = part(0), end = part(kNW);
  const int wlo = part(warp), whi = part(warp + 1), n_mine = whi - wlo;
  const FlatMap map{prefix, a.units};
  WarpStream<P, F, FlatMap> ws(a, &tmK, &tmV, sm8, &full[0][0], map, warp, lane, wlo, n_mine);
  ws.begin();
  int u = n_mine > 0 ? owner_of(prefix, a.units, wlo) : 0;
  for (int pos = wlo; pos < whi;) {
    while (prefix[u + 1] <= pos) ++u;  // the next unit with steps
    const int hi = min(whi, prefix[u + 1]);
    uint32_t qb[8][2];
    float qf[2];
    load_q8(a, u, lane, qb, qf);
    State st;
    float2* own = ws.run(hi - wlo, qb, qf, st);
    __syncwarp();
    if (pos == prefix[u] && hi == prefix[u + 1]) {  // whole: finished here
      CpuPart8 next = load_cpu8(a, u, 0, lane);
      for (int h = 0; h < a.G; ++h) {
        const float m0 = __shfl_sync(0xffffffffu, st.m[0], h >> 1), m1 = __shfl_sync(0xffffffffu, st.m[1], h >> 1);
        const float l0 = __shfl_sync(0xffffffffu, st.l[0], h >> 1), l1 = __shfl_sync(0xffffffffu, st.l[1], h >> 1);
        const float M0 = __shfl_sync(0xffffffffu, st.M[0], h >> 1), M1 = __shfl_sync(0xffffffffu, st.M[1], h >> 1);
        const Joined j = join_one(h & 1 ? m1 : m0, h & 1 ? l1 : l0, h & 1 ? M1 : M0);
        float2 o[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float2 v = own[state_at(h, (lane + 32 * x) >> 3, lane & 7)];
          o[x] = make_float2(j.f * v.x * j.pow, j.f * v.y * j.pow);
        }
        const CpuPart8 cpu = next;
        if (h + 1 < a.G) next = load_cpu8(a, u, h + 1, lane);
        write_head(a, u, h, lane, j.lse, o, cpu);
      }
    } else {
      const float2* where = own;
      if (hi < whi) {  // a first piece with more to come: out of the ring's way
        float4* dst = reinterpret_cast<float4*>(a.piece_O + ((int64_t)c * kNW + warp) * (kMaxG * kD));
        for (int e = lane; e < a.G * (kD / 4); e += 32) dst[e] = reinterpret_cast<const float4*>(own)[e];
        where = reinterpret_cast<const float2*>(dst);
      }
      pieces.put(warp, pos == wlo ? 0 : 1, lane, where, st);
    }
    if (hi < whi) ws.release(own);
    pos = hi;
  }
  ws.drain();
  release_dependents();
  if (CL && snap) {
    join_in_cluster(a, prefix, pieces, lo, len, c, rank, warp, lane);
    return;
  }
  __syncthreads();

  // What boundaries cut, a (unit, head) a warp.  First the units cut by the CTA's ends (at most two):
  // their pieces go to the workspace, and after one fence they are counted; while the answers
  // come back, the units inside that only warp boundaries cut are joined (phase 1).
  const int v0 = owner_of(prefix, a.units, start), v1 = owner_of(prefix, a.units, end - 1);
  const bool cut0 = prefix[v0] < start || prefix[v0 + 1] > end, cut1 = v1 != v0 && prefix[v1 + 1] > end;
  const int n_cut = ((int)cut0 + (int)cut1) * a.G;
  auto cut_unit = [&](int q) { return q < a.G && cut0 ? v0 : v1; };  // of task q: unit, then q % G the head
  auto piece_of = [&](int v, int h, int cc) {
    return (cc * 2 + (prefix[v] <= ranges.first(cc) ? 0 : 1)) * kMaxG + h;
  };
  int arrived = -1;  // of lane k: the count before it of this warp's k-th task
#pragma unroll 1
  for (int phase1 = 0; phase1 < 2; ++phase1) {
    const int tasks = phase1 ? (v1 - v0 + 1) * a.G : n_cut;
#pragma unroll 1
    for (int q = warp; q < tasks; q += kNW) {
      const int h = q % a.G, v = phase1 ? v0 + q / a.G : cut_unit(q);
      const int plo = max(start, prefix[v]), phi = min(end, prefix[v + 1]);
      if (plo >= phi) continue;
      // the warps whose parts hold its ends here
      const int wl = lane & (kNW - 1), lo_w = part(wl);
      const int w0 = __popc(__ballot_sync(0xffffffffu, lane < kNW && lo_w <= plo)) - 1;
      const int w1 = __popc(__ballot_sync(0xffffffffu, lane < kNW && lo_w < phi)) - 1;
      // phase 1: not the cut ones again, nor those that one warp has finished
      if (phase1 && (prefix[v] < start || prefix[v + 1] > end || w0 == w1)) continue;
      CpuPart8 cpu;
      if (phase1) cpu = load_cpu8(a, v, h, lane);
      float2 o[2];
      const float lse = pieces.join_head(h, lane, wl >= w0 && wl <= w1 && lo_w < part(wl + 1),
                                         [&](int w) { return part(w) >= plo ? 0 : 1; }, o);
      if (phase1) {
        write_head(a, v, h, lane, lse, o, cpu);
      } else {
        const int mine = piece_of(v, h, c);
        reinterpret_cast<float2*>(a.slot_O + (int64_t)mine * kD)[lane] = o[0];
        reinterpret_cast<float2*>(a.slot_O + (int64_t)mine * kD)[lane + 32] = o[1];
        if (lane == 0) a.slot_lse[mine] = lse;
      }
    }
    if (phase1 == 0 && warp < n_cut) {
      __threadfence();
      __syncwarp();
      const int q = warp + kNW * lane;  // two tasks a warp at most
      if (lane < 2 && q < n_cut) arrived = atomicAdd(a.counters + (int64_t)cut_unit(q) * kMaxG + q % a.G, 1);
    }
  }
  // a unit of several CTAs: the last to count itself merges the pieces, in the order of the ranges
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    const int q = warp + kNW * k;
    if (q >= n_cut) break;
    const int v = cut_unit(q), h = q % a.G;
    const CpuPart8 cpu = load_cpu8(a, v, h, lane);
    const int c0 = ranges.holder(prefix[v]), c1 = ranges.holder(prefix[v + 1] - 1);
    if (__shfl_sync(0xffffffffu, arrived, k) != c1 - c0) continue;
    __threadfence();
    float m = -INFINITY, L = 0.f;
    float2 o[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
    for (int b0 = c0; b0 <= c1; b0 += kPieces) {  // all loads of a batch together
      const int nb = min(kPieces, c1 - b0 + 1);
      const int e_lane = lane & (kPieces - 1), at_lane = piece_of(v, h, b0 + min(e_lane, nb - 1));
      const float lse = e_lane < nb ? __ldcg(a.slot_lse + at_lane) : -INFINITY;
      int at_piece[kPieces];
#pragma unroll
      for (int e = 0; e < kPieces; ++e) at_piece[e] = __shfl_sync(0xffffffffu, at_lane, e);
      add_parts(lse, nb, lane,
                [&](int e, int x) {
                  return __ldcg(reinterpret_cast<const float2*>(a.slot_O + (int64_t)at_piece[e] * kD) + lane + 32 * x);
                },
                m, L, o);
    }
    write_parts(a, v, h, lane, m, L, o, cpu);
    if (lane == 0) a.counters[(int64_t)v * kMaxG + h] = 0;  // ready for the next call
  }
}

// Few units with short lists: the CTAs of a cluster take equal parts of one unit and join them through
// distributed shared memory, which costs one cluster barrier where the even split's pieces take a
// fence, a count and a read through L2; no prefix over the units is needed either.
template <int P, int F>
__global__ void __launch_bounds__(kThreads8, kCtasPerSm) attn8_cluster_kernel(const __grid_constant__ CUtensorMap tmK,
                                                                                  const __grid_constant__ CUtensorMap tmV,
                                                                                  const Attn8Args a, int cs) {
  extern __shared__ uint8_t smem_raw8[];
  uint8_t* sm8 = smem_raw8 + ((1024u - (smem_u32(smem_raw8) & 1023u)) & 1023u);
  __shared__ uint64_t full[kNW][kHalves];
  __shared__ Pieces pieces;
  __shared__ __align__(16) float2 part_o[kMaxG][kD / 2];  // this CTA's part, head by head
  __shared__ float part_lse[kMaxG];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < kNW * kHalves) mbar_init(&full[0][0] + tid, 1);
  if (tid < kNW * kHalves) fence_mbar_init();
  if (tid == 64) {
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  wait_prerequisites();
  const int u = (int)blockIdx.x / cs, rank = (int)cluster_rank();
  const int n = steps_of<P>(min(max(a.res_count[u], 0), a.k));
  const int start = (int)((int64_t)n * rank / cs), end = (int)((int64_t)n * (rank + 1) / cs), len = end - start;
  auto part = [&](int w) { return start + (int)(((int64_t)len * w) >> 3); };
  const int wlo = part(warp), n_mine = part(warp + 1) - wlo;
  __syncthreads();  // the barriers are ready
  const UnitMap map{u};
  WarpStream<P, F, UnitMap> ws(a, &tmK, &tmV, sm8, &full[0][0], map, warp, lane, wlo, n_mine);
  ws.begin();
  if (n_mine > 0) {
    uint32_t qb[8][2];
    float qf[2];
    load_q8(a, u, lane, qb, qf);
    State st;
    const float2* own = ws.run(n_mine, qb, qf, st);
    pieces.put(warp, 0, lane, own, st);
  }
  ws.drain();
  release_dependents();
  __syncthreads();
  if (warp < a.G) {  // warp h: head h of this CTA's part
    const int wl = lane & (kNW - 1);
    float2 o[2];
    const float lse = pieces.join_head(warp, lane, part(wl) < part(wl + 1), [](int) { return 0; }, o);
    part_o[warp][lane] = o[0];
    part_o[warp][lane + 32] = o[1];
    if (lane == 0) part_lse[warp] = lse;
  }
  // warp w of CTA r finishes head r + cs w
  const int h = rank + cs * warp;
  CpuPart8 cpu;
  if (h < a.G) cpu = load_cpu8(a, u, h, lane);
  cluster_barrier();
  if (h < a.G) {
    float m = -INFINITY, L = 0.f;
    float2 o[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    const int e_lane = lane & (kPieces - 1);
    const float lse = e_lane < cs ? ld_cluster(in_rank(smem_u32(&part_lse[h]), (uint32_t)e_lane)) : -INFINITY;
    add_parts(lse, cs, lane,
              [&](int e, int x) { return ld_cluster2(in_rank(smem_u32(&part_o[h][lane + 32 * x]), (uint32_t)e)); }, m, L, o);
    write_parts(a, u, h, lane, m, L, o, cpu);
  }
  cluster_barrier();  // no CTA leaves while another reads its part
}

// The workspace's layout does not depend on the call's shape: the counters that one call leaves zero
// are those that the next one, of any shape, finds.
constexpr size_t kCounters8 = (size_t)kMaxUnits8 * kMaxG * sizeof(int32_t);
static_assert(kCounters8 == SCOUT_SPARSE_ATTN8_ZERO_BYTES, "as the header says");
// shared memory of the largest launch: two such CTAs fit an SM
constexpr size_t kMostSmem = 1024 + (size_t)kRingBytes8 + kTileBytes + (size_t)(kMaxUnits8 + 1) * 4;
static_assert(kCtasPerSm * (kMostSmem + 8 * 1024) <= 228 * 1024, "two CTAs an SM");
constexpr size_t kSlotLse8 = (size_t)kMaxGrid8 * 2 * kMaxG * sizeof(float);
constexpr size_t kSlotO8 = (size_t)kMaxGrid8 * 2 * kMaxG * kD * sizeof(float);
constexpr size_t kPieceO8 = (size_t)kMaxGrid8 * kNW * kMaxG * kD * sizeof(float);

// The pool as rows of 128 bytes; a box is the rows of a step that lie in one page.
bool make_rows_map(CUtensorMap* map, const void* pool, int64_t rows, int box_rows) {
  const cuuint64_t dims[2] = {kD, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {kD};
  const cuuint32_t box[2] = {kD, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(pool), dims, strides, box, estr,
                      CU_TENSOR_MAP_SWIZZLE_128B) == CUDA_SUCCESS;
}

// Clusters of kSnap CTAs that the current device holds at once (0 if it cannot say): a property of the
// device and the kernel, asked once for each.
template <int P, int F>
int snap_clusters() {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];  // 0: not asked yet, n + 1: n
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return 0;
  const int k = known[dev].load(std::memory_order_relaxed);
  if (k > 0) return k - 1;
  auto kern = attn8_kernel<P, F, true>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kSnap);
  cfg.blockDim = dim3(kThreads8);
  cfg.dynamicSmemBytes = kMostSmem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = kSnap;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMostSmem) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess)
    n = 0;
  cudaGetLastError();
  n = min(n, kMaxGrid8 / kSnap);
  known[dev].store(n + 1, std::memory_order_relaxed);
  return n;
}

template <int P, int F>
int launch_attn8(const Attn8Args& a, const scout_launch* launch, cudaStream_t stream) {
  CUtensorMap tmK, tmV;
  constexpr int kBox = P == 16 ? 16 : 32;
  if (!make_rows_map(&tmK, a.K_pool, a.n_slots * P, kBox) || !make_rows_map(&tmV, a.V_pool, a.n_slots * P, kBox))
    return SCOUT_ERR_UNSUPPORTED;
  const int max_ctas = launch != nullptr ? launch->max_ctas : 0;
  const int limit = max_ctas > 0 ? max_ctas : sm_count() * kCtasPerSm;
  // CTAs a unit, for lists as long as they may be: as many as fit (up to 8) and find a step for each warp
  const int64_t steps = P == 16 ? ((int64_t)a.k + 1) / 2 : P == 32 ? (int64_t)a.k : 2 * (int64_t)a.k;
  int cs = 1;
  while (cs < kMaxCluster && (int64_t)a.units * cs * 2 <= limit && steps > cs * kNW) cs *= 2;
  const bool cluster = cs > 1 && steps <= (int64_t)cs * kNW * kClusterSteps;
  const size_t smem = 1024 + (size_t)kRingBytes8 + kTileBytes + (cluster ? 0 : (size_t)(a.units + 1) * 4);
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads8);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[3];
  cfg.attrs = attr;
  cfg.numAttrs = early_start_attrs(launch, attr, 0);
  auto clusters_of = [&](int n) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = (unsigned)n;
    attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  };
  // the limit is the same for every call, so that calls on several host threads do not lower it for
  // one another
  auto ready = [&](const void* kern) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMostSmem) == cudaSuccess;
  };
  bool sent;
  if (cluster) {
    auto kern = attn8_cluster_kernel<P, F>;
    cfg.gridDim = dim3((unsigned)(a.units * cs));
    clusters_of(cs);
    sent = ready(reinterpret_cast<const void*>(kern)) && cudaLaunchKernelEx(&cfg, kern, tmK, tmV, a, cs) == cudaSuccess;
  } else {
    const int resident = snap_clusters<P, F>();
    const int clusters = max_ctas > 0 ? (max_ctas / kSnap < resident ? max_ctas / kSnap : resident) : resident;
    if (clusters > 0 && a.units >= kSnapUnits * clusters) {
      auto kern = attn8_kernel<P, F, true>;
      cfg.gridDim = dim3((unsigned)(clusters * kSnap));
      clusters_of(kSnap);
      sent = ready(reinterpret_cast<const void*>(kern)) && cudaLaunchKernelEx(&cfg, kern, tmK, tmV, a) == cudaSuccess;
    } else {
      auto kern = attn8_kernel<P, F, false>;
      cfg.gridDim = dim3((unsigned)min(kMaxGrid8, limit));
      sent = ready(reinterpret_cast<const void*>(kern)) && cudaLaunchKernelEx(&cfg, kern, tmK, tmV, a) == cudaSuccess;
    }
  }
  if (!sent) {
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
  if (launch != nullptr && (launch->max_ctas < 0 || (launch->inject != SCOUT_INJECT_NONE &&
                                                     launch->inject != SCOUT_INJECT_ABANDON)))
    return SCOUT_ERR_INVALID_ARG;
  const int64_t units = (int64_t)B * Hkv;
  const int G = Hq / Hkv;
  if (D != kD || !valid_P(P) || G > kMaxG || units > kMaxUnits8 || !aligned16(K_pool) || !aligned16(V_pool) ||
      (reinterpret_cast<uintptr_t>(q) & 7u) || n_slots > 0x7fffffffLL || n_slots * P > 0x7fffffffLL ||
      units * k > kMaxEntries8)
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
  a.slot_lse = reinterpret_cast<float*>(ws + kCounters8);
  a.slot_O = reinterpret_cast<float*>(ws + kCounters8 + kSlotLse8);
  a.piece_O = reinterpret_cast<float*>(ws + kCounters8 + kSlotLse8 + kSlotO8);
  a.status = dev_status;
  a.inject = launch != nullptr ? launch->inject : SCOUT_INJECT_NONE;
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
  return scout::kCounters8 + scout::kSlotLse8 + scout::kSlotO8 + scout::kPieceO8;
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
