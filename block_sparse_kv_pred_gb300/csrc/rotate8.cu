// scout_append_rotated_kv8: new keys normalised, turned and quantised on their way into 8-bit pools with
// their values, and the same tokens' queries normalised and turned beside them.
//
// Eight lanes hold a token's row (rotate.cuh).  A warp takes the K or the V of a touched block of one KV head: its new rows
// sit in registers, four a step, are read once, turned, rounded to bf16, their maximum is taken, and the codes are made
// from the registers.  Two kernels, by how many new tokens a sequence has:
//
// Many: a CTA takes a block and some or all of its KV heads.  Its cosines and sines, which all heads share, are made
// once, into shared memory, while the first heads' rows are on their way.  Other CTAs take the queries, a warp four
// tokens and up to 16 heads, their cosines in registers.
//
// Few (a decode step): a warp takes one head of a block, or one query head of four tokens, with no barrier and little code.
//
// GB300, 8 prompts of up to 16K tokens, 8 KV and 32 query heads: 260 us for 1.57 GB (6.0 TB/s, 0.90 of the measured
// copy bandwidth; blocks of 16 tokens 258, of 64 266), bound by how well 16 warps an SM overlap arithmetic and
// loads (the keys and values alone: 90 us, against 70 of scout_append_kv8 without turns).  A warp that made its own rows'
// cosines for each head: 351 us; a CTA's warps holding four rows each of all heads, joined by its barrier: 302; half as
// many rows a warp: 262, but 26 us instead of 24 for 8 prompts of 1,000 tokens.  A decode step of 40 sequences: 4.2 us, a
// chain of dependent reads (lengths, slot and rows, scale).
#include "fp8.cuh"
#include "rotate.cuh"

namespace scout {

int check_heads(const void* x, int64_t ld_x, const void* out, int64_t ld_out, int heads, int D, const scout_rope* rope,
                const void* norm, float eps);  // rotate.cu

namespace {

constexpr int kR8Warps = 4;
constexpr int kR8PerSm = 4;  // CTAs of the first kernel an SM (128 registers)
// GB300, 8 prompts of up to 16K tokens (8 KV, 32 query heads): 265 us with four times as many CTAs as run at a time, for the
// hardware to deal out; 294 with once, 267 with sixteen times.
constexpr int kR8Waves = 4;
constexpr int kR8Heads = 16;  // query heads of a warp, one turn made for them
// New tokens a sequence up to which a call is the second kernel's.  40 sequences (8 KV, 40 query heads), us, first / second
// kernel: one token 11.2 / 4.1, 8: 11.7 / 7.0, 16: 12.9 / 12.3, 24: 15.3 / 17.6, 32: 17.3 / 23.9.  The mean decides, so a
// chunk among many single tokens is the second kernel's as well: 255 of them and 3,800 tokens of another sequence (8 KV, 32 query
// heads) take 61.5 us in one call, 9.4 and 22.2 in two.
constexpr int kFewTokens = 16;
constexpr int kHold = 8;  // row steps that a warp holds: a larger block is a set of warps'

struct Rot8Args {
  const __nv_bfloat16 *kv[2], *q;  // new rows
  int64_t ld[2], ld_q, ld_q_out;
  __nv_bfloat16* q_out;
  const __nv_bfloat16 *k_norm, *q_norm;
  uint8_t* pool[2];
  float* scale[2];
  const int32_t *positions, *prev_len, *seq_len, *page_table;
  int n_tokens, B, Hkv, Hq, nblk_cap;
  int kv_heads, kv_ctas;  // KV heads of a CTA's item, CTAs that take them
  int q_per, q_parts;     // query heads of a warp, warps of four tokens
  int64_t n_slots;
  Rope rope;
  float eps;
  int32_t* status;
};

// The lane's position of token row i (its index in the sequence where none are given).
__device__ __forceinline__ uint32_t position_of(const Rot8Args& a, int64_t i, int index, bool live, int sub) {
  if (a.positions == nullptr || !live) return (uint32_t)max(index, 0);
  const int pos = a.positions[i];
  if (pos < 0 && sub == 0) report(a.status, SCOUT_DEV_BAD_INDEX);
  return (uint32_t)max(pos, 0);
}

__device__ __forceinline__ uint32_t max_finite(uint32_t m, const uint4& x) {
  return max_abs2(max_abs2(max_abs2(max_abs2(m, finite2(x.x)), finite2(x.y)), finite2(x.z)), finite2(x.w));
}
__device__ __forceinline__ uint32_t max_all(uint32_t m, const uint4& x) {
  return max_abs2(max_abs2(max_abs2(max_abs2(m, x.x), x.y), x.z), x.w);
}
__device__ __forceinline__ uint32_t warp_max(uint32_t m) {
  return __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
}

// A touched block: its sequence's part, the same for all its heads.
struct Block {
  int b, j, r0, r1;  // new rows [r0, r1)
  int64_t i0;        // token row of its row 0
};
template <int P>
__device__ __forceinline__ Block block_of(const Rot8Args& a, const int* tok, const int* tou, int blk) {
  Block k;
  k.b = owner_of(tou, a.B, blk);
  const SeqSpan s = seq_span(a.prev_len, a.seq_len, k.b, a.nblk_cap * P);
  k.j = s.prev / P + blk - tou[k.b];
  k.r0 = max(s.prev - k.j * P, 0);
  k.r1 = min(s.seq - k.j * P, P);
  k.i0 = (int64_t)tok[k.b] + (k.j * P - s.prev);
  return k;
}

// The N warps of a set meet (at a barrier of their own: sets do not wait for one another).
template <int N>
__device__ __forceinline__ void set_sync() {
  if (N > 1) asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)threadIdx.x / (N * 32)), "n"(N * 32) : "memory");
}

// The K or V of one head of a block, by a set of N warps that hold an Nth of it each (`top`: the maxima of the CTA's warps, two
// rounds of them).  H: steps held (of four rows each, from row `first`); with MORE the others, up to `steps`, are read again.
// load(g, x, y) reads the rows of a step (zeros for rows that are not new), turn(g, x, y) turns them.
template <int P, int F, int H, bool MORE, int N, class Load, class Turner>
__device__ __forceinline__ void quantise(const Rot8Args& a, const Block& k, bool is_v, int slot, const int2& at, int first,
                                         int steps, uint4 (&x)[H], uint4 (&y)[H], uint32_t* top, Load load, Turner turn) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane & 7;
  const bool in_pool = slot >= 0 && slot < a.n_slots;
  float* scale_at = a.scale[is_v] + (in_pool ? slot : 0);
  const float old = in_pool && k.r0 > 0 ? *scale_at : 0.f;
  if (!is_v) {
#pragma unroll
    for (int g = 0; g < H; ++g) turn(g, x[g], y[g]);
  }
  // rows that are not new hold zeros, or what a norm without eps makes of them (NaN, which the maxima pass over)
  uint32_t m = 0u, fin = 0u;
#pragma unroll
  for (int g = 0; g < H; ++g) m = max_all(max_all(m, x[g]), y[g]);
  for (int g = H; MORE && g < steps; ++g) {
    uint4 lo, hi;
    load(g, lo, hi);
    if (!is_v) turn(g, lo, hi);
    m = max_all(max_all(m, lo), hi);
    fin = max_finite(max_finite(fin, lo), hi);
  }
  auto join = [&](uint32_t v, int round) {
    v = warp_max(v);
    if (N == 1) return v;
    if (lane == 0) top[round * kR8Warps + warp] = v;
    set_sync<N>();
#pragma unroll
    for (int i = 0; i < N; ++i) v = max(v, top[round * kR8Warps + warp / N * N + i]);
    return v;
  };
  uint32_t big = join(m, 0);
  if (big == 0x7f80u) {  // an infinity among them: the largest of the others (rare)
#pragma unroll
    for (int g = 0; g < H; ++g) fin = max_finite(max_finite(fin, x[g]), y[g]);
    big = join(fin, 1);
  }
  if (!in_pool) {
    if (lane == 0) report(a.status, SCOUT_DEV_BAD_INDEX);
  } else {
    uint8_t* page = a.pool[is_v] + (int64_t)slot * (P * kD);
    const float need = pow2_biased(scale_exponent<F>(__uint_as_float(big << 16)));
    const bool grows = k.r0 > 0 && need > old;  // the scale of a block with cached tokens never shrinks
    const float scale = k.r0 > 0 && !grows ? old : need;
    const float inv = 1.f / scale;  // exact where the scale is a power of two (1 / 2^-126 = 2^126 is finite)
    if (grows) {
      const float ratio = old / need;
#pragma unroll 1
      for (int r = warp % N * 4 + (lane >> 3); r < k.r0; r += 4 * N) {
        uint4* p = reinterpret_cast<uint4*>(page + r * kD + sub * 16);
        const uint4 c = *p;
        *p = make_uint4(recode4<F>(c.x, ratio), recode4<F>(c.y, ratio), recode4<F>(c.z, ratio), recode4<F>(c.w, ratio));
      }
    }
    auto store = [&](int g, const uint4& lo, const uint4& hi) {
      const int r = first + 4 * g + (lane >> 3);
      if (r < k.r0 || r >= k.r1) return;
      *reinterpret_cast<uint2*>(page + r * kD + at.x) = encode8<F>(lo, inv);
      *reinterpret_cast<uint2*>(page + r * kD + at.y) = encode8<F>(hi, inv);
    };
#pragma unroll
    for (int g = 0; g < H; ++g) store(g, x[g], y[g]);
    for (int g = H; MORE && g < steps; ++g) {
      uint4 lo, hi;
      load(g, lo, hi);
      if (!is_v) turn(g, lo, hi);
      store(g, lo, hi);
    }
    __syncwarp();  // every lane has read the old scale, and a set's other warps before they met this one
    if (lane == 0 && warp % N == 0 && (k.r0 == 0 || grows)) *scale_at = scale;
  }
  set_sync<N>();  // the maxima have been read: the next ones may be written
}

// Query rows: four tokens of a warp, heads [h0, h1), U of them in flight together.
template <int LAYOUT, int U>
__device__ __forceinline__ void turn_queries(const Rot8Args& a, const int* tok, int64_t i, int rows, int h0, int h1,
                                             int cap_tokens) {
  const int sub = threadIdx.x & 7;
  const bool live = i < rows;
  const int2 at = lane_chunks<LAYOUT>(sub, a.rope.n);
  const __nv_bfloat16* src = a.q + i * a.ld_q;
  __nv_bfloat16* dst = a.q_out + i * a.ld_q_out;
  Turn t;
  Weights w;
  auto prepare = [&] {
    int index = 0;
    if (a.positions == nullptr && live) {
      const int b = owner_of(tok, a.B, (int)i);
      index = seq_span(a.prev_len, a.seq_len, b, cap_tokens).prev + (int)i - tok[b];
    }
    if (a.q_norm != nullptr) w = lane_weights(a.q_norm, at);
    t = lane_turn(a.rope, sub, position_of(a, i, index, live, sub));
  };
  if (U > 1) prepare();  // (one head: its loads first)
  for (int h = h0; h < h1; h += U) {
    uint4 x[U], y[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!live || h + u >= h1) continue;
      x[u] = ld_stream(src + (h + u) * kD + at.x);
      y[u] = ld_stream(src + (h + u) * kD + at.y);
    }
    if (U == 1) prepare();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float v[16];
      unpack16(x[u], y[u], v);
      if (a.q_norm != nullptr) norm_head(v, w, a.eps);
      turn_head<LAYOUT>(v, t, sub < a.rope.n);
      pack16(v, x[u], y[u]);
      if (!live || h + u >= h1) continue;
      *reinterpret_cast<uint4*>(dst + (h + u) * kD + at.x) = x[u];
      *reinterpret_cast<uint4*>(dst + (h + u) * kD + at.y) = y[u];
    }
  }
}

// tok [B + 1]: new tokens before sequence b; tou [B + 1]: touched blocks (of one KV head) before it.
template <int P>
__device__ __forceinline__ void prefixes(const Rot8Args& a, int* tok, int* tou, int* partial) {
  const int cap_tokens = a.nblk_cap * P;
  int* const out[2] = {tok, tou};
  cta_prefixes<2>(a.B, out, partial, [&](int b, int (&x)[2]) {
    const SeqSpan s = seq_span(a.prev_len, a.seq_len, b, cap_tokens);
    x[0] = s.seq - s.prev;
    x[1] = s.seq > s.prev ? (s.seq + P - 1) / P - s.prev / P : 0;
  });
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.B; b += blockDim.x) report_span(a.status, a.prev_len, a.seq_len, b, cap_tokens);
}

template <int P, int F, int LAYOUT>
__global__ void __launch_bounds__(kR8Warps * 32, kR8PerSm) rotate8_kernel(const Rot8Args a) {
  constexpr int H = P / 4 < kHold ? P / 4 : kHold, kSet = P / 4 / H;  // warps of one head's K or V
  constexpr int kSets = kR8Warps / kSet;
  static_assert(kSets % 2 == 0, "a head's K and V are of one round of the sets: exactly one of them is V");
  start_dependent();
  extern __shared__ int sm[];
  __shared__ int partial[2 * 32];
  __shared__ uint32_t top[2 * kR8Warps];
  __shared__ float4 table[4][P][8];  // [quarter of a lane's pairs: c, c, s, s][row][lane]
  int *tok = sm, *tou = sm + (a.B + 1);
  prefixes<P>(a, tok, tou, partial);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, sub = lane & 7;
  const int rows = min(tok[a.B], a.n_tokens), first = warp % kSet * (4 * H);  // the warp's first row of a block
  if ((int)blockIdx.x >= a.kv_ctas) {  // queries
    const int64_t wn = (int64_t)(gridDim.x - a.kv_ctas) * kR8Warps;
    const int64_t items = (int64_t)((rows + 3) / 4) * a.q_parts;
    for (int64_t it = (int64_t)(blockIdx.x - a.kv_ctas) * kR8Warps + warp; it < items; it += wn) {
      const int64_t group = (uint64_t)it / (unsigned)a.q_parts;
      const int h0 = (int)(it - group * a.q_parts) * a.q_per;
      turn_queries<LAYOUT, 4>(a, tok, group * 4 + (lane >> 3), rows, h0, min(a.Hq, h0 + a.q_per), a.nblk_cap * P);
    }
    return;
  }
  const unsigned parts = ((unsigned)a.Hkv + a.kv_heads - 1) / a.kv_heads;
  const int64_t items = (int64_t)tou[a.B] * parts;
  for (int64_t it = blockIdx.x; it < items; it += a.kv_ctas) {
    const int blk = (int)((uint64_t)it / parts), part = (int)(it - (int64_t)blk * parts);
    const Block k = block_of<P>(a, tok, tou, blk);
    if (k.i0 + k.r1 > a.n_tokens) {  // the same for the CTA
      if (tid == 0) report(a.status, SCOUT_DEV_BAD_INDEX);
      continue;
    }
    // K and V of the part's heads, dealt to the sets of warps so that each gets as many of either
    const int p1 = 2 * min(a.Hkv, (part + 1) * a.kv_heads);
    bool made = false;
    for (int p = 2 * part * a.kv_heads + warp / kSet; p < p1 || !made; p += kSets) {
      const bool mine = p < p1;
      const int h = p >> 1;
      const bool is_v = (p + p / kSets) & 1;
      const int2 at = is_v ? make_int2(sub * 16, sub * 16 + 8) : lane_chunks<LAYOUT>(sub, a.rope.n);
      const int64_t ld = a.ld[is_v];
      const __nv_bfloat16* src = a.kv[is_v] + k.i0 * ld + h * kD;
      auto load = [&](int g, uint4& lo, uint4& hi) {
        const int r = first + 4 * g + (lane >> 3);
        lo = hi = make_uint4(0u, 0u, 0u, 0u);
        if (r < k.r0 || r >= k.r1) return;
        lo = ldg_stream(src + r * ld + at.x);
        hi = ldg_stream(src + r * ld + at.y);
      };
      uint4 x[H], y[H];
      int slot = -1;
      if (mine) {
        slot = a.page_table[((int64_t)k.b * a.Hkv + h) * a.nblk_cap + k.j];  // in flight with the rows
#pragma unroll
        for (int g = 0; g < H; ++g) load(g, x[g], y[g]);
      }
      if (!made) {
        made = true;
        __syncthreads();  // the last item's table has been read
        for (int g = warp; g < P / 4; g += kR8Warps) {
          const int r = 4 * g + (lane >> 3);
          const bool live = r >= k.r0 && r < k.r1;
          const Turn t = lane_turn(a.rope, sub, position_of(a, k.i0 + r, k.j * P + r, live, sub));
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            table[i][r][sub] = make_float4(t.c[4 * i], t.c[4 * i + 1], t.c[4 * i + 2], t.c[4 * i + 3]);
            table[2 + i][r][sub] = make_float4(t.s[4 * i], t.s[4 * i + 1], t.s[4 * i + 2], t.s[4 * i + 3]);
          }
        }
        __syncthreads();
        if (!mine) break;
      }
      Weights w;
      const bool norm = !is_v && a.k_norm != nullptr;
      if (norm) w = lane_weights(a.k_norm, at);
      auto turn = [&](int g, uint4& lo, uint4& hi) {
        const int r = first + 4 * g + (lane >> 3);
        Pairs v = unpack_pairs<LAYOUT>(lo, hi);
        if (norm) norm_pairs<LAYOUT>(v, w, a.eps);
        if (sub < a.rope.n) {
          f2 c[4], s[4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const auto co = *reinterpret_cast<const ulonglong2*>(&table[i][r][sub]);
            const auto si = *reinterpret_cast<const ulonglong2*>(&table[2 + i][r][sub]);
            c[2 * i] = co.x, c[2 * i + 1] = co.y;
            s[2 * i] = si.x, s[2 * i + 1] = si.y;
          }
          turn_pairs(v, c, s);
        }
        pack_pairs<LAYOUT>(v, lo, hi);
      };
      quantise<P, F, H, false, kSet>(a, k, is_v, slot, at, first, H, x, y, top, load, turn);
    }
  }
}

template <int P, int F, int LAYOUT>
__global__ void __launch_bounds__(kR8Warps * 32, 4) rotate8_few_kernel(const Rot8Args a) {
  start_dependent();
  extern __shared__ int sm[];
  __shared__ int partial[2 * 32];
  int *tok = sm, *tou = sm + (a.B + 1);
  prefixes<P>(a, tok, tou, partial);
  const int lane = threadIdx.x & 31, sub = lane & 7;
  const int64_t wn = (int64_t)gridDim.x * kR8Warps;
  const unsigned sets = 2 * (unsigned)a.Hkv;
  const int64_t n_kv = (int64_t)tou[a.B] * sets;
  const int rows = min(tok[a.B], a.n_tokens);
  const int64_t items = n_kv + (int64_t)((rows + 3) / 4) * a.Hq;
  for (int64_t it = (int64_t)blockIdx.x * kR8Warps + (threadIdx.x >> 5); it < items; it += wn) {
    if (it >= n_kv) {
      const int64_t group = (uint64_t)(it - n_kv) / (unsigned)a.Hq;
      const int h = (int)(it - n_kv - group * a.Hq);
      turn_queries<LAYOUT, 1>(a, tok, group * 4 + (lane >> 3), rows, h, h + 1, a.nblk_cap * P);
      continue;
    }
    const int blk = (int)((uint64_t)it / sets), p = (int)(it - (int64_t)blk * sets);
    const int h = p >> 1;
    const bool is_v = p & 1;
    const Block k = block_of<P>(a, tok, tou, blk);
    if (k.i0 + k.r1 > a.n_tokens) {
      if (lane == 0) report(a.status, SCOUT_DEV_BAD_INDEX);
      continue;
    }
    const int slot = a.page_table[((int64_t)k.b * a.Hkv + h) * a.nblk_cap + k.j];  // in flight with the rows
    const int2 at = is_v ? make_int2(sub * 16, sub * 16 + 8) : lane_chunks<LAYOUT>(sub, a.rope.n);
    const int64_t ld = a.ld[is_v];
    const __nv_bfloat16* src = a.kv[is_v] + k.i0 * ld + h * kD;
    Weights w;
    const bool norm = !is_v && a.k_norm != nullptr;
    if (norm) w = lane_weights(a.k_norm, at);
    auto load = [&](int g, uint4& lo, uint4& hi) {
      const int r = k.r0 + 4 * g + (lane >> 3);
      lo = hi = make_uint4(0u, 0u, 0u, 0u);
      if (r >= k.r1) return;
      lo = ldg_stream(src + r * ld + at.x);
      hi = ldg_stream(src + r * ld + at.y);
    };
    auto turn = [&](int g, uint4& lo, uint4& hi) {
      const int r = k.r0 + 4 * g + (lane >> 3);
      const Turn t = lane_turn(a.rope, sub, position_of(a, k.i0 + r, k.j * P + r, r < k.r1, sub));
      float v[16];
      unpack16(lo, hi, v);
      if (norm) norm_head(v, w, a.eps);
      turn_head<LAYOUT>(v, t, sub < a.rope.n);
      pack16(v, lo, hi);
    };
    uint4 x[1], y[1];
    load(0, x[0], y[0]);
    quantise<P, F, 1, true, 1>(a, k, is_v, slot, at, k.r0, (k.r1 - k.r0 + 3) / 4, x, y, nullptr, load, turn);
  }
}

// the prefixes' static part, the two rows of the largest batch and the largest table: what a CTA may have without a request
constexpr size_t kStatic8 = (2 * 32 + 2 * kR8Warps) * sizeof(int), kTable8 = 4 * 8 * 16;

template <int P, int F, int LAYOUT>
int launch_rotate8(Rot8Args& a, cudaStream_t st) {
  // at most n_tokens / P + 2 B blocks of a head are touched (each span's two ends partly)
  const int64_t blocks = (int64_t)a.n_tokens / P + 2 * (int64_t)(a.B < a.n_tokens ? a.B : a.n_tokens);
  const size_t smem = (size_t)(2 * a.B + 2) * sizeof(int);
  const int64_t groups = ((int64_t)a.n_tokens + 3) / 4, none = a.n_tokens == 0;  // (without rows: the report alone)
  if (a.n_tokens <= kFewTokens * (int64_t)a.B) {
    const int64_t want = (blocks * 2 * a.Hkv + groups * a.Hq + kR8Warps - 1) / kR8Warps + none;
    const int64_t most = (int64_t)sm_count() * 8;
    return launch_dependent(rotate8_few_kernel<P, F, LAYOUT>, want < most ? want : most, kR8Warps * 32, smem, st, a);
  }
  if (smem + kStatic8 + kTable8 * P > 48 * 1024 &&
      cudaFuncSetAttribute(rotate8_kernel<P, F, LAYOUT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (2 * kMaxBatch + 2) * (int)sizeof(int)) != cudaSuccess)
    return SCOUT_ERR_CUDA;
  const int64_t most = (int64_t)sm_count() * kR8PerSm;  // CTAs at a time
  // the CTAs by the bytes that the keys and values, and the queries, move
  const float share = 768.f * a.Hkv / (768.f * a.Hkv + 512.f * a.Hq);
  const int64_t kv_most = (int64_t)max(1, (int)(most * share));
  a.kv_heads = max(1, (int)(a.Hkv / max((int64_t)1, kv_most / blocks)));
  const int64_t kv_want = blocks * ((a.Hkv + a.kv_heads - 1) / a.kv_heads);
  a.kv_ctas = (int)(kv_want < kv_most * kR8Waves ? kv_want : kv_most * kR8Waves);
  a.q_per = kR8Heads;
  a.q_parts = (a.Hq + a.q_per - 1) / a.q_per;
  const int64_t q_want = (groups * a.q_parts + kR8Warps - 1) / kR8Warps, q_most = max((int64_t)1, most - kv_most) * kR8Waves;
  const int grid = a.kv_ctas + (int)(q_want < q_most ? q_want : q_most);
  return launch_dependent(rotate8_kernel<P, F, LAYOUT>, grid, kR8Warps * 32, smem, st, a);
}

template <int P, int F>
int dispatch_rotate8(int layout, Rot8Args& a, cudaStream_t st) {
  return layout == SCOUT_ROPE_HALF ? launch_rotate8<P, F, SCOUT_ROPE_HALF>(a, st)
                                   : launch_rotate8<P, F, SCOUT_ROPE_INTERLEAVED>(a, st);
}

template <int F>
int dispatch_rotate8(int P, int layout, Rot8Args& a, cudaStream_t st) {
  switch (P) {
    case 16: return dispatch_rotate8<16, F>(layout, a, st);
    case 32: return dispatch_rotate8<32, F>(layout, a, st);
    default: return dispatch_rotate8<64, F>(layout, a, st);
  }
}

}  // namespace
}  // namespace scout

extern "C" int scout_append_rotated_kv8(int fmt, const void* K_new, int64_t ld_k, const void* V_new, int64_t ld_v,
                                        int n_tokens, const int32_t* positions, const scout_rope* rope,
                                        const void* k_norm, float eps, const int32_t* prev_len, const int32_t* seq_len,
                                        const int32_t* page_table, int B, int Hkv, int D, int P, int nblk_cap,
                                        void* K_pool, void* V_pool, float* K_scale, float* V_scale, int64_t n_slots,
                                        const void* q, int64_t ld_q, int Hq, const void* q_norm, void* q_out,
                                        int64_t ld_q_out, int32_t* dev_status, cudaStream_t stream) {
  using namespace scout;
  if (seq_len == nullptr || page_table == nullptr || K_pool == nullptr || V_pool == nullptr || K_scale == nullptr ||
      V_scale == nullptr || (n_tokens > 0 && V_new == nullptr))
    return SCOUT_ERR_INVALID_ARG;
  if (!valid_fp8(fmt) || n_tokens < 0 || B <= 0 || Hkv <= 0 || Hq < 0 || nblk_cap <= 0 || n_slots <= 0 ||
      ld_v < (int64_t)Hkv * D)
    return SCOUT_ERR_INVALID_ARG;
  // (without rows there is no K_new either: the pool stands in for it)
  int rc = check_heads(n_tokens > 0 ? K_new : K_pool, ld_k, K_pool, ld_k, Hkv, D, rope, k_norm, eps);
  if (rc == SCOUT_OK && Hq > 0 && n_tokens > 0) rc = check_heads(q, ld_q, q_out, ld_q_out, Hq, D, rope, q_norm, eps);
  if (rc != SCOUT_OK) return rc;
  if (!valid_P(P) || B > kMaxBatch || nblk_cap > kMaxNblk || n_slots > 0x7fffffffLL ||
      (int64_t)B * nblk_cap * P > 0x7fffffffLL || (int64_t)B * Hkv * nblk_cap > 0x7fffffffLL || ld_v % 8 != 0 ||
      !aligned16(V_new) || !aligned16(V_pool) || (reinterpret_cast<uintptr_t>(positions) & 3u))
    return SCOUT_ERR_UNSUPPORTED;
  if (n_tokens == 0 && dev_status == nullptr) return SCOUT_OK;  // no rows, and nowhere to say that some were due
  Rot8Args a = {};
  a.kv[0] = static_cast<const __nv_bfloat16*>(K_new);
  a.kv[1] = static_cast<const __nv_bfloat16*>(V_new);
  a.ld[0] = ld_k;
  a.ld[1] = ld_v;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.ld_q = ld_q;
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.ld_q_out = ld_q_out;
  a.k_norm = static_cast<const __nv_bfloat16*>(k_norm);
  a.q_norm = static_cast<const __nv_bfloat16*>(q_norm);
  a.pool[0] = static_cast<uint8_t*>(K_pool);
  a.pool[1] = static_cast<uint8_t*>(V_pool);
  a.scale[0] = K_scale;
  a.scale[1] = V_scale;
  a.positions = positions;
  a.prev_len = prev_len;
  a.seq_len = seq_len;
  a.page_table = page_table;
  a.n_tokens = n_tokens;
  a.B = B;
  a.Hkv = Hkv;
  a.Hq = Hq;
  a.nblk_cap = nblk_cap;
  a.n_slots = n_slots;
  a.rope = rope_of(rope);
  a.eps = eps;
  a.status = dev_status;
  return fmt == SCOUT_FP8_E4M3 ? dispatch_rotate8<SCOUT_FP8_E4M3>(P, rope->layout, a, stream)
                               : dispatch_rotate8<SCOUT_FP8_E5M2>(P, rope->layout, a, stream);
}

