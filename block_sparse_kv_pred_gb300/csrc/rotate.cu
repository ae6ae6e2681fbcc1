// scout_rotate and scout_append_rotated_kv: heads normalised and turned by their positions, and keys
// on their way into a bf16 paged cache with their values.
//
// One kernel: a warp takes four tokens and some heads of one kind (queries row to row, keys and values by slot map).
// Its rows' cosines are made once, in registers, while the first heads' rows are on their way; four heads are in flight
// together.  Bound by DRAM: GB300, 8 prompts of up to 16K tokens, 8 KV and 32 query heads, 264 us for 1.72 GB (6.5 TB/s, 0.97 of the
// measured copy bandwidth) at 20 warps an SM and half of its issue slots; two heads in flight 282 us, eight 336 (registers); the
// next heads read before the present ones are turned 280.  A decode step of 40 sequences 2.2 us, 8 x 32 heads 1.75 us:
// the launch and one read.
#include "rotate.cuh"

namespace scout {
namespace {

constexpr int kRotThreads = 128;

struct HeadRows {  // heads of a token side by side, tokens ld elements apart
  const __nv_bfloat16* src;
  int64_t ld;
  __nv_bfloat16* dst;
  int64_t ld_dst;
  const __nv_bfloat16* norm;
  int heads;
};

struct RotArgs {
  HeadRows q;             // rows to rows
  HeadRows kv[2];         // K and V rows to the pools (dst), by slot_map; V is copied
  const int64_t* slot_map;
  int64_t pool_rows;
  const int32_t* positions;
  int n_tokens;
  int per;                // heads of a warp
  int parts_q, parts_kv;  // warps of a group of four tokens: of the queries, of K and of V each
  Rope rope;
  float eps;
  int32_t* status;
};

// A warp takes four tokens and `per` of their heads of one kind, the warps of a CTA consecutive tokens.
// U heads are in flight together.
template <int LAYOUT, int U>
__global__ void __launch_bounds__(kRotThreads, 5) rotate_kernel(const RotArgs a) {
  start_dependent();
  const int lane = threadIdx.x & 31, sub = lane & 7;
  const unsigned parts = (unsigned)a.parts_q + 2 * (unsigned)a.parts_kv;
  const unsigned block = blockIdx.x / parts;
  int part = (int)(blockIdx.x - block * parts);
  const int64_t i = ((int64_t)block * (kRotThreads / 32) + (threadIdx.x >> 5)) * 4 + (lane >> 3);
  const int pos = i < a.n_tokens ? a.positions[i] : -1;
  const bool is_q = part < a.parts_q;
  const bool is_v = part >= a.parts_q + a.parts_kv;
  part -= is_q ? 0 : is_v ? a.parts_q + a.parts_kv : a.parts_q;
  const HeadRows& r = is_q ? a.q : a.kv[is_v];
  const int h0 = part * a.per, h1 = min(r.heads, h0 + a.per);
  const int2 at = is_v ? make_int2(sub * 8, 64 + sub * 8) : lane_chunks<LAYOUT>(sub, a.rope.n);
  const __nv_bfloat16* src = r.src + i * r.ld;
  const bool norm = r.norm != nullptr;
  Turn t;
  Weights w;
  auto prepare = [&] {
    if (is_v) return;
    if (norm) w = lane_weights(r.norm, at);
    t = lane_turn(a.rope, sub, (uint32_t)max(pos, 0));
  };
  // One head a warp: its loads go out before the position is there (8 x 32 heads 2.05 -> 1.75 us, a decode step's write 2.65 ->
  // 2.2; with more heads, whose loads then hold registers meanwhile, 266 -> 269 us).
  if (U > 1) prepare();
  for (int h = h0; h < h1; h += U) {
    uint4 x[U], y[U];
    int64_t to[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      to[u] = -1;
      if ((U > 1 ? pos < 0 : i >= a.n_tokens) || h + u >= h1) continue;
      to[u] = is_q ? i * r.ld_dst + (h + u) * kD : a.slot_map[i * r.heads + h + u];
      x[u] = ld_stream(src + (h + u) * kD + at.x);
      y[u] = ld_stream(src + (h + u) * kD + at.y);
    }
    if (U == 1) prepare();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!is_q) {
        if (to[u] >= a.pool_rows) {
          if (sub == 0 && pos >= 0) report(a.status, SCOUT_DEV_BAD_INDEX);
          to[u] = -1;
        }
        if (to[u] >= 0) to[u] *= kD;
      }
      if (!is_v) {
        float v[16];
        unpack16(x[u], y[u], v);
        if (norm) norm_head(v, w, a.eps);
        turn_head<LAYOUT>(v, t, sub < a.rope.n);
        pack16(v, x[u], y[u]);
      }
      if (to[u] < 0 || pos < 0) continue;
      *reinterpret_cast<uint4*>(r.dst + to[u] + at.x) = x[u];
      *reinterpret_cast<uint4*>(r.dst + to[u] + at.y) = y[u];
    }
  }
}
// Heads of a warp.  The fewer, the shorter a call of few rows (a warp's heads follow one another, four at a time) and
// the more often a token's cosines are made.  GB300, 40 (8) heads, us, with 1 / 4 / 8 / 16 a warp:
//   200 tokens 3.2 / 3.7 / 5.0 / 8.0 (2.5 / 3.5 / 4.9), 800: 6.5 / 5.0 / 5.8 / 8.1, 3,200 (8 heads): 5.5 / 4.3 / 5.7,
//   6,400: 40.7 / 25.1 / 23.9 / 25.5, 20,000: 132 / 79.8 / 71.0 / 70.6
// One where its warps are one wave (20 of them an SM at its registers), four likewise, then eight, and sixteen where
// there are many or where that is all the heads (9,001 tokens of 12 heads: 14.2 us with eight, 12.9 with all).
inline int heads_of_warp(int64_t steps, int heads) {
  const int64_t wave = 20 * (int64_t)sm_count();
  return steps <= wave ? 1 : steps <= 4 * wave ? 4 : steps <= 32 * wave && heads > 16 ? 8 : 16;
}

template <int LAYOUT>
int launch_rotate(RotArgs& a, cudaStream_t st) {
  const int64_t groups = ((int64_t)a.n_tokens + 3) / 4;
  const int most = max(a.q.heads, a.kv[0].heads);
  a.per = heads_of_warp(groups * ((int64_t)a.q.heads + 2 * (int64_t)a.kv[0].heads), most);
  a.parts_q = (a.q.heads + a.per - 1) / a.per;
  a.parts_kv = (a.kv[0].heads + a.per - 1) / a.per;
  const int64_t grid = (groups + kRotThreads / 32 - 1) / (kRotThreads / 32) * ((int64_t)a.parts_q + 2 * (int64_t)a.parts_kv);
  if (grid > 0x7fffffffLL) return SCOUT_ERR_UNSUPPORTED;
  return launch_dependent(a.per == 1 ? rotate_kernel<LAYOUT, 1> : rotate_kernel<LAYOUT, 4>, grid, kRotThreads, 0, st, a);
}

int launch_rotate(RotArgs& a, int layout, cudaStream_t st) {
  return layout == SCOUT_ROPE_HALF ? launch_rotate<SCOUT_ROPE_HALF>(a, st) : launch_rotate<SCOUT_ROPE_INTERLEAVED>(a, st);
}

}  // namespace

int check_heads(const void* x, int64_t ld_x, const void* out, int64_t ld_out, int heads, int D, const scout_rope* rope,
                const void* norm, float eps) {
  if (x == nullptr || out == nullptr || heads <= 0 || !valid_rope(rope) || !valid_eps(eps) ||
      ld_x < (int64_t)heads * D || ld_out < (int64_t)heads * D)
    return SCOUT_ERR_INVALID_ARG;
  if (D != kD || heads > (1 << 20) || !supported_rope(rope) || ld_x % 8 != 0 || ld_out % 8 != 0 || !aligned16(x) || !aligned16(out) ||
      !aligned16(norm))
    return SCOUT_ERR_UNSUPPORTED;
  return SCOUT_OK;
}

}  // namespace scout

extern "C" int scout_rotate(const void* x, int64_t ld_x, void* out, int64_t ld_out, const int32_t* positions,
                            int n_tokens, int heads, int D, const scout_rope* rope, const void* norm, float eps,
                            cudaStream_t stream) {
  using namespace scout;
  if (positions == nullptr || n_tokens < 0) return SCOUT_ERR_INVALID_ARG;
  const int rc = check_heads(x, ld_x, out, ld_out, heads, D, rope, norm, eps);
  if (rc != SCOUT_OK) return rc;
  if (reinterpret_cast<uintptr_t>(positions) & 3u) return SCOUT_ERR_UNSUPPORTED;
  if (n_tokens == 0) return SCOUT_OK;
  RotArgs a = {};
  a.q = HeadRows{static_cast<const __nv_bfloat16*>(x), ld_x, static_cast<__nv_bfloat16*>(out), ld_out,
                 static_cast<const __nv_bfloat16*>(norm), heads};
  a.positions = positions;
  a.n_tokens = n_tokens;
  a.rope = rope_of(rope);
  a.eps = eps;
  return launch_rotate(a, rope->layout, stream);
}

extern "C" int scout_append_rotated_kv(const void* K_new, int64_t ld_k, const void* V_new, int64_t ld_v,
                                       const int32_t* positions, const scout_rope* rope, const void* k_norm, float eps,
                                       const int64_t* slot_map, int n_tokens, int Hkv, int D, int P, void* K_pool,
                                       void* V_pool, int64_t n_slots, const void* q, int64_t ld_q, int Hq,
                                       const void* q_norm, void* q_out, int64_t ld_q_out, int32_t* dev_status,
                                       cudaStream_t stream) {
  using namespace scout;
  if (V_new == nullptr || positions == nullptr || slot_map == nullptr || V_pool == nullptr) return SCOUT_ERR_INVALID_ARG;
  if (n_tokens < 0 || Hkv <= 0 || Hq < 0 || n_slots <= 0 || ld_v < (int64_t)Hkv * D) return SCOUT_ERR_INVALID_ARG;
  int rc = check_heads(K_new, ld_k, K_pool, ld_k, Hkv, D, rope, k_norm, eps);
  if (rc == SCOUT_OK && Hq > 0) rc = check_heads(q, ld_q, q_out, ld_q_out, Hq, D, rope, q_norm, eps);
  if (rc != SCOUT_OK) return rc;
  if (!valid_P(P) || !aligned16(V_new) || !aligned16(V_pool) || ld_v % 8 != 0 ||
      (reinterpret_cast<uintptr_t>(slot_map) & 7u) || (reinterpret_cast<uintptr_t>(positions) & 3u) ||
      n_slots > 0x7fffffffLL)
    return SCOUT_ERR_UNSUPPORTED;
  if (n_tokens == 0) return SCOUT_OK;
  RotArgs a = {};
  if (Hq > 0)
    a.q = HeadRows{static_cast<const __nv_bfloat16*>(q), ld_q, static_cast<__nv_bfloat16*>(q_out), ld_q_out,
                   static_cast<const __nv_bfloat16*>(q_norm), Hq};
  a.kv[0] = HeadRows{static_cast<const __nv_bfloat16*>(K_new), ld_k, static_cast<__nv_bfloat16*>(K_pool), 0,
                     static_cast<const __nv_bfloat16*>(k_norm), Hkv};
  a.kv[1] = HeadRows{static_cast<const __nv_bfloat16*>(V_new), ld_v, static_cast<__nv_bfloat16*>(V_pool), 0, nullptr, Hkv};
  a.slot_map = slot_map;
  a.pool_rows = n_slots * P;
  a.positions = positions;
  a.n_tokens = n_tokens;
  a.rope = rope_of(rope);
  a.eps = eps;
  a.status = dev_status;
  return launch_rotate(a, rope->layout, stream);
}
