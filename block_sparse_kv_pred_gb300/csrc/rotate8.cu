// scout_append_rotated_kv8: new keys normalised, turned and quantised on their way into 8-bit pools with
// their values, and the same tokens' queries normalised and turned beside them.
//
// A CTA takes a touched block and a part of its heads: kHeads KV heads, K and V, or up to kQHeads query heads.
// Eight lanes hold a token's row (rotate.cuh), so its P / 4 warps hold a whole block of each of those
// heads in registers: read once, turned, rounded to bf16, the block's maximum joined through shared
// memory, and the codes made from the registers.  A lane's token is the same for every head, so its cosines and sines
// are made once a block.  A range of consecutive (block, part) items goes to each CTA.
#include "fp8.cuh"
#include "rotate.cuh"

namespace scout {

int check_heads(const void* x, int64_t ld_x, const void* out, int64_t ld_out, int heads, int D, const scout_rope* rope,
                const void* norm, float eps);  // rotate.cu

namespace {

constexpr int kHeads = 2;   // KV heads of an item
constexpr int kQHeads = 8;  // query heads of an item

struct Rot8Args {
  const __nv_bfloat16 *kv[2], *q;  // new rows
  int64_t ld[2], ld_q, ld_q_out;
  __nv_bfloat16* q_out;
  const __nv_bfloat16 *k_norm, *q_norm;
  uint8_t* pool[2];
  float* scale[2];
  const int32_t *positions, *prev_len, *seq_len, *page_table;
  int n_tokens, B, Hkv, Hq, nblk_cap;
  int kv_parts, q_parts;
  int64_t n_slots;
  Rope rope;
  float eps;
  int32_t* status;
};

template <int P, int F, int LAYOUT>
__global__ void __launch_bounds__(P * 8) rotate8_kernel(const Rot8Args a) {
  constexpr int kWarps = P / 4, kSets = 2 * kHeads;
  extern __shared__ int sm[];
  __shared__ int partial[2 * 32];
  __shared__ uint32_t top[2][kSets][kWarps];  // largest magnitudes, a buffer for every other item
  const int B = a.B;
  int* tok = sm;            // [B + 1] new tokens before sequence b
  int* tou = sm + (B + 1);  // [B + 1] touched blocks (of one KV head) before it
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, sub = lane & 7;
  const int cap_tokens = a.nblk_cap * P;
  int* const out[2] = {tok, tou};
  cta_prefixes<2>(B, out, partial, [&](int b, int (&x)[2]) {
    const SeqSpan s = seq_span(a.prev_len, a.seq_len, b, cap_tokens);
    x[0] = s.seq - s.prev;
    x[1] = s.seq > s.prev ? (s.seq + P - 1) / P - s.prev / P : 0;
  });
  if (blockIdx.x == 0)
    for (int b = tid; b < B; b += blockDim.x) report_span(a.status, a.prev_len, a.seq_len, b, cap_tokens);
  const int parts = a.kv_parts + a.q_parts;
  const int64_t items = (int64_t)tou[B] * parts;
  const int64_t first = items * blockIdx.x / gridDim.x, last = items * (blockIdx.x + 1) / gridDim.x;
  const int r = warp * 4 + (lane >> 3);  // the lane's row of a block
  const int2 at_k = lane_chunks<LAYOUT>(sub, a.rope.n), at_v = make_int2(sub * 16, sub * 16 + 8);
  const bool turns = sub < a.rope.n;
  int blk = (int)(first / parts), part = (int)(first - (int64_t)blk * parts) - 1;
  int b = 0, j = 0, r0 = 0, r1 = 0, buf = 0;
  int64_t row = 0;
  bool rows_ok = false, fresh = false;
  Turn t;
  for (int64_t it = first; it < last; ++it) {
    bool enter = it == first;
    if (++part == parts) {
      part = 0;
      ++blk;
      enter = true;
    }
    if (enter) {
      b = owner_of(tou, B, blk);
      const SeqSpan s = seq_span(a.prev_len, a.seq_len, b, cap_tokens);
      j = s.prev / P + blk - tou[b];
      r0 = max(s.prev - j * P, 0), r1 = min(s.seq - j * P, P);  // the block's new rows
      const int64_t i0 = (int64_t)tok[b] + (j * P - s.prev);     // token row of its row 0
      row = i0 + r;
      rows_ok = i0 + r1 <= a.n_tokens;
      fresh = rows_ok && r >= r0 && r < r1;
      int pos = j * P + r;
      if (a.positions != nullptr && fresh) {
        pos = a.positions[row];
        if (pos < 0) {
          if (sub == 0) report(a.status, SCOUT_DEV_BAD_INDEX);
          pos = 0;
        }
      }
      t = lane_turn(a.rope, sub, (uint32_t)pos);
    }
    if (!rows_ok) {
      if (tid == 0) report(a.status, SCOUT_DEV_BAD_INDEX);
      break;  // the rows are packed: those of the items that follow end no earlier
    }
    if (part >= a.kv_parts) {  // query heads
      const int h0 = (part - a.kv_parts) * kQHeads, h1 = min(a.Hq, h0 + kQHeads);
      float w[16];
      if (a.q_norm != nullptr)
        unpack16(__ldg(reinterpret_cast<const uint4*>(a.q_norm + at_k.x)),
                 __ldg(reinterpret_cast<const uint4*>(a.q_norm + at_k.y)), w);
      for (int h = h0; h < h1; h += 2) {
        uint4 x[2], y[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (!fresh || h + u >= h1) continue;
          const __nv_bfloat16* src = a.q + row * a.ld_q + (h + u) * kD;
          x[u] = ld_stream(src + at_k.x);
          y[u] = ld_stream(src + at_k.y);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float v[16];
          unpack16(x[u], y[u], v);
          if (a.q_norm != nullptr) norm_head(v, w, a.eps);
          turn_head<LAYOUT>(v, t, turns);
          pack16(v, x[u], y[u]);
          if (!fresh || h + u >= h1) continue;
          __nv_bfloat16* dst = a.q_out + row * a.ld_q_out + (h + u) * kD;
          *reinterpret_cast<uint4*>(dst + at_k.x) = x[u];
          *reinterpret_cast<uint4*>(dst + at_k.y) = y[u];
        }
      }
      continue;
    }
    // K and V of kHeads heads: set 2 u + s is head u's K (s = 0) or V
    const int h0 = part * kHeads;
    uint4 x[kSets], y[kSets];
    int slot[kHeads];
    float old[kSets];
#pragma unroll
    for (int u = 0; u < kHeads; ++u) {
      slot[u] = -2;
      if (h0 + u < a.Hkv) slot[u] = a.page_table[((int64_t)b * a.Hkv + h0 + u) * a.nblk_cap + j];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int2 at = s ? at_v : at_k;
        x[2 * u + s] = y[2 * u + s] = make_uint4(0u, 0u, 0u, 0u);
        if (!fresh || h0 + u >= a.Hkv) continue;
        const __nv_bfloat16* src = a.kv[s] + row * a.ld[s] + (h0 + u) * kD;
        x[2 * u + s] = ldg_stream(src + at.x);
        y[2 * u + s] = ldg_stream(src + at.y);
      }
    }
#pragma unroll
    for (int u = 0; u < kHeads; ++u) {
      if (slot[u] < 0 || slot[u] >= a.n_slots) {
        if (tid == 0 && h0 + u < a.Hkv) report(a.status, SCOUT_DEV_BAD_INDEX);
        slot[u] = -1;
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) old[2 * u + s] = r0 > 0 && slot[u] >= 0 ? a.scale[s][slot[u]] : 0.f;
    }
    {
      float w[16];
      if (a.k_norm != nullptr)
        unpack16(__ldg(reinterpret_cast<const uint4*>(a.k_norm + at_k.x)),
                 __ldg(reinterpret_cast<const uint4*>(a.k_norm + at_k.y)), w);
#pragma unroll
      for (int u = 0; u < kHeads; ++u) {
        float v[16];
        unpack16(x[2 * u], y[2 * u], v);
        if (a.k_norm != nullptr) norm_head(v, w, a.eps);
        turn_head<LAYOUT>(v, t, turns);
        pack16(v, x[2 * u], y[2 * u]);
      }
    }
    bool infinite = false;
#pragma unroll
    for (int i = 0; i < kSets; ++i) {
      uint32_t m = max_abs2(max_abs2(max_abs2(max_abs2(0u, x[i].x), x[i].y), x[i].z), x[i].w);
      m = max_abs2(max_abs2(max_abs2(max_abs2(m, y[i].x), y[i].y), y[i].z), y[i].w);
      // rows that are not new hold zeros (a zero stays zero through norm and turn)
      const uint32_t big = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
      if (lane == 0) top[buf][i][warp] = big;
    }
    __syncthreads();  // also: every thread has read the old scales
    uint32_t big[kSets];
#pragma unroll
    for (int i = 0; i < kSets; ++i) {
      big[i] = 0u;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) big[i] = max(big[i], top[buf][i][k]);
      infinite |= big[i] == 0x7f80u;
    }
    buf ^= 1;
    if (infinite) {  // the same for the CTA: the largest of the finite values (rare)
#pragma unroll
      for (int i = 0; i < kSets; ++i) {
        uint32_t m = max_abs2(max_abs2(max_abs2(max_abs2(0u, finite2(x[i].x)), finite2(x[i].y)), finite2(x[i].z)), finite2(x[i].w));
        m = max_abs2(max_abs2(max_abs2(max_abs2(m, finite2(y[i].x)), finite2(y[i].y)), finite2(y[i].z)), finite2(y[i].w));
        const uint32_t v = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
        if (lane == 0) top[buf][i][warp] = v;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kSets; ++i) {
        big[i] = 0u;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) big[i] = max(big[i], top[buf][i][k]);
      }
      buf ^= 1;
    }
#pragma unroll
    for (int u = 0; u < kHeads; ++u) {
      if (slot[u] < 0) continue;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int i = 2 * u + s;
        const int2 at = s ? at_v : at_k;
        const float need = pow2_biased(scale_exponent<F>(__uint_as_float(big[i] << 16)));
        // the scale of a block with cached tokens never shrinks
        const bool grows = r0 > 0 && need > old[i];
        const float scale = r0 > 0 && !grows ? old[i] : need;
        uint8_t* page = a.pool[s] + (int64_t)slot[u] * (P * kD) + r * kD;
        if (r < r0 && grows) {
          const float ratio = old[i] / need;
          uint2 *p0 = reinterpret_cast<uint2*>(page + at.x), *p1 = reinterpret_cast<uint2*>(page + at.y);
          const uint2 c0 = *p0, c1 = *p1;
          *p0 = make_uint2(recode4<F>(c0.x, ratio), recode4<F>(c0.y, ratio));
          *p1 = make_uint2(recode4<F>(c1.x, ratio), recode4<F>(c1.y, ratio));
        }
        if (fresh) {
          const float inv = 1.f / scale;  // exact where the scale is a power of two (1 / 2^-126 = 2^126 is finite)
          *reinterpret_cast<uint2*>(page + at.x) = encode8<F>(x[i], inv);
          *reinterpret_cast<uint2*>(page + at.y) = encode8<F>(y[i], inv);
        }
        if (tid == 0 && (r0 == 0 || grows)) a.scale[s][slot[u]] = scale;
      }
    }
  }
}

// the two rows of the largest batch, the prefixes' part and the maxima: within what needs no request
static_assert((2 * 32 + 2 * kMaxBatch + 2 + 4 * kHeads * 16) * sizeof(int) <= 48 * 1024, "48 KB of shared memory");

template <int P, int F>
int launch_rotate8(int layout, const Rot8Args& a, int grid, size_t smem, cudaStream_t st) {
  if (layout == SCOUT_ROPE_HALF)
    rotate8_kernel<P, F, SCOUT_ROPE_HALF><<<grid, P * 8, smem, st>>>(a);
  else
    rotate8_kernel<P, F, SCOUT_ROPE_INTERLEAVED><<<grid, P * 8, smem, st>>>(a);
  return launch_status();
}

template <int F>
int dispatch_rotate8(int P, int layout, const Rot8Args& a, int grid, size_t smem, cudaStream_t st) {
  switch (P) {
    case 16: return launch_rotate8<16, F>(layout, a, grid, smem, st);
    case 32: return launch_rotate8<32, F>(layout, a, grid, smem, st);
    default: return launch_rotate8<64, F>(layout, a, grid, smem, st);
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
  a.kv_parts = (Hkv + kHeads - 1) / kHeads;
  a.q_parts = (Hq + kQHeads - 1) / kQHeads;
  a.n_slots = n_slots;
  a.rope = rope_of(rope);
  a.eps = eps;
  a.status = dev_status;
  // at most n_tokens / P + 2 B blocks of a head are touched (each span's two ends partly)
  const int64_t blocks = (int64_t)n_tokens / P + 2 * (int64_t)(B < n_tokens ? B : n_tokens);
  const int64_t want = blocks * (a.kv_parts + a.q_parts) + (n_tokens == 0);  // (without rows: the report alone)
  const int most = sm_count() * (1024 / (P * 8));
  const int grid = (int)(want < most ? want : most);
  const size_t smem = (size_t)(2 * B + 2) * sizeof(int);
  return fmt == SCOUT_FP8_E4M3 ? dispatch_rotate8<SCOUT_FP8_E4M3>(P, rope->layout, a, grid, smem, stream)
                               : dispatch_rotate8<SCOUT_FP8_E5M2>(P, rope->layout, a, grid, smem, stream);
}
