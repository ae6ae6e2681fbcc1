// scout_append_kv8: new bf16 K/V rows into 8-bit pools with one power-of-two scale per slot (a
// block of one KV head), quantised as they are written.
//
// One warp per (touched block, KV head, K or V).  Sixteen lanes hold a token's 128 channels (16
// bytes each), so a warp instruction moves two rows, and a whole block's new rows sit in
// registers (64 of a lane's at P = 32): they are read once, their maximum is taken, and the codes
// are made from the registers.  Items go in (sequence, block, head) order, so that neighbouring
// warps read neighbouring head rows of the same tokens.  The page-table slot is in flight with
// the rows, which do not depend on it.
//
// Cached tokens of a sequence's last block are read only when the block's scale grows: their
// codes are then rounded to the new scale (a power of two coarser: exact but for codes that fall
// below the normal range).
//
// Bound by DRAM for prompts: GB300, 8 of up to 16K tokens, 8 KV heads, 70.4 us for 428 MB (6.1 TB/s,
// 0.90 of the measured copy bandwidth); a decode step of 40 sequences takes 3.9 us, a chain of
// dependent reads (lengths, slot and rows, scale).
#include "fp8.cuh"

namespace scout {
namespace {

constexpr int kA8Warps = 8;

struct App8Args {
  const __nv_bfloat16 *K, *V;  // new rows
  int64_t ld_k, ld_v;          // elements from a token to the next
  uint8_t *K_pool, *V_pool;
  float *K_scale, *V_scale;
  const int32_t* prev_len;
  const int32_t* seq_len;
  const int32_t* page_table;
  int n_tokens, B, Hkv, nblk_cap;
  int64_t n_slots;
  int32_t* status;
};

template <int P, int F>
__global__ void __launch_bounds__(kA8Warps * 32) append8_kernel(const App8Args a) {
  extern __shared__ int sm[];
  __shared__ int partial[2 * 32];
  const int B = a.B;
  int* tok = sm;            // [B + 1] new tokens before sequence b
  int* tou = sm + (B + 1);  // [B + 1] touched blocks (of one KV head) before it
  const int tid = threadIdx.x, lane = tid & 31;
  const int cap_tokens = a.nblk_cap * P;
  int* const out[2] = {tok, tou};
  cta_prefixes<2>(B, out, partial, [&](int b, int (&x)[2]) {
    const SeqSpan s = seq_span(a.prev_len, a.seq_len, b, cap_tokens);
    x[0] = s.seq - s.prev;
    x[1] = s.seq > s.prev ? (s.seq + P - 1) / P - s.prev / P : 0;
  });
  if (blockIdx.x == 0)
    for (int b = tid; b < B; b += blockDim.x) report_span(a.status, a.prev_len, a.seq_len, b, cap_tokens);
  const int64_t items = (int64_t)tou[B] * a.Hkv * 2;
  const int half = lane >> 4, chunk = lane & 15;
  const int64_t wn = (int64_t)gridDim.x * kA8Warps;
  for (int64_t it = (int64_t)blockIdx.x * kA8Warps + (tid >> 5); it < items; it += wn) {
    const bool is_v = (it & 1) != 0;
    const int bh = (int)(it >> 1), blk = (int)((unsigned)bh / (unsigned)a.Hkv), h = bh - blk * a.Hkv;
    const int b = owner_of(tou, B, blk);
    const SeqSpan s = seq_span(a.prev_len, a.seq_len, b, cap_tokens);
    const int j = s.prev / P + blk - tou[b];
    const int r0 = max(s.prev - j * P, 0), r1 = min(s.seq - j * P, P);  // the block's new rows
    const int64_t i0 = (int64_t)tok[b] + (j * P - s.prev);              // token row of its row 0
    const int slot = a.page_table[((int64_t)b * a.Hkv + h) * a.nblk_cap + j];  // in flight with the rows
    const int64_t ld = is_v ? a.ld_v : a.ld_k;
    const bool rows_ok = i0 + r1 <= a.n_tokens;
    const __nv_bfloat16* src = (is_v ? a.V : a.K) + i0 * ld + h * kD + chunk * 8;
    uint4 v[P / 2];
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      const int r = 2 * i + half;
      v[i] = r >= r0 && r < r1 && rows_ok ? ldg_stream(src + (int64_t)r * ld) : make_uint4(0u, 0u, 0u, 0u);
    }
    if (!rows_ok || slot < 0 || slot >= a.n_slots) {
      if (lane == 0) report(a.status, SCOUT_DEV_BAD_INDEX);
      if (!rows_ok) break;  // the rows are packed: those of the items that follow end no earlier
      continue;
    }
    uint8_t* page = (is_v ? a.V_pool : a.K_pool) + (int64_t)slot * (P * kD) + chunk * 8;
    float* scale_at = (is_v ? a.V_scale : a.K_scale) + slot;
    const float old = r0 > 0 ? *scale_at : 0.f;
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < P / 2; ++i) m = max_abs2(max_abs2(max_abs2(max_abs2(m, v[i].x), v[i].y), v[i].z), v[i].w);
    uint32_t big = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
    if (big == 0x7f80u) {  // an infinity among them: the largest of the others (rare)
      m = 0u;
#pragma unroll 1
      for (int r = r0 + half; r < r1; r += 2) {  // the same rows, from memory (L2)
        const uint4 x = ldg_stream(src + (int64_t)r * ld);
        m = max_abs2(max_abs2(max_abs2(max_abs2(m, finite2(x.x)), finite2(x.y)), finite2(x.z)), finite2(x.w));
      }
      big = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
    }
    const float need = pow2_biased(scale_exponent<F>(__uint_as_float(big << 16)));
    // the scale of a block with cached tokens never shrinks
    const bool grows = r0 > 0 && need > old;
    const float scale = r0 > 0 && !grows ? old : need;
    // exact where the scale is a power of two (1 / 2^-126 = 2^126 is finite)
    const float inv = 1.f / scale;
    if (grows) {
      const float ratio = old / need;
#pragma unroll 1
      for (int r = half; r < r0; r += 2) {
        uint2* at = reinterpret_cast<uint2*>(page + r * kD);
        const uint2 c = *at;
        *at = make_uint2(recode4<F>(c.x, ratio), recode4<F>(c.y, ratio));
      }
    }
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      const int r = 2 * i + half;
      if (r >= r0 && r < r1) *reinterpret_cast<uint2*>(page + r * kD) = encode8<F>(v[i], inv);
    }
    if (lane == 0 && (r0 == 0 || grows)) *scale_at = scale;
  }
}

// the prefixes' static part and the two rows of the largest batch: within what needs no request
static_assert((2 * 32 + 2 * kMaxBatch + 2) * sizeof(int) <= 48 * 1024, "48 KB of shared memory");

template <int P, int F>
int launch_append8(const App8Args& a, int grid, size_t smem, cudaStream_t st) {
  append8_kernel<P, F><<<grid, kA8Warps * 32, smem, st>>>(a);
  return launch_status();
}

template <int F>
int dispatch_append8(int P, const App8Args& a, int grid, size_t smem, cudaStream_t st) {
  switch (P) {
    case 16: return launch_append8<16, F>(a, grid, smem, st);
    case 32: return launch_append8<32, F>(a, grid, smem, st);
    default: return launch_append8<64, F>(a, grid, smem, st);
  }
}

}  // namespace
}  // namespace scout

extern "C" int scout_append_kv8(int fmt, const void* K_new, int64_t ld_k, const void* V_new, int64_t ld_v,
                                int n_tokens, const int32_t* prev_len, const int32_t* seq_len,
                                const int32_t* page_table, int B, int Hkv, int D, int P, int nblk_cap, void* K_pool,
                                void* V_pool, float* K_scale, float* V_scale, int64_t n_slots, int32_t* dev_status,
                                cudaStream_t stream) {
  using namespace scout;
  if ((n_tokens > 0 && (K_new == nullptr || V_new == nullptr)) || seq_len == nullptr || page_table == nullptr ||
      K_pool == nullptr || V_pool == nullptr || K_scale == nullptr || V_scale == nullptr)
    return SCOUT_ERR_INVALID_ARG;
  if (!valid_fp8(fmt) || n_tokens < 0 || B <= 0 || Hkv <= 0 || nblk_cap <= 0 || n_slots <= 0 ||
      ld_k < (int64_t)Hkv * D || ld_v < (int64_t)Hkv * D)
    return SCOUT_ERR_INVALID_ARG;
  if (D != kD || !valid_P(P) || B > kMaxBatch || nblk_cap > kMaxNblk || n_slots > 0x7fffffffLL ||
      (int64_t)B * nblk_cap * P > 0x7fffffffLL || (int64_t)B * Hkv * nblk_cap > 0x7fffffffLL || ld_k % 8 != 0 ||
      ld_v % 8 != 0 || !aligned16(K_new) || !aligned16(V_new) || !aligned16(K_pool) || !aligned16(V_pool))
    return SCOUT_ERR_UNSUPPORTED;
  if (n_tokens == 0 && dev_status == nullptr) return SCOUT_OK;  // no rows, and nowhere to say that some were due
  App8Args a;
  a.K = static_cast<const __nv_bfloat16*>(K_new);
  a.V = static_cast<const __nv_bfloat16*>(V_new);
  a.ld_k = ld_k;
  a.ld_v = ld_v;
  a.K_pool = static_cast<uint8_t*>(K_pool);
  a.V_pool = static_cast<uint8_t*>(V_pool);
  a.K_scale = K_scale;
  a.V_scale = V_scale;
  a.prev_len = prev_len;
  a.seq_len = seq_len;
  a.page_table = page_table;
  a.n_tokens = n_tokens;
  a.B = B;
  a.Hkv = Hkv;
  a.nblk_cap = nblk_cap;
  a.n_slots = n_slots;
  a.status = dev_status;
  // at most n_tokens / P + 2 B blocks of a head are touched (each span's two ends partly)
  const int64_t warps = ((int64_t)n_tokens / P + 2 * (int64_t)(B < n_tokens ? B : n_tokens)) * Hkv * 2;
  const int64_t want = (warps + kA8Warps - 1) / kA8Warps + (n_tokens == 0);  // (without rows: the report alone)
  const int grid = (int)(want < sm_count() * 8 ? want : sm_count() * 8);
  const size_t smem = (size_t)(2 * B + 2) * sizeof(int);
  return fmt == SCOUT_FP8_E4M3 ? dispatch_append8<SCOUT_FP8_E4M3>(P, a, grid, smem, stream)
                               : dispatch_append8<SCOUT_FP8_E5M2>(P, a, grid, smem, stream);
}
