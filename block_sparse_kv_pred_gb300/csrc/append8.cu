// scout_append_kv8: new bf16 K/V rows into 8-bit pools with one power-of-two scale per slot (a
// block of one KV head), quantised as they are written.
//
// One warp per (touched block, KV head, K or V).  Sixteen lanes hold a token's 128 channels (16
// bytes each), so a warp instruction moves two rows, and a whole block's new rows sit in
// registers (64 of a lane's at P = 32): they are read once, their maximum is
// taken, and the codes are made from the registers.  Items go in (sequence, block, head) order, so
// that neighbouring warps read neighbouring head rows of the same tokens.
//
// Cached tokens of a sequence's last block are read only when the block's scale grows: their
// codes are then rounded to the new scale (a power of two coarser: exact but for codes that fall
// below the normal range).
#include "fp8.cuh"

namespace scout {
namespace {

constexpr int kA8Warps = 8;

struct App8Args {
  const __nv_bfloat16* src[2];  // K, V rows
  int64_t ld[2];                // elements from a token to the next
  uint8_t* pool[2];
  float* scale[2];
  const int32_t* prev_len;
  const int32_t* seq_len;
  const int32_t* page_table;
  int n_tokens, B, Hkv, nblk_cap;
  int64_t n_slots;
  int32_t* status;
};

// largest finite |x| of the eight bf16 of v, into the running pair maximum m (packed magnitudes):
// bf16 magnitudes order as integers; infinities and NaN count as zero
__device__ __forceinline__ uint32_t finite_max(uint32_t m, const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t a = w[i] & 0x7fff7fffu;
    a = __vminu2(a, 0x7f807f80u);            // NaN magnitudes become infinity's
    a &= ~__vcmpeq2(a, 0x7f807f80u);         // and those zero
    m = __vmaxu2(m, a);
  }
  return m;
}

template <int F>
__device__ __forceinline__ uint2 encode8(const uint4& v, float inv) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = Fp8<F>::pack(bf16_lo(w[i]) * inv, bf16_hi(w[i]) * inv);
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// Codes at the old scale -> codes at the new one; ratio = old / new.
template <int F>
__device__ __forceinline__ uint32_t recode4(uint32_t w, float ratio) {
  uint32_t lo, hi;
  unpack4<F>(w, lo, hi);
  const float2 a = half2_floats(lo), b = half2_floats(hi);
  return (uint32_t)Fp8<F>::pack(a.x * ratio, a.y * ratio) |
         ((uint32_t)Fp8<F>::pack(b.x * ratio, b.y * ratio) << 16);
}

template <int P, int F>
__global__ void __launch_bounds__(kA8Warps * 32) append8_kernel(const App8Args a) {
  extern __shared__ int sm[];
  __shared__ int partial[32];
  const int B = a.B;
  int* tok = sm;            // [B + 1] new tokens before sequence b
  int* tou = sm + (B + 1);  // [B + 1] touched blocks (of one KV head) before it
  const int tid = threadIdx.x, lane = tid & 31;
  const int cap_tokens = a.nblk_cap * P;
  for (int b = tid; b < B; b += blockDim.x) {
    const SeqSpan s = seq_span(a.prev_len, a.seq_len, b, cap_tokens);
    tok[b] = s.seq - s.prev;
    tou[b] = s.seq > s.prev ? (s.seq + P - 1) / P - s.prev / P : 0;
    if (blockIdx.x == 0) report_span(a.status, a.prev_len, a.seq_len, b, cap_tokens);
  }
  __syncthreads();
  cta_exclusive_prefix(tok, B, partial);
  cta_exclusive_prefix(tou, B, partial);
  const int64_t items = (int64_t)tou[B] * a.Hkv * 2;
  const int half = lane >> 4, chunk = lane & 15;
  const int64_t wn = (int64_t)gridDim.x * kA8Warps;
  for (int64_t it = (int64_t)blockIdx.x * kA8Warps + (tid >> 5); it < items; it += wn) {
    const int which = (int)(it & 1);
    const int64_t bh = it >> 1;
    const int blk = (int)(bh / a.Hkv), h = (int)(bh - (int64_t)blk * a.Hkv);
    const int b = owner_of(tou, B, blk);
    const SeqSpan s = seq_span(a.prev_len, a.seq_len, b, cap_tokens);
    const int j = s.prev / P + blk - tou[b];
    const int r0 = max(s.prev - j * P, 0), r1 = min(s.seq - j * P, P);  // the block's new rows
    const int64_t i0 = (int64_t)tok[b] + (j * P - s.prev);              // token row of its row 0
    const int slot = a.page_table[((int64_t)b * a.Hkv + h) * a.nblk_cap + j];
    if (slot < 0 || slot >= a.n_slots || i0 + r1 > a.n_tokens) {
      if (lane == 0) report(a.status, SCOUT_DEV_BAD_INDEX);
      continue;
    }
    const __nv_bfloat16* src = a.src[which] + i0 * a.ld[which] + h * kD + chunk * 8;
    uint8_t* page = a.pool[which] + (int64_t)slot * (P * kD) + chunk * 8;
    const float old = r0 > 0 ? a.scale[which][slot] : 0.f;
    uint4 v[P / 2];
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      const int r = 2 * i + half;
      v[i] = r >= r0 && r < r1 ? ldg_stream(src + (int64_t)r * a.ld[which]) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < P / 2; ++i) m = finite_max(m, v[i]);
    const uint32_t big = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
    const uint32_t e = scale_exponent<F>(__uint_as_float(big << 16));
    const float need = pow2_biased(e);
    // the scale of a block with cached tokens never shrinks
    const bool grows = r0 > 0 && need > old;
    const float scale = r0 > 0 && !grows ? old : need;
    // both factors are exact where the scales are powers of two (1 / 2^-126 = 2^126 is finite)
    const float inv = 1.f / scale;
    if (grows) {
      const float ratio = old / need;
      for (int i = 0; i < P / 2; ++i) {
        const int r = 2 * i + half;
        if (r >= r0) continue;
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
    if (lane == 0 && (r0 == 0 || grows)) a.scale[which][slot] = scale;
  }
}

template <int P, int F>
int launch_append8(const App8Args& a, int grid, size_t smem, cudaStream_t st) {
  if (smem > 48 * 1024 && cudaFuncSetAttribute(append8_kernel<P, F>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)smem) != cudaSuccess)
    return SCOUT_ERR_CUDA;
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
  if (K_new == nullptr || V_new == nullptr || seq_len == nullptr || page_table == nullptr || K_pool == nullptr ||
      V_pool == nullptr || K_scale == nullptr || V_scale == nullptr)
    return SCOUT_ERR_INVALID_ARG;
  if (!valid_fp8(fmt) || n_tokens < 0 || B <= 0 || Hkv <= 0 || nblk_cap <= 0 || n_slots <= 0 ||
      ld_k < (int64_t)Hkv * D || ld_v < (int64_t)Hkv * D)
    return SCOUT_ERR_INVALID_ARG;
  if (D != kD || !valid_P(P) || B > kMaxBatch || nblk_cap > kMaxNblk || n_slots > 0x7fffffffLL ||
      (int64_t)B * nblk_cap * P > 0x7fffffffLL || ld_k % 8 != 0 || ld_v % 8 != 0 || !aligned16(K_new) ||
      !aligned16(V_new) || !aligned16(K_pool) || !aligned16(V_pool))
    return SCOUT_ERR_UNSUPPORTED;
  if (n_tokens == 0) return SCOUT_OK;
  App8Args a;
  a.src[0] = static_cast<const __nv_bfloat16*>(K_new);
  a.src[1] = static_cast<const __nv_bfloat16*>(V_new);
  a.ld[0] = ld_k;
  a.ld[1] = ld_v;
  a.pool[0] = static_cast<uint8_t*>(K_pool);
  a.pool[1] = static_cast<uint8_t*>(V_pool);
  a.scale[0] = K_scale;
  a.scale[1] = V_scale;
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
  const int64_t want = (warps + kA8Warps - 1) / kA8Warps;
  const int grid = (int)(want < sm_count() * 8 ? want : sm_count() * 8);
  const size_t smem = (size_t)(2 * B + 2) * sizeof(int);
  return fmt == SCOUT_FP8_E4M3 ? dispatch_append8<SCOUT_FP8_E4M3>(P, a, grid, smem, stream)
                               : dispatch_append8<SCOUT_FP8_E5M2>(P, a, grid, smem, stream);
}
