// scout_read_kv and scout_read_kv8: blocks of a paged cache back as bf16 rows in token order.
//
// A warp takes a block of one KV head, its K or its V.  Sixteen lanes hold a row (16 bytes of bf16, 8 of codes a lane), all of
// the block's loads are in flight together, and 16-byte stores write whole rows.
#include "fp8.cuh"

namespace scout {
namespace {

constexpr int kReadWarps = 8;

struct ReadArgs {
  const uint8_t* pool[2];
  const float* scale[2];
  int64_t n_slots;
  const int32_t* page_table;
  const int32_t* seq_len;
  int B, Hkv, nblk_cap;
  const int32_t* block_list;
  int64_t n_items;  // blocks
  __nv_bfloat16* out[2];
  int64_t stride_b, stride_h, stride_t, T;
  int heads_inner;  // order of all the blocks: (b, j, h) or (b, h, j)
  int32_t* status;
};

constexpr int kCopy = -1;  // the format of a bf16 pool

template <int F>
__device__ __forceinline__ uint4 widen8(const uint2& c, float scale) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t lo, hi;
    unpack4<F>(i ? c.y : c.x, lo, hi);
    const float2 a = half2_floats(lo), b = half2_floats(hi);
    o[2 * i] = pack_bf16(a.x * scale, a.y * scale);
    o[2 * i + 1] = pack_bf16(b.x * scale, b.y * scale);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int P, int F>
__global__ void __launch_bounds__(kReadWarps * 32) read_kernel(const ReadArgs a) {
  const int lane = threadIdx.x & 31, half = lane >> 4, chunk = lane & 15;
  const int64_t wn = (int64_t)gridDim.x * kReadWarps;
  for (int64_t w = (int64_t)blockIdx.x * kReadWarps + (threadIdx.x >> 5); w < 2 * a.n_items; w += wn) {
    const int64_t it = w >> 1;
    const int kv = (int)(w & 1);
    int b, h, j;
    if (a.block_list != nullptr) {
      const int2 e = __ldg(reinterpret_cast<const int2*>(a.block_list) + it);
      if (e.x == -1 && e.y == -1) continue;
      if (e.x < 0 || e.x >= a.B * a.Hkv || e.y < 0 || e.y >= a.nblk_cap) {
        if (lane == 0) report(a.status, SCOUT_DEV_BAD_INDEX);
        continue;
      }
      b = e.x / a.Hkv;
      h = e.x - b * a.Hkv;
      j = e.y;
    } else {
      const unsigned n = (unsigned)it, heads = (unsigned)a.Hkv, cap = (unsigned)a.nblk_cap;
      const unsigned q = a.heads_inner ? n / heads : n / cap, m = a.heads_inner ? n - q * heads : n - q * cap;
      b = (int)(a.heads_inner ? q / cap : q / heads);
      h = (int)(a.heads_inner ? m : q - b * heads);
      j = (int)(a.heads_inner ? q - b * cap : m);
    }
    const int64_t t0 = (int64_t)j * P, n = a.seq_len[b];
    if (t0 >= n) continue;
    const int slot = a.page_table[((int64_t)b * a.Hkv + h) * a.nblk_cap + j];
    if (slot < 0 || slot >= a.n_slots) {
      if (lane == 0 && (a.block_list != nullptr || slot != -1)) report(a.status, SCOUT_DEV_BAD_INDEX);
      continue;
    }
    int rows = (int)(n - t0 < P ? n - t0 : P);
    if (t0 + rows > a.T) {
      if (lane == 0) report(a.status, SCOUT_DEV_OVERFLOW);
      rows = (int)(a.T > t0 ? a.T - t0 : 0);
    }
    __nv_bfloat16* dst = a.out[kv] + b * a.stride_b + h * a.stride_h + (t0 + half) * a.stride_t + chunk * 8;
    const int64_t step = 2 * a.stride_t;
    if constexpr (F == kCopy) {
      const uint4* src = reinterpret_cast<const uint4*>(a.pool[kv]) + (int64_t)slot * (P * 16) + lane;
      uint4 v[P / 2];
#pragma unroll
      for (int i = 0; i < P / 2; ++i)
        if (2 * i + half < rows) v[i] = ldg_stream(src + i * 32);
#pragma unroll
      for (int i = 0; i < P / 2; ++i)
        if (2 * i + half < rows) *reinterpret_cast<uint4*>(dst + i * step) = v[i];
    } else {
      const uint2* src = reinterpret_cast<const uint2*>(a.pool[kv]) + (int64_t)slot * (P * 16) + lane;
      const float scale = a.scale[kv][slot];
      uint2 v[P / 2];
#pragma unroll
      for (int i = 0; i < P / 2; ++i)
        if (2 * i + half < rows) v[i] = __ldg(src + i * 32);
#pragma unroll
      for (int i = 0; i < P / 2; ++i)
        if (2 * i + half < rows) *reinterpret_cast<uint4*>(dst + i * step) = widen8<F>(v[i], scale);
    }
  }
}

template <int F>
int launch_read(int P, const ReadArgs& a, cudaStream_t st) {
  const int64_t want = (2 * a.n_items + kReadWarps - 1) / kReadWarps;
  const int grid = (int)(want < sm_count() * 8 ? want : sm_count() * 8);
  switch (P) {
    case 16: read_kernel<16, F><<<grid, kReadWarps * 32, 0, st>>>(a); break;
    case 32: read_kernel<32, F><<<grid, kReadWarps * 32, 0, st>>>(a); break;
    default: read_kernel<64, F><<<grid, kReadWarps * 32, 0, st>>>(a); break;
  }
  return launch_status();
}

int read_blocks(int fmt, const void* K_pool, const void* V_pool, const float* K_scale, const float* V_scale,
                int64_t n_slots, const int32_t* page_table, const int32_t* seq_len, int B, int Hkv, int D, int P,
                int nblk_cap, const int32_t* block_list, int n_list, void* K_out, void* V_out, int64_t stride_b,
                int64_t stride_h, int64_t stride_t, int64_t T, int host_out, int32_t* dev_status, cudaStream_t stream) {
  if (K_pool == nullptr || V_pool == nullptr || page_table == nullptr || seq_len == nullptr || K_out == nullptr ||
      V_out == nullptr || (fmt != kCopy && (K_scale == nullptr || V_scale == nullptr)))
    return SCOUT_ERR_INVALID_ARG;
  if (n_slots <= 0 || B <= 0 || Hkv <= 0 || nblk_cap <= 0 || T <= 0 || stride_b < 0 || stride_h < 0 || stride_t < 0 ||
      (block_list != nullptr && n_list < 0) || host_out < 0 || host_out > 1)
    return SCOUT_ERR_INVALID_ARG;
  if (D != kD || !valid_P(P) || nblk_cap > kMaxNblk || n_slots > 0x7fffffffLL ||
      (int64_t)B * Hkv > 0x7fffffffLL / nblk_cap || stride_b % 8 != 0 || stride_h % 8 != 0 || stride_t % 8 != 0 ||
      !aligned16(K_pool) || !aligned16(V_pool) || !aligned16(K_out) || !aligned16(V_out) ||
      (reinterpret_cast<uintptr_t>(block_list) & 7u))
    return SCOUT_ERR_UNSUPPORTED;
  if (block_list != nullptr && n_list == 0) return SCOUT_OK;
  if (host_out) {
    // the last row's end, in elements; a host copy that does not fit 62 bits is not mapped
    const __int128 end = (__int128)(B - 1) * stride_b + (__int128)(Hkv - 1) * stride_h + (__int128)(T - 1) * stride_t + D;
    if (end > (__int128)1 << 61) return SCOUT_ERR_UNSUPPORTED;
    K_out = mapped_address(K_out, (size_t)end * 2);
    V_out = mapped_address(V_out, (size_t)end * 2);
    if (K_out == nullptr || V_out == nullptr) return SCOUT_ERR_UNSUPPORTED;
  }
  ReadArgs a;
  a.pool[0] = static_cast<const uint8_t*>(K_pool);
  a.pool[1] = static_cast<const uint8_t*>(V_pool);
  a.scale[0] = K_scale;
  a.scale[1] = V_scale;
  a.n_slots = n_slots;
  a.page_table = page_table;
  a.seq_len = seq_len;
  a.B = B;
  a.Hkv = Hkv;
  a.nblk_cap = nblk_cap;
  a.block_list = block_list;
  a.n_items = block_list != nullptr ? n_list : (int64_t)B * Hkv * nblk_cap;
  a.out[0] = static_cast<__nv_bfloat16*>(K_out);
  a.out[1] = static_cast<__nv_bfloat16*>(V_out);
  a.stride_b = stride_b;
  a.stride_h = stride_h;
  a.stride_t = stride_t;
  a.T = T;
  a.heads_inner = stride_h < stride_t;
  a.status = dev_status;
  switch (fmt) {
    case kCopy: return launch_read<kCopy>(P, a, stream);
    case SCOUT_FP8_E4M3: return launch_read<SCOUT_FP8_E4M3>(P, a, stream);
    default: return launch_read<SCOUT_FP8_E5M2>(P, a, stream);
  }
}

}  // namespace
}  // namespace scout

extern "C" int scout_read_kv(const void* K_pool, const void* V_pool, int64_t n_slots, const int32_t* page_table,
                             const int32_t* seq_len, int B, int Hkv, int D, int P, int nblk_cap,
                             const int32_t* block_list, int n_list, void* K_out, void* V_out, int64_t stride_b,
                             int64_t stride_h, int64_t stride_t, int64_t T, int host_out, int32_t* dev_status,
                             cudaStream_t stream) {
  using namespace scout;
  return read_blocks(kCopy, K_pool, V_pool, nullptr, nullptr, n_slots, page_table, seq_len, B, Hkv, D, P, nblk_cap,
                     block_list, n_list, K_out, V_out, stride_b, stride_h, stride_t, T, host_out, dev_status, stream);
}

extern "C" int scout_read_kv8(int fmt, const void* K_pool, const void* V_pool, const float* K_scale,
                              const float* V_scale, int64_t n_slots, const int32_t* page_table, const int32_t* seq_len,
                              int B, int Hkv, int D, int P, int nblk_cap, const int32_t* block_list, int n_list,
                              void* K_out, void* V_out, int64_t stride_b, int64_t stride_h, int64_t stride_t, int64_t T,
                              int host_out, int32_t* dev_status, cudaStream_t stream) {
  using namespace scout;
  if (!valid_fp8(fmt)) return SCOUT_ERR_INVALID_ARG;
  return read_blocks(fmt, K_pool, V_pool, K_scale, V_scale, n_slots, page_table, seq_len, B, Hkv, D, P, nblk_cap,
                     block_list, n_list, K_out, V_out, stride_b, stride_h, stride_t, T, host_out, dev_status, stream);
}
