// scout_read_kv and scout_read_kv8: blocks of a paged cache back as bf16 rows in token order.
//
// A warp takes 16 or 32 rows of a block of one KV head, of its K or its V.  Eight lanes hold a row, 32 bytes of bf16 each: all
// of the item's loads are in flight together, and a lane stores its 32 bytes at once, a whole sector (with two 16-byte
// stores the prompts below take 81 us, with sixteen lanes and 16-byte accesses 73).  One item a warp: a grid of resident
// CTAs that stride over the items takes 10% longer.
//
// Bound by DRAM: GB300, 8 prompts of up to 16K tokens, 8 KV heads, out of an 8-bit cache: 65.4 us for 428 MB (6.5 TB/s, 0.98 of
// the measured copy bandwidth), out of a bf16 one 85.5 us for 570 MB; 320 blocks by list: 2.8 us, the launch and two dependent reads.
// Into pinned host memory by the link: 365 MB of rows 1,887 us (193 GB/s, as a plain copy's), 320 blocks 16.5 us (173), out of
// either cache and in either order of the rows.
#include "fp8.cuh"

namespace scout {
namespace {

constexpr int kReadWarps = 2;
constexpr int kMaxItems = 1 << 29;  // blocks of a call

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

// R: rows of a warp's item.
template <int P, int F, int R>
__global__ void __launch_bounds__(kReadWarps * 32) read_kernel(const ReadArgs a) {
  constexpr int kParts = P / R;  // items of a block's K or V
  start_dependent();
  const int lane = threadIdx.x & 31, quad = lane >> 3, sub = lane & 7;
  const int64_t w = (int64_t)blockIdx.x * kReadWarps + (threadIdx.x >> 5);
  if (w >= 2 * kParts * a.n_items) return;
  const int64_t it = w / (2 * kParts);
  const int kv = (int)(w & 1), part = (int)(w / 2 % kParts);
  int b, h, j;
  if (a.block_list != nullptr) {
    const int2 e = __ldg(reinterpret_cast<const int2*>(a.block_list) + it);
    if (e.x == -1 && e.y == -1) return;
    if (e.x < 0 || e.x >= a.B * a.Hkv || e.y < 0 || e.y >= a.nblk_cap) {
      if (lane == 0) report(a.status, SCOUT_DEV_BAD_INDEX);
      return;
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
  const int64_t t0 = (int64_t)j * P + part * R, n = a.seq_len[b];
  if (lane == 0 && n < 0) report(a.status, SCOUT_DEV_BAD_INDEX);
  if (lane == 0 && n > (int64_t)a.nblk_cap * P) report(a.status, SCOUT_DEV_OVERFLOW);
  // a listed block needs a slot whether or not it has tokens; without a list entries past the end are not looked at
  if (a.block_list == nullptr && t0 >= n) return;
  const int slot = a.page_table[((int64_t)b * a.Hkv + h) * a.nblk_cap + j];
  if (slot < 0 || slot >= a.n_slots) {
    if (lane == 0 && (a.block_list != nullptr || slot != -1)) report(a.status, SCOUT_DEV_BAD_INDEX);
    return;
  }
  if (t0 >= n) return;
  int rows = (int)(n - t0 < R ? n - t0 : R);
  if (t0 + rows > a.T) {
    if (lane == 0) report(a.status, SCOUT_DEV_OVERFLOW);
    rows = (int)(a.T > t0 ? a.T - t0 : 0);
  }
  __nv_bfloat16* dst = a.out[kv] + b * a.stride_b + h * a.stride_h + (t0 + quad) * a.stride_t + sub * 16;
  const int64_t step = 4 * a.stride_t, row = (int64_t)slot * P + part * R + quad;
  if constexpr (F == kCopy) {
    const uint8_t* src = a.pool[kv] + row * (kD * 2) + sub * 32;
    uint4 x[R / 4], y[R / 4];
#pragma unroll
    for (int i = 0; i < R / 4; ++i)
      if (4 * i + quad < rows) ld32(src + i * (4 * kD * 2), x[i], y[i]);
#pragma unroll
    for (int i = 0; i < R / 4; ++i)
      if (4 * i + quad < rows) st32(dst + i * step, x[i], y[i]);
  } else {
    const uint8_t* src = a.pool[kv] + row * kD + sub * 16;
    const float scale = a.scale[kv][slot];
    uint4 v[R / 4];
#pragma unroll
    for (int i = 0; i < R / 4; ++i)
      if (4 * i + quad < rows) v[i] = ldg_stream(src + i * (4 * kD));
#pragma unroll
    for (int i = 0; i < R / 4; ++i)
      if (4 * i + quad < rows)
        st32(dst + i * step, widen8<F>(make_uint2(v[i].x, v[i].y), scale), widen8<F>(make_uint2(v[i].z, v[i].w), scale));
  }
}

template <int P, int F, int R>
int launch_read(const ReadArgs& a, cudaStream_t st) {
  const int64_t grid = (2 * (P / R) * a.n_items + kReadWarps - 1) / kReadWarps;  // at most twice kMaxItems
  return launch_dependent(read_kernel<P, F, R>, grid, kReadWarps * 32, 0, st, a);
}

template <int P, int F>
int launch_read(const ReadArgs& a, cudaStream_t st) {
  // Items of 16 rows where they are few (320 blocks: 2.9 us against 3.1 of 32 rows), otherwise of 32 (all blocks into
  // [B][T][Hkv][D] rows: 67.2 us against 69.0).
  if (P == 16 || 2 * (P / 16) * a.n_items <= 32 * (int64_t)sm_count()) return launch_read<P, F, 16>(a, st);
  return launch_read<P, F, P == 16 ? 16 : 32>(a, st);
}

template <int F>
int launch_read(int P, const ReadArgs& a, cudaStream_t st) {
  switch (P) {
    case 16: return launch_read<16, F>(a, st);
    case 32: return launch_read<32, F>(a, st);
    default: return launch_read<64, F>(a, st);
  }
}

inline bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

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
      (int64_t)B * Hkv > kMaxItems / nblk_cap || (block_list != nullptr && n_list > kMaxItems) || stride_b % 16 != 0 || stride_h % 16 != 0 || stride_t % 16 != 0 ||
      !aligned(K_pool, fmt == kCopy ? 32 : 16) || !aligned(V_pool, fmt == kCopy ? 32 : 16) || !aligned(K_out, 32) ||
      !aligned(V_out, 32) ||
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
