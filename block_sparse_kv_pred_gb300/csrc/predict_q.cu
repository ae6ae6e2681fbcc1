// scout_predict_q: layer-ahead query prediction Q_pred = X W_Q^T on the 5th-generation
// tensor cores.  ScoutAttention (arXiv HTML), section 3.3 and Algorithm 1 (query
// prediction): the next layer's query projection applied to the current layer's input.
//
// Decode batches are small (M = 1..256 rows of X) while W_Q is large, so the GEMM is
// computed swapped: D[n][m] = sum_k W[n][k] X[m][k].  A CTA owns 128 rows of W (the
// MMA's M = 128 TMEM lanes); the batch, padded to a multiple of 16, is the MMA's N.
// W and X tiles (64 k-columns, 128-byte swizzle) stream in by TMA through a ring of
// shared-memory stages guarded by mbarriers, up to four k-blocks per stage (measured on
// GB300: one k-block per stage streams ~25% slower, the barrier round trip of a stage
// being paid per 22 KB instead of per 88 KB); one thread issues tcgen05.mma into a
// TMEM accumulator and frees each stage with tcgen05.commit.  The K dimension is
// split over the CTAs of a thread-block cluster so that about one CTA runs per SM.
// The batch columns of the accumulator are dealt out over the cluster's CTAs: each
// CTA stores the columns another CTA owns straight into that CTA's shared memory
// (distributed shared memory), then sums the partials of its own columns and writes
// them as bf16 Q.  No global scratch is used.

//
// scout_predict_q_rotated is the same kernel with another last step: a tile is one head, so a
// CTA holds whole heads of its batch columns.  The sums go to shared memory in fp32, eight lanes
// take a head (rotate.cuh), normalise and turn it, and store it rounded once, 16 bytes a lane.
// The cosines and sines are made, and the norm's weights read, while W streams in (read in the last step, the weights
// alone cost 1.3 us).  GB300: 14.0 us for 40 x 5120 x 5120 and 10.5 us for 8 x 4096 x 4096 (3.8 and 3.2 TB/s of W: the
// launch, ~1.8 us to the first product, the stream at about 6 TB/s, 1.3 and 1.1 us of exchange, 1.2 and 0.6 of last step).
// 128 and 256 x 5120 x 5120: 17.8 and 25.5 us (2.9 and 2.1 TB/s of W: X's tiles take up to two thirds of the ring, and what is
// exchanged grows with the rows).

#include "rotate.cuh"

namespace scout {
namespace {

constexpr int kBM = 128;      // W rows per CTA (MMA M)
constexpr int kBK = 64;       // k columns per k-block (one 128-byte swizzle atom of bf16)
constexpr int kMaxKps = 4;    // k-blocks per ring stage, at most
constexpr int kStages = 16;  // upper bound; the ring takes what shared memory holds
constexpr int kThreadsQ = 128;
constexpr int kMaxN = 256;    // padded batch (MMA N) limit
constexpr int kWTileBytes = kBM * kBK * 2;  // 16 KiB
constexpr int kRingBytes = 224 * 1024;      // of shared memory, at most, the exchange included
constexpr int kApartBytes = 32 * 1024;      // an exchange that lies beside the ring, at most

// --- cluster PTX --------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
__device__ __forceinline__ uint32_t map_peer(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void st_peer(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// Instruction descriptor: fp32 accumulate, bf16 A and B, both K-major, M = 128, N = n.
__host__ __device__ constexpr uint32_t idesc_bf16(int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kBM >> 4) << 24);
}

struct GemmArgs {
  __nv_bfloat16* Q;
  int M, N, n_pad, tmem_cols, kblocks, stages, x_tile_bytes;
  int kps;     // k-blocks per ring stage
  int recv_at; // bytes from the ring's start to what peers write: past the ring, or 0 (in it, once it is idle)
  int32_t* status;
  // of the rotated form
  const int32_t* positions;
  const __nv_bfloat16* norm;
  Rope rope;
  float eps;
  bool early;  // W may be read before the kernel before this one has finished
};

constexpr int kPlain = -1;  // no rotary layout: the sums are the result

// A ring stage holds nk <= kps consecutive k-blocks: their W tiles first, then their X tiles.
// One arrival expects both; the W and the X copies may be issued apart.
__device__ __forceinline__ void load_w(uint8_t* st, const CUtensorMap* tmW, const GemmArgs& a, int tile, int kb,
                                       int nk, uint64_t* bar) {
  mbar_arrive_tx(bar, (uint32_t)(nk * (kWTileBytes + a.x_tile_bytes)));
  for (int j = 0; j < nk; ++j) tma_load_2d(st + j * kWTileBytes, tmW, (kb + j) * kBK, tile * kBM, bar);
}
__device__ __forceinline__ void load_x(uint8_t* st, const CUtensorMap* tmX, const GemmArgs& a, int kb, int nk,
                                       uint64_t* bar) {
  for (int j = 0; j < nk; ++j)
    tma_load_2d(st + a.kps * kWTileBytes + j * a.x_tile_bytes, tmX, (kb + j) * kBK, 0, bar);
}

template <int LAYOUT>
__global__ void __launch_bounds__(kThreadsQ, 1) predict_q_kernel(const __grid_constant__ CUtensorMap tmW,
                                                                 const __grid_constant__ CUtensorMap tmX,
                                                                 const GemmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full_bar[kStages], empty_bar[kStages], done_bar;
  __shared__ uint32_t tmem_slot;
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* base = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const int stage_bytes = a.kps * (kWTileBytes + a.x_tile_bytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tile = blockIdx.x;
  const uint32_t S = gridDim.y, rank = cluster_rank();
  const int kb0 = (int)(rank * a.kblocks / S), kb1 = (int)((rank + 1) * a.kblocks / S);
  const int nst = (kb1 - kb0 + a.kps - 1) / a.kps;  // ring stages of this CTA's k range
  auto nk_of = [&](int i) { return min(a.kps, kb1 - kb0 - i * a.kps); };
  // A kernel that starts early after this one (scout_score_topk) may take SMs as they free up.  It waits for this grid to
  // finish before it reads Q, but what it reads before that has to be complete by now.  So the rotated form without
  // pdl, which is scheduled before its predecessor has finished all the same, lets it start after its own wait, further down
  // (GB300: behind the CTA's barrier 10.5 and 14.0 us for the sizes above, each thread right after its wait 10.6 and 14.2).
  if (LAYOUT == kPlain || a.early) release_dependents();

  // the first pass over the ring needs no free slot: issue it before the TMEM allocation.  W
  // does not depend on an earlier kernel; X may be written by the one this launch follows, so
  // an early start waits for it between the two
  const int first = min(a.stages, nst);
  if (tid == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(&full_bar[i], 1);
      mbar_init(&empty_bar[i], 1);
    }
    mbar_init(&done_bar, 1);
    fence_mbar_init();
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmX);
    if (LAYOUT != kPlain && !a.early) wait_prerequisites();
    for (int i = 0; i < first; ++i)
      load_w(base + i * stage_bytes, &tmW, a, tile, kb0 + i * a.kps, nk_of(i), &full_bar[i]);
    wait_prerequisites();
    for (int i = 0; i < first; ++i) load_x(base + i * stage_bytes, &tmX, a, kb0 + i * a.kps, nk_of(i), &full_bar[i]);
  }
  if (warp == 2) tmem_alloc(&tmem_slot, (uint32_t)a.tmem_cols);
  // rotated: the CTA's column k (of its groups, in order) is batch row m_of(k); eight lanes take one
  const int sub = lane & 7;
  auto m_of = [&](int k) { return ((int)rank + (k >> 3) * (int)S) * 8 + (k & 7); };
  int pos = -1;  // and turn: of the lane's column among the CTA's first 16
  Turn turn;
  Weights w;
  if constexpr (LAYOUT != kPlain) {
    wait_prerequisites();  // the positions may be an earlier kernel's, as X
    const int m = m_of(warp * 4 + (lane >> 3));
    pos = m < a.M ? a.positions[m] : -1;
    if (a.norm != nullptr) w = lane_weights(a.norm, lane_chunks<LAYOUT>(sub, a.rope.n));
    turn = lane_turn(a.rope, sub, (uint32_t)max(pos, 0));
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  if (LAYOUT != kPlain && !a.early) release_dependents();
  const bool apart = LAYOUT != kPlain && a.recv_at > 0;
  if (apart) cluster_arrive();  // this CTA runs: its shared memory may be written

  if (warp == 0 && lane == 0) {
    // TMA producer: the rest of the k range, each stage once the MMAs have freed it
    int issued = first;
    for (int i = first; i < nst; ++i) {
      const int st = i % a.stages;
      if (!mbar_wait(&empty_bar[st], ((i / a.stages) & 1) ^ 1)) {
        report(a.status, SCOUT_DEV_TIMEOUT);
        break;
      }
      load_w(base + st * stage_bytes, &tmW, a, tile, kb0 + i * a.kps, nk_of(i), &full_bar[st]);
      load_x(base + st * stage_bytes, &tmX, a, kb0 + i * a.kps, nk_of(i), &full_bar[st]);
      issued = i + 1;
    }
    // every issued copy lands before the CTA can retire
    for (int r = 0; r < a.stages && r < issued; ++r) {
      const int last = issued - 1 - r;
      if (!mbar_wait(&full_bar[last % a.stages], (last / a.stages) & 1)) report(a.status, SCOUT_DEV_TIMEOUT);
    }
  } else if (warp == 1 && lane == 0) {
    // MMA issuer
    const uint32_t idesc = idesc_bf16(a.n_pad);
    for (int i = 0; i < nst; ++i) {
      const int st = i % a.stages;
      if (!mbar_wait(&full_bar[st], (i / a.stages) & 1)) {
        report(a.status, SCOUT_DEV_TIMEOUT);
        break;
      }
      tc_fence_after();
      const uint32_t s0 = smem_u32(base + st * stage_bytes);
      const int nk = nk_of(i);
      for (int j = 0; j < nk; ++j) {
        const uint32_t sW = s0 + j * kWTileBytes, sX = s0 + a.kps * kWTileBytes + j * a.x_tile_bytes;
#pragma unroll
        for (int kk = 0; kk < kBK / 16; ++kk)
          umma_bf16(tmem, sw128_desc(sW + kk * 32), sw128_desc(sX + kk * 32), idesc,
                    (i > 0 || j > 0 || kk > 0) ? 1u : 0u);
      }
      umma_commit(&empty_bar[st]);
    }
    umma_commit(&done_bar);
  }
  __syncwarp();

  // ---- epilogue: thread (warp w, lane l) owns W row tile*128 + 32w + l (TMEM lane) ----
  // Column group g (8 batch columns) belongs to CTA g % S of the cluster.  recv holds, for
  // every source CTA s and every group this CTA owns, s's partial: [S][owned][8][128] fp32.
  if (!mbar_wait(&done_bar, 0)) report(a.status, SCOUT_DEV_TIMEOUT);
  tc_fence_after();
  const int r_local = warp * 32 + lane;
  const int row = tile * kBM + r_local;
  const uint32_t trow = tmem + ((uint32_t)(warp * 32) << 16);
  const int ngroups = a.n_pad / 8;
  const int owned = (ngroups + (int)S - 1) / (int)S;
  float* recv = reinterpret_cast<float*>(base + a.recv_at);
  float* mine = recv + (int)rank * owned * 8 * kBM;  // this CTA's own slots: no peer writes them
  float v[8];
  if (S > 1) {
    if (apart) cluster_wait();
    else cluster_sync();  // every CTA of the cluster is done with its ring: it may be written
    for (int g = 0; g < ngroups; ++g) {
      const uint32_t owner = (uint32_t)g % S;
      if (owner == rank) continue;
      tmem_ld8(trow + (uint32_t)(g * 8), v);
      const int slot = ((int)rank * owned + g / (int)S) * 8;
      const uint32_t dst = map_peer(smem_u32(recv + slot * kBM + r_local), owner);
#pragma unroll
      for (int e = 0; e < 8; ++e) st_peer(dst + (uint32_t)(e * kBM * 4), v[e]);
    }
    cluster_sync();  // the partials have landed (release/acquire across the cluster)
  }
  for (int g = (int)rank; g < ngroups; g += (int)S) {
    tmem_ld8(trow + (uint32_t)(g * 8), v);
    for (uint32_t s = 0; s < S; ++s) {
      if (s == rank) continue;
      const float* src = recv + ((int)s * owned + g / (int)S) * 8 * kBM + r_local;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += src[e * kBM];
    }
    if constexpr (LAYOUT == kPlain) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int m = g * 8 + e;
        if (m < a.M && row < a.N) a.Q[(int64_t)m * a.N + row] = __float2bfloat16_rn(v[e]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) mine[((g / (int)S) * 8 + e) * kBM + r_local] = v[e];
    }
  }
  if constexpr (LAYOUT != kPlain) {
    __syncthreads();
    const int2 at = lane_chunks<LAYOUT>(sub, a.rope.n);
    const int columns = (ngroups - (int)rank + (int)S - 1) / (int)S * 8;  // of this CTA
    for (int k0 = 0; k0 < columns; k0 += 16) {
      const int k = k0 + warp * 4 + (lane >> 3);
      const int m = m_of(k);
      const bool live = k < columns && m < a.M;
      if (k0 > 0) {
        pos = live ? a.positions[m] : -1;
        turn = lane_turn(a.rope, sub, (uint32_t)max(pos, 0));
      }
      float x[16];
      const float4* src = reinterpret_cast<const float4*>(mine + (live ? k : 0) * kBM);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 f = src[((i < 2 ? at.x : at.y) >> 2) + (i & 1)];
        x[4 * i] = f.x;
        x[4 * i + 1] = f.y;
        x[4 * i + 2] = f.z;
        x[4 * i + 3] = f.w;
      }
      if (a.norm != nullptr) norm_head(x, w, a.eps);
      turn_head<LAYOUT>(x, turn, sub < a.rope.n);
      uint4 lo, hi;
      pack16(x, lo, hi);
      if (live && pos >= 0) {
        __nv_bfloat16* dst = a.Q + (int64_t)m * a.N + tile * kBM;
        *reinterpret_cast<uint4*>(dst + at.x) = lo;
        *reinterpret_cast<uint4*>(dst + at.y) = hi;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) tmem_dealloc(tmem, (uint32_t)a.tmem_cols);
}

bool make_map(CUtensorMap* map, const void* ptr, int rows, int cols, int box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)cols * 2};
  const cuuint32_t box[2] = {(cuuint32_t)kBK, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, estr,
                      CU_TENSOR_MAP_SWIZZLE_128B) == CUDA_SUCCESS;
}

template <int LAYOUT>
int predict(const void* X, const void* W, void* Q, int M, int N, int K, const int32_t* positions, const scout_rope* rope,
            const void* norm, float eps, int32_t* dev_status, const scout_launch* launch, cudaStream_t stream) {
  if (X == nullptr || W == nullptr || Q == nullptr || M <= 0 || N <= 0 || K <= 0) return SCOUT_ERR_INVALID_ARG;
  if (launch != nullptr && launch->max_ctas < 0) return SCOUT_ERR_INVALID_ARG;
  if (M > kMaxN || N % kBM != 0 || K % kBK != 0 || !aligned16(X) || !aligned16(W) || !aligned16(Q))
    return SCOUT_ERR_UNSUPPORTED;
  GemmArgs a = {};
  a.Q = static_cast<__nv_bfloat16*>(Q);
  a.M = M;
  a.N = N;
  a.n_pad = (M + 15) / 16 * 16;
  a.tmem_cols = 32;
  while (a.tmem_cols < a.n_pad) a.tmem_cols <<= 1;
  a.kblocks = K / kBK;
  a.x_tile_bytes = (a.n_pad * 128 + 1023) / 1024 * 1024;
  a.status = dev_status;
  if constexpr (LAYOUT != kPlain) {
    a.positions = positions;
    a.norm = static_cast<const __nv_bfloat16*>(norm);
    a.rope = rope_of(rope);
    a.eps = eps;
    a.early = launch != nullptr && launch->pdl;
  }
  const int tiles = N / kBM;
  const int cap = launch != nullptr && launch->max_ctas > 0 ? launch->max_ctas : sm_count();
  const int S = max(1, min(min(8, a.kblocks), cap / tiles));  // split-K so tiles x S fits the CTA budget
  const int owned = (a.n_pad / 8 + S - 1) / S;                  // column groups per CTA in the reduction
  // ~180 to 220 KB in flight per SM, in stages of up to kMaxKps k-blocks (the fewer the stages, the fewer
  // barrier round trips per byte) but at least two, so that copies and MMAs overlap.  The rotated form keeps what the
  // cluster's CTAs exchange beside the ring, where it is small, so that a CTA sends without waiting for its peers' rings, and
  // takes three stages where they hold two k-blocks each.  Alone that is faster (GB300, 40 x 5120 x 5120:
  // 1.5 us, of which the stages 0.2), but not beside the other kernels of a decode step (57.0 us a step against 56.9,
  // 57.4 with the stages), which calls the plain form.
  const int exchange = S * owned * 8 * kBM * 4, tile_bytes = kWTileBytes + a.x_tile_bytes;
  const int room = kRingBytes - (LAYOUT != kPlain && S > 1 && exchange <= kApartBytes ? exchange : 0);
  a.kps = max(1, min(kMaxKps, room / 2 / tile_bytes));
  if (LAYOUT != kPlain && room / 3 / tile_bytes >= 2) a.kps = min(kMaxKps, room / 3 / tile_bytes);
  const int stage_bytes = a.kps * tile_bytes;
  a.stages = min(kStages, room / stage_bytes);
  const int ring = a.stages * stage_bytes;
  a.recv_at = room < kRingBytes ? ring : 0;
  const size_t smem = 1024 + (size_t)(a.recv_at > 0 ? ring + exchange : max(ring, exchange));
  CUtensorMap tmW, tmX;
  if (!make_map(&tmW, W, N, K, kBM) || !make_map(&tmX, X, M, K, a.n_pad)) return SCOUT_ERR_UNSUPPORTED;
  // the same limit for every call: calls on several host threads do not lower it for one another (the
  // exchange, at most (n_pad / 8 + S - 1) * 4 KB, is smaller than the ring's bound)
  static_assert((kMaxN / 8 + 7) * 8 * kBM * 4 <= kRingBytes, "the exchange fits where the ring does");
  if (cudaFuncSetAttribute(predict_q_kernel<LAYOUT>, cudaFuncAttributeMaxDynamicSharedMemorySize, 1024 + kRingBytes) !=
      cudaSuccess)
    return SCOUT_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)tiles, (unsigned)S, 1);
  cfg.blockDim = dim3(kThreadsQ, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[3];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = (unsigned)S;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = early_start_attrs(launch, attr, 1);
  if (LAYOUT != kPlain && !a.early) {  // scheduled, and set up, while the kernel before it ends
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  if (cudaLaunchKernelEx(&cfg, predict_q_kernel<LAYOUT>, tmW, tmX, a) != cudaSuccess) return SCOUT_ERR_CUDA;
  return launch_status();
}

}  // namespace
}  // namespace scout

extern "C" int scout_predict_q(const void* X, const void* W, void* Q, int M, int N, int K, int32_t* dev_status,
                               const scout_launch* launch, cudaStream_t stream) {
  return scout::predict<scout::kPlain>(X, W, Q, M, N, K, nullptr, nullptr, nullptr, 0.f, dev_status, launch, stream);
}

extern "C" int scout_predict_q_rotated(const void* X, const void* W, void* Q, int M, int N, int K,
                                       const int32_t* positions, const scout_rope* rope, const void* norm, float eps,
                                       int32_t* dev_status, const scout_launch* launch, cudaStream_t stream) {
  using namespace scout;
  if (positions == nullptr || !valid_rope(rope) || !valid_eps(eps)) return SCOUT_ERR_INVALID_ARG;
  if (!supported_rope(rope) || !aligned16(norm) || (reinterpret_cast<uintptr_t>(positions) & 3u))
    return SCOUT_ERR_UNSUPPORTED;
  auto* const call = rope->layout == SCOUT_ROPE_HALF ? predict<SCOUT_ROPE_HALF> : predict<SCOUT_ROPE_INTERLEAVED>;
  return call(X, W, Q, M, N, K, positions, rope, norm, eps, dev_status, launch, stream);
}
