// scout_build_tables: page table, residency bits, slot map and touched-block list of a batch from
// its request lengths; scout_append_kv: new bf16 K/V rows into a paged pool by that slot map.
// The pages leave the paging open (ScoutAttention (arXiv HTML), section 3.2 takes the KV blocks
// as given); the tables here are the ones the library's other entry points read.
//
// Tables: every CTA makes the same three prefixes over the batch (new tokens, touched blocks, new
// blocks) in shared memory, and after that no item depends on another: a warp takes a word of 32
// blocks of a unit (one coalesced row piece, one ballot for the residency word), a touched block
// of a sequence (its tokens x heads are one contiguous piece of the slot map, stored as pairs of
// heads where their number is a power of two), or 32 list entries.  One launch, no atomics.  GB300, device
// time: 13.7 us for 40 prompts (3.3 TB/s into L2), bound by the issue of this index arithmetic, some 120
// instructions for each 512 bytes of map; 5.5 us for a decode step of 40 sequences, the launch and
// three sections in turn of two dependent reads each (a length, then a free slot or a table entry).
//
// Append: bound by DRAM.  8 prompts of up to 16K tokens, 8 KV heads: 89.1 us for 575 MB (6.5 TB/s, 0.95
// of the measured copy bandwidth); 2.6 us for a decode step of 8 sequences.
#include "fp8.cuh"

namespace scout {
namespace {

constexpr int kTabWarps = 8;
constexpr int kTabPartials = 3 * 32;  // ints of static shared memory, for the prefixes

struct TabArgs {
  const int32_t* prev_len;
  const int32_t* seq_len;
  const int32_t* free_slots;
  int n_free;
  int64_t n_slots;
  int B, Hkv, P, nblk_cap, words;
  int32_t* page_table;
  uint32_t* bits;
  int32_t* cu_tokens;
  int64_t* slot_map;
  int max_tokens;
  int32_t* block_list;
  int max_list;
  int32_t* counts;
  int32_t* status;
};

// Items of a warp whose free slots are in flight together, and CTAs an SM.  GB300, the tables of 40
// prompts of up to 32K tokens, 8 KV heads (45 MB written): 13.8 us with two and four; 14.2 with four
// items, 15.6 with eight (more instructions than they hide), 15.3 with three CTAs, 16.0 with eight.
constexpr int kBatch = 2;
constexpr int kTabPerSm = 4;

// Slot of the i-th new block of the batch (kNoSlot past the free list), unchecked: the read is in
// flight when this returns.
constexpr int kNoSlot = -2;
__device__ __forceinline__ int take_slot(const TabArgs& a, int i) {
  if (i >= a.n_free) return kNoSlot;
  return a.free_slots != nullptr ? max(a.free_slots[i], -1) : i;
}
// The slot of a lane that has one, -1 (reported) where it is none of the pool's.
__device__ __forceinline__ int checked(const TabArgs& a, bool has, int s) {
  if (!has) return -1;
  if (s >= 0 && s < a.n_slots) return s;
  report(a.status, s == kNoSlot ? SCOUT_DEV_OVERFLOW : SCOUT_DEV_BAD_INDEX);
  return -1;
}

__global__ void __launch_bounds__(kTabWarps * 32) tables_kernel(const TabArgs a) {
  extern __shared__ int sm[];
  __shared__ int partial[kTabPartials];
  const int B = a.B, P = a.P;
  int* tok = sm;              // [B + 1] new tokens before sequence b
  int* tou = sm + (B + 1);    // [B + 1] touched blocks (of one KV head)
  int* neu = tou + (B + 1);   // [B + 1] new blocks (of one KV head)
  int* prv = neu + (B + 1);   // [B] clamped previous lengths
  int* seq = prv + B;         // [B] clamped lengths
  const int tid = threadIdx.x, lane = tid & 31;
  const int cap_tokens = a.nblk_cap * P;
  const int lg = P == 16 ? 4 : P == 32 ? 5 : 6;  // P = 2^lg
  int* const out[3] = {tok, tou, neu};
  cta_prefixes<3>(B, out, partial, [&](int b, int (&x)[3]) {
    const SeqSpan s = seq_span(a.prev_len, a.seq_len, b, cap_tokens);
    prv[b] = s.prev;
    seq[b] = s.seq;
    const int nb = (s.seq + P - 1) >> lg;
    x[0] = s.seq - s.prev;
    x[1] = s.seq > s.prev ? nb - (s.prev >> lg) : 0;
    x[2] = nb - ((s.prev + P - 1) >> lg);
  });
  if (blockIdx.x == 0)
    for (int b = tid; b < B; b += blockDim.x) report_span(a.status, a.prev_len, a.seq_len, b, cap_tokens);
  const int n_tok = tok[B], n_tou = tou[B];
  const int64_t n_list = (int64_t)n_tou * a.Hkv;
  if (blockIdx.x == 0) {
    if (a.cu_tokens != nullptr)
      for (int b = tid; b <= B; b += blockDim.x) a.cu_tokens[b] = tok[b];
    if (tid == 0) {
      if (a.counts != nullptr) {
        a.counts[0] = n_tok;
        a.counts[1] = (int32_t)n_list;
        a.counts[2] = neu[B] * a.Hkv;
      }
      if ((a.slot_map != nullptr && n_tok > a.max_tokens) || (a.block_list != nullptr && n_list > a.max_list))
        report(a.status, SCOUT_DEV_OVERFLOW);
    }
  }
  const int64_t w0 = (int64_t)blockIdx.x * kTabWarps + (tid >> 5), wn = (int64_t)gridDim.x * kTabWarps;

  // rows of the page table, a word of 32 blocks at a time; a grown row gets its new blocks only.
  // kBatch items of a warp together: their free slots are all in flight before the first is stored.
  const int64_t n_words = (int64_t)B * a.Hkv * a.words;
  for (int64_t it0 = w0; it0 < n_words; it0 += kBatch * wn) {
    int slot[kBatch];
    bool fresh[kBatch], mine[kBatch];  // a new block; a word with one (or any word, made anew)
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      const int64_t it = it0 + y * wn;
      fresh[y] = mine[y] = false;
      slot[y] = -1;
      if (it >= n_words) continue;
      const int u = (int)((unsigned)it / (unsigned)a.words), w = (int)it - u * a.words;
      const int b = u / a.Hkv, h = u - b * a.Hkv;
      const int j0 = (prv[b] + P - 1) >> lg, j1 = (seq[b] + P - 1) >> lg;  // new blocks
      mine[y] = a.prev_len == nullptr || (w * 32 + 32 > j0 && w * 32 < j1);
      const int j = w * 32 + lane;
      fresh[y] = j >= j0 && j < j1;
      if (fresh[y]) slot[y] = take_slot(a, neu[b] * a.Hkv + h * (j1 - j0) + (j - j0));
    }
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      const int64_t it = it0 + y * wn;
      const int u = (int)((unsigned)it / (unsigned)a.words), j = ((int)it - u * a.words) * 32 + lane;
      slot[y] = checked(a, fresh[y], slot[y]);
      const uint32_t m = __ballot_sync(0xffffffffu, slot[y] >= 0), made = __ballot_sync(0xffffffffu, fresh[y]);
      if (!mine[y]) continue;
      if (j < a.nblk_cap && (fresh[y] || a.prev_len == nullptr)) a.page_table[(int64_t)u * a.nblk_cap + j] = slot[y];
      if (lane == 0) {
        a.bits[it] = a.prev_len == nullptr ? m : (a.bits[it] & ~made) | m;  // a word is one warp's alone
      }
    }
  }

  // slot map: the tokens of one touched block of a sequence, all heads: one contiguous piece, 32
  // entries at a time; (r, hh) = (token, head) of a lane's entry, stepped without a division
  if (a.slot_map != nullptr) {
    const bool aligned = (reinterpret_cast<uintptr_t>(a.slot_map) & 15u) == 0;
    for (int h0 = 0; h0 < a.Hkv; h0 += 32) {
      const int hn = min(32, a.Hkv - h0), dr = 32 / hn, dh = 32 - dr * hn;
      const int r_first = lane / hn, h_first = lane - r_first * hn;
      const bool pairs = hn == a.Hkv && hn >= 2 && (hn & (hn - 1)) == 0 && aligned;
      for (int64_t it0 = w0; it0 < n_tou; it0 += kBatch * wn) {
        int slot[kBatch], off[kBatch], i0[kBatch], rows[kBatch];
#pragma unroll
        for (int y = 0; y < kBatch; ++y) {
          const int64_t it = it0 + y * wn;
          rows[y] = 0;
          if (it >= n_tou) continue;
          const int b = owner_of(tou, B, (int)it);
          const int p = prv[b], j = (p >> lg) + ((int)it - tou[b]);
          const int t0 = max(j << lg, p), t1 = min((j + 1) << lg, seq[b]);
          const int j0 = (p + P - 1) >> lg, nb = ((seq[b] + P - 1) >> lg) - j0;
          i0[y] = tok[b] + t0 - p;  // first of its tokens
          rows[y] = min(t1 - t0, a.max_tokens - i0[y]);
          off[y] = t0 - (j << lg);
          const int h = h0 + lane;
          if (lane < hn)  // a new block's slot, or that of the partly filled last block
            slot[y] = j >= j0 ? take_slot(a, neu[b] * a.Hkv + h * nb + (j - j0))
                              : max(a.page_table[((int64_t)b * a.Hkv + h) * a.nblk_cap + j], -1);
        }
#pragma unroll
        for (int y = 0; y < kBatch; ++y) {
          if (rows[y] <= 0) continue;
          const int s = checked(a, lane < hn, slot[y]);
          const int64_t first = s < 0 ? -1 : ((int64_t)s << lg) + off[y];  // pool row of its first token
          int64_t* dst = a.slot_map + (int64_t)i0[y] * a.Hkv + h0;
          if (pairs) {  // 32 entry pairs at a time, always the same two heads a lane
            const int64_t f0 = __shfl_sync(0xffffffffu, first, (2 * lane) & (hn - 1));
            const int64_t f1 = __shfl_sync(0xffffffffu, first, (2 * lane + 1) & (hn - 1));
            longlong2* d2 = reinterpret_cast<longlong2*>(dst) + lane;
            const int dr2 = 64 / hn;
#pragma unroll 4
            for (int r = 2 * lane / hn; r < rows[y]; r += dr2, d2 += 32)
              *d2 = make_longlong2(f0 < 0 ? -1 : f0 + r, f1 < 0 ? -1 : f1 + r);
            continue;
          }
          int r = r_first, hh = h_first;
          for (int e = 0; e < rows[y] * hn; e += 32) {
            const int64_t f = __shfl_sync(0xffffffffu, first, hh);
            if (r < rows[y]) dst[(int64_t)r * a.Hkv + hh] = f < 0 ? -1 : f + r;
            r += dr;
            hh += dh;
            if (hh >= hn) {
              hh -= hn;
              ++r;
            }
          }
        }
      }
    }
    // rows past the last new token hold -1: a padded batch's rows are skipped
    const int64_t from = (int64_t)min(n_tok, a.max_tokens) * a.Hkv, to = (int64_t)a.max_tokens * a.Hkv;
    for (int64_t e = from + w0 * 32 + lane; e < to; e += wn * 32) a.slot_map[e] = -1;
  }

  // touched blocks in (sequence, head, block) order, -1 past the last
  if (a.block_list != nullptr) {
    for (int64_t i = w0 * 32 + lane; i < a.max_list; i += wn * 32) {
      int u = -1, j = -1;
      if (i < n_list) {
        const int b = owner_of(tou, B, (int)((unsigned)i / (unsigned)a.Hkv));
        const int nt = tou[b + 1] - tou[b], r = (int)(i - (int64_t)tou[b] * a.Hkv);
        const int h = r / nt;
        u = b * a.Hkv + h;
        j = (prv[b] >> lg) + (r - h * nt);
      }
      reinterpret_cast<int2*>(a.block_list)[i] = make_int2(u, j);
    }
  }
}

// Sixteen lanes move one (token, KV head) row of K and of V, 16 bytes a lane; four rows of each a
// lane are in flight together.
constexpr int kAppThreads = 256, kAppRows = 4;

__global__ void __launch_bounds__(kAppThreads) append_kernel(const __nv_bfloat16* __restrict__ K,
                                                             const __nv_bfloat16* __restrict__ V, int64_t ld_k,
                                                             int64_t ld_v, const int64_t* __restrict__ slot_map,
                                                             int64_t n_items, int Hkv, __nv_bfloat16* K_pool,
                                                             __nv_bfloat16* V_pool, int64_t pool_rows, int32_t* status) {
  const int chunk = threadIdx.x & 15;
  constexpr int kGroups = kAppThreads / 16;
  const int64_t first = (int64_t)blockIdx.x * kGroups * kAppRows + (threadIdx.x >> 4);
  int64_t row[kAppRows];
  uint4 k[kAppRows], v[kAppRows];
#pragma unroll
  for (int r = 0; r < kAppRows; ++r) {
    const int64_t it = first + r * kGroups;
    row[r] = it < n_items ? slot_map[it] : -1;
  }
#pragma unroll
  for (int r = 0; r < kAppRows; ++r) {
    if (row[r] >= pool_rows) {
      if (chunk == 0) report(status, SCOUT_DEV_BAD_INDEX);
      row[r] = -1;
    }
    if (row[r] < 0) continue;
    const int64_t it = first + r * kGroups, i = it / Hkv;
    const int h = (int)(it - i * Hkv);
    k[r] = ldg_stream(K + i * ld_k + h * kD + chunk * 8);
    v[r] = ldg_stream(V + i * ld_v + h * kD + chunk * 8);
  }
#pragma unroll
  for (int r = 0; r < kAppRows; ++r) {
    if (row[r] < 0) continue;
    *reinterpret_cast<uint4*>(K_pool + row[r] * kD + chunk * 8) = k[r];
    *reinterpret_cast<uint4*>(V_pool + row[r] * kD + chunk * 8) = v[r];
  }
}

}  // namespace
}  // namespace scout

extern "C" int scout_build_tables(const int32_t* prev_len, const int32_t* seq_len, const int32_t* free_slots,
                                  int n_free, int64_t n_slots, int B, int Hkv, int P, int nblk_cap,
                                  int32_t* page_table, uint32_t* resident_bits, int32_t* cu_tokens, int64_t* slot_map,
                                  int max_tokens, int32_t* block_list, int max_list, int32_t* counts,
                                  int32_t* dev_status, cudaStream_t stream) {
  using namespace scout;
  if (seq_len == nullptr || page_table == nullptr || resident_bits == nullptr) return SCOUT_ERR_INVALID_ARG;
  if (B <= 0 || Hkv <= 0 || nblk_cap <= 0 || n_slots <= 0 || n_free < 0 || max_tokens < 0 || max_list < 0)
    return SCOUT_ERR_INVALID_ARG;
  if (!valid_P(P) || B > kMaxBatch || nblk_cap > kMaxNblk || n_slots > 0x7fffffffLL ||
      (int64_t)B * nblk_cap * P > 0x7fffffffLL || (int64_t)B * Hkv * nblk_cap > 0x7fffffffLL ||
      (reinterpret_cast<uintptr_t>(block_list) & 7u) || (reinterpret_cast<uintptr_t>(slot_map) & 7u))
    return SCOUT_ERR_UNSUPPORTED;
  TabArgs a;
  a.prev_len = prev_len;
  a.seq_len = seq_len;
  a.free_slots = free_slots;
  a.n_free = n_free;
  a.n_slots = n_slots;
  a.B = B;
  a.Hkv = Hkv;
  a.P = P;
  a.nblk_cap = nblk_cap;
  a.words = (nblk_cap + 31) / 32;
  a.page_table = page_table;
  a.bits = resident_bits;
  a.cu_tokens = cu_tokens;
  a.slot_map = slot_map;
  a.max_tokens = max_tokens;
  a.block_list = block_list;
  a.max_list = max_list;
  a.counts = counts;
  a.status = dev_status;
  const int64_t warps = (int64_t)B * Hkv * a.words + max_tokens / P + B + max_list / 32 + 1;
  const int64_t want = (warps + kTabWarps - 1) / kTabWarps;
  const int grid = (int)(want < sm_count() * kTabPerSm ? want : sm_count() * kTabPerSm);
  const size_t smem = (size_t)(5 * B + 3) * sizeof(int);
  // More than 48 KB, the static part included, has to be asked for.  (The same limit for every call: calls
  // on several host threads do not lower it for one another.)
  if (smem + kTabPartials * sizeof(int) > 48 * 1024 &&
      cudaFuncSetAttribute(tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (5 * kMaxBatch + 3) * (int)sizeof(int)) != cudaSuccess)
    return SCOUT_ERR_CUDA;
  tables_kernel<<<grid, kTabWarps * 32, smem, stream>>>(a);
  return launch_status();
}

extern "C" int scout_append_kv(const void* K_new, int64_t ld_k, const void* V_new, int64_t ld_v,
                               const int64_t* slot_map, int n_tokens, int Hkv, int D, int P, void* K_pool,
                               void* V_pool, int64_t n_slots, int32_t* dev_status, cudaStream_t stream) {
  using namespace scout;
  if (K_new == nullptr || V_new == nullptr || slot_map == nullptr || K_pool == nullptr || V_pool == nullptr)
    return SCOUT_ERR_INVALID_ARG;
  if (n_tokens < 0 || Hkv <= 0 || n_slots <= 0 || ld_k < (int64_t)Hkv * D || ld_v < (int64_t)Hkv * D)
    return SCOUT_ERR_INVALID_ARG;
  if (D != kD || !valid_P(P) || !aligned16(K_new) || !aligned16(V_new) || !aligned16(K_pool) || !aligned16(V_pool) ||
      ld_k % 8 != 0 || ld_v % 8 != 0 || (reinterpret_cast<uintptr_t>(slot_map) & 7u) || n_slots > 0x7fffffffLL)
    return SCOUT_ERR_UNSUPPORTED;
  const int64_t items = (int64_t)n_tokens * Hkv;
  if (items == 0) return SCOUT_OK;
  constexpr int kPerCta = kAppThreads / 16 * kAppRows;
  const int64_t grid = (items + kPerCta - 1) / kPerCta;
  if (grid > 0x7fffffffLL) return SCOUT_ERR_UNSUPPORTED;
  append_kernel<<<(unsigned)grid, kAppThreads, 0, stream>>>(
      static_cast<const __nv_bfloat16*>(K_new), static_cast<const __nv_bfloat16*>(V_new), ld_k, ld_v, slot_map, items,
      Hkv, static_cast<__nv_bfloat16*>(K_pool), static_cast<__nv_bfloat16*>(V_pool), n_slots * P, dev_status);
  return launch_status();
}
