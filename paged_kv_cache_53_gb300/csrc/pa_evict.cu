// Eviction from a paged cache by accumulated attention weight.
//
// Per (sequence, KV head), of n cached positions the k = min(n, keep) that rank highest stay,
// in their order: the first `sinks` and last `recent` positions before all others, then by
// mass (NaN lowest), the lower position among equals.  Their K and V rows move to positions
// 0 .. k-1, their mass with them.  Two launches:
//   1. select -- a CTA, or a cluster of up to eight, per (sequence, KV head) holds the row of
//                mass in registers (read once, so it may be compacted in place), finds the k-th
//                largest key by radix selection (11 + 11 + 10 bits; every CTA adds the bins it
//                has filled to each CTA's own copy of the pass's histogram, through distributed
//                shared memory), and writes the kept positions in order, their mass, and zeros
//                behind.  The scan order is warp, then 32 positions at a time, so ranks come from
//                ballots.  Protected positions are counted, not sorted.
//   2. move   -- CTAs take tiles of kept rows (32 KiB of K and V) by tickets: read a tile, say so,
//                wait until every lower tile of the (sequence, KV head) is read, store.  Kept
//                position i comes from s_i >= i with s increasing, so what a tile overwrites
//                (positions up to its last row) is read by this tile or a lower one.  Lower tiles
//                have lower tickets: the CTA that has one is running, and waits only for lower
//                ones still.  (A CTA per column slice of a head that walks all of its rows needs
//                no flags, and takes 34 us a call where tiles take 22 for 8 heads of 32,769 cut
//                to an eighth, 189 against 167 for 256 heads of 8,192 cut by half.)
// Bound: HBM (mass read once, kept rows read and written once; 64 sequences of up to 8,192 tokens
// cut by half 221 us, 0.84 of a copy's rate, the move alone 0.93); for few sequences the chain of
// dependent steps.
#include <algorithm>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_launch.h"

namespace pa {
namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMostKeys = 64;   // keys a thread can hold
constexpr int kMaxCluster = 8;  // portable cluster size
static_assert(kMaxEvictCtx == kSelThreads * kMostKeys * kMaxCluster, "row in registers");
constexpr int kBins = 2048;                  // of a pass; the third needs 1,024
constexpr int kOwnBins = 2 * kBins + 1024;  // of the three passes

// What the move kernel needs of one (sequence, KV head).
struct EvictRec {
  int k;     // kept positions, -1: leave the sequence as it is
  int same;  // leading kept positions that stay where they are
  int n;     // context length before
  int pad;
};

struct SelectParams {
  const float* mass;
  float* new_mass;
  long long stride;
  const int32_t* rows;
  int num_rows;
  const int32_t* context_lens;
  const int32_t* keep_lens;
  int32_t* kept;  // [seqs, H_kv, max_keep]
  EvictRec* recs;
  int* ticket;      // zeroed here for the move kernel, like
  uint32_t* done;   // [(sequence, KV head)][done_words] a bit per tile that has been read
  int32_t* status;
  int ctx_cap, max_keep, sinks, recent, num_kv_heads, done_words;
};

// Order-preserving map of a mass to an unsigned key: larger mass, larger key; NaN lowest.
__device__ __forceinline__ uint32_t mass_key(float m) {
  const uint32_t u = __float_as_uint(m + 0.f);  // (-0 counts as 0)
  if (m != m) return 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ uint32_t ld_dsmem(const void* local, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];"
               : "=r"(v)
               : "r"(mapa_shared(smem_addr(local), rank))
               : "memory");
  return v;
}

__device__ __forceinline__ void add_dsmem(const void* local, uint32_t rank, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(
                   mapa_shared(smem_addr(local), rank)),
               "r"(v)
               : "memory");
}

__device__ __forceinline__ uint32_t cluster_nctas() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
  return r;
}

// KPT: keys a thread holds.
template <int KPT>
__global__ void __launch_bounds__(kSelThreads, KPT == 4 ? 3 : KPT == 16 ? 2 : 1)
    evict_select_kernel(const SelectParams p) {
  // a histogram per pass, so that one barrier a pass suffices; in a cluster, `own` is filled
  // first and its bins then added to every CTA's s_hist
  __shared__ __align__(16) uint32_t s_hist[kOwnBins];
  extern __shared__ __align__(16) uint32_t s_own[];  // [kOwnBins] in a cluster
  __shared__ uint32_t s_warp[kSelWarps], s_weq[kSelWarps];
  __shared__ uint32_t s_digit, s_above, s_inbin, s_gt, s_eq, s_first;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t nc = cluster_nctas(), rank = cluster_ctarank();
  const int h = blockIdx.y, b = blockIdx.z;
  // the CTAs of the cluster, or the CTA alone, meet
  auto meet = [&] {
    if (nc > 1) cluster_sync();
    else __syncthreads();
  };
  for (int i = tid; i < kOwnBins / 4; i += kSelThreads) {
    reinterpret_cast<uint4*>(s_hist)[i] = make_uint4(0, 0, 0, 0);
    if (nc > 1) reinterpret_cast<uint4*>(s_own)[i] = make_uint4(0, 0, 0, 0);
  }
  griddep_wait();
  griddep_launch_dependents();

  int n = __ldg(p.context_lens + b), k = __ldg(p.keep_lens + b);
  const int row = p.rows != nullptr ? __ldg(p.rows + b) : b;
  bool bad = n < 0 || n > p.ctx_cap || k < 0;
  n = min(max(n, 0), p.ctx_cap);
  k = min(max(k, 0), n);
  if (k > p.max_keep) {
    bad = true;
    k = p.max_keep;
  }
  const bool skip = row < 0 || row >= p.num_rows;
  if ((bad || skip) && tid == 0 && rank == 0) flag_status(p.status, PA_STATUS_BAD_CONTEXT);
  const size_t bh = (size_t)b * p.num_kv_heads + h;
  if (rank == 0) {
    if (bh == 0 && tid == 0) *p.ticket = 0;
    for (int i = tid; i < p.done_words; i += kSelThreads) p.done[bh * p.done_words + i] = 0;
  }
  int32_t* kept = p.kept + bh * p.max_keep;
  // (every CTA of the cluster takes these branches alike)
  for (int i = (skip ? 0 : k) + rank * kSelThreads + tid; i < p.max_keep; i += nc * kSelThreads)
    kept[i] = -1;
  if (skip) {
    if (tid == 0 && rank == 0) p.recs[bh] = EvictRec{-1, 0, n, 0};
    return;
  }
  const float* mass = p.mass + ((size_t)row * p.num_kv_heads + h) * p.stride;
  float* out = p.new_mass + ((size_t)row * p.num_kv_heads + h) * p.stride;

  // warp gw of the cluster's owns positions [first, first + 32 its)
  const int gw = (int)rank * kSelWarps + warp;
  const int its = (n + (int)nc * kSelThreads - 1) / ((int)nc * kSelThreads);  // <= KPT
  const int first = gw * its * 32;
  float m[KPT];
#pragma unroll
  for (int i = 0; i < KPT; ++i) {
    const int pos = first + 32 * i + lane;
    m[i] = i < its && pos < n ? mass[pos] : 0.f;
  }
  auto is_protected = [&](int pos) { return pos < p.sinks || pos >= n - p.recent; };

  // radix selection among the positions that are not protected: the digits of the need-th
  // largest key from the top
  const int safe = (int)min((long long)n, (long long)min(p.sinks, n) + min(p.recent, n));
  uint32_t prefix = 0, mask = 0;  // digits found so far
  uint32_t need = (uint32_t)max(0, k - safe);  // keys still to take among those with the prefix
  bool whole = need == 0 || k == n;            // take all keys with the prefix
  if (nc > 1) cluster_sync();  // the histograms are zero
  else __syncthreads();
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    if (whole) break;  // (the whole cluster agrees)
    uint32_t* sums = s_hist + pass * kBins;
    uint32_t* hist = nc > 1 ? s_own + pass * kBins : sums;
    const bool has_bins = pass < 2 || 4 * tid < kOwnBins - 2 * kBins;
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t digits = pass == 2 ? 1023u : 2047u;
#pragma unroll
    for (int i = 0; i < KPT; ++i) {
      if (i >= its) break;
      const int pos = first + 32 * i + lane;
      const uint32_t key = mass_key(m[i]);
      if (pos < n && (key & mask) == prefix && !is_protected(pos))
        atomicAdd(hist + ((key >> shift) & digits), 1u);
    }
    if (nc > 1) {
      __syncthreads();
      const uint4 v = has_bins ? reinterpret_cast<const uint4*>(hist)[tid] : make_uint4(0, 0, 0, 0);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (w[j] != 0)
          for (uint32_t r = 0; r < nc; ++r) add_dsmem(sums + 4 * tid + j, r, w[j]);
    }
    meet();
    // four bins per thread
    const uint4 sum = has_bins ? reinterpret_cast<const uint4*>(sums)[tid] : make_uint4(0, 0, 0, 0);
    const uint32_t c[4] = {sum.x, sum.y, sum.z, sum.w};
    const uint32_t own = (c[0] + c[1]) + (c[2] + c[3]);
    uint32_t suf = own;  // of this thread's bins and those above, within the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_down_sync(~0u, suf, o);
      if (lane + o < 32) suf += v;
    }
    if (lane == 0) s_warp[warp] = suf;
    __syncthreads();
    const uint32_t others = lane > warp && lane < kSelWarps ? s_warp[lane] : 0u;
    uint32_t above = __reduce_add_sync(~0u, others) + suf - own;  // in bins above this thread's
#pragma unroll
    for (int j = 3; j >= 0; --j) {
      if (above < need && above + c[j] >= need) {
        s_digit = 4 * tid + j;
        s_above = above;
        s_inbin = c[j];
      }
      above += c[j];
    }
    __syncthreads();
    prefix |= s_digit << shift;
    mask |= digits << shift;
    need -= s_above;
    whole = s_inbin == need;
  }
  // kept: protected positions, keys above the prefix, and of those with it all (whole) or the first
  // `quota`; with k <= safe, the first k protected positions
  const bool few = k <= safe && k < n;
  const uint32_t quota = few ? (uint32_t)k : need;
  if (few) whole = false;
  auto is_above = [&](int i, int pos) {  // kept whatever its rank
    if (pos >= n || few) return false;
    const uint32_t key = mass_key(m[i]) & mask;
    return is_protected(pos) || (whole ? key >= prefix : key > prefix);
  };
  auto is_equal = [&](int i, int pos) {  // kept by rank
    if (pos >= n) return false;
    if (few) return is_protected(pos);
    return !is_protected(pos) && (mass_key(m[i]) & mask) == prefix;
  };

  uint32_t gt = 0, eq = 0;
#pragma unroll
  for (int i = 0; i < KPT; ++i) {
    if (i >= its) break;
    const int pos = first + 32 * i + lane;
    gt += __popc(__ballot_sync(~0u, is_above(i, pos)));
    if (!whole) eq += __popc(__ballot_sync(~0u, is_equal(i, pos)));
  }
  if (tid == 0) s_first = (uint32_t)n;
  __syncthreads();  // s_warp is spent
  if (lane == 0) {
    s_warp[warp] = gt;
    s_weq[warp] = eq;
  }
  __syncthreads();
  if (warp == 0) {
    const uint32_t a = __reduce_add_sync(~0u, lane < kSelWarps ? s_warp[lane] : 0u);
    const uint32_t e = __reduce_add_sync(~0u, lane < kSelWarps ? s_weq[lane] : 0u);
    if (lane == 0) {
      s_gt = a;
      s_eq = e;
    }
  }
  gt = __reduce_add_sync(~0u, lane < warp ? s_warp[lane] : 0u);
  eq = __reduce_add_sync(~0u, lane < warp ? s_weq[lane] : 0u);
  meet();  // every mass of the row is in registers, the counts are complete
  if (rank > 0) {
    gt += __reduce_add_sync(~0u, lane < (int)rank ? ld_dsmem(&s_gt, lane) : 0u);
    eq += __reduce_add_sync(~0u, lane < (int)rank ? ld_dsmem(&s_eq, lane) : 0u);
  }
  const unsigned below = (1u << lane) - 1;
  uint32_t hole = (uint32_t)n;  // the first position not kept
#pragma unroll
  for (int i = 0; i < KPT; ++i) {
    if (i >= its) break;
    const int pos = first + 32 * i + lane;
    bool keep = is_above(i, pos);
    const unsigned ba = __ballot_sync(~0u, keep);
    uint32_t at = gt + __popc(ba & below);
    gt += __popc(ba);
    if (!whole) {
      const bool e = is_equal(i, pos);
      const unsigned be = __ballot_sync(~0u, e);
      const uint32_t q = eq + __popc(be & below);
      eq += __popc(be);
      keep = keep || (e && q < quota);
      at += min(q, quota);
    }
    if (keep) {
      kept[at] = pos;
      out[at] = m[i];
    } else if (pos < n) {
      hole = min(hole, (uint32_t)pos);
    }
  }
  for (int i = k + (int)rank * kSelThreads + tid; i < n; i += (int)nc * kSelThreads) out[i] = 0.f;
  hole = __reduce_min_sync(~0u, hole);
  if (lane == 0) atomicMin(&s_first, hole);
  meet();
  if (rank == 0 && warp == 0) {
    uint32_t f = s_first;
    if (nc > 1)
      f = __reduce_min_sync(~0u, lane < (int)nc ? ld_dsmem(&s_first, lane) : (uint32_t)n);
    if (lane == 0) p.recs[bh] = EvictRec{k, min((int)f, k), n, 0};
  }
  if (nc > 1) cluster_sync();  // no CTA leaves while another reads its shared memory
}

struct MoveParams {
  uint4* k_cache;
  uint4* v_cache;
  const int32_t* block_tables;
  const int32_t* new_block_tables;
  const int32_t* kept;
  const EvictRec* recs;
  int* ticket;
  uint32_t* done;
  int32_t* new_context_lens;
  int32_t* status;
  int max_blocks, new_max_blocks, max_keep, num_kv_heads, block_log2, num_blocks, in_place;
  int num_seqs;
  int heads;       // (sequence, KV head) pairs
  int tiles;       // of the longest list
  int done_words;
};

constexpr int kMoveThreads = 256;
constexpr int kMoveCtasPerSm = 5;  // 221 us where four take 229 (64 sequences cut by half)
constexpr int kMoveVecs = 8;  // 16-byte vectors a thread moves per tile: half K, half V
constexpr int tile_rows(int row_vecs) { return kMoveThreads * kMoveVecs / 2 / row_vecs; }

// VECS: 16-byte vectors of a row.
template <int VECS>
__global__ void __launch_bounds__(kMoveThreads, kMoveCtasPerSm)
    evict_move_kernel(const MoveParams p) {
  constexpr int kRows = tile_rows(VECS), kHalf = kMoveVecs / 2, kStep = kMoveThreads / VECS;
  __shared__ int s_src[kRows], s_dst[kRows];  // cache rows, -1: nothing to move
  __shared__ int s_ticket, s_k, s_start, s_go;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bs_mask = (1 << p.block_log2) - 1;
  const int r0 = tid / VECS, c = tid % VECS;
  griddep_wait();
  griddep_launch_dependents();
  for (int i = blockIdx.x * kMoveThreads + tid; i < p.num_seqs; i += gridDim.x * kMoveThreads) {
    const EvictRec rec = p.recs[(size_t)i * p.num_kv_heads];
    p.new_context_lens[i] = rec.k < 0 ? rec.n : rec.k;
  }
  // tickets run over the first tile of every head, then the second of every head, ..
  const long long tickets = (long long)p.heads * p.tiles;
  for (;;) {
    __syncthreads();  // the last tile's s_src and s_dst are spent
    if (tid == 0) {
      const int i = atomicAdd(p.ticket, 1);
      s_ticket = i;
      if (i < tickets) {
        const EvictRec rec = p.recs[i % p.heads];
        // rows that stay where they are need no move unless the table changes their block
        s_start = (p.in_place ? rec.same : 0) + i / p.heads * kRows;
        s_k = rec.k;
      }
    }
    __syncthreads();
    if (s_ticket >= tickets) return;
    const int bh = s_ticket % p.heads, tile = s_ticket / p.heads;
    const int b = bh / p.num_kv_heads, h = bh - b * p.num_kv_heads;
    const int k = s_k, t = s_start;
    if (t >= k) continue;
    if (tid < kRows) {
      const int i = t + tid;
      int src = -1, dst = -1;
      if (i < k) {
        const int s = __ldcg(p.kept + (size_t)bh * p.max_keep + i);
        const int sb = s >> p.block_log2, db = i >> p.block_log2;
        const int src_id = __ldg(p.block_tables + (size_t)b * p.max_blocks + sb);
        const int dst_id =
            db < p.new_max_blocks ? __ldg(p.new_block_tables + (size_t)b * p.new_max_blocks + db)
                                  : -1;
        if (src_id < 0 || src_id >= p.num_blocks || dst_id < 0 || dst_id >= p.num_blocks) {
          flag_status(p.status, PA_STATUS_BAD_BLOCK);
        } else {  // (num_blocks * H_kv * block_size fits 31 bits)
          src = ((src_id * p.num_kv_heads + h) << p.block_log2) + (s & bs_mask);
          dst = ((dst_id * p.num_kv_heads + h) << p.block_log2) + (i & bs_mask);
          if (src == dst) dst = -1;
        }
      }
      s_src[tid] = src;
      s_dst[tid] = dst;
    }
    __syncthreads();
    uint4 v[kMoveVecs];
#pragma unroll
    for (int u = 0; u < kHalf; ++u) {
      const int j = u * kStep + r0;
      if (s_dst[j] >= 0) {
        const size_t at = (size_t)s_src[j] * VECS + c;
        v[u] = p.k_cache[at];
        v[kHalf + u] = p.v_cache[at];
      }
    }
    __syncthreads();
    if (warp == 0) {
      uint32_t* done = p.done + (size_t)bh * p.done_words;
      if (lane == 0) {
        // the barrier orders every thread's loads before this fence, and the fence before the bit:
        // no store that follows the bit's reading can reach them
        __threadfence();
        atomicOr(done + (tile >> 5), 1u << (tile & 31));
      }
      // every lower tile too
      const uint64_t t0 = global_timer_ns();
      bool ok = true;
      for (int w0 = 0; w0 <= tile >> 5 && ok; w0 += 32) {
        const int w = w0 + lane;
        const uint32_t want = w < tile >> 5 ? ~0u : w == tile >> 5 ? (1u << (tile & 31)) - 1 : 0u;
        for (;;) {
          uint32_t got = 0;
          if (want != 0) got = (uint32_t)ld_acquire_gpu(reinterpret_cast<const int*>(done + w));
          if (__all_sync(~0u, (got & want) == want)) break;
          if (__any_sync(~0u, global_timer_ns() - t0 > kWaitTimeoutNs)) {
            ok = false;
            break;
          }
        }
      }
      if (lane == 0) {
        if (!ok) flag_status(p.status, PA_STATUS_TIMEOUT);
        s_go = ok;
      }
    }
    __syncthreads();
    if (!s_go) return;
#pragma unroll
    for (int u = 0; u < kHalf; ++u) {
      const int d = s_dst[u * kStep + r0];
      if (d >= 0) {
        const size_t at = (size_t)d * VECS + c;
        p.k_cache[at] = v[u];
        p.v_cache[at] = v[kHalf + u];
      }
    }
  }
}

using MoveKernel = void (*)(MoveParams);
MoveKernel move_kernel_for(int row_vecs) {
  return row_vecs == 8    ? evict_move_kernel<8>
         : row_vecs == 16 ? evict_move_kernel<16>
                          : evict_move_kernel<32>;
}

struct Layout {
  size_t ticket, recs, done, total;
};
// The workspace for any element type: tiles of the widest rows (512 bytes) are the most.
Layout layout(int num_seqs, int num_kv_heads, int max_keep) {
  const size_t heads = (size_t)num_seqs * num_kv_heads;
  const size_t words = ((size_t)max_keep / tile_rows(32) + 32) / 32;
  Layout l;
  l.ticket = 0;
  l.recs = 256;
  l.done = align_up(l.recs + sizeof(EvictRec) * heads, 256);
  l.total = align_up(l.done + sizeof(uint32_t) * heads * words, 256);
  return l;
}

}  // namespace

size_t evict_workspace_bytes(int num_seqs, int num_kv_heads, int, int max_keep) {
  return layout(num_seqs, num_kv_heads, max_keep).total;
}

bool evict_fits(int num_seqs, int num_kv_heads, int max_keep) {
  // (tickets of the smallest tiles, and one more per CTA, fit 31 bits)
  const long long tiles = max_keep / tile_rows(32) + 1;
  return num_seqs <= 65535 && num_kv_heads <= 65535 &&
         (long long)num_seqs * num_kv_heads * tiles <= 0x40000000ll;
}

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
  const Layout l = layout(a.num_seqs, a.num_kv_heads, a.max_keep);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  const int sms = std::max(1, sm_count());
  const int row_vecs = (int)(a.head_dim * a.elem_bytes / 16);
  const int tiles = (a.max_keep + tile_rows(row_vecs) - 1) / tile_rows(row_vecs);
  const long long heads = (long long)a.num_kv_heads * a.num_seqs;

  SelectParams s;
  s.mass = a.mass;
  s.new_mass = a.new_mass;
  s.stride = a.mass_stride;
  s.rows = a.mass_rows;
  s.num_rows = a.num_mass_rows;
  s.context_lens = a.context_lens;
  s.keep_lens = a.keep_lens;
  s.kept = a.kept;
  s.recs = reinterpret_cast<EvictRec*>(ws + l.recs);
  s.ticket = reinterpret_cast<int*>(ws + l.ticket);
  s.done = reinterpret_cast<uint32_t*>(ws + l.done);
  s.status = a.status;
  s.ctx_cap = a.ctx_cap;
  s.max_keep = a.max_keep;
  s.sinks = a.sinks;
  s.recent = a.recent;
  s.num_kv_heads = a.num_kv_heads;
  s.done_words = (tiles + 31) / 32;
  // a cluster as large as the SMs allow, since its steps are short and dependent, but not
  // beyond four keys a thread; larger where the row needs it
  auto holds = [&](int cluster, int keys) {
    return (long long)cluster * kSelThreads * keys >= a.ctx_cap;
  };
  int cluster = 1;
  while (cluster < kMaxCluster && !holds(cluster, 4) && 2 * cluster * heads <= 2ll * sms)
    cluster *= 2;
  while (cluster < kMaxCluster && !holds(cluster, kMostKeys)) cluster *= 2;
  auto select = holds(cluster, 4)    ? evict_select_kernel<4>
                : holds(cluster, 16) ? evict_select_kernel<16>
                                     : evict_select_kernel<kMostKeys>;
  const size_t own = cluster > 1 ? kOwnBins * sizeof(uint32_t) : 0;
  cudaError_t e = launch_pdl_cluster(select,
                                     dim3((unsigned)cluster, (unsigned)a.num_kv_heads,
                                          (unsigned)a.num_seqs),
                                     dim3(kSelThreads), own, stream, cluster, s);
  if (e != cudaSuccess) return e;
  MoveParams m;
  m.k_cache = static_cast<uint4*>(a.k_cache);
  m.v_cache = static_cast<uint4*>(a.v_cache);
  m.block_tables = a.block_tables;
  m.new_block_tables = a.new_block_tables;
  m.kept = a.kept;
  m.recs = s.recs;
  m.ticket = s.ticket;
  m.done = s.done;
  m.new_context_lens = a.new_context_lens;
  m.status = a.status;
  m.max_blocks = a.max_blocks;
  m.new_max_blocks = a.new_max_blocks;
  m.max_keep = a.max_keep;
  m.num_kv_heads = a.num_kv_heads;
  m.block_log2 = a.block_size == 16 ? 4 : 5;
  m.num_blocks = a.num_blocks;
  m.in_place = a.new_block_tables == a.block_tables && a.new_max_blocks == a.max_blocks;
  m.num_seqs = a.num_seqs;
  m.heads = (int)heads;
  m.tiles = tiles;
  m.done_words = s.done_words;
  const long long tickets = heads * tiles;
  const long long wave = (long long)kMoveCtasPerSm * sms;  // all resident
  return launch_pdl(move_kernel_for(row_vecs),
                    dim3((unsigned)std::max<long long>(1, std::min(tickets, wave))),
                    dim3(kMoveThreads), 0, stream, m);
}

}  // namespace pa
