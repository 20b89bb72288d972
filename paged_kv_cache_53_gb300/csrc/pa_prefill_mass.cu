// Attention weights that a prefill chunk's queries give each cached position, summed over the
// queries and the query heads of a KV head, on sm_103a tensor cores (tcgen05).
//
// With lse_t = log2 sum_j 2^(c q_t . k_j), c = scale * log2(e), which the chunked-prefill
// kernel leaves for every query row t, the weight of position j is
//     w_j = sum_t 2^(c k_j . q_t - lse_t)        over the rows t that see j.
// The product is taken transposed, S^T = K Q^T, keys as rows: a key's whole sum then belongs
// to one thread (its TMEM lane), which adds it up in registers and updates its position of
// the mass once.  No reduction across threads, no atomics, a fixed order of addition.
//
// A cluster of two CTAs on two SMs shares every product (tcgen05 cta_group::2, M = 256 keys):
// each CTA holds 128 of a tile's keys and 64 of a query tile's 128 rows, so that a product's
// operands take 96 bytes a clock of each SM's shared memory (128, all of it, with one CTA per
// product; the keys in tensor memory instead took 85 clocks of the tensor core where 64 do) and
// a query row is read from L2 by one of the two SMs.  An item is KT tiles of 256 keys of one
// (sequence, KV head); pair c takes items c, c + pairs, .. of the list whose per-sequence starts
// the plan kernel left.  Warp roles in each CTA:
//   warp 0     TMA: its half of the query tiles (128 / G tokens of a KV head's group) into a ring
//   warp 1     MMA issuer (first CTA only): for each query tile, a product per key tile, into
//              four S buffers, two for each key tile in turn
//   warp 2     -lse / c of its rows of each query tile, as four bf16 terms (32 bits), into a
//              16-column operand beside the tile: against a column operand of ones, one more
//              k-step makes S the exponent itself, c (k . q - lse / c), and no warp has to fetch
//              the 128 values for its columns (which cost more than the 2^x)
//   warp 3     items, and TMA of their keys, an item ahead
//   warps 4-11 a warpgroup per key tile: S into registers (which frees its buffer), a packed
//              product and two 2^x per pair of columns, added up
// Bound: one 2^x per (key, query row), 32 a clock and SM, which for a 128 x 128 tile are the 512
// clocks its product takes the tensor core; the two overlap (8 chunks of 512 over contexts of up to
// 16,896 tokens, 32 heads: 108 us where either alone would take 60; the rest is the hand-over of
// the S buffers between two SMs).  Queries before the first that sees
// the item's first key, and those not observed, are never loaded, and no product is taken of
// tiles wholly above the diagonal.
#include <algorithm>
#include <cmath>
#include <mutex>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_launch.h"
#include "pa_tcgen05.cuh"

namespace pa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

struct PrefillMassParams {
  const float* lse;        // [H_kv, num_tokens, group], log2 units
  const int* tile_starts;  // [num_seqs + 1] first item (of a head) of each sequence
  const int32_t* block_tables;
  const int32_t* cu_q_lens;
  const int32_t* context_lens;
  const int32_t* observe;  // null: every query of a chunk
  int32_t* status;
  MassTarget mass;
  int max_blocks, num_seqs, num_tokens, num_kv_heads, group, group_log2, block_log2, num_blocks;
  float scale_log2;  // c; 1 with no_scores
  float inv_scale;   // 1 / c
  int no_scores;     // c is 0 or next to it: the exponent is -lse alone
};

// One item as warp 3 hands it to the other warps of its CTA.
struct MassItem {
  int valid;                 // 0: no more items
  int h, row, key0, ctx, ctx0, i0;  // i0: the first query of the chunk that counts
  int q_row;                 // its token
  int n_rows, n_qt;          // query rows from there on, and tiles of them
  int pad0, pad1;
};

template <int D, int KT>
struct MassCfg {
  static constexpr int BK = 128;  // keys of a tile per CTA (TMEM lanes)
  static constexpr int BQ = 128;  // query rows per tile
  static constexpr int kItemKeys = KT * 2 * BK;
  static constexpr int kHalves = D / 64;
  static constexpr int kKHalfBytes = BK * 128;
  static constexpr int kKBytes = kHalves * kKHalfBytes;  // a CTA's keys of a tile
  static constexpr int kQHalfBytes = BQ / 2 * 128;
  static constexpr int kQBytes = kHalves * kQHalfBytes;  // a CTA's rows of a query tile
  static constexpr int kOnesBytes = BK * 128;       // the operand of ones, 32 bytes of each row used
  static constexpr int kBiasBytes = BQ / 2 * 128;   // -lse / c of a CTA's rows of a tile, likewise
  static constexpr int kStages = D == 64 ? 6 : KT == 1 ? 5 : 3;
  static constexpr int kThreads = 384;
  static constexpr int kTmemCols = 512;  // four S buffers
  static constexpr int kSums = KT == 1 ? 1 : 0;
  // barriers: q_full, q_empty [stages], s_full[4], s_empty[4], item_full[2], item_empty[2],
  // k_full[2], k_empty[2], join_full, join_empty
  static constexpr int kBars = 2 * kStages + 18;
  static constexpr size_t kSmem = 1024 + 2 * KT * (size_t)kKBytes +
                                  kStages * (size_t)(kQBytes + kBiasBytes) + kOnesBytes +
                                  kSums * BK * 4 + 2 * sizeof(MassItem) + kBars * 8 + 16;
};

// 2^x that the compiler may move and interleave (fast_exp2 is volatile).
__device__ __forceinline__ float exp2_free(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Waits for the tensor-memory loads issued so far; `v` is what the last one reads, named so
// that nothing uses it earlier.
__device__ __forceinline__ void tmem_landed(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]),
                 "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]),
                 "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]),
                 "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                 "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]));
  asm volatile("" : "+f"(v[29]), "+f"(v[30]), "+f"(v[31]));
}

template <typename T>
constexpr int kFmt = 0;
template <>
constexpr int kFmt<__nv_bfloat16> = 1;

template <typename T, int D, int KT>
__global__ void __launch_bounds__(384, 1)
    prefill_mass_kernel(const __grid_constant__ CUtensorMap tmq,
                        const __grid_constant__ CUtensorMap tmk, const PrefillMassParams p) {
  using C = MassCfg<D, KT>;
  constexpr int ST = C::kStages, BK = C::BK, BQ = C::BQ;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sK = base;                                              // [slot][tile][half][128][128 B]
  uint8_t* sQ = sK + 2 * KT * C::kKBytes;                          // [stage][half][64][128 B]
  uint8_t* sB = sQ + ST * C::kQBytes;                              // [stage][64][128 B], -lse / c
  uint8_t* sOne = sB + ST * C::kBiasBytes;                         // [128][128 B]
  float* sX = reinterpret_cast<float*>(sOne + C::kOnesBytes);      // [128], KT = 1
  MassItem* items = reinterpret_cast<MassItem*>(sX + C::kSums * BK);
  uint64_t* bars = reinterpret_cast<uint64_t*>(items + 2);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kBars);
  // the first CTA's q_full and k_full count both CTAs' copies (and -lse), its s_empty both readers;
  // commits arrive in both CTAs; everything else is each CTA's own
  uint64_t* q_full = bars;
  uint64_t* q_empty = q_full + ST;
  uint64_t* s_full = q_empty + ST;
  uint64_t* s_empty = s_full + 4;
  uint64_t* item_full = s_empty + 4;
  uint64_t* item_empty = item_full + 2;
  uint64_t* k_full = item_empty + 2;
  uint64_t* k_empty = k_full + 2;
  uint64_t* join_full = k_empty + 2;
  uint64_t* join_empty = join_full + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(smem_addr(q_full + i), 3);  // the copies, warp 2 of each CTA
      mbar_init(smem_addr(q_empty + i), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_addr(s_full + i), 1);
      mbar_init(smem_addr(s_empty + i), 8);  // four warps of each CTA
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(item_full + i), 1);
      mbar_init(smem_addr(item_empty + i), leader ? 11 : 10);  // readers: all but warp 3, and
                                                               // the issuer in the first CTA only
      mbar_init(smem_addr(k_full + i), 1);
      mbar_init(smem_addr(k_empty + i), 1);
    }
    mbar_init(smem_addr(join_full), 4);
    mbar_init(smem_addr(join_empty), 4);
    fence_mbar_init();
    prefetch_tensormap(&tmq);
    prefetch_tensormap(&tmk);
  }
  // the operand of ones: 1 in columns 0 .. 3 of 16, the rest 0 (16-byte pieces swizzled by the row);
  // and zeros where warp 2 leaves columns 8 .. 15 alone
  for (int i = threadIdx.x; i < C::kOnesBytes / 16; i += C::kThreads) {
    const int row = i >> 3, piece = (i & 7) ^ (row & 7);
    const uint32_t ones = 0x3f803f80u;
    reinterpret_cast<uint4*>(sOne)[i] = piece == 0 ? make_uint4(ones, ones, 0, 0) : make_uint4(0, 0, 0, 0);
  }
  for (int i = threadIdx.x; i < ST * C::kBiasBytes / 16; i += C::kThreads)
    reinterpret_cast<uint4*>(sB)[i] = make_uint4(0, 0, 0, 0);
  tc::fence_proxy_async_smem();
  if (warp == 1) {
    tc::tmem_alloc_pair(smem_addr(tmem_slot), C::kTmemCols);
    tc::tmem_relinquish_pair();
  }
  tc::fence_before_sync();
  cluster_sync();  // both CTAs' barriers exist before either uses them
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();  // the plan and the lse of every query row are written
  griddep_launch_dependents();
  const int G = p.group, gl = p.group_log2;
  bool ok = true;
  // by whole warps; barriers the peer may complete take cluster-scope acquire
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(~0u, mbar_wait_cluster(smem_addr(bar), parity));
  };
  auto lead = [](uint64_t* bar) { return mapa_shared(smem_addr(bar), 0); };
  // the first query tile with a row that sees a key of the pair's tile kt, and whether any does:
  // if not, the tile is neither loaded nor used
  auto first_tile = [&](const MassItem& m, int kt) {
    return (max(0, m.key0 + kt * 2 * BK - m.ctx0 - m.i0) << gl) / BQ;
  };
  auto used = [&](const MassItem& m, int kt) { return first_tile(m, kt) < m.n_qt; };
  // an item for a consuming warp, which arrives on item_empty when it has it in registers
  auto take = [&](int n, MassItem& m) {
    if (!wait(item_full + (n & 1), (n >> 1) & 1)) {
      ok = false;
      return false;
    }
    m = items[n & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(item_empty + (n & 1)));
    return m.valid != 0;
  };

  if (warp == 0) {
    // ------------------------------ queries ------------------------------
    const uint64_t keep = l2_policy_evict_last();  // queries are read by many items
    int qt = 0;  // query tiles loaded
    MassItem m;
    for (int n = 0; take(n, m) && ok; ++n) {
      for (int j = 0; j < m.n_qt; ++j, ++qt) {
        const int s = qt % ST;
        if (!wait(q_empty + s, ((qt / ST) & 1) ^ 1)) { ok = false; break; }
        if (lane == 0) {
          if (leader) mbar_arrive_expect_tx(smem_addr(q_full + s), 2 * C::kQBytes);
#pragma unroll
          for (int hb = 0; hb < C::kHalves; ++hb)
            tma_load_3d_pair(smem_addr(sQ + s * C::kQBytes + hb * C::kQHalfBytes), &tmq, hb * 64,
                             m.h * G, m.q_row + ((2 * j + rank) * (BQ / 2) >> gl),
                             lead(q_full + s), keep);
        }
        __syncwarp();
      }
      if (!ok) break;
    }
  } else if (warp == 1) {
    // ------------------------------ MMA issuer ------------------------------
    if (leader) {
      const uint32_t idesc = tc::idesc_f16(kFmt<T>, 2 * BK, BQ, false, false);
      const uint64_t dk0 = tc::smem_desc_sw128(smem_addr(sK), 16, 1024);
      const uint64_t dq0 = tc::smem_desc_sw128(smem_addr(sQ), 16, 1024);
      const uint32_t idesc_bias = tc::idesc_f16(kFmt<__nv_bfloat16>, 2 * BK, BQ, false, false);
      const uint64_t dones = tc::smem_desc_sw128(smem_addr(sOne), 16, 1024);
      const uint64_t dbias0 = tc::smem_desc_sw128(smem_addr(sB), 16, 1024);
      const bool scores = p.no_scores == 0;
      uint32_t done[2] = {0, 0};  // products for each pair of S buffers so far
      int kn = 0, qt = 0;         // items with keys, query tiles
      MassItem m;
      for (int n = 0; take(n, m) && ok; ++n) {
        if (m.n_qt == 0) continue;
        int from[KT];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) from[kt] = first_tile(m, kt);
        const int slot = kn & 1;
        if (!wait(k_full + slot, (kn >> 1) & 1)) { ok = false; break; }
        ++kn;
        const uint64_t dk = tc::desc_advance(dk0, slot * KT * C::kKBytes);
        for (int j = 0; j < m.n_qt && ok; ++j, ++qt) {
          const int s = qt % ST;
          if (!wait(q_full + s, (qt / ST) & 1)) { ok = false; break; }
          tc::fence_after_sync();
          const uint64_t dq = tc::desc_advance(dq0, s * C::kQBytes);
#pragma unroll
          for (int kt = 0; kt < KT; ++kt) {
            if (j < from[kt]) continue;
            const int w = KT == 1 ? qt & 1 : kt;
            const int buf = 2 * w + (done[w] & 1);
            if (!wait(s_empty + buf, ((done[w] >> 1) & 1) ^ 1)) { ok = false; break; }
            ++done[w];
            tc::fence_after_sync();
            if (scores) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                tc::mma_ss_warp<true>(
                    tmem + buf * BQ,
                    tc::desc_advance(dk,
                                     kt * C::kKBytes + (kk >> 2) * C::kKHalfBytes + (kk & 3) * 32),
                    tc::desc_advance(dq, (kk >> 2) * C::kQHalfBytes + (kk & 3) * 32), idesc, kk > 0);
            }
            // last, when the sum has its full size
            tc::mma_ss_warp<true>(tmem + buf * BQ, dones, tc::desc_advance(dbias0, s * C::kBiasBytes),
                                  idesc_bias, scores);
            tc::commit_warp<true>(smem_addr(s_full + buf));
          }
          tc::commit_warp<true>(smem_addr(q_empty + s));
        }
        tc::commit_warp<true>(smem_addr(k_empty + slot));
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------ -lse / c of each query tile ------------------------------
    int qt = 0;
    MassItem m;
    for (int n = 0; take(n, m) && ok; ++n) {
      const float* lse = p.lse + ((size_t)m.h * p.num_tokens + m.q_row) * G;
      for (int j = 0; j < m.n_qt; ++j, ++qt) {
        const int s = qt % ST;
        float v[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int i = j * BQ + rank * (BQ / 2) + lane + 32 * u;
          // (the columns of rows past the chunk are masked below)
          v[u] = i < m.n_rows ? -__ldcg(lse + i) * p.inv_scale : 0.f;
        }
        if (!wait(q_empty + s, ((qt / ST) & 1) ^ 1)) { ok = false; break; }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float x = v[u];
          uint32_t term[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat16 y = __float2bfloat16_rn(x);
            term[e] = __bfloat16_as_ushort(y);
            x -= __bfloat162float(y);
          }
          const int row = lane + 32 * u;
          *reinterpret_cast<uint4*>(sB + s * C::kBiasBytes + row * 128 + ((row & 7) << 4)) =
              make_uint4(term[0] | term[1] << 16, term[2] | term[3] << 16, 0, 0);
        }
        tc::fence_proxy_async_smem();  // the tensor core reads what the lanes wrote
        __syncwarp();
        if (lane == 0) {
          if (leader) mbar_arrive(smem_addr(q_full + s));
          else mbar_arrive_remote(lead(q_full + s));
        }
      }
      if (!ok) break;
    }
  } else if (warp == 3) {
    // ------------------------------ items and keys ------------------------------
    const uint64_t once = l2_policy_evict_first();
    const int bs = 1 << p.block_log2, pairs = (int)gridDim.x / 2;
    const int total = __ldcg(p.tile_starts + p.num_seqs) * p.num_kv_heads;
    int kn = 0;  // items with keys loaded
    int i = (int)blockIdx.x / 2;
    for (int n = 0;; ++n, i += pairs) {
      MassItem m = {};
      int b = 0;
      if (i < total) {
        m.valid = 1;
        const int tile = i / p.num_kv_heads;
        m.h = i - tile * p.num_kv_heads;
        // the sequence: the last with tile_starts[b] <= tile, 32 probes a round
        int cnt = p.num_seqs;
        while (cnt > 1) {
          const int step = (cnt + 31) / 32;
          const bool le = lane * step < cnt && __ldcg(p.tile_starts + b + lane * step) <= tile;
          const int last = 31 - __clz(__ballot_sync(~0u, le) | 1u);
          cnt = min(step, cnt - last * step);
          b += last * step;
        }
        m.key0 = (tile - __ldcg(p.tile_starts + b)) * C::kItemKeys;
        const int q_begin = __ldg(p.cu_q_lens + b);
        const int chunk = __ldg(p.cu_q_lens + b + 1) - q_begin;
        m.ctx = __ldg(p.context_lens + b);
        m.row = p.mass.rows != nullptr ? __ldg(p.mass.rows + b) : b;
        const int seen = p.observe != nullptr ? max(0, __ldg(p.observe + b)) : chunk;
        m.ctx0 = m.ctx - chunk;
        m.i0 = max(max(0, m.key0 - m.ctx0), chunk - min(seen, chunk));
        m.q_row = q_begin + m.i0;
        m.n_rows = max(0, chunk - m.i0) << gl;
        if (m.row < 0 || m.row >= p.mass.num_rows) {  // nothing is added or written
          if (lane == 0) flag_status(p.status, PA_STATUS_BAD_CONTEXT);
          m.row = -1;
          m.n_rows = 0;
        }
        m.n_qt = (m.n_rows + BQ - 1) / BQ;
      }
      if (!wait(item_empty + (n & 1), ((n >> 1) & 1) ^ 1)) { ok = false; break; }
      if (lane == 0) {
        items[n & 1] = m;
        mbar_arrive(smem_addr(item_full + (n & 1)));
      }
      if (!m.valid) break;
      if (m.n_qt == 0) continue;
      // this CTA's keys: 128 of each tile's 256
      const int per_tile = BK >> p.block_log2;
      int id = -1;  // of this CTA's block `lane` (KT * BK / block_size <= 32 of them)
      const int key = m.key0 + lane / per_tile * 2 * BK + rank * BK +
                      (lane % per_tile << p.block_log2);
      if (lane < KT * per_tile && key < m.ctx) {
        id = __ldg(p.block_tables + (size_t)b * p.max_blocks + (key >> p.block_log2));
        if (id < 0 || id >= p.num_blocks) {
          flag_status(p.status, PA_STATUS_BAD_BLOCK);
          id = -1;
        }
      }
      const int slot = kn & 1;
      const int tiles = KT > 1 && used(m, KT - 1) ? KT : 1;
      if (!wait(k_empty + slot, ((kn >> 1) & 1) ^ 1)) { ok = false; break; }
      ++kn;
      if (lane == 0 && leader)
        mbar_arrive_expect_tx(smem_addr(k_full + slot), tiles * 2 * C::kKBytes);
      for (int x = 0; x < tiles * per_tile; ++x) {
        const int idx = __shfl_sync(~0u, id, x);
        if (lane == 0) {
          // blocks past the context (and bad ids) read a box wholly outside: zeros
          const int y = idx < 0 ? -bs : (idx * p.num_kv_heads + m.h) << p.block_log2;
          uint8_t* dst = sK + (slot * KT + x / per_tile) * C::kKBytes +
                         (x % per_tile << p.block_log2) * 128;
#pragma unroll
          for (int hb = 0; hb < C::kHalves; ++hb)
            tma_load_2d_pair(smem_addr(dst + hb * C::kKHalfBytes), &tmk, hb * 64, y,
                             lead(k_full + slot), once);
        }
      }
      __syncwarp();
    }
  } else {
    // ------------------------------ weights ------------------------------
    const int w = (warp - 4) >> 2;  // pair of S buffers
    const int r = threadIdx.x & 127;
    const uint32_t tS = tmem + ((uint32_t)((warp & 3) * 32) << 16) + w * 2 * BQ;
    const uint64_t sc2 = f2(p.scale_log2, p.scale_log2);
    // (what a masked column becomes: c times it is -inf whatever the sign of c)
    const float minus_inf = p.scale_log2 > 0.f ? -__builtin_huge_valf() : __builtin_huge_valf();
    uint32_t done = 0;  // S tiles of these warpgroups so far
    int qt = 0;
    MassItem m;
    for (int n = 0; take(n, m) && ok; ++n) {
      float total = 0.f;
      const int kt = KT == 1 ? 0 : w;
      const int from = first_tile(m, kt);
      const int key = m.key0 + kt * 2 * BK + rank * BK + r;
      float* mass = p.mass.mass + ((size_t)m.row * p.num_kv_heads + m.h) * p.mass.stride + key;
      const bool mine = key < m.ctx && m.row >= 0 && (KT > 1 || w == 0);
      const float old = mine && p.mass.decay != 0.f ? *mass : 0.f;
      for (int j = 0; j < m.n_qt && ok; ++j, ++qt) {
        if (KT == 1 && (qt & 1) != w) continue;
        if (j < from) continue;
        // columns from lo on see this thread's key, those from hi on lie past the chunk
        const int lo = (max(0, key - m.ctx0 - m.i0) << gl) - j * BQ;
        const int hi = m.n_rows - j * BQ;
        // the warp's smallest and largest lo: its keys are consecutive
        const int lo_min = __shfl_sync(~0u, lo, 0), lo_max = __shfl_sync(~0u, lo, 31);
        const int buf = 2 * w + (done & 1);
        if (!wait(s_full + buf, (done >> 1) & 1)) { ok = false; break; }
        tc::fence_after_sync();
        const uint32_t at = tS + (done & 1) * BQ;
        ++done;
        float x[4][32];
#pragma unroll
        for (int k = 0; k < 4; ++k) tc::tmem_ld32(at + 32 * k, x[k]);
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_landed(x[k]);
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) {  // the scores are in registers
          if (leader) mbar_arrive(smem_addr(s_empty + buf));
          else mbar_arrive_remote(lead(s_empty + buf));
        }
        uint64_t acc[4] = {0, 0, 0, 0};  // pairs of zeros
        auto add = [&](const float (&v)[32]) {
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; e += 2)
              f2_split(f2_mul(f2(v[i + e], v[i + e + 1]), sc2), y[e], y[e + 1]);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = exp2_free(y[e]);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = f2_add(acc[e], f2(y[2 * e], y[2 * e + 1]));
          }
        };
        // (two paths: branches between the chunks of the plain one would keep the compiler from
        // interleaving them)
        if (lo_max <= 0 && hi >= BQ) {
#pragma unroll
          for (int k = 0; k < 4; ++k) add(x[k]);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (lo_min >= 32 * k + 32 || hi <= 32 * k) continue;  // no lane sees any of the columns
            if (lo_max > 32 * k || hi < 32 * k + 32) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                x[k][i] = 32 * k + i >= lo && 32 * k + i < hi ? x[k][i] : minus_inf;
            }
            add(x[k]);
          }
        }
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x0, x1;
          f2_split(acc[e], x0, x1);
          sum += x0 + x1;
        }
        total += sum;
      }
      if (!ok) break;
      if constexpr (KT == 1) {  // both warpgroups hold a part of the same keys' sums
        if (w == 1) {
          sX[r] = total;
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(join_full));
          if (!wait(join_empty, n & 1)) { ok = false; break; }
        } else {
          if (!wait(join_full, n & 1)) { ok = false; break; }
          total += sX[r];
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(join_empty));
        }
      }
      if (mine && (m.n_qt > 0 || p.mass.decay != 1.f)) *mass = fmaf(p.mass.decay, old, total);
    }
  }
  if (!ok && lane == 0) flag_status(p.status, PA_STATUS_TIMEOUT);
  tc::fence_before_sync();
  __syncwarp();
  cluster_sync();  // neither CTA frees its tensor memory or leaves while the other uses it
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc_pair(tmem, C::kTmemCols);
  }
}

// A call without queries: decay alone, over every context.  The same product, rounded once, as the
// weights of an item without query tiles end on.  Bound by HBM, at few positions by the launch (64
// contexts of 8,192, 8 heads: 5.6 us of mostly L2 traffic, 0.90 of a copy's rate; 3 of 200: 1.6).
constexpr int kDecayThreads = 256, kDecayPerThread = 4;
__global__ void __launch_bounds__(kDecayThreads)
    mass_decay_kernel(const MassTarget mass, const int32_t* context_lens, int num_kv_heads,
                      int ctx_cap, int32_t* status) {
  griddep_wait();
  griddep_launch_dependents();
  const int h = blockIdx.y, b = blockIdx.z;
  const int ctx = __ldg(context_lens + b);
  if (ctx == 0) return;
  const int row = mass.rows != nullptr ? __ldg(mass.rows + b) : b;
  if (ctx < 0 || ctx > ctx_cap || row < 0 || row >= mass.num_rows) {
    if (threadIdx.x == 0) flag_status(status, PA_STATUS_BAD_CONTEXT);
    return;
  }
  float* m = mass.mass + ((size_t)row * num_kv_heads + h) * mass.stride;
  const long long first = (long long)blockIdx.x * kDecayThreads * kDecayPerThread + threadIdx.x;
#pragma unroll
  for (int i = 0; i < kDecayPerThread; ++i) {
    const long long at = first + i * kDecayThreads;
    if (at < ctx) m[at] = mass.decay != 0.f ? mass.decay * m[at] : 0.f;  // (0: not read)
  }
}

constexpr int kMaxDev = 64;
std::mutex g_mutex;

template <typename T, int D, int KT>
int launch_kt(const PrefillArgs& a, const PrefillMassParams& p, int ctx_cap,
              cudaStream_t stream) {
  using C = MassCfg<D, KT>;
  static_assert(C::kSmem <= 232448, "shared memory per CTA");
  static_assert(KT * C::BK / 16 <= 32, "a lane per block of an item");
  static bool configured[kMaxDev] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= kMaxDev)
    return fail(PA_ERR_CUDA, "pa_prefill_mass: no usable device");
  {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (!configured[dev]) {
      if (cudaFuncSetAttribute(prefill_mass_kernel<T, D, KT>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)C::kSmem) != cudaSuccess)
        return fail(PA_ERR_CUDA, "pa_prefill_mass: shared-memory configuration failed");
      configured[dev] = true;
    }
  }
  CUtensorMap tmq, tmk;
  const int r0 = encode_query_map(&tmq, a.q, a.dtype, a.num_tokens, a.num_q_heads, a.head_dim,
                                  p.group, C::BQ / 2 / p.group);
  const int r1 = encode_cache_map(&tmk, a.k_cache, a.dtype, a.num_blocks, a.num_kv_heads,
                                  a.block_size, a.head_dim);
  if (r0 != CUDA_SUCCESS || r1 != CUDA_SUCCESS)
    return fail(PA_ERR_CUDA, "pa_prefill_mass: cuTensorMapEncodeTiled failed (%d, %d)", r0, r1);
  // at most one pair per two SMs, and no more than there may be items
  const long long items = (long long)((std::max(1, ctx_cap) + C::kItemKeys - 1) / C::kItemKeys) *
                          a.num_kv_heads * a.num_seqs;
  const unsigned pairs = (unsigned)std::min<long long>(items, std::max(1, sm_count() / 2));
  const cudaError_t e = launch_pdl_cluster(prefill_mass_kernel<T, D, KT>, dim3(2 * pairs),
                                           dim3(C::kThreads), C::kSmem, stream, 2, tmq, tmk, p);
  if (e != cudaSuccess) return fail(PA_ERR_CUDA, "pa_prefill_mass: %s", cudaGetErrorString(e));
  return PA_OK;
}

template <typename T, int D>
int launch_t(const PrefillArgs& a, const PrefillMassParams& p, int ctx_cap, int item_keys,
             cudaStream_t stream) {
  return item_keys == MassCfg<D, 2>::kItemKeys ? launch_kt<T, D, 2>(a, p, ctx_cap, stream)
                                               : launch_kt<T, D, 1>(a, p, ctx_cap, stream);
}

template <typename T>
int dispatch(const PrefillArgs& a, const PrefillMassParams& p, int ctx_cap, int item_keys,
             cudaStream_t stream) {
  return a.head_dim == 128 ? launch_t<T, 128>(a, p, ctx_cap, item_keys, stream)
                           : launch_t<T, 64>(a, p, ctx_cap, item_keys, stream);
}

}  // namespace

int launch_prefill_mass(const PrefillArgs& a, const int32_t* observe, const MassTarget& mass,
                        cudaStream_t stream) {
  PrefillMassParams p;
  p.lse = a.lse;
  p.tile_starts = a.tile_starts;
  p.block_tables = a.block_tables;
  p.cu_q_lens = a.cu_q_lens;
  p.context_lens = a.context_lens;
  p.observe = observe;
  p.status = a.status;
  p.mass = mass;
  p.max_blocks = a.max_blocks;
  p.num_seqs = a.num_seqs;
  p.num_tokens = a.num_tokens;
  p.num_kv_heads = a.num_kv_heads;
  p.group = a.num_q_heads / a.num_kv_heads;
  p.group_log2 = 0;
  while ((1 << p.group_log2) < p.group) ++p.group_log2;
  p.block_log2 = a.block_size == 16 ? 4 : 5;
  p.num_blocks = a.num_blocks;
  const float c = a.scale * kLog2e;
  // (below 2^-120, lse / c could pass fp32's range; the scores are then 0 to fp32's last bit unless
  // a product of a query and a key is larger than 2^90)
  p.no_scores = std::fabs(c) < 0x1p-120f;
  p.scale_log2 = p.no_scores ? 1.f : c;
  p.inv_scale = 1.f / p.scale_log2;
  const int ctx_cap = (int)std::min<long long>(a.max_ctx, (long long)a.max_blocks * a.block_size);
  return a.dtype == PA_BF16 ? dispatch<__nv_bfloat16>(a, p, ctx_cap, a.tile_keys, stream)
                            : dispatch<__half>(a, p, ctx_cap, a.tile_keys, stream);
}

cudaError_t launch_mass_decay(const MassTarget& mass, const int32_t* context_lens, int num_seqs,
                              int num_kv_heads, int ctx_cap, int32_t* status,
                              cudaStream_t stream) {
  constexpr int kPositions = kDecayThreads * kDecayPerThread;
  // (a context's status is looked at even where none may have a position)
  const unsigned x = (unsigned)std::max(1, ctx_cap / kPositions + (ctx_cap % kPositions != 0));
  return launch_pdl(mass_decay_kernel, dim3(x, (unsigned)num_kv_heads, (unsigned)num_seqs),
                    dim3(kDecayThreads), 0, stream, mass, context_lens, num_kv_heads, ctx_cap,
                    status);
}

int prefill_mass_item_keys(int num_seqs, int num_kv_heads, int max_ctx) {
  // items of 512 keys read the queries from L2 half as often; with fewer of them than pairs of
  // SMs, 256
  const long long items = (long long)((max_ctx + 511) / 512) * num_kv_heads * num_seqs;
  return 2 * items >= std::max(1, sm_count()) ? 512 : 256;
}

}  // namespace pa
