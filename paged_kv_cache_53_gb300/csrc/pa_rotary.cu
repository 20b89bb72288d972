// Rotary positions with any number of axes, applied to a step's queries and keys, with the
// cache write of the rotated keys and the values in the same launch.
//
// Pair i of a head is the plane (x, y) = elements (i, i + r/2), or (2i, 2i + 1) interleaved,
// of its first r elements, and is turned by the angle a = position[axis(i)] * freq[i]:
//     (x, y) -> (x cos a - y sin a, y cos a + x sin a).
// Angles.  A turn count in 64-bit fixed point, freq / 2 pi * 2^64, multiplied by the integer
// position wraps at whole turns exactly, so the angle's error does not grow with the
// position (fp32 would be off by 0.03 rad at position 1,000,000).  The top 32 bits are the
// angle as a signed fraction of a turn; the sine and cosine are taken of that, once per
// (token, pair) for all heads.
// Bound: every element is read and written once (HBM for prompts, launch latency for a few
// tokens).  A CTA takes one token, or four where there are plenty: its threads load their first
// vectors and, meanwhile, a warp per token finds the token's sequence and slot, three or four
// loads that wait for one another, and the other warps the sines.  (With one token per CTA
// that chain held a prompt's tokens to half of HBM's rate; now 25k tokens of 32 + 8 heads of 128,
// bf16, take 107 us, 0.86 of a copy's rate, and 256 tokens 4 us.)
#include <cmath>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_launch.h"

namespace pa {
namespace {

constexpr int kThreads = 256;

struct RotaryParams {
  const void* q;
  const void* k_new;
  const void* v_new;
  void* q_out;
  void* k_cache;
  void* v_cache;
  int64_t* slots;
  const int32_t* block_tables;
  const int32_t* cu_q_lens;  // null: token t belongs to sequence t
  const int32_t* context_lens;
  const int32_t* positions;  // [axes, num_tokens]
  int32_t* status;
  long long q_stride, k_stride, v_stride;  // elements between tokens
  int max_blocks, num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim, block_log2,
      num_blocks, half;  // half: rotated pairs of a head
  unsigned long long turns[kMaxRotaryPairs];  // freq / 2 pi in units of 2^-64 turns
  unsigned char axis[kMaxRotaryPairs];
};

// The sequence of token t by one warp: the last b with cu[b] <= t, 32 probes a round (the last
// sequence for tokens past the end).
__device__ __forceinline__ int find_sequence(const int32_t* cu, int num_seqs, int t, int lane) {
  int lo = 0, n = num_seqs;  // the answer lies in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const bool le = lane * step < n && __ldg(cu + lo + lane * step) <= t;
    const int last = 31 - __clz(__ballot_sync(~0u, le) | 1u);
    n = min(step, n - last * step);
    lo += last * step;
  }
  return lo;
}

template <typename T>
__device__ __forceinline__ float to_f32(T x) { return static_cast<float>(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x) { return static_cast<T>(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

template <typename T>
__device__ __forceinline__ void turn(T& x, T& y, float2 cs) {
  const float a = to_f32(x), b = to_f32(y);
  x = from_f32<T>(a * cs.x - b * cs.y);
  y = from_f32<T>(b * cs.x + a * cs.y);
}

// A 16-byte vector of elements.
template <typename T>
union Vec {
  static constexpr int N = 16 / sizeof(T);
  uint4 u;
  T e[N];
  __device__ Vec() {}
};

// How a head's elements are cut into work items of up to two 16-byte vectors (or, kScalar,
// two elements).  kSplit: the vectors at c and half + c of a rotated head; kInterleaved: two
// vectors of whole pairs, half a head apart; kScalar: half-split pairs whose halves do not
// start on vectors, an element a load (25k tokens of 32 + 8 heads, bf16: 348 us with 24 of 64
// elements turned, 528 with 126 of 128, 0.12 and 0.17 of a copy's rate).
enum Mode { kSplit, kInterleaved, kScalar };

constexpr int kAhead = 3;  // items a thread has in flight

// TOK: tokens per CTA.
template <typename T, Mode M, int TOK>
__global__ void __launch_bounds__(kThreads) rotary_append_kernel(
    const __grid_constant__ RotaryParams p) {
  using V = Vec<T>;
  constexpr int N = V::N;
  __shared__ float2 s_cs[TOK][kMaxRotaryPairs];
  __shared__ long long s_slot[TOK];
  const int t0 = blockIdx.x * TOK, ntok = min(TOK, p.num_tokens - t0);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int D = p.head_dim, half = p.half, rot = 2 * half;
  griddep_wait();
  griddep_launch_dependents();

  // rows are heads: a token's q heads, k heads and v heads, then the next token's.  A row is
  // `per_row` items wide (a v head may need fewer); a thread keeps its place in the row and
  // moves on by the rows that the CTA covers at once.
  const int per_row = M == kSplit ? half / N + (D - rot) / N : M == kInterleaved ? D / N / 2 : D - half;
  const int v_items = M == kScalar ? D / N : D / N / 2;
  const int heads = p.num_q_heads + 2 * p.num_kv_heads;
  const int rows_at_once = kThreads / per_row;
  const int c = tid % per_row;
  int row = tid / per_row;
  const int rows = row < rows_at_once ? ntok * heads : 0;  // (the last threads may be left over)
  // the item's places in a rotated head and in a v head (the second < 0: none), and whether
  // it is turned
  const bool turned = M == kSplit ? c < half / N : M == kInterleaved ? true : c < half;
  const int a = M == kSplit ? (turned ? c * N : rot + (c - half / N) * N)
                            : M == kInterleaved ? c * N : (turned ? c : half + c);
  const int b = M == kSplit ? (turned ? half + c * N : -1)
                            : M == kInterleaved ? D / 2 + c * N : (turned ? half + c : -1);
  const int va = c < v_items ? c * N : -1;
  const int vb = M == kScalar || va < 0 ? -1 : D / 2 + c * N;

  // a scalar item's elements ride in a vector's first places
  auto load = [&](int r, V& x, V& y) {
    const int tk = r / heads, head = r - tk * heads;
    const long long t = t0 + tk;
    if (head < p.num_q_heads + p.num_kv_heads) {
      const T* s = head < p.num_q_heads
                       ? static_cast<const T*>(p.q) + t * p.q_stride + (long long)head * D
                       : static_cast<const T*>(p.k_new) + t * p.k_stride +
                             (long long)(head - p.num_q_heads) * D;
      if constexpr (M == kScalar) {
        x.e[0] = s[a];
        if (b >= 0) y.e[0] = s[b];
      } else {
        x.u = *reinterpret_cast<const uint4*>(s + a);
        if (b >= 0) y.u = *reinterpret_cast<const uint4*>(s + b);
      }
    } else if (va >= 0) {
      const T* s = static_cast<const T*>(p.v_new) + t * p.v_stride +
                   (long long)(head - p.num_q_heads - p.num_kv_heads) * D;
      x.u = *reinterpret_cast<const uint4*>(s + va);
      if (vb >= 0) y.u = *reinterpret_cast<const uint4*>(s + vb);
    }
  };
  auto finish = [&](int r, V& x, V& y) {
    const int tk = r / heads, head = r - tk * heads;
    const long long slot = s_slot[tk];
    if (slot == -2) return;  // past the last sequence: no row of the token is written
    const bool is_v = head >= p.num_q_heads + p.num_kv_heads;
    T* d;
    if (head < p.num_q_heads) {
      d = static_cast<T*>(p.q_out) + ((long long)(t0 + tk) * p.num_q_heads + head) * D;
    } else {
      if (slot < 0) return;
      const int h = head - p.num_q_heads - (is_v ? p.num_kv_heads : 0);
      const long long blk = slot >> p.block_log2, off = slot & ((1 << p.block_log2) - 1);
      d = static_cast<T*>(is_v ? p.v_cache : p.k_cache) +
          (((blk * p.num_kv_heads + h) << p.block_log2) + off) * D;
    }
    if (is_v) {
      if (va >= 0) *reinterpret_cast<uint4*>(d + va) = x.u;
      if (vb >= 0) *reinterpret_cast<uint4*>(d + vb) = y.u;
      return;
    }
    const float2* cs = s_cs[tk];
    if constexpr (M == kSplit) {
      if (turned) {
#pragma unroll
        for (int e = 0; e < N; ++e) turn(x.e[e], y.e[e], cs[a + e]);
      }
    } else if constexpr (M == kInterleaved) {
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        if (a + e < rot) turn(x.e[e], x.e[e + 1], cs[(a + e) >> 1]);
        if (b + e < rot) turn(y.e[e], y.e[e + 1], cs[(b + e) >> 1]);
      }
    } else {
      if (turned) turn(x.e[0], y.e[0], cs[a]);
    }
    if constexpr (M == kScalar) {
      d[a] = x.e[0];
      if (b >= 0) d[b] = y.e[0];
    } else {
      *reinterpret_cast<uint4*>(d + a) = x.u;
      if (b >= 0) *reinterpret_cast<uint4*>(d + b) = y.u;
    }
  };

  V x[kAhead], y[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if (row + k * rows_at_once < rows) load(row + k * rows_at_once, x[k], y[k]);

  if (warp < TOK) {
    const int t = t0 + warp;
    if (warp < ntok) {
      const int s = p.cu_q_lens == nullptr ? min(t, p.num_seqs - 1)
                                           : find_sequence(p.cu_q_lens, p.num_seqs, t, lane);
      if (lane == 0) {
        const int first = p.cu_q_lens != nullptr ? __ldg(p.cu_q_lens + s) : s;
        const int end = p.cu_q_lens != nullptr ? __ldg(p.cu_q_lens + s + 1) : s + 1;
        const long long pos = (long long)__ldg(p.context_lens + s) - end + t;
        long long slot = -1;
        if (s == p.num_seqs - 1 && t >= end) {
          slot = -2;
        } else if (t < first || t >= end || pos < 0 ||
                   pos >= ((long long)p.max_blocks << p.block_log2)) {
          flag_status(p.status, PA_STATUS_BAD_CONTEXT);
        } else {
          const int blk = __ldg(p.block_tables + (size_t)s * p.max_blocks + (pos >> p.block_log2));
          if (blk < 0 || blk >= p.num_blocks)
            flag_status(p.status, PA_STATUS_BAD_BLOCK);
          else
            slot = ((long long)blk << p.block_log2) + (pos & ((1 << p.block_log2) - 1));
        }
        if (p.slots != nullptr && slot != -2) p.slots[t] = slot;
        s_slot[warp] = slot;
      }
    }
  } else {
    for (int j = tid - 32 * TOK; j < ntok * half; j += kThreads - 32 * TOK) {
      const int tk = j / half, i = j - tk * half;
      const long long pos = __ldg(p.positions + (size_t)p.axis[i] * p.num_tokens + t0 + tk);
      const unsigned long long turns = (unsigned long long)pos * p.turns[i];
      // a signed fraction of a turn, in [-1/2, 1/2), as half-turns
      const float f = (float)(int)(turns >> 32) * 0x1p-31f;
      float sn, cn;
      sincospif(f, &sn, &cn);
      s_cs[tk][i] = make_float2(cn, sn);
    }
  }
  __syncthreads();
  for (;;) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (row + k * rows_at_once < rows) finish(row + k * rows_at_once, x[k], y[k]);
    row += kAhead * rows_at_once;
    if (row >= rows) break;
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (row + k * rows_at_once < rows) load(row + k * rows_at_once, x[k], y[k]);
  }
}

// A frequency in radians as turns in 64-bit fixed point, whole turns dropped.  1 / 2 pi is
// carried as the sum of two doubles, good to 2^-107 of itself: up to kMaxRotaryFreq that is far
// below the two truncations (2^-64 turns each), so that a position of 2^31 still has its angle to
// 2^-32 turns.
unsigned long long turns_per_position(double freq) {
  const double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
  const double q = freq * hi;
  const double r = std::fma(freq, hi, -q) + freq * lo;
  auto fixed = [](double x) -> unsigned long long {  // x modulo 1, in units of 2^-64
    const double f = (x - std::trunc(x)) * 0x1p64;   // (both steps are exact)
    return f < 0.0 ? 0ull - (unsigned long long)-f : (unsigned long long)f;
  };
  return fixed(q) + fixed(r);
}

template <typename T, Mode M>
cudaError_t launch_mode(const RotaryParams& p, cudaStream_t stream) {
  // four tokens per CTA once that still gives every SM several CTAs
  if (p.num_tokens >= 32 * sm_count())
    return launch_pdl(rotary_append_kernel<T, M, 4>, dim3((unsigned)((p.num_tokens + 3) / 4)),
                      dim3(kThreads), 0, stream, p);
  return launch_pdl(rotary_append_kernel<T, M, 1>, dim3((unsigned)p.num_tokens), dim3(kThreads), 0,
                    stream, p);
}

template <typename T>
cudaError_t launch(const RotaryParams& p, bool interleaved, cudaStream_t stream) {
  if (interleaved) return launch_mode<T, kInterleaved>(p, stream);
  if (p.half % Vec<T>::N == 0) return launch_mode<T, kSplit>(p, stream);
  return launch_mode<T, kScalar>(p, stream);
}

}  // namespace

cudaError_t launch_rotary_append(const RotaryArgs& a, cudaStream_t stream) {
  RotaryParams p;
  p.q = a.q;
  p.k_new = a.k_new;
  p.v_new = a.v_new;
  p.q_out = a.q_out;
  p.k_cache = a.k_cache;
  p.v_cache = a.v_cache;
  p.slots = a.slots;
  p.block_tables = a.block_tables;
  p.cu_q_lens = a.cu_q_lens;
  p.context_lens = a.context_lens;
  p.positions = a.positions;
  p.status = a.status;
  p.q_stride = a.q_stride;
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  p.max_blocks = a.max_blocks;
  p.num_seqs = a.num_seqs;
  p.num_tokens = a.num_tokens;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.head_dim = a.head_dim;
  p.block_log2 = a.block_size == 16 ? 4 : 5;
  p.num_blocks = a.num_blocks;
  p.half = a.rotary_dim / 2;
  for (int i = 0; i < p.half; ++i) {
    p.turns[i] = turns_per_position(a.inv_freq[i]);
    p.axis[i] = (unsigned char)a.pair_axis[i];
  }
  switch (a.dtype) {
    case PA_F32: return launch<float>(p, a.interleaved, stream);
    case PA_F16: return launch<__half>(p, a.interleaved, stream);
    default: return launch<__nv_bfloat16>(p, a.interleaved, stream);
  }
}

}  // namespace pa
