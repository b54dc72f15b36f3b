// What the kernels of basiskv_dense_attn share: the parameter block, which keys
// a row sees, what becomes of a raw score, and the joining of a split axis.
//
// A row is one (new token t, query head h) of a sequence; its position is
// i = L - n_new + t.  Its score for key j and what it does with it:
//   s = scale q.k_j;  s = cap tanh(s / cap) (cap > 0);  s -= slope_h |i - j|
//   sees j:  j < L and ((j <= i and (window = 0 or i - j < window)) or j < prefix)
//   o = sum_j softmax(s)_j C_j,  lse = log sum_j exp(s_j)
// Scores are kept in units of log 2, so that a weight is one exp2.
#pragma once

#include "common.cuh"

namespace bkv {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct DenseParams {
  const void* q;               // [B][n_new][Hq][d]
  const void* k_raw;
  const void* c_lat;
  const int32_t* block_table;
  const int32_t* seq_len;
  const float* slopes;         // [Hq] or NULL
  const int32_t* prefix_len;   // [B] or NULL
  float* o;                    // [B][n_new][Hq][r]
  float* lse;                  // [B][n_new][Hq] or NULL
  int32_t* err;
  float* part;                 // partial results of splits: per row (max, sum, acc[r])
  int32_t* cnt;                // finished splits of each row tile, or of each CTA's last group; zero between calls
  int batch, n_new, Hq, Hkv, G, d, r, page, max_pages, num_phys;
  int window;
  int mc;                      // row swizzle of C pages (swz())
  int splits;
  float scale;                 // plain scores: scale log2(e); capped: scale / cap
  float cap;                   // 0, or cap log2(e)
};

// 2^x by the hardware's instruction (2 units in the last place; results below the normal range are 0,
// which no sum of weights around 1 notices).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh(x) = x P(x^2) on |x| <= 1: P interpolates tanh(sqrt t) / sqrt t at the
// Chebyshev points of [0, 1] (degree 6; within 5e-8 of tanh, and 1.2e-7 as fp32 rounds it, that is
// 1.2e-7 cap in a score).  Beyond 1, 1 - 2 / (1 + e^2x) loses nothing: 2e-7.
constexpr int kTanhTop = 6;
__host__ __device__ constexpr float tanh_coef(int k) {
  return k == 0 ? 0.999999949f : k == 1 ? -0.33332828f : k == 2 ? 0.133250761f : k == 3 ? -0.0534516464f
       : k == 4 ? 0.0202797083f : k == 5 ? -0.00619432483f : 0.0010380251f;
}
__device__ __forceinline__ float tanh_far(float x) { return 1.f - __fdividef(2.f, 1.f + ex2(x * (2.f * kLog2e))); }
__device__ __forceinline__ float cap_score(float x, float cap) {  // x = s / cap
  const float t = x * x;
  float y = tanh_coef(kTanhTop);
#pragma unroll
  for (int k = kTanhTop - 1; k >= 0; --k) y = fmaf(y, t, tanh_coef(k));
  return cap * (t <= 1.f ? x * y : tanh_far(x));
}

// Raw score -> score in units of log 2.
__device__ __forceinline__ float mod_score(float raw, float scale, float cap, float slope2, int i, int j) {
  float s = raw * scale;
  if (cap > 0.f) s = cap_score(s, cap);
  return s - slope2 * fabsf((float)(i - j));
}

__device__ __forceinline__ bool sees(int i, int j, int L, int window, int prefix) {
  return j < L && ((j <= i && (window == 0 || i - j < window)) || j < prefix);
}

// Keys that rows at positions [i0, i1] of a sequence see, as tiles of `tile`
// keys: tiles [0, na) and [nb, ne), na <= nb.
struct KeyTiles {
  int na, nb, ne;
  __device__ __forceinline__ int count() const { return na + ne - nb; }
  __device__ __forceinline__ int tile(int x) const { return x < na ? x : x - na + nb; }
};
__device__ __forceinline__ KeyTiles key_tiles(int i0, int i1, int L, int window, int prefix, int tile) {
  KeyTiles k;
  const int end = min(L, max(i1 + 1, prefix));
  k.ne = (end + tile - 1) / tile;
  const int lo = window > 0 ? max(0, i0 - window + 1) : 0;
  k.na = min(k.ne, (min(prefix, end) + tile - 1) / tile);
  k.nb = min(k.ne, max(k.na, lo / tile));
  return k;
}

// A sequence as the kernels take it: its length (0: nothing to attend over),
// its prefix clamped to the length.
struct DenseSeq {
  int L, prefix;
};
__device__ __forceinline__ DenseSeq dense_seq(const DenseParams& p, int b, bool report) {
  DenseSeq s{p.seq_len[b], 0};
  if (s.L < 0 || (s.L > 0 && s.L < p.n_new) || s.L > p.max_pages * p.page) {
    if (report) set_err(p.err, BASISKV_DEVERR_SEQ_LEN);
    s.L = 0;
  }
  if (p.prefix_len) s.prefix = max(0, min(s.L, p.prefix_len[b]));
  return s;
}

// physical page of a logical page, -1 (reported) where the table's entry is out of range
__device__ __forceinline__ int dense_page(const DenseParams& p, int b, int page) {
  const int id = p.block_table[(size_t)b * p.max_pages + page];
  if (id < 0 || id >= p.num_phys) {
    set_err(p.err, BASISKV_DEVERR_BLOCK_TABLE);
    return -1;
  }
  return id;
}

// Counts this CTA among the splits of its unit; true in every thread of the
// last one, which joins their results.  The counter is left at zero.  One that
// did not start there is reported where it shows: below zero, or past the end.
__device__ __forceinline__ bool dense_last_split(int32_t* cnt, int splits, int32_t* err, int* s_last) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    const int prev = atomicAdd(cnt, 1);
    if (prev < 0 || prev >= splits) set_err(err, BASISKV_DEVERR_WORKSPACE);
    *s_last = prev == splits - 1;
    if (*s_last) {
      *cnt = 0;
      __threadfence();
    }
  }
  __syncthreads();
  return *s_last != 0;
}

// A warp's fold of a row's partial results, `stride` floats apart, in order:
// M = max m_s, l = sum 2^(m_s - M) l_s (whole warp), acc likewise (columns
// lane + 32 k).  Eight results' loads are in flight at a time.
struct DenseFold {
  float M, l, acc[4];
};
__device__ __forceinline__ DenseFold dense_fold(const float* part, size_t stride, int splits, int r, int lane) {
  constexpr int kAt = 8;
  DenseFold f{-INFINITY, 0.f, {0.f, 0.f, 0.f, 0.f}};
  for (int s0 = 0; s0 < splits; s0 += kAt) {
    const int n = min(kAt, splits - s0);
    const float* at = part + s0 * stride;
    float m = -INFINITY, l = 0.f, x[kAt][4];
    if (lane < n) {
      m = __ldcg(at + lane * stride);
      l = __ldcg(at + lane * stride + 1);
    }
#pragma unroll
    for (int s = 0; s < kAt; ++s)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        x[s][k] = (s < n && lane + 32 * k < r) ? __ldcg(at + s * stride + 2 + lane + 32 * k) : 0.f;
    const float M = fmaxf(f.M, warp_max(m));
    // while nothing has been seen, sums are 0, or NaN where all scores were
    const float c = M == -INFINITY ? 1.f : exp2f(f.M - M), w = M == -INFINITY ? 1.f : exp2f(m - M);
    f.l = f.l * c + warp_sum(lane < n ? l * w : 0.f);
#pragma unroll
    for (int k = 0; k < 4; ++k) f.acc[k] *= c;
#pragma unroll
    for (int s = 0; s < kAt; ++s) {
      const float ws = __shfl_sync(kFull, w, s);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (s < n) f.acc[k] = fmaf(ws, x[s][k], f.acc[k]);
    }
    f.M = M;
  }
  return f;
}

// The fold as one partial result.  failed: a wait gave up on the way; the sum
// is NaN then, and with it every output that it goes into.
__device__ __forceinline__ void dense_fold_row(const float* part, size_t stride, int splits, int r, float* to,
                                               bool failed, int lane) {
  const DenseFold f = dense_fold(part, stride, splits, r, lane);
  if (lane == 0) {
    to[0] = f.M;
    to[1] = failed ? __int_as_float(0x7fc00000) : f.l;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (lane + 32 * k < r) to[2 + lane + 32 * k] = f.acc[k];
}

// The fold as the row's result.
__device__ __forceinline__ void dense_join_row(const float* part, size_t stride, int splits, int r, float* o,
                                               float* lse, int lane, bool failed) {
  const DenseFold f = dense_fold(part, stride, splits, r, lane);
  const float l = failed ? __int_as_float(0x7fc00000) : f.l;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (lane + 32 * k < r) o[lane + 32 * k] = l > 0.f ? f.acc[k] / l : (l == l ? 0.f : l);
  if (lse && lane == 0) *lse = l > 0.f ? (f.M + log2f(l)) * kLn2 : (l == l ? -INFINITY : l);
}

}  // namespace bkv
