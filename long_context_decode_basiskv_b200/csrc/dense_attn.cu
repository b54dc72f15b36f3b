// Attention of the new tokens over the whole paged cache, on the CUDA cores:
// fp32 caches, and bf16 caches whose rows are not swizzled (ranks that are no
// multiple of 16).  dense_attn_mma.cu and dense_attn_tc.cu hold the
// tensor-core kernels of the others.
//
// One CTA of four warps per (row tile, KV head, sequence, share of the keys).
// The rows of a tile are consecutive new tokens' G heads of the KV head, so a
// key tile that is staged in shared memory serves them all.  Each warp keeps a
// quarter of the rows: a lane scores one key of the tile for each of them, the
// running maximum and sum are per row (fp32), and for the weighted sum a lane
// holds the latent columns lane + 32 k.
#include <algorithm>

#include "dense_attn.cuh"
#include "kernels.cuh"

namespace bkv {

constexpr int kDcKeys = 32;      // keys per tile: one per lane
constexpr int kDcThreads = 128;

template <typename T, int D, int RT>
__global__ void __launch_bounds__(kDcThreads) dense_attn_kernel(DenseParams p) {
  constexpr int RW = RT / 4;         // rows of a warp
  constexpr int KP = D + 4;          // padded key row: 16-byte reads of 8 lanes in different banks
  extern __shared__ __align__(16) float sm[];
  __shared__ int s_ok[kDcKeys];
  __shared__ int s_last;
  const int r = p.r, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  float* sQ = sm;                    // [RT][D]
  float* sK = sQ + RT * D;           // [keys][KP]
  float* sC = sK + kDcKeys * KP;     // [keys][r]
  const int tiles = (p.n_new * p.G + RT - 1) / RT;
  const int split = blockIdx.x % p.splits;
  // the last row tiles of a causal prompt see the most keys: they start first
  const int rt = tiles - 1 - (int)(blockIdx.x / p.splits);
  const int g = blockIdx.y, b = blockIdx.z;
  const DenseSeq sq = dense_seq(p, b, tid == 0 && g == 0);
  const int row0 = rt * RT, rows = min(RT, p.n_new * p.G - row0);
  const int pos0 = sq.L - p.n_new;
  const T* q = static_cast<const T*>(p.q);
  const T* kr = static_cast<const T*>(p.k_raw);
  const T* cl = static_cast<const T*>(p.c_lat);

  KeyTiles kt{0, 0, 0};
  if (sq.L > 0)
    kt = key_tiles(pos0 + row0 / p.G, pos0 + (row0 + rows - 1) / p.G, sq.L, p.window, sq.prefix, kDcKeys);
  const int lo = (int)((long long)kt.count() * split / p.splits);
  const int hi = (int)((long long)kt.count() * (split + 1) / p.splits);
  const int see_lo = p.window > 0 ? pos0 + row0 / p.G - p.window + 1 : 0;  // first key past the prefix that a row sees
  const int see_hi = max(pos0 + (row0 + rows - 1) / p.G + 1, sq.prefix);

  for (int x = tid; x < rows * D; x += kDcThreads) {
    const int row = row0 + x / D;
    sQ[x] = Elem<T>::to_f(q[(((size_t)b * p.n_new + row / p.G) * p.Hq + (size_t)g * p.G + row % p.G) * D + x % D]);
  }
  float m[RW], l[RW], acc[RW][4], slope[RW];
#pragma unroll
  for (int y = 0; y < RW; ++y) {
    m[y] = -INFINITY;
    l[y] = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[y][k] = 0.f;
    const int row = row0 + warp * RW + y;
    slope[y] = p.slopes ? p.slopes[g * p.G + row % p.G] * kLog2e : 0.f;
  }

  for (int x = lo; x < hi; ++x) {
    const int j0 = kt.tile(x) * kDcKeys;
    __syncthreads();
    // this tile's rows; keys that no row of the CTA sees are not read (zeros stand for them)
    if (warp == 0) {
      const int j = j0 + lane;
      int ok = -1;
      if (j < sq.L && j < see_hi && (j >= see_lo || j < sq.prefix)) ok = dense_page(p, b, j / p.page);
      s_ok[lane] = ok;
    }
    __syncthreads();
    for (int y = tid; y < kDcKeys * D; y += kDcThreads) {
      const int jj = y / D, slot = (j0 + jj) % p.page;
      sK[jj * KP + y % D] = s_ok[jj] < 0 ? 0.f
          : Elem<T>::to_f(kr[(((size_t)s_ok[jj] * p.Hkv + g) * p.page + slot) * D + y % D]);
    }
    for (int y = tid; y < kDcKeys * r; y += kDcThreads) {
      const int jj = y / r, slot = (j0 + jj) % p.page;
      sC[y] = s_ok[jj] < 0 ? 0.f : Elem<T>::to_f(cl[(((size_t)s_ok[jj] * p.Hkv + g) * p.page + slot) * r + y % r]);
    }
    __syncthreads();
    float s[RW];
#pragma unroll
    for (int y = 0; y < RW; ++y) s[y] = 0.f;
    for (int e = 0; e < D; e += 4) {
      const float4 kv = *reinterpret_cast<const float4*>(sK + lane * KP + e);
#pragma unroll
      for (int y = 0; y < RW; ++y) {
        const float4 qv = *reinterpret_cast<const float4*>(sQ + (warp * RW + y) * D + e);
        s[y] = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y, fmaf(qv.z, kv.z, fmaf(qv.w, kv.w, s[y]))));
      }
    }
    const int j = j0 + lane;
    const bool have = s_ok[lane] >= 0;
#pragma unroll
    for (int y = 0; y < RW; ++y) {
      const int row = row0 + warp * RW + y, i = pos0 + row / p.G;
      float v = -INFINITY;
      if (have && warp * RW + y < rows && sees(i, j, sq.L, p.window, sq.prefix))
        v = mod_score(s[y], p.scale, p.cap, slope[y], i, j);
      const float mn = fmaxf(m[y], warp_max(v));
      float w = v != v ? v : 0.f, corr = 1.f;  // a row of nothing but NaN keeps a maximum of -inf
      if (mn != -INFINITY) {
        w = exp2f(v - mn);
        corr = exp2f(m[y] - mn);
      }
      m[y] = mn;
      l[y] = l[y] * corr + w;
      s[y] = w;
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[y][k] *= corr;
    }
    for (int jj = 0; jj < kDcKeys; ++jj) {
      float c[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) c[k] = lane + 32 * k < r ? sC[jj * r + lane + 32 * k] : 0.f;
#pragma unroll
      for (int y = 0; y < RW; ++y) {
        const float w = __shfl_sync(kFull, s[y], jj);
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[y][k] = fmaf(w, c[k], acc[y][k]);
      }
    }
  }

  const size_t unit = ((size_t)b * p.Hkv + g) * tiles + rt;
  const size_t stride = (size_t)RT * (r + 2);  // between the splits of a row
  float* part = p.part + unit * p.splits * stride;
#pragma unroll
  for (int y = 0; y < RW; ++y) {
    const int rr = warp * RW + y, row = row0 + rr;
    const float ls = warp_sum(l[y]);
    if (rr >= rows) continue;
    if (p.splits > 1) {
      float* out = part + split * stride + (size_t)rr * (r + 2);
      if (lane == 0) {
        out[0] = m[y];
        out[1] = ls;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (lane + 32 * k < r) out[2 + lane + 32 * k] = acc[y][k];
    } else {
      const size_t at = ((size_t)b * p.n_new + row / p.G) * p.Hq + (size_t)g * p.G + row % p.G;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (lane + 32 * k < r) p.o[at * r + lane + 32 * k] = ls > 0.f ? acc[y][k] / ls : (ls == ls ? 0.f : ls);
      if (p.lse && lane == 0) p.lse[at] = ls > 0.f ? (m[y] + log2f(ls)) * kLn2 : (ls == ls ? -INFINITY : ls);
    }
  }
  if (p.splits == 1 || !dense_last_split(p.cnt + unit, p.splits, p.err, &s_last)) return;
  for (int rr = warp; rr < rows; rr += 4) {
    const int row = row0 + rr;
    const size_t at = ((size_t)b * p.n_new + row / p.G) * p.Hq + (size_t)g * p.G + row % p.G;
    dense_join_row(part + (size_t)rr * (r + 2), stride, p.splits, r, p.o + at * r, p.lse ? p.lse + at : nullptr, lane,
                   false);
  }
}

// rows of a tile: a decode step's few, or 32
static int core_rows(int rows) { return rows <= 8 ? 8 : 32; }

// Splits: enough CTAs for two on every SM, each with at least 4 key tiles of a
// cache that fills its block table.
DensePlan dense_plan(int batch, int n_new, int Hq, int Hkv, int d, int r, int page, int max_pages, bool bf16,
                     int num_sms) {
  DensePlan pl{};
  const long long rows = (long long)n_new * (Hq / Hkv);
  if (kc_swizzled(bf16, d, r)) {
    pl.row_tile = rows <= 16 ? 0 : -1;
    if (rows <= 16) dense_plan_mma(&pl, batch, (int)rows, Hkv, d, r, page, max_pages, num_sms);
    else dense_plan_tc(&pl, batch, rows, Hkv, r, page, max_pages, num_sms);
    return pl;
  }
  pl.row_tile = core_rows((int)std::min(rows, 1000LL));
  const long long tiles = (rows + pl.row_tile - 1) / pl.row_tile;
  const long long units = tiles * Hkv * batch;
  const long long key_tiles = ((long long)max_pages * page + kDcKeys - 1) / kDcKeys;
  pl.splits = (int)std::max(1LL, std::min({2LL * num_sms / units, key_tiles / 4, 256LL}));
  size_t off = 0;
  pl.cnt_off = off;
  off += ((size_t)units * 4 + 255) & ~(size_t)255;
  pl.part_off = off;
  if (pl.splits > 1) off += (size_t)units * pl.splits * pl.row_tile * (r + 2) * 4;
  pl.bytes = (off + 255) & ~(size_t)255;
  return pl;
}

template <typename T, int D, int RT>
static cudaError_t launch_core_t(const DenseParams& p, cudaStream_t st) {
  const size_t smem = ((size_t)RT * D + kDcKeys * (D + 4) + (size_t)kDcKeys * p.r) * sizeof(float);
  cudaError_t e = ensure_smem((const void*)dense_attn_kernel<T, D, RT>, smem);
  if (e != cudaSuccess) return e;
  const int tiles = (p.n_new * p.G + RT - 1) / RT;
  dense_attn_kernel<T, D, RT><<<dim3(tiles * p.splits, p.Hkv, p.batch), kDcThreads, smem, st>>>(p);
  return cudaGetLastError();
}

template <typename T, int D>
static cudaError_t launch_core(const DenseParams& p, int row_tile, cudaStream_t st) {
  return row_tile == 8 ? launch_core_t<T, D, 8>(p, st) : launch_core_t<T, D, 32>(p, st);
}

cudaError_t launch_dense_attn(const DensePlan& pl, DenseParams p, bool bf16, void* scratch, cudaStream_t st) {
  char* base = static_cast<char*>(scratch);
  p.cnt = reinterpret_cast<int32_t*>(base + pl.cnt_off);
  p.part = reinterpret_cast<float*>(base + pl.part_off);
  p.splits = pl.splits;
  if (pl.row_tile == 0) return launch_dense_mma(p, st);
  if (pl.row_tile < 0) return launch_dense_tc(p, st);
  if (bf16)
    return p.d == 128 ? launch_core<__nv_bfloat16, 128>(p, pl.row_tile, st)
                      : launch_core<__nv_bfloat16, 64>(p, pl.row_tile, st);
  return p.d == 128 ? launch_core<float, 128>(p, pl.row_tile, st) : launch_core<float, 64>(p, pl.row_tile, st);
}

}  // namespace bkv
