// Attention of the new tokens over the whole paged cache, on the CUDA cores:
// fp32 caches, and bf16 caches whose rows are not swizzled (ranks that are no
// multiple of 16).  dense_attn_mma.cu and dense_attn_tc.cu hold the
// tensor-core kernels of the others.
//
// One CTA of four warps per (row tile, KV head, sequence, share of the keys).
// The rows of a tile are consecutive new tokens' G heads of the KV head, so a
// key tile that is staged in shared memory serves them all; the next tile is
// on its way (cp.async, two buffers) while one is worked on.  Each warp keeps a
// quarter of the rows: a lane scores one key of the tile for each of them, the
// running maximum and sum are per row (fp32); the weights cross to the other
// lanes through shared memory, four keys to a load, and for the weighted sum a
// lane holds the latent columns lane + 32 k.  Few rows: bound by latency, so
// the keys are split over the SMs; many: by shared-memory reads (9 to 32 FMAs).
//
// Measured (fp32, d 64, rank 16, 8 heads over 2): one sequence of 2048 tokens
// 13.2 us (1.3 MB: a launch, a split's 2 key tiles, the join of 32 splits); 512
// tokens after 1536 others 213 us (5.5 TFLOP/s).  bf16, d 128, 8 heads over 2: 300
// tokens after 5700, rank 24 500 us, rank 40 552 us (8.5 TFLOP/s).
#include <algorithm>

#include "dense_attn.cuh"
#include "kernels.cuh"

namespace bkv {

constexpr int kDcKeys = 32;      // keys per tile: one per lane
constexpr int kDcThreads = 128;

// bytes of a staged K row (16 more than the row: the 16-byte reads of 8 lanes fall in different banks), C row
template <typename T, int D>
__host__ __device__ constexpr int dc_krow() { return D * (int)sizeof(T) + 16; }
__host__ __device__ inline int dc_crow(int r, int es) { return (r * es + 15) & ~15; }
template <typename T, int D>
__host__ __device__ inline int dc_stage(int r) { return kDcKeys * (dc_krow<T, D>() + dc_crow(r, sizeof(T))); }

template <typename T, int D, int RT, int CU>
__global__ void __launch_bounds__(kDcThreads) dense_attn_kernel(DenseParams p) {
  constexpr int RW = RT / 4;              // rows of a warp
  constexpr int KP = dc_krow<T, D>(), E = 16 / (int)sizeof(T), KC = D / E;  // elements of a chunk, chunks of a row
  extern __shared__ __align__(16) unsigned char sm[];
  __shared__ int s_last;
  const int r = p.r, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, P = p.page;
  const int CP = dc_crow(r, sizeof(T)), stage = dc_stage<T, D>(r);
  float* sQ = reinterpret_cast<float*>(sm);                 // [RT][D]
  float (*s_w)[kDcKeys] = reinterpret_cast<float (*)[kDcKeys]>(sQ + RT * D);  // [RT] weights of the tile
  unsigned char* sKC = sm + (size_t)RT * (D + kDcKeys) * sizeof(float);  // two of: K [keys][KP], C [keys][CP]
  const int tiles = (p.n_new * p.G + RT - 1) / RT;
  const int split = blockIdx.x % p.splits;
  // the last row tiles of a causal prompt see the most keys: they start first
  const int rt = tiles - 1 - (int)(blockIdx.x / p.splits);
  const int g = blockIdx.y, b = blockIdx.z;
  grid_dep_wait();     // the append may still be running when this grid starts
  allow_dependents();  // the out-projection may start and stage its weights
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
  const int see_hi = min(sq.L, max(pos0 + (row0 + rows - 1) / p.G + 1, sq.prefix));

  // the page of key `lane` of tile x, -1 where no row of the CTA sees the key (zeros stand for it then)
  auto page_of = [&](int x) {
    int id = -1;
    if (x < hi) {
      const int j = kt.tile(x) * kDcKeys + lane;
      if (j < see_hi && (j >= see_lo || j < sq.prefix)) id = dense_page(p, b, j / P);
    }
    return id;
  };
  const bool c_chunks = r * (int)sizeof(T) % 16 == 0;
  auto copy = [&](int x, int ids) {
    if (x >= hi) return;
    unsigned char* dst = sKC + (size_t)((x - lo) & 1) * stage;
    const int slot0 = kt.tile(x) * kDcKeys % P;  // of the tile's first key: tiles and pages are multiples of 16
    for (int y = tid; y < kDcKeys * KC; y += kDcThreads) {
      const int jj = y / KC, c = y - jj * KC, id = __shfl_sync(kFull, ids, jj);
      const size_t at = id < 0 ? 0 : (((size_t)id * p.Hkv + g) * P + (slot0 + jj) % P) * D + c * E;
      cp_async16_zfill(dst + jj * KP + c * 16, kr + at, id >= 0);
    }
    dst += kDcKeys * KP;
    if (c_chunks) {
      const int cc = r / E;
      for (int y0 = 0; y0 < kDcKeys * cc; y0 += kDcThreads) {
        const int y = y0 + tid, jj = min(y / cc, kDcKeys - 1), c = y - jj * cc, id = __shfl_sync(kFull, ids, jj);
        if (y >= kDcKeys * cc) continue;
        const size_t at = id < 0 ? 0 : (((size_t)id * p.Hkv + g) * P + (slot0 + jj) % P) * r + c * E;
        cp_async16_zfill(dst + jj * CP + c * 16, cl + at, id >= 0);
      }
    } else {  // rows that are no multiple of 16 bytes
      for (int y0 = 0; y0 < kDcKeys * r; y0 += kDcThreads) {
        const int y = y0 + tid, jj = min(y / r, kDcKeys - 1), c = y - jj * r, id = __shfl_sync(kFull, ids, jj);
        if (y >= kDcKeys * r) continue;
        T v{};
        if (id >= 0) v = cl[(((size_t)id * p.Hkv + g) * P + (slot0 + jj) % P) * r + c];
        *reinterpret_cast<T*>(dst + jj * CP + c * sizeof(T)) = v;
      }
    }
  };

  int ids = page_of(lo), next = page_of(lo + 1);
  copy(lo, ids);
  cp_async_commit_group();
  for (int x = tid; x < rows * D; x += kDcThreads) {
    const int row = row0 + x / D;
    sQ[x] = Elem<T>::to_f(q[(((size_t)b * p.n_new + row / p.G) * p.Hq + (size_t)g * p.G + row % p.G) * D + x % D]);
  }
  float m[RW], l[RW], acc[RW][CU], slope[RW];
#pragma unroll
  for (int y = 0; y < RW; ++y) {
    m[y] = -INFINITY;
    l[y] = 0.f;
#pragma unroll
    for (int k = 0; k < CU; ++k) acc[y][k] = 0.f;
    const int row = row0 + warp * RW + y;
    slope[y] = p.slopes ? p.slopes[g * p.G + row % p.G] * kLog2e : 0.f;
  }

  for (int x = lo; x < hi; ++x) {
    const bool have = ids >= 0;
    const int after = page_of(x + 2);
    copy(x + 1, next);
    cp_async_commit_group();
    ids = next;
    next = after;
    cp_async_wait_group<1>();
    __syncthreads();
    const int j = kt.tile(x) * kDcKeys + lane;
    const unsigned char* sK = sKC + (size_t)((x - lo) & 1) * stage;
    const unsigned char* sC = sK + kDcKeys * KP;
    if (warp * RW < rows) {
      float s[RW];
#pragma unroll
      for (int y = 0; y < RW; ++y) s[y] = 0.f;
#pragma unroll 4
      for (int c = 0; c < KC; ++c) {
        const uint4 w = *reinterpret_cast<const uint4*>(sK + lane * KP + c * 16);
        float kv[E];
        if constexpr (sizeof(T) == 4) {
          kv[0] = __uint_as_float(w.x);
          kv[1] = __uint_as_float(w.y);
          kv[2] = __uint_as_float(w.z);
          kv[3] = __uint_as_float(w.w);
        } else {
          kv[0] = bf16lo(w.x);
          kv[1] = bf16hi(w.x);
          kv[2] = bf16lo(w.y);
          kv[3] = bf16hi(w.y);
          kv[4] = bf16lo(w.z);
          kv[5] = bf16hi(w.z);
          kv[6] = bf16lo(w.w);
          kv[7] = bf16hi(w.w);
        }
#pragma unroll
        for (int y = 0; y < RW; ++y)
#pragma unroll
          for (int e = 0; e < E; e += 4) {
            const float4 qv = *reinterpret_cast<const float4*>(sQ + (warp * RW + y) * D + c * E + e);
            s[y] = fmaf(qv.x, kv[e], fmaf(qv.y, kv[e + 1], fmaf(qv.z, kv[e + 2], fmaf(qv.w, kv[e + 3], s[y]))));
          }
      }
#pragma unroll
      for (int y = 0; y < RW; ++y) {
        const int row = row0 + warp * RW + y, i = pos0 + row / p.G;
        float v = -INFINITY;
        if (have && warp * RW + y < rows && sees(i, j, sq.L, p.window, sq.prefix))
          v = mod_score(s[y], p.scale, p.cap, slope[y], i, j);
        const float mn = fmaxf(m[y], warp_max(v));
        float w = v != v ? v : 0.f, corr = 1.f;  // a row of nothing but NaN keeps a maximum of -inf
        if (mn != -INFINITY) {
          w = ex2(v - mn);
          corr = ex2(m[y] - mn);
        }
        m[y] = mn;
        l[y] = l[y] * corr + w;
        s_w[warp * RW + y][lane] = w;
#pragma unroll
        for (int k = 0; k < CU; ++k) acc[y][k] *= corr;
      }
      __syncwarp();
#pragma unroll 2
      for (int jj = 0; jj < kDcKeys; jj += 4) {
        float c[4][CU];
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int k = 0; k < CU; ++k)
            c[u][k] = lane + 32 * k < r
                ? Elem<T>::to_f(*reinterpret_cast<const T*>(sC + (jj + u) * CP + (lane + 32 * k) * sizeof(T))) : 0.f;
#pragma unroll
        for (int y = 0; y < RW; ++y) {
          const float4 w = *reinterpret_cast<const float4*>(&s_w[warp * RW + y][jj]);
#pragma unroll
          for (int k = 0; k < CU; ++k)
            acc[y][k] = fmaf(w.x, c[0][k], fmaf(w.y, c[1][k], fmaf(w.z, c[2][k], fmaf(w.w, c[3][k], acc[y][k]))));
        }
      }
    }
    __syncthreads();  // the buffer is free for the tile after the next
  }
  cp_async_wait_group<0>();

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
      for (int k = 0; k < CU; ++k)
        if (lane + 32 * k < r) out[2 + lane + 32 * k] = acc[y][k];
    } else {
      const size_t at = ((size_t)b * p.n_new + row / p.G) * p.Hq + (size_t)g * p.G + row % p.G;
#pragma unroll
      for (int k = 0; k < CU; ++k)
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

// rows of a tile: a decode step's few (a row or two per warp), or 32
static int core_rows(int rows) { return rows <= 4 ? 4 : rows <= 8 ? 8 : 32; }

// Splits: enough CTAs for two on every SM, each with at least 2 key tiles of a
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
  pl.splits = (int)std::max(1LL, std::min({2LL * num_sms / units, key_tiles / 2, 256LL}));
  pl.part_off = pl.bytes = dense_counter_bytes(num_sms);
  if (pl.splits > 1) pl.bytes += ((size_t)units * pl.splits * pl.row_tile * (r + 2) * 4 + 255) & ~(size_t)255;
  return pl;
}

template <typename T, int D, int RT, int CU>
static cudaError_t launch_core_t(const DenseParams& p, cudaStream_t st) {
  const size_t smem = (size_t)RT * (D + kDcKeys) * sizeof(float) + 2 * (size_t)dc_stage<T, D>(p.r);
  // (the limit without an attribute counts static shared memory too)
  cudaError_t e = ensure_smem((const void*)dense_attn_kernel<T, D, RT, CU>, smem + 1024);
  if (e != cudaSuccess) return e;
  const int tiles = (p.n_new * p.G + RT - 1) / RT;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles * p.splits, p.Hkv, p.batch);
  cfg.blockDim = dim3(kDcThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, dense_attn_kernel<T, D, RT, CU>, p);
}

template <typename T, int D, int RT>
static cudaError_t launch_core_r(const DenseParams& p, cudaStream_t st) {
  if (p.r <= 32) return launch_core_t<T, D, RT, 1>(p, st);
  if (p.r <= 64) return launch_core_t<T, D, RT, 2>(p, st);
  if constexpr (D > 64) return p.r <= 96 ? launch_core_t<T, D, RT, 3>(p, st) : launch_core_t<T, D, RT, 4>(p, st);
  return cudaErrorInvalidValue;  // the rank is at most the head's width
}

template <typename T, int D>
static cudaError_t launch_core(const DenseParams& p, int row_tile, cudaStream_t st) {
  return row_tile == 4 ? launch_core_r<T, D, 4>(p, st)
       : row_tile == 8 ? launch_core_r<T, D, 8>(p, st) : launch_core_r<T, D, 32>(p, st);
}

cudaError_t launch_dense_attn(const DensePlan& pl, DenseParams p, bool bf16, void* scratch, cudaStream_t st) {
  p.cnt = static_cast<int32_t*>(scratch);
  p.part = reinterpret_cast<float*>(static_cast<char*>(scratch) + pl.part_off);
  p.splits = pl.splits;
  if (pl.row_tile == 0) return launch_dense_mma(p, st);
  if (pl.row_tile < 0) return launch_dense_tc(p, st);
  if (bf16)
    return p.d == 128 ? launch_core<__nv_bfloat16, 128>(p, pl.row_tile, st)
                      : launch_core<__nv_bfloat16, 64>(p, pl.row_tile, st);
  return p.d == 128 ? launch_core<float, 128>(p, pl.row_tile, st) : launch_core<float, 64>(p, pl.row_tile, st);
}

}  // namespace bkv
