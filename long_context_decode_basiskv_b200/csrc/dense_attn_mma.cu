// Attention of a few new tokens over the whole paged cache (bf16, swizzled
// rows): up to 16 rows (new tokens x heads of a KV head), the decode step.
//
// HBM-bound: at 4 heads per KV head there are 16 flops to a byte of K and C, so
// the kernel is a stream of the cache with the arithmetic beside it.  The
// 16-token tiles of every (sequence, KV head), those its rows see, are laid end
// to end and cut into equal runs, one per warp: no CTA or SM has more bytes
// than another, whatever the lengths, and a warp needs nothing from its
// neighbours until its run ends.  Each warp streams its run through a private
// ring of 1-D bulk copies (a tile of K and of C is contiguous in its page) and
// works a tile on the tensor cores, the few rows as the N of mma.sync m16n8k16
// (8 of them; tcgen05's shapes would be mostly padding): S^T = K Q^T, running
// maximum and sum, O^T += C^T P^T, the weights turned by movmatrix between the
// two.  The fp32 weights enter the second product as three bf16 terms (24
// mantissa bits: o_lat is fp32), for MMAs that the stream hides.  A row's
// reference is its maximum at the last tile where some score passed it by more
// than 2^8: most tiles need no reduction across the lanes and no rescaling.
//
// Measured (bf16, d 128, rank 64, 8 KV heads, 4 heads each): 131 us for 8
// sequences of 32 k (805 MB, 6.1 TB/s), 139 us for 64 ragged ones with a window
// and capped scores (806 MB, 5.8 TB/s); 3 and 4 tokens of 8 sequences of 16 k, 12
// and 16 rows, 82 and 84 us (403 MB).  With the rows as M (half of it padding)
// the first took 133 us and 138 us against 136 in a loop of calls; at 16 rows,
// where nothing is padding, that layout is 4% the faster one (ranks 48 to 96
// spill in both, at the 128 registers of two CTAs an SM).  Six warps a CTA, for
// more registers and a deeper ring, cost a single sequence of 8 k 20 us instead
// of 14: its runs no longer end where the sequence's heads do.
//
// Where a run ends inside a sequence, the warp leaves (max, sum, acc) in its
// slot: run w and group g meet in slot w + g, since along the tiles each step
// from one piece to the next raises one of the two.  A CTA joins its warps'
// pieces of a group, and the last CTA of a group the CTAs' pieces (counters;
// the order of the sums is fixed, so the result is reproducible).
#include <algorithm>

#include "dense_attn.cuh"
#include "kernels.cuh"

namespace bkv {

constexpr int kDmTile = 16;   // tokens per tile
constexpr int kDmWarps = 8;
constexpr float kDmRaise = 8.f;  // how far (log2) a score may pass its row's reference before that is raised

constexpr uint32_t dm_stage(int d, int r) { return ((uint32_t)kDmTile * (d + r) * 2 + 127u) & ~127u; }
// ring depth with `ctas` CTAs on an SM (its 228 KB, less 1 KB reserved and the barriers for each), at most 4
constexpr int dm_fit(int d, int r, int ctas) {
  const int fit = (int)((228 * 1024 / ctas - 1024 - 512) / (kDmWarps * dm_stage(d, r)));
  return fit > 4 ? 4 : fit;
}
// two CTAs on an SM where each holds two tiles per warp
constexpr int dm_ctas(int d, int r) { return dm_fit(d, r, 2) >= 2 ? 2 : 1; }
constexpr int dm_slots(int d, int r) { return dm_fit(d, r, dm_ctas(d, r)); }

__device__ __forceinline__ void dm_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void dm_ldsm(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void dm_ldsm_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
// an 8 x 8 matrix of b16, two neighbouring elements of a row to a lane, transposed
__device__ __forceinline__ uint32_t dm_transpose(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t dm_pack(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// two fp32 values as a bf16 pair, what it leaves of them as another, and what that leaves as a third: 24 bits
__device__ __forceinline__ void dm_split(float a, float b, uint32_t& x, uint32_t& y, uint32_t& z) {
  x = dm_pack(a, b);
  a -= bf16lo(x);
  b -= bf16hi(x);
  y = dm_pack(a, b);
  z = dm_pack(a - bf16lo(y), b - bf16hi(y));
}

// One sequence's rows and the tiles they see.
struct DmSeq {
  int L, prefix, pos0;
  KeyTiles kt;
};
__device__ __forceinline__ DmSeq dm_seq(const DenseParams& p, int b, bool report) {
  const DenseSeq s = dense_seq(p, b, report);
  DmSeq q{s.L, s.prefix, s.L - p.n_new, {0, 0, 0}};
  if (s.L > 0) q.kt = key_tiles(q.pos0, s.L - 1, s.L, p.window, s.prefix, kDmTile);
  return q;
}

// A place in the laid-out tiles: tile x of group (b, g).
struct DmCursor {
  int b, g, x, n;  // n: tiles of the group
  DmSeq s;
  __device__ __forceinline__ void set(const DenseParams& p, int b_) {
    b = b_;
    s = dm_seq(p, b, false);
    n = s.kt.count();
  }
  // the next group; only called while tiles are left, so there is one
  __device__ __forceinline__ void next_group(const DenseParams& p) {
    x = 0;
    if (++g < p.Hkv) return;
    g = 0;
    do set(p, b + 1);
    while (n == 0);
  }
};

template <int D, int NT, bool ROWS16>
__global__ void __launch_bounds__(32 * kDmWarps, dm_ctas(D, NT * 8)) dense_mma_kernel(DenseParams p) {
  constexpr int KS = D / 16, R = NT * 8, SW = dm_slots(D, R);
  constexpr uint32_t k_bytes = kDmTile * D * 2, c_bytes = kDmTile * R * 2, stage_bytes = dm_stage(D, R);
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int meta_all[kDmWarps][SW];
  __shared__ int warp_tot[32];
  __shared__ int s_start[kDmWarps + 1][2];  // sequence of each warp's first tile, tiles before it
  __shared__ int s_last, s_fail;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int rows = p.n_new * p.G;
  unsigned char* ring = smem + (size_t)w * SW * stage_bytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + (size_t)kDmWarps * SW * stage_bytes) + w * SW;
  int* meta = meta_all[w];
  if (lane == 0) {
    for (int s = 0; s < SW; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
  }
  if (tid == 0) s_fail = 0;
  if (tid < 2 * (kDmWarps + 1)) (&s_start[0][0])[tid] = 0;
  __syncthreads();
  grid_dep_wait();     // the append may still be running when this grid starts
  allow_dependents();  // the out-projection may start and stage its weights

  // the tiles of every sequence: total, and where this CTA's warps start
  const int per_thr = (p.batch + blockDim.x - 1) / blockDim.x;
  const int b0 = min(p.batch, tid * per_thr), b1 = min(p.batch, b0 + per_thr);
  int mine = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = dm_seq(p, b, blockIdx.x == 0).kt.count();
    mine += n;
  }
  // sequences with nothing to see: zeros, written by the CTAs in turn
  for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
    if (dm_seq(p, b, false).kt.count() != 0) continue;
    const size_t at = (size_t)b * p.n_new * p.Hq;
    for (int x = tid; x < p.n_new * p.Hq * R; x += blockDim.x) p.o[at * R + x] = 0.f;
    if (p.lse)
      for (int x = tid; x < p.n_new * p.Hq; x += blockDim.x) p.lse[at + x] = -INFINITY;
  }
  int total;
  int before = block_exclusive_scan(mine, warp_tot, total);
  // runs of the laid-out tiles (64 bits: 65535 sequences of 3 M tokens times heads)
  const long long T = (long long)total * p.Hkv;
  const long long per = (T + (long long)gridDim.x * kDmWarps - 1) / ((long long)gridDim.x * kDmWarps);
  const long long cta_lo = min(T, per * kDmWarps * blockIdx.x), cta_hi = min(T, cta_lo + per * kDmWarps);
  if (cta_lo >= cta_hi) return;
  for (int b = b0; b < b1; ++b) {
    const int n = dm_seq(p, b, false).kt.count();
    const long long a = (long long)before * p.Hkv, e = a + (long long)n * p.Hkv;
    if (a < cta_hi && e > cta_lo)
      for (int y = 0; y < kDmWarps; ++y) {
        const long long lo = cta_lo + y * per;
        if (lo >= a && lo < e) {
          s_start[y][0] = b;
          s_start[y][1] = before;
        }
      }
    before += n;
  }
  __syncthreads();
  const long long lo = min(cta_hi, cta_lo + w * per), hi = min(cta_hi, lo + per);
  const int tiles = (int)(hi - lo);

  const __nv_bfloat16* kbase = static_cast<const __nv_bfloat16*>(p.k_raw);
  const __nv_bfloat16* cbase = static_cast<const __nv_bfloat16*>(p.c_lat);
  const uint64_t pol = l2_evict_first();
  const int gr = lane >> 2, tq = lane & 3;
  const int mi = lane >> 3, rr = lane & 7;
  constexpr int mk = 7;
  const int mc = swz_mask(R);
  bool ok = true;
  int issued = 0, consumed = 0;

  if (tiles > 0) {
    DmCursor in, out;  // where copies are issued, where tiles are consumed
    out.set(p, s_start[w][0]);
    {
      const long long off = lo - (long long)s_start[w][1] * p.Hkv;
      out.g = (int)(off / out.n);
      out.x = (int)(off - (long long)out.g * out.n);
    }
    in = out;
    // physical pages of the next tiles of one group, lane j's tile batch_x + j;
    // -1: not to be read
    int page_of_lane = -1, batch_n = 0, batch_at = 0;
    auto load_batch = [&]() {
      if (in.x == in.n) in.next_group(p);
      batch_n = min(32, min(in.n - in.x, tiles - issued));
      batch_at = 0;
      page_of_lane = -1;
      if (lane < batch_n) page_of_lane = dense_page(p, in.b, in.s.kt.tile(in.x + lane) * kDmTile / p.page);
    };
    auto issue = [&]() {
      if (batch_at == batch_n) load_batch();
      const int id = __shfl_sync(kFull, page_of_lane, batch_at);
      if (lane == 0) {
        const int s = issued % SW;
        meta[s] = id;
        unsigned char* st = ring + (size_t)s * stage_bytes;
        fence_proxy_async_smem();
        if (id >= 0) {
          const int slot = in.s.kt.tile(in.x) * kDmTile % p.page;
          const size_t row0 = ((size_t)id * p.Hkv + in.g) * p.page + slot;
          mbar_arrive_expect_tx(&full[s], k_bytes + c_bytes);
          bulk_g2s_hint(st, kbase + row0 * D, k_bytes, &full[s], pol);
          bulk_g2s_hint(st + k_bytes, cbase + row0 * R, c_bytes, &full[s], pol);
        } else {
          mbar_arrive_expect_tx(&full[s], 0);
        }
      }
      ++batch_at;
      ++in.x;
      ++issued;
    };
    while (issued < SW && issued < tiles) issue();

    while (consumed < tiles && ok) {
      if (out.x == out.n) out.next_group(p);
      const int first = out.x, last = (int)min((long long)out.n, (long long)first + (tiles - consumed));
      // this piece's queries (B operand, rows as its columns), and per row of this lane (2 tq, 2 tq + 1 of
      // each block of 8) the score's slope and the state
      constexpr int RB = ROWS16 ? 2 : 1;
      uint32_t qb[KS][RB][2];
      float slope[RB][2], m[RB][2], l[RB][2];
      int pos[RB][2];
      bool on[RB][2];
#pragma unroll
      for (int y = 0; y < RB; ++y) {
        const int row = gr + 8 * y, t = row < rows ? row / p.G : 0, h = out.g * p.G + (row < rows ? row - t * p.G : 0);
        const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(p.q) + (((size_t)out.b * p.n_new + t) * p.Hq + h) * D;
#pragma unroll
        for (int s2 = 0; s2 < KS; ++s2)
#pragma unroll
          for (int u = 0; u < 2; ++u)
            qb[s2][y][u] = row < rows ? *reinterpret_cast<const uint32_t*>(qr + 16 * s2 + 8 * u + 2 * tq) : 0u;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r2 = 8 * y + 2 * tq + e;
          on[y][e] = r2 < rows;
          const int t2 = on[y][e] ? r2 / p.G : 0, h2 = out.g * p.G + (on[y][e] ? r2 - t2 * p.G : 0);
          pos[y][e] = out.s.pos0 + t2;
          slope[y][e] = p.slopes ? p.slopes[h2] * kLog2e : 0.f;
          m[y][e] = -INFINITY;
          l[y][e] = 0.f;
        }
      }
      float acc[R / 16][RB][4];  // latents 16 i + gr (elements 0, 1: the lane's rows) and + 8 (2, 3)
#pragma unroll
      for (int i = 0; i < R / 16; ++i)
#pragma unroll
        for (int y = 0; y < RB; ++y) acc[i][y][0] = acc[i][y][1] = acc[i][y][2] = acc[i][y][3] = 0.f;
      const bool mod = p.cap > 0.f || p.slopes;

      for (; out.x < last; ++out.x) {
        const int s = consumed % SW;
        if (!__all_sync(kFull, mbar_wait_bounded(&full[s], (uint32_t)((consumed / SW) & 1)))) {
          ok = false;
          break;
        }
        if (meta[s] >= 0) {
          unsigned char* st = ring + (size_t)s * stage_bytes;
          const uint32_t kaddr = smem_u32(st), caddr = smem_u32(st + k_bytes);
          const int j0 = out.s.kt.tile(out.x) * kDmTile;
          // seen whole by every row?
          const bool whole = j0 + kDmTile <= out.s.prefix ||
              (j0 + kDmTile - 1 <= out.s.pos0 && (p.window == 0 || out.s.L - 1 - j0 < p.window));
          if (!whole) {
            // tokens that no row sees: their latents, which may be anything, become zero
            const int seen_lo = p.window > 0 ? out.s.pos0 - p.window + 1 : 0;
            for (int y = lane; y < kDmTile * R / 8; y += 32) {
              const int j = j0 + y / (R / 8);
              if (j >= out.s.L || (j < seen_lo && j >= out.s.prefix))
                reinterpret_cast<uint4*>(st + k_bytes)[y] = make_uint4(0u, 0u, 0u, 0u);
            }
            __syncwarp();
          }
          float sc[2][RB][4];  // [chain][row block][fragment: tokens gr, gr + 8 by the lane's rows]
#pragma unroll
          for (int y = 0; y < 8 * RB; ++y) (&sc[0][0][0])[y] = 0.f;
          {
            const int tok = (mi & 1) * 8 + rr;
            const uint32_t rowaddr = kaddr + (uint32_t)(tok * D * 2);
#pragma unroll
            for (int s2 = 0; s2 < KS; ++s2) {
              uint32_t ka[4];
              dm_ldsm(ka, rowaddr + (uint32_t)(((2 * s2 + (mi >> 1)) ^ (tok & mk)) << 4));
#pragma unroll
              for (int y = 0; y < RB; ++y) dm_mma(sc[s2 & 1][y], ka[0], ka[1], ka[2], ka[3], qb[s2][y][0], qb[s2][y][1]);
            }
          }
          // the scores; does one lie more than 2^kDmRaise above its row's reference?
          auto each_score = [&](auto f) {  // f(score, its row's block and number in it, its token)
#pragma unroll
            for (int y = 0; y < RB; ++y)
#pragma unroll
              for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int u = 0; u < 2; ++u) f(sc[0][y][2 * u + e], y, e, j0 + 8 * u + gr);
          };
#pragma unroll
          for (int y = 0; y < RB; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[0][y][e] += sc[1][y][e];
          if (mod)
            each_score([&](float& v, int y, int e, int j) { v = mod_score(v, p.scale, p.cap, slope[y][e], pos[y][e], j); });
          else
            each_score([&](float& v, int, int, int) { v *= p.scale; });
          if (!whole)
            each_score([&](float& v, int y, int e, int j) {
              if (!sees(pos[y][e], j, out.s.L, p.window, out.s.prefix)) v = -INFINITY;
            });
          bool above = false;
          each_score([&](float& v, int y, int e, int) { above |= v > m[y][e] + kDmRaise; });
          if (__any_sync(kFull, above)) {  // the references become the maxima so far, and the sums follow
#pragma unroll
            for (int y = 0; y < RB; ++y) {
              float corr[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float mx = fmaxf(sc[0][y][e], sc[0][y][2 + e]);
                mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 16));
                mx = fmaxf(m[y][e], mx);
                corr[e] = mx == -INFINITY ? 1.f : ex2(m[y][e] - mx);
                m[y][e] = mx;
                l[y][e] *= corr[e];
              }
#pragma unroll
              for (int i = 0; i < R / 16; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][y][e] *= corr[e & 1];
            }
          }
          uint32_t pw[3][RB][2];  // [term][row block][8 tokens]: weights as B operand
#pragma unroll
          for (int y = 0; y < RB; ++y) {
            float pr[2][2];  // [token gr, gr + 8][row]
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const bool none = m[y][e] == -INFINITY;  // nothing seen, or nothing but NaN
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const float v = sc[0][y][2 * u + e];
                pr[u][e] = none ? (v != v ? v : 0.f) : ex2(v - m[y][e]);
              }
              l[y][e] += pr[0][e] + pr[1][e];
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              uint32_t w[3];
              dm_split(pr[u][0], pr[u][1], w[0], w[1], w[2]);
#pragma unroll
              for (int z = 0; z < 3; ++z) pw[z][y][u] = dm_transpose(w[z]);
            }
          }
          {
            const int tok = (mi >> 1) * 8 + rr;
            const uint32_t rowaddr = caddr + (uint32_t)(tok * R * 2);
#pragma unroll
            for (int i = 0; i < R / 16; ++i) {
              uint32_t ca[4];
              dm_ldsm_t(ca, rowaddr + (uint32_t)(((2 * i + (mi & 1)) ^ (tok & mc)) << 4));
#pragma unroll
              for (int y = 0; y < RB; ++y) {
                // the tile's products on their own, then added in fp32: tensor cores cut off what they add
                // up, which over a long run's tiles would cost more than the three terms keep
                float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int z = 0; z < 3; ++z) dm_mma(t, ca[0], ca[1], ca[2], ca[3], pw[z][y][0], pw[z][y][1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][y][e] += t[e];
              }
            }
          }
        }
        __syncwarp();  // every lane is done with the slot
        ++consumed;
        if (issued < tiles) issue();
      }

      // the piece's result: final where the piece is the whole group, else this run's slot
      const bool whole_group = first == 0 && last == out.n;
#pragma unroll
      for (int y = 0; y < RB; ++y) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float ls = l[y][e];
          ls += __shfl_xor_sync(kFull, ls, 4);
          ls += __shfl_xor_sync(kFull, ls, 8);
          ls += __shfl_xor_sync(kFull, ls, 16);
          if (!on[y][e] || !ok) continue;
          const int row = 8 * y + 2 * tq + e;
          if (whole_group) {
            const int t = row / p.G, h = out.g * p.G + row - t * p.G;
            const size_t at = ((size_t)out.b * p.n_new + t) * p.Hq + h;
#pragma unroll
            for (int i = 0; i < R / 16; ++i)
#pragma unroll
              for (int u = 0; u < 2; ++u)
                p.o[at * R + 16 * i + 8 * u + gr] = ls > 0.f ? acc[i][y][2 * u + e] / ls : (ls == ls ? 0.f : ls);
            if (p.lse && gr == 0) p.lse[at] = ls > 0.f ? (m[y][e] + log2f(ls)) * kLn2 : (ls == ls ? -INFINITY : ls);
          } else {
            const size_t slot = (size_t)blockIdx.x * kDmWarps + w + (size_t)out.b * p.Hkv + out.g;
            float* o = p.part + (slot * rows + row) * (R + 2);
            if (gr == 0) *reinterpret_cast<float2*>(o) = make_float2(m[y][e], ls);
#pragma unroll
            for (int i = 0; i < R / 16; ++i)
#pragma unroll
              for (int u = 0; u < 2; ++u) o[2 + 16 * i + 8 * u + gr] = acc[i][y][2 * u + e];
          }
        }
      }
    }
    if (!ok && lane == 0) {
      // a wait gave up: let the copies still in flight land before the ring is released
      s_fail = 1;
      set_err(p.err, BASISKV_DEVERR_TIMEOUT);
      for (int t = consumed; t < issued; ++t) mbar_wait_bounded(&full[t % SW], (uint32_t)((t / SW) & 1));
    }
  }
  __syncthreads();  // every warp's pieces are written

  // join the pieces: of this CTA's warps, then of the CTAs
  const size_t pstride = (size_t)rows * (R + 2);
  const long long nw = (long long)gridDim.x * kDmWarps;
  float* cta_part = p.part + (size_t)(nw + (long long)p.batch * p.Hkv) * pstride;
  DmCursor c;
  c.set(p, s_start[0][0]);
  const long long off = cta_lo - (long long)s_start[0][1] * p.Hkv;
  c.g = (int)(off / c.n);
  c.x = 0;
  for (long long a = (long long)s_start[0][1] * p.Hkv + (long long)c.g * c.n; a < cta_hi;) {
    const long long e = a + c.n;
    const long long slot = (long long)c.b * p.Hkv + c.g;
    const int w0 = (int)((max(a, cta_lo) - cta_lo) / per), w1 = (int)((min(e, cta_hi) - 1 - cta_lo) / per);
    const bool spans = a < cta_lo || e > cta_hi;  // other CTAs hold pieces too
    auto out_at = [&](int row) {
      const int t = row / p.G;
      return ((size_t)c.b * p.n_new + t) * p.Hq + (size_t)c.g * p.G + row - t * p.G;
    };
    if (spans || w1 > w0) {
      for (int row = w; row < rows; row += kDmWarps) {
        const float* from = p.part + (size_t)((long long)blockIdx.x * kDmWarps + w0 + slot) * pstride + (size_t)row * (R + 2);
        if (spans) {
          float* to = cta_part + (size_t)((long long)blockIdx.x + slot) * pstride + (size_t)row * (R + 2);
          dense_fold_row(from, pstride, w1 - w0 + 1, R, to, s_fail != 0, lane);
        } else {
          const size_t at = out_at(row);
          dense_join_row(from, pstride, w1 - w0 + 1, R, p.o + at * R, p.lse ? p.lse + at : nullptr, lane, s_fail != 0);
        }
      }
    }
    if (spans) {
      const long long per_cta = per * kDmWarps;
      const int c0 = (int)(a / per_cta), c1 = (int)((e - 1) / per_cta);
      // the counter of its first CTA, of which it is the last group: no other group counts there
      if (dense_last_split(p.cnt + c0, c1 - c0 + 1, p.err, &s_last)) {
        for (int row = w; row < rows; row += kDmWarps) {
          const size_t at = out_at(row);
          dense_join_row(cta_part + (size_t)(c0 + slot) * pstride + (size_t)row * (R + 2), pstride, c1 - c0 + 1, R,
                         p.o + at * R, p.lse ? p.lse + at : nullptr, lane, false);
        }
      }
      __syncthreads();  // s_last is free again
    }
    a = e;
    if (a < cta_hi) c.next_group(p);
  }
}

static long long dm_grid(int batch, int Hkv, int d, int r, int page, int max_pages, int num_sms) {
  const long long most = (long long)batch * Hkv * ((long long)max_pages * page / kDmTile);
  return std::max(1LL, std::min((long long)dm_ctas(d, r) * num_sms, most / kDmWarps));
}

void dense_plan_mma(DensePlan* pl, int batch, int rows, int Hkv, int d, int r, int page, int max_pages, int num_sms) {
  const long long groups = (long long)batch * Hkv, grid = dm_grid(batch, Hkv, d, r, page, max_pages, num_sms);
  pl->splits = (int)grid;
  const size_t slots = (size_t)(grid * kDmWarps + groups) + (size_t)(grid + groups);
  pl->part_off = dense_counter_bytes(num_sms);
  pl->bytes = pl->part_off + ((slots * rows * (r + 2) * 4 + 255) & ~(size_t)255);
}

template <int D, int NT, bool ROWS16>
static cudaError_t launch_dm(const DenseParams& p, cudaStream_t st) {
  constexpr int SW = dm_slots(D, NT * 8);
  static_assert(SW >= 2, "a ring of at least two tiles");
  constexpr size_t smem = (size_t)kDmWarps * SW * (dm_stage(D, NT * 8) + 8);
  cudaError_t e = ensure_smem((const void*)dense_mma_kernel<D, NT, ROWS16>, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.splits);
  cfg.blockDim = dim3(32 * kDmWarps);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, dense_mma_kernel<D, NT, ROWS16>, p);
}

template <int D, int NT>
static cudaError_t launch_dm_rows(const DenseParams& p, cudaStream_t st) {
  return p.n_new * p.G <= 8 ? launch_dm<D, NT, false>(p, st) : launch_dm<D, NT, true>(p, st);
}

template <int D>
static cudaError_t launch_dm_r(const DenseParams& p, cudaStream_t st) {
  switch (p.r / 16) {
    case 1: return launch_dm_rows<D, 2>(p, st);
    case 2: return launch_dm_rows<D, 4>(p, st);
    case 3: return launch_dm_rows<D, 6>(p, st);
    case 4: return launch_dm_rows<D, 8>(p, st);
    default: break;
  }
  if constexpr (D == 128) {  // the rank is at most the head's width
    switch (p.r / 16) {
      case 5: return launch_dm_rows<D, 10>(p, st);
      case 6: return launch_dm_rows<D, 12>(p, st);
      case 7: return launch_dm_rows<D, 14>(p, st);
      case 8: return launch_dm_rows<D, 16>(p, st);
      default: break;
    }
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_dense_mma(const DenseParams& p, cudaStream_t st) {
  return p.d == 128 ? launch_dm_r<128>(p, st) : launch_dm_r<64>(p, st);
}

}  // namespace bkv
