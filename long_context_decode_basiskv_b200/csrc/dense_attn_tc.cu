// Attention of many new tokens over the whole paged cache (bf16, swizzled
// rows) on the tcgen05 tensor cores: prompts, chunks of them, and the few
// tokens that dense_attn_mma.cu has too few rows for.
//
// One CTA per (256 rows, KV head, sequence, share of the keys): rows are
// consecutive new tokens' G heads of the KV head, in tiles of M = 128.  Per row
// tile and tile of 128 keys
//
//   S [128 x 128] = Q [128 x d] . K^T          operands in shared memory, S in tensor memory
//   P = 2^(S c - m), m the running row maximum   a thread owns a row: no shuffles
//   O [128 x r]   = P [128 x 128] . C            P in tensor memory (over S), C in shared memory
//
// The products of four key tiles add up in tensor memory; then the thread adds
// O to its row's fp32 accumulators.  Tensor cores cut off what they add up, an
// error that over 64 MMAs stays near fp32's own (2.4e-6 of the result over 8192
// keys, 2.8e-6 over 16384) and over a whole context would not; each tile by
// itself cost 631 us where four together cost 621.  P, fp32, is multiplied as
// two bf16 terms (hi + lo, 16 mantissa bits), like every chained product of
// this library: o_lat is fp32 and the out-projection takes it so.
//
// m is a reference, not always the maximum: any value keeps the result as long
// as the weights stay in range, so it is raised only when a tile's sums show
// that it is too low, and O is then rescaled.
//
// Two softmax warpgroups, each with its own O, and S tiles (with P over them)
// that they take in turn: three where the rank leaves room beside the two O's
// in the 512 columns (r <= 64), so that one warpgroup's next S is under way
// while it is in its exponentials; else two.  The warpgroups take the two row
// tiles of the CTA, which then share every K and C tile; where there are at
// most 128 rows they take the even and the odd key tiles of the one row tile
// and join at the end.  Warp 8 copies K pages (and C pages where their rows are
// whole swizzle atoms, r a multiple of 64) by TMA straight from the paged cache:
// the stored row swizzle is the operand's.  Warps 9-11 copy the other C tiles
// by 16-byte cp.async: ranks that are no multiple of 64, and tiles with tokens
// that no row of the CTA sees, which become zeros so that nothing in them
// reaches a sum.  Warp 12 issues the MMAs.
//
// Bound by the softmax: a pair of 128 x 128 tiles takes about 4600 cycles, of
// which the exponentials alone are 2048 (16 a cycle) and the MMAs, beside them,
// 2112.  Measured (bf16, d 128): a prompt of 8192 tokens, 32 heads over 8, rank
// 64, 582 us (708 TFLOP/s, P C counted once: 0.43 of the measured peak; 626 once
// the power cap holds the clocks down); 1021 tokens after 15360 others, 64 heads
// over 8, rank 96, capped scores, 1241 us (378 TFLOP/s, the tanh beside the
// exponentials).  One S tile for each of the two warpgroups took 704 us for the
// first; three warpgroups of 128 rows 597, and a prompt of 2048 tokens 68 instead
// of 58.
#include <cuda.h>

#include <algorithm>

#include "dense_attn.cuh"
#include "kernels.cuh"
#include "tcgen05.cuh"

namespace bkv {

constexpr int kDtM = 128;       // rows of an MMA
constexpr int kDtRows = 256;    // rows of a CTA
constexpr int kDtKeys = 128;    // keys per tile
constexpr int kDtThreads = 512; // 4 warpgroups: softmax, softmax, copies, MMA (one warp of it)
constexpr int kDtK = 3;         // K stages
constexpr int kDtMasks = 8;     // tiles whose page bits are kept: more than the copies run ahead
constexpr int kDtDrain = 4;      // tiles whose products add up in tensor memory
constexpr float kDtAhead = 8.f;  // a reference is this far below a row's largest score at most, in a masked or modified
constexpr float kDtMost = 65536.f; // tile; and the sum of 32 weights of a tile seen whole is at most this
constexpr uint32_t kDtAtom = kDtKeys * 128;  // 128 rows x 128 bytes

// C stages, and registers of a softmax thread: 512 x 128 at launch = 256 x softmax + 256 x (256 - softmax)
template <int RMAX> constexpr int dt_cstages() { return RMAX <= 64 ? 3 : 2; }
template <int RMAX> constexpr int dt_regs() { return RMAX <= 64 ? 208 : RMAX <= 96 ? 216 : 224; }

struct DtLayout {
  uint32_t q, k, c, bar, total;
};
template <int D, int RMAX>
__host__ __device__ constexpr DtLayout dt_layout() {
  DtLayout l{};
  uint32_t o = 0;
  l.q = o; o += 2 * (D / 64) * kDtAtom;
  l.k = o; o += kDtK * (D / 64) * kDtAtom;
  l.c = o; o += dt_cstages<RMAX>() * ((RMAX + 63) / 64) * kDtAtom;
  l.bar = o; o += 256;
  l.total = o;
  return l;
}

// ---------------------------------------------------------------------------
// tensor cores and tensor memory
// ---------------------------------------------------------------------------
// Issued by a whole warp, for which `leader` is set in one lane: the warp stays converged, so that the
// descriptors are formed in uniform registers (inside a one-lane branch each MMA took 70 to 100 cycles to issue).
__device__ __forceinline__ uint32_t elect_leader() {
  uint32_t x;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(x));
  return x;
}
__device__ __forceinline__ void dt_mma_ss(uint32_t leader, uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                          bool accum) {
  asm volatile("{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
               "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem), "l"(a), "l"(b),
               "r"(idesc), "r"((uint32_t)accum), "r"(leader) : "memory");
}
__device__ __forceinline__ void dt_mma_ts(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                          bool accum) {
  asm volatile("{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
               "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem), "r"(a_tmem), "l"(b),
               "r"(idesc), "r"((uint32_t)accum), "r"(leader) : "memory");
}
__device__ __forceinline__ void dt_commit(uint32_t leader, uint64_t* bar) {
  asm volatile("{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
               "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
               "r"(leader) : "memory");
}
__device__ __forceinline__ void tc_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tc_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// 8 columns of hi pairs and the 8 of their lo pairs, 16 columns on
__device__ __forceinline__ void tc_ld16u(uint32_t taddr, uint32_t (&r)[16]) {
#pragma unroll
  for (int h = 0; h < 16; h += 8)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[h]), "=r"(r[h + 1]), "=r"(r[h + 2]), "=r"(r[h + 3]), "=r"(r[h + 4]), "=r"(r[h + 5]),
                   "=r"(r[h + 6]), "=r"(r[h + 7])
                 : "r"(taddr + 2 * h));
}
__device__ __forceinline__ void tc_st16u(uint32_t taddr, const uint32_t (&r)[16]) {
#pragma unroll
  for (int h = 0; h < 16; h += 8)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr + 2 * h),
                 "r"(r[h]), "r"(r[h + 1]), "r"(r[h + 2]), "r"(r[h + 3]), "r"(r[h + 4]), "r"(r[h + 5]), "r"(r[h + 6]),
                 "r"(r[h + 7])
                 : "memory");
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_st16(uint32_t taddr, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
      "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// the C tile as B operand: the columns of a key contiguous (MN-major), 64 of them per swizzled 128-byte
// row, 8-key groups 1024 bytes apart, 64-column atoms kDtAtom apart
__device__ __forceinline__ uint64_t dt_cdesc(const unsigned char* base) {
  return ((smem_u32(base) >> 4) & 0x3fffull) | ((uint64_t)(kDtAtom >> 4) << 16) | (64ull << 32) | (1ull << 46) |
         (2ull << 61);
}

// a page's rows of one 64-column half -> 128-byte rows in shared memory
__device__ __forceinline__ void dt_tma(void* dst, const CUtensorMap* map, int half, int block, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(smem_u32(dst)), "l"(map), "r"(0), "r"(half), "r"(0), "r"(block), "r"(smem_u32(bar))
      : "memory");
}

// two fp32 operations in one instruction
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max32(const uint32_t (&s)[32]) {
  float a = __uint_as_float(s[0]), b = __uint_as_float(s[1]);
#pragma unroll
  for (int x = 2; x < 32; x += 4) {
    a = max3(a, __uint_as_float(s[x]), __uint_as_float(s[x + 1]));
    if (x + 2 < 32) b = max3(b, __uint_as_float(s[x + 2]), __uint_as_float(s[x + 3]));
  }
  return fmaxf(a, b);
}
// two fp32 values as a bf16 pair, and what it leaves of them as another
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  const __nv_bfloat162 l = __floats2bfloat162_rn(a - bf16lo(hi), b - bf16hi(hi));
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

// Barrier operations of a whole warp.  It waits together, the verdict a vote, so that it stays converged; and one
// lane arrives for it (32 arrivals at one barrier take their turns in shared memory).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  if (__all_sync(kFull, mbar_try_wait(bar, parity))) return true;
  const long long t0 = clock64();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (__all_sync(kFull, mbar_try_wait(bar, parity))) return true;
    if (__any_sync(kFull, clock64() - t0 > 2000000000LL)) return false;  // about a second
  }
}
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
  __syncwarp();
}

// named barrier.  0: __syncthreads; 1: the softmax warps; 2: warps 9-11 (below); 3: the CTA, before the registers
// go back to the launch count
template <int ID, int THREADS>
__device__ __forceinline__ void dt_bar() {
  asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(THREADS) : "memory");
}

// barrier of the 96 threads of warps 9-11: whether `x` holds in all of them
__device__ __forceinline__ bool all_of_96(bool x) {
  uint32_t y;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
               "barrier.cta.red.and.pred p, 2, 96, q;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(y) : "r"((uint32_t)x) : "memory");
  return y != 0;
}

// bits [lo, hi) of a 32-bit word (bounds of any size)
__device__ __forceinline__ uint32_t bit_range(int lo, int hi) {
  const uint32_t below_hi = hi >= 32 ? 0xffffffffu : hi <= 0 ? 0u : (1u << hi) - 1u;
  const uint32_t below_lo = lo >= 32 ? 0xffffffffu : lo <= 0 ? 0u : (1u << lo) - 1u;
  return below_hi & ~below_lo;
}

// MOD: scores are capped or biased
template <int D, int RMAX, bool MOD>
__global__ void __launch_bounds__(kDtThreads, 1)
    dense_tc_kernel(const __grid_constant__ DenseParams p, const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap cmap) {
  constexpr int CS = dt_cstages<RMAX>();
  constexpr int KA = D / 64, CA = (RMAX + 63) / 64;  // atoms of a K row, of a C row
  constexpr int NB = RMAX <= 64 ? 3 : 2;             // S buffers: what 512 columns hold beside two O
  constexpr uint32_t tO0 = NB * 128, tOstep = NB == 3 ? 64 : 128;
  constexpr uint32_t k_stage = KA * kDtAtom, c_stage = CA * kDtAtom;
  constexpr DtLayout lay = dt_layout<D, RMAX>();
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint32_t s_tmem;
  __shared__ int s_last;
  __shared__ uint32_t s_pages[kDtMasks];  // bit x: page x of the tile is there
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = p.r, P = p.page, psh = 31 - __clz(P), np = kDtKeys >> psh;
  unsigned char* sQ = smem + lay.q;
  uint64_t* kfull = reinterpret_cast<uint64_t*>(smem + lay.bar);
  uint64_t* kempty = kfull + kDtK;
  uint64_t* cfull = kempty + kDtK;
  uint64_t* cempty = cfull + CS;
  uint64_t* cturn = cempty + CS;   // per C stage: free, and its next tile not TMA's
  uint64_t* qfull = cturn + CS;
  uint64_t* sfull = qfull + 1;     // per S buffer: S there
  uint64_t* pfull = sfull + NB;    // per S buffer: P there, and the O that its product overwrites taken
  uint64_t* ofull = pfull + NB;    // per warpgroup: O there
  uint64_t* odone = ofull + 2;     // every product

  // this CTA's rows and keys; the last row tiles of a prompt see the most keys and start first
  const int tiles = (int)(((long long)p.n_new * p.G + kDtRows - 1) / kDtRows);
  const int split = blockIdx.x % p.splits;
  int u = blockIdx.x / p.splits;
  const int g = u % p.Hkv;
  u /= p.Hkv;
  const int b = u % p.batch, rt = tiles - 1 - u / p.batch;
  const int row0 = rt * kDtRows;  // of the sequence: n_new G < 2^25
  const int rows = min(kDtRows, p.n_new * p.G - row0);
  const bool two = rows > kDtM;   // two row tiles; else two shares of the key tiles
  const DenseSeq sq = dense_seq(p, b, tid == 0 && g == 0);
  const int pos0 = sq.L - p.n_new;
  const int t_lo = row0 / p.G, t_hi = (row0 + rows - 1) / p.G;
  KeyTiles kt{0, 0, 0};
  if (sq.L > 0) kt = key_tiles(pos0 + t_lo, pos0 + t_hi, sq.L, p.window, sq.prefix, kDtKeys);
  const int lo = (int)((long long)kt.count() * split / p.splits);
  const int n = (int)((long long)kt.count() * (split + 1) / p.splits) - lo;  // key tiles of this CTA
  // Key tiles are taken from the last to the first: the first one then has the rows' own positions, where a
  // distance bias leaves the scores highest, and its maximum serves as reference for the others.
  auto tile_at = [&](int j) { return kt.tile(lo + n - 1 - j); };
  // keys that some row of the CTA sees: [0, prefix) and [see_lo, see_hi)
  const int see_lo = p.window > 0 ? pos0 + t_lo - p.window + 1 : 0;
  const int see_hi = min(sq.L, max(pos0 + t_hi + 1, sq.prefix));

  if (tid == 0) {
    for (int s = 0; s < kDtK; ++s) {
      mbar_init(&kfull[s], 1);
      mbar_init(&kempty[s], 1);
    }
    for (int s = 0; s < CS; ++s) {
      mbar_init(&cfull[s], 1);
      mbar_init(&cempty[s], 1);
      mbar_init(&cturn[s], 1);
    }
    mbar_init(qfull, two ? 8 : 4);
    for (int x = 0; x < NB; ++x) {
      mbar_init(&sfull[x], 1);
      mbar_init(&pfull[x], 4);
    }
    mbar_init(&ofull[0], 1);
    mbar_init(&ofull[1], 1);
    mbar_init(odone, 1);
    fence_mbar_init();
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  bool ok = true;

  if (warp < 8) {
    // ------------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(dt_regs<RMAX>()));
    const int m = warp >> 2;
    const uint32_t tw = tmem + ((uint32_t)((warp & 3) * 32) << 16), tO = tw + tO0 + (uint32_t)m * tOstep;
    const int row = two ? tid : tid & 127;  // of the CTA
    const int mine = two ? n : (n + 1 - m) / 2;  // key tiles of this warpgroup
    const int srow = row0 + min(row, rows - 1);
    const int t = srow / p.G, h = g * p.G + srow - t * p.G;
    const int pos = pos0 + t;
    if (two || m == 0) {  // the row's query, as A operand
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + (((size_t)b * p.n_new + t) * p.Hq + h) * D;
      unsigned char* dst = sQ + (size_t)m * k_stage + (row & 127) * 128;
#pragma unroll
      for (int c = 0; c < D / 8; ++c)
        cp_async16_zfill(dst + (c >> 3) * kDtAtom + (((c & 7) ^ (row & 7)) << 4), q + c * 8, row < rows);
      cp_async_commit_group();
      cp_async_wait_group<0>();
      fence_proxy_async_smem();
      warp_arrive(qfull, lane);
    }
    const bool work = (row & ~31) < rows;  // this warp holds rows
    // first and last position of the warpgroup's rows
    const int m0 = two ? m * kDtM : 0;
    const int i0 = pos0 + (row0 + min(m0, rows - 1)) / p.G;
    const int i1 = pos0 + (row0 + min(m0 + kDtM - 1, rows - 1)) / p.G;
    const float slope = p.slopes ? p.slopes[h] * kLog2e : 0.f;
    const float c1 = MOD ? 1.f : p.scale;
    const uint64_t c2 = pack2(c1, c1);
    // Weights are 2^(s - ref) (log 2 units).  Any reference is right that keeps them in range, so ref is a
    // maximum that is brought up to date only when a score passes it by kDtAhead: the rescaling of l, acc
    // and O that goes with it is rare, and tiles that are seen whole need no pass for their maximum.
    float ref = -INFINITY, l = 0.f;
    float acc[RMAX];
#pragma unroll
    for (int c = 0; c < RMAX; ++c) acc[c] = 0.f;

    // acc += O
    auto add_o = [&]() {
#pragma unroll
      for (int c0 = 0; c0 < RMAX; c0 += 32) {
        if (c0 < r) {  // r is a multiple of 16: the last 16 of 32 columns may be unused
          uint32_t o[32];
          tc_ld32(tO + (uint32_t)c0, o);
          tc_wait_ld();
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const uint64_t v = add2(pack2(acc[c0 + c], acc[c0 + c + 1]),
                                    pack2(__uint_as_float(o[c]), __uint_as_float(o[c + 1])));
            unpack2(v, acc[c0 + c], acc[c0 + c + 1]);
          }
        }
      }
    };
    auto o_there = [&](int j) {  // the product of this warpgroup's tile j is in O
      const bool there = warp_wait(&ofull[m], (uint32_t)(j & 1));
      tc_fence_after();
      return there;
    };

    for (int j = 0; j < mine; ++j) {
      const int x = 2 * j + m;  // the item: S buffer x % NB, for the x / NB th time
      const uint32_t tS = tw + (uint32_t)(x % NB) * 128;
      if (!warp_wait(&sfull[x % NB], (uint32_t)((x / NB) & 1))) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (work) {
        uint32_t sa[32];
        tc_ld32(tS, sa);
        const int jt = two ? j : x;
        const int j0 = tile_at(jt) * kDtKeys;
        const uint32_t pages = s_pages[jt % kDtMasks];
        const bool whole = pages == (1u << np) - 1u &&
            (j0 + kDtKeys <= sq.prefix || (j0 + kDtKeys - 1 <= i0 && (p.window == 0 || i1 - j0 < p.window)));
        // raw scores of columns 32 c on -> capped and biased, in units of log 2
        auto modify = [&](int c, uint32_t (&s)[32]) {
          if (p.cap > 0.f) {
            const uint64_t sc2 = pack2(p.scale, p.scale), cap2 = pack2(p.cap, p.cap);
            float far = 0.f;  // the largest x^2: beyond 1 the polynomial does not hold
#pragma unroll
            for (int y = 0; y < 32; y += 2) {
              const uint64_t v = mul2(pack2(__uint_as_float(s[y]), __uint_as_float(s[y + 1])), sc2);
              const uint64_t v2 = mul2(v, v);
              uint64_t t2 = pack2(tanh_coef(kTanhTop), tanh_coef(kTanhTop));
#pragma unroll
              for (int k = kTanhTop - 1; k >= 0; --k) t2 = fma2(t2, v2, pack2(tanh_coef(k), tanh_coef(k)));
              float y0, y1;
              unpack2(v2, y0, y1);
              far = max3(far, y0, y1);
              unpack2(mul2(mul2(t2, v), cap2), y0, y1);
              s[y] = __float_as_uint(y0);
              s[y + 1] = __float_as_uint(y1);
            }
            if (__any_sync(kFull, far > 1.f)) {  // rare: from the raw scores again, which still stand in S
              tc_ld32(tS + 32 * c, s);
              tc_wait_ld();
#pragma unroll
              for (int y = 0; y < 32; ++y) s[y] = __float_as_uint(cap_score(__uint_as_float(s[y]) * p.scale, p.cap));
            }
          } else {
#pragma unroll
            for (int y = 0; y < 32; ++y) s[y] = __float_as_uint(__uint_as_float(s[y]) * p.scale);
          }
          if (p.slopes) {
            const float far = (float)(pos - j0 - 32 * c);
#pragma unroll
            for (int y = 0; y < 32; ++y)
              s[y] = __float_as_uint(fmaf(-slope, fabsf(far - (float)y), __uint_as_float(s[y])));
          }
        };
        // A new reference: f takes what was summed relative to the old one to it.  O of the tiles since the
        // last one that went to acc is rescaled where it is.
        auto rebase = [&](float nref) {
          const float f = ref == -INFINITY ? 1.f : ex2(ref - nref);  // nothing summed yet, or only NaN
          ref = nref;
          l *= f;
#pragma unroll
          for (int c = 0; c < RMAX; ++c) acc[c] *= f;
          if (j > 0) {
            if (!o_there(j - 1)) ok = false;
#pragma unroll 1
            for (int c0 = 0; c0 < r; c0 += 16) {
              float o[16];
              tc_ld16(tO + (uint32_t)c0, o);
#pragma unroll
              for (int c = 0; c < 16; ++c) o[c] *= f;
              tc_st16(tO + (uint32_t)c0, o);
            }
            tc_wait_st();
          }
          return f;
        };
        const bool first_pass = !whole || __any_sync(kFull, ref == -INFINITY);
        if (first_pass) {
          // scores as they count, written back over S, and their maximum.  Seen keys of the tile, as bits:
          // the range that the row's position and window give, and the prefix
          float top = -INFINITY;
          const int e = min(sq.L, pos + 1) - j0, a = p.window > 0 ? pos - p.window + 1 - j0 : 0, pr = sq.prefix - j0;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t s[32];
            tc_ld32(tS + 32 * c, s);
            uint32_t bits = bit_range(a - 32 * c, e - 32 * c) | bit_range(0, pr - 32 * c);
            if (P == 16) bits &= ((pages >> (2 * c) & 1u) ? 0x0000ffffu : 0u) | ((pages >> (2 * c + 1) & 1u) ? 0xffff0000u : 0u);
            else if (!((pages >> ((32 * c) >> psh)) & 1u)) bits = 0;
            tc_wait_ld();
            if (MOD) modify(c, s);
            if (!whole) {
#pragma unroll
              for (int y = 0; y < 32; ++y)
                if (!((bits >> y) & 1u)) s[y] = __float_as_uint(-INFINITY);
            }
            top = fmaxf(top, max32(s));
            tc_st32(tS + 32 * c, s);
          }
          tc_wait_st();
          tc_ld32(tS, sa);
          top *= c1;
          if (__any_sync(kFull, top > ref + kDtAhead)) rebase(fmaxf(ref, top));
        }
        // weights, 32 columns at a time, in place
        const uint64_t minus = pack2(-1.f, -1.f);
        float base = ref == -INFINITY ? 0.f : ref;  // nothing seen yet: scores are -inf or NaN, weights 0 or NaN
        uint64_t total = 0;  // (0, 0)
        auto weights = [&](int c, uint32_t (&s)[32]) {
          if (MOD && !first_pass) modify(c, s);
          uint32_t w[32];  // 16 words of hi pairs, 16 of lo pairs
          uint64_t sum0 = 0, sum1 = 0;
          const uint64_t nb = pack2(-base, -base);
#pragma unroll
          for (int y = 0; y < 16; ++y) {
            float a, e;
            unpack2(fma2(pack2(__uint_as_float(s[2 * y]), __uint_as_float(s[2 * y + 1])), c2, nb), a, e);
            a = ex2(a);
            e = ex2(e);
            const uint64_t w2 = pack2(a, e);
            if (y & 1) sum1 = add2(sum1, w2); else sum0 = add2(sum0, w2);
            const __nv_bfloat162 hi = __floats2bfloat162_rn(a, e);
            w[y] = *reinterpret_cast<const uint32_t*>(&hi);
            unpack2(fma2(pack2(bf16lo(w[y]), bf16hi(w[y])), minus, w2), a, e);
            const __nv_bfloat162 low = __floats2bfloat162_rn(a, e);
            w[16 + y] = *reinterpret_cast<const uint32_t*>(&low);
          }
          sum0 = add2(sum0, sum1);
          float a, e;
          unpack2(sum0, a, e);
          if (__any_sync(kFull, a + e > kDtMost)) return false;
          total = add2(total, sum0);
          tc_st32(tS + 32 * c, w);
          return true;
        };
        // some weight of columns 32 c on is too large: a new reference from their scores, to which the
        // weights of the columns before are brought
        auto raise = [&](int c) {
          uint32_t s[32];
          tc_ld32(tS + 32 * c, s);
          tc_wait_ld();
          if (MOD && !first_pass) modify(c, s);
          const float f = rebase(fmaxf(ref, max32(s) * c1));
          base = ref;
          total = mul2(total, pack2(f, f));
          tc_wait_st();
#pragma unroll 1
          for (int y = 0; y < 2 * c; ++y) {
            uint32_t w[16];
            tc_ld16u(tS + 32 * (y >> 1) + 8 * (y & 1), w);
            tc_wait_ld();
#pragma unroll
            for (int z = 0; z < 8; ++z)
              split2((bf16lo(w[z]) + bf16lo(w[8 + z])) * f, (bf16hi(w[z]) + bf16hi(w[8 + z])) * f, w[z], w[8 + z]);
            tc_st16u(tS + 32 * (y >> 1) + 8 * (y & 1), w);
          }
          tc_wait_st();
        };
        auto columns = [&](int c, uint32_t (&s)[32]) {
          if (!weights(c, s)) {
            raise(c);
            tc_ld32(tS + 32 * c, s);
            tc_wait_ld();
            weights(c, s);  // the largest is 1 now (or NaN)
          }
        };
        if constexpr (RMAX <= 64) {  // the next columns on their way meanwhile, where registers hold them
          uint32_t sb[32];
#pragma unroll 1
          for (int c = 0; c < 4; c += 2) {
            tc_wait_ld();
            tc_ld32(tS + 32 * (c + 1), sb);
            columns(c, sa);
            tc_wait_ld();
            if (c == 0) tc_ld32(tS + 64, sa);
            columns(c + 1, sb);
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            tc_wait_ld();
            columns(c, sa);
            if (c < 3) tc_ld32(tS + 32 * (c + 1), sa);
          }
        }
        float sum0, sum1;
        unpack2(total, sum0, sum1);
        l += sum0 + sum1;
        tc_wait_st();
      }
      // every kDtDrain tiles O goes to acc, and this tile's product starts it anew
      if (j > 0 && j % kDtDrain == 0) {
        if (!o_there(j - 1)) ok = false;
        if (work && ok) add_o();
      }
      if (!__all_sync(kFull, ok)) {
        ok = false;
        break;
      }
      tc_fence_before();
      warp_arrive(&pfull[x % NB], lane);
    }
    if (n > 0 && ok) {
      if (!warp_wait(odone, 0)) ok = false;
      tc_fence_after();
      if (ok && work && mine > 0) add_o();
    }
    float mx = ref;  // what l and acc are relative to
    if (!ok) l = __int_as_float(0x7fc00000);
    if (!two) {
      // the odd key tiles' result joins the even ones'; every product is done, so the K stages are free
      float* x = reinterpret_cast<float*>(smem + lay.k) + (row & 127);
      if (m == 1) {
        x[0] = mx;
        x[128] = l;
#pragma unroll
        for (int c = 0; c < RMAX; ++c)
          if (c < r) x[128 * (2 + c)] = acc[c];
      }
      dt_bar<1, 256>();
      if (m == 0) {
        const float mo = x[0], lo2 = x[128];
        const float mn = fmaxf(mx, mo);
        const float fa = mn == -INFINITY ? 1.f : ex2(mx - mn), fb = mn == -INFINITY ? 1.f : ex2(mo - mn);
        mx = mn;
        l = l * fa + lo2 * fb;
#pragma unroll
        for (int c = 0; c < RMAX; ++c)
          if (c < r) acc[c] = acc[c] * fa + x[128 * (2 + c)] * fb;
      }
    }
    if ((two || m == 0) && row < rows) {
      if (p.splits > 1) {
        const size_t unit = blockIdx.x / p.splits;
        float* out = p.part + ((unit * p.splits + split) * kDtRows + row) * (size_t)(r + 2);
        *reinterpret_cast<float2*>(out) = make_float2(mx, l);
#pragma unroll
        for (int c = 0; c < RMAX; c += 2)
          if (c < r) *reinterpret_cast<float2*>(out + 2 + c) = make_float2(acc[c], acc[c + 1]);
      } else {
        const size_t at = ((size_t)b * p.n_new + t) * p.Hq + h;
        const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
#pragma unroll
        for (int c = 0; c < RMAX; c += 4)
          if (c < r)
            *reinterpret_cast<float4*>(p.o + at * r + c) =
                make_float4(acc[c] * inv, acc[c + 1] * inv, acc[c + 2] * inv, acc[c + 3] * inv);
        if (p.lse) p.lse[at] = l > 0.f ? (mx + log2f(l)) * kLn2 : (l == l ? -INFINITY : l);
      }
    }
    // What follows is common code, for which every warp has the registers it was compiled with.  The other
    // warps take theirs back only behind a barrier of the whole CTA that stands after this branch's release:
    // taken any earlier, they could be the ones that a softmax warp still waits for at its start.  The
    // barrier before it brings each warpgroup together between its two changes, as the instruction asks.
    __syncwarp();
    dt_bar<1, 256>();
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(128));
    dt_bar<3, kDtThreads>();
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(256 - dt_regs<RMAX>()));
    // physical page of lane x < np of key tile j: -1 where no row sees any of it, or for a bad entry
    auto pages_of = [&](int j) {
      int id = -1;
      if (j < n && lane < np) {
        const int first = tile_at(j) * kDtKeys + (lane << psh);
        if (first < see_hi && (first + P > see_lo || first < sq.prefix)) id = dense_page(p, b, first >> psh);
      }
      return id;
    };
    // C tile j comes by TMA: whole swizzle atoms, every token seen by some row
    auto c_by_tma = [&](int j, uint32_t bits) {
      const int j0 = tile_at(j) * kDtKeys;
      return r % 64 == 0 && bits == (1u << np) - 1u && j0 + kDtKeys <= see_hi &&
             (j0 >= see_lo || j0 + kDtKeys <= sq.prefix);
    };
    if (warp == 8) {
      // ---------------------------------------------------------------- copies by TMA
      int ids = pages_of(0), ids_c = -1;
      uint32_t bits_c = 0;
      int issued = 0, last_c = -1;  // K tiles issued, the last C tile issued here
      for (int j = 0; j <= n && ok; ++j) {
        const int next = pages_of(j + 1);
        const uint32_t bits = __ballot_sync(kFull, ids >= 0);
        if (j < n) {
          const int s = j % kDtK;
          if (j >= kDtK && !warp_wait(&kempty[s], (uint32_t)((j / kDtK - 1) & 1))) {
            ok = false;
            break;
          }
          issued = j + 1;
          if (lane == 0) {
            s_pages[j % kDtMasks] = bits;
            mbar_arrive_expect_tx(&kfull[s], (uint32_t)__popc(bits) * P * D * 2);
          }
          __syncwarp();
          if (ids >= 0) {
#pragma unroll
            for (int a = 0; a < KA; ++a)
              dt_tma(smem + lay.k + (size_t)s * k_stage + a * kDtAtom + ((lane * 128) << psh), &kmap, a,
                     ids * p.Hkv + g, &kfull[s]);
          }
        }
        // A parity says nothing two phases on, so one role only waits for a C stage to be free, for every tile:
        // this one where any tile may come by TMA, handing the stage on for the others.
        if (r % 64 == 0 && j > 0) {
          const int s = (j - 1) % CS;
          if (j - 1 >= CS && !warp_wait(&cempty[s], (uint32_t)(((j - 1) / CS - 1) & 1))) {
            ok = false;
            break;
          }
          if (c_by_tma(j - 1, bits_c)) {
            last_c = j - 1;
            if (lane == 0) mbar_arrive_expect_tx(&cfull[s], (uint32_t)kDtKeys * r * 2);
            __syncwarp();
            if (ids_c >= 0)
              for (int a = 0; a < r / 64; ++a)
                dt_tma(smem + lay.c + (size_t)s * c_stage + a * kDtAtom + ((lane * 128) << psh), &cmap, a,
                       ids_c * p.Hkv + g, &cfull[s]);
          } else {
            warp_arrive(&cturn[s], lane);
          }
        }
        ids_c = ids;
        bits_c = bits;
        ids = next;
      }
      // no copy is on its way when the CTA ends, whatever became of the other warps
      for (int j = max(0, issued - kDtK); j < issued; ++j) warp_wait(&kfull[j % kDtK], (uint32_t)((j / kDtK) & 1));
      // (a C stage that a later tile took was read, so its copy had landed)
      for (int j = max(0, (ok ? n : last_c + 1) - CS); j <= last_c; ++j)
        warp_wait(&cfull[j % CS], (uint32_t)((j / CS) & 1));
    } else if (warp < 12) {
      // ---------------------------------------------------------------- the other C tiles, by 96 threads
      const int ct = tid - 288, cc = r / 8;
      const __nv_bfloat16* cl = static_cast<const __nv_bfloat16*>(p.c_lat);
      const int dr = 96 / cc, dc = 96 - dr * cc;
      int ids = pages_of(0);
      uint32_t turns = 0;  // bit s: the parity of cturn[s]'s next phase
      for (int j = 0; j < n && ok; ++j) {
        const int next = pages_of(j + 1);
        const uint32_t bits = __ballot_sync(kFull, ids >= 0);
        const int s = j % CS;
        if (!c_by_tma(j, bits)) {
          bool free = true;
          if (r % 64 == 0) {  // one phase for each of these tiles, and the last one of this stage was filled here
            free = warp_wait(&cturn[s], (turns >> s) & 1u);
            turns ^= 1u << s;
          } else if (j >= CS) {
            free = warp_wait(&cempty[s], (uint32_t)((j / CS - 1) & 1));
          }
          ok = all_of_96(free);  // the three warps give up together
          if (!ok) break;
          const int j0 = tile_at(j) * kDtKeys;
          unsigned char* dst = smem + lay.c + (size_t)s * c_stage;
          int row = ct / cc, ch = ct - row * cc;
#pragma unroll 4
          for (int x = ct; x < kDtKeys * cc + (96 - kDtKeys * cc % 96) % 96; x += 96) {
            const int id = __shfl_sync(kFull, ids, min(row, kDtKeys - 1) >> psh);
            if (row < kDtKeys) {
              const int key = j0 + row;
              const bool valid = id >= 0 && key < see_hi && (key >= see_lo || key < sq.prefix);
              const size_t src = valid ? (((size_t)id * p.Hkv + g) * P + (row & (P - 1))) * r + (size_t)ch * 8 : 0;
              const int c = ch ^ (row & p.mc);  // the chunk that is stored here
              cp_async16_zfill(dst + (c >> 3) * kDtAtom + row * 128 + (((c & 7) ^ (row & 7)) << 4), cl + src, valid);
            }
            row += dr;
            ch += dc;
            if (ch >= cc) {
              ch -= cc;
              ++row;
            }
          }
          cp_async_commit_group();
          cp_async_wait_group<0>();
          fence_proxy_async_smem();
          all_of_96(true);
          if (ct == 0) mbar_arrive(&cfull[s]);
        }
        ids = next;
      }
    } else if (warp == 12 && n > 0) {
      // ---------------------------------------------------------------- MMA
      // items x = 0, 1, ...: warpgroup x & 1, its key tile; PV(x) frees x's buffer for S(x + NB)
      const uint32_t leader = elect_leader();
      const uint32_t id_s = idesc_bf16(kDtM, kDtKeys);
      const uint32_t id_o = idesc_bf16(kDtM, r) | (1u << 16);  // B with its columns contiguous
      const uint64_t qdesc = smem_desc_sw128(sQ), kdesc = smem_desc_sw128(smem + lay.k), cdesc = dt_cdesc(smem + lay.c);
      const int items = two ? 2 * n : n;
      ok = warp_wait(qfull, 0);
      for (int x = -NB; x < items && ok; ++x) {
        if (x >= 0) {
          const int j = two ? x >> 1 : x, s = j % CS, m = x & 1, buf = x % NB;
          if (!warp_wait(&cfull[s], (uint32_t)((j / CS) & 1)) ||
              !warp_wait(&pfull[buf], (uint32_t)((x / NB) & 1))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t bd = cdesc + (uint64_t)((uint32_t)s * c_stage >> 4);
          const bool join = (x >> 1) % kDtDrain != 0;  // onto the O of the tiles before
          const uint32_t o = tmem + tO0 + (uint32_t)m * tOstep, pa = tmem + (uint32_t)buf * 128;
#pragma unroll
          for (int y = 0; y < kDtKeys / 16; ++y) {
            const uint32_t at = pa + (y >> 1) * 32 + (y & 1) * 8;
            dt_mma_ts(leader, o, at, bd + y * 128, id_o, y > 0 || join);
            dt_mma_ts(leader, o, at + 16, bd + y * 128, id_o, true);
          }
          dt_commit(leader, &ofull[m]);
          if (!two || m == 1) dt_commit(leader, &cempty[s]);
        }
        const int z = x + NB;
        if (z < items) {
          const int j = two ? z >> 1 : z, s = j % kDtK, m = z & 1, buf = z % NB;
          if (!warp_wait(&kfull[s], (uint32_t)((j / kDtK) & 1))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ad = qdesc + (uint64_t)(two ? ((uint32_t)m * k_stage >> 4) : 0u);
          const uint64_t bd = kdesc + (uint64_t)((uint32_t)s * k_stage >> 4);
#pragma unroll
          for (int y = 0; y < D / 16; ++y) {
            const uint64_t step = (uint64_t)(((y >> 2) * kDtAtom + (y & 3) * 32) >> 4);
            dt_mma_ss(leader, tmem + (uint32_t)buf * 128, ad + step, bd + step, id_s, y > 0);
          }
          dt_commit(leader, &sfull[buf]);
          if (!two || m == 1) dt_commit(leader, &kempty[s]);
        }
      }
      // every product, or after a failed wait what was issued
      dt_commit(leader, odone);
      if (!warp_wait(odone, 0)) ok = false;
    }
    __syncwarp();
    dt_bar<3, kDtThreads>();  // the softmax warps have had their registers and given them back
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(128));
  }
  if (!ok) set_err(p.err, BASISKV_DEVERR_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
  if (p.splits == 1) return;
  const size_t unit = blockIdx.x / p.splits;
  if (!dense_last_split(p.cnt + unit, p.splits, p.err, &s_last)) return;
  const size_t stride = (size_t)kDtRows * (r + 2);
  for (int row = warp; row < rows; row += kDtThreads / 32) {
    const int sr = row0 + row, t = sr / p.G;
    const size_t at = ((size_t)b * p.n_new + t) * p.Hq + (size_t)g * p.G + (sr - t * p.G);
    dense_join_row(p.part + unit * p.splits * stride + (size_t)row * (r + 2), stride, p.splits, r, p.o + at * r,
                   p.lse ? p.lse + at : nullptr, lane, false);
  }
}

void dense_plan_tc(DensePlan* pl, int batch, long long rows, int Hkv, int r, int page, int max_pages, int num_sms) {
  const long long units = (rows + kDtRows - 1) / kDtRows * Hkv * batch;
  const long long key_tiles = ((long long)max_pages * page + kDtKeys - 1) / kDtKeys;
  // where there are fewer units than SMs, each is split over its keys, four tiles to a split at least
  pl->splits = (int)std::max(1LL, std::min((long long)num_sms / units, key_tiles / 4));
  pl->part_off = pl->bytes = dense_counter_bytes(num_sms);
  if (pl->splits > 1) pl->bytes += ((size_t)units * pl->splits * kDtRows * (r + 2) * 4 + 255) & ~(size_t)255;
}

// ---------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------
// The driver's tensor-map encoder, looked up through the runtime (the library does not link libcuda).
typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
static EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiled>(f);
  }();
  return fn;
}

// [blocks][P][cols] bf16 pages (a block: one KV head of a physical page) as (64 columns, halves, rows, blocks),
// copied a half of a block at a time; no swizzle: the rows are stored swizzled
static cudaError_t page_map(CUtensorMap* map, const void* base, int cols, int page, long long blocks) {
  const EncodeTiled enc = encode_tiled();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t dims[4] = {64, (cuuint64_t)(cols / 64), (cuuint64_t)page, (cuuint64_t)blocks};
  const cuuint64_t strides[3] = {128, (cuuint64_t)cols * 2, (cuuint64_t)cols * 2 * page};
  const cuuint32_t box[4] = {64, 1, (cuuint32_t)page, 1}, one[4] = {1, 1, 1, 1};
  const CUresult e = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, one,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return e == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D, int RMAX, bool MOD>
static cudaError_t launch_dt(const DenseParams& p, cudaStream_t st) {
  constexpr size_t smem = dt_layout<D, RMAX>().total + 1024;
  static_assert(smem <= 227 * 1024, "shared memory of a CTA");
  cudaError_t e = ensure_smem((const void*)dense_tc_kernel<D, RMAX, MOD>, smem);
  if (e != cudaSuccess) return e;
  CUtensorMap kmap{}, cmap{};
  const long long blocks = (long long)p.num_phys * p.Hkv;
  if ((e = page_map(&kmap, p.k_raw, D, p.page, blocks)) != cudaSuccess) return e;
  if (p.r % 64 == 0 && (e = page_map(&cmap, p.c_lat, p.r, p.page, blocks)) != cudaSuccess) return e;
  const long long units = ((long long)p.n_new * p.G + kDtRows - 1) / kDtRows * p.Hkv * p.batch;
  dense_tc_kernel<D, RMAX, MOD><<<(unsigned)(units * p.splits), kDtThreads, smem, st>>>(p, kmap, cmap);
  return cudaGetLastError();
}

template <bool MOD>
static cudaError_t launch_dt_shape(const DenseParams& p, cudaStream_t st) {
  if (p.d == 64) return launch_dt<64, 64, MOD>(p, st);
  return p.r <= 64 ? launch_dt<128, 64, MOD>(p, st)
       : p.r <= 96 ? launch_dt<128, 96, MOD>(p, st) : launch_dt<128, 128, MOD>(p, st);
}

cudaError_t launch_dense_tc(const DenseParams& p, cudaStream_t st) {
  return p.cap > 0.f || p.slopes ? launch_dt_shape<true>(p, st) : launch_dt_shape<false>(p, st);
}

}  // namespace bkv
