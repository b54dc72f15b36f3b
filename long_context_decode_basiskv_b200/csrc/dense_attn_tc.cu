// Attention of many new tokens over the whole paged cache (bf16, swizzled
// rows) on the tcgen05 tensor cores: prompts, and chunks of them.
//
// One CTA per (256 rows, KV head, sequence, share of the keys): rows are
// consecutive new tokens' G heads of the KV head, two M = 128 tiles that share
// every key tile of 128 tokens.  Per row tile and key tile
//
//   S [128 x 128] = Q [128 x d] . K^T          operands in shared memory, S in tensor memory
//   P = 2^(S c - m), m the running row maximum   a thread owns a row: no shuffles
//   O [128 x r]   = P [128 x 128] . C            P in tensor memory (over S), C in shared memory
//
// and the thread adds O to its row's fp32 accumulators, rescaled by the change
// of the maximum.  O is not left to accumulate in tensor memory: a sum over
// hundreds of MMAs there loses more than the fp32 result may (measured in the
// table of the design notes), 16 MMAs do not, and adding it in registers makes
// the rescaling one FMA that is needed anyway.  P, fp32, is multiplied as two
// bf16 terms (hi + lo, 16 mantissa bits), like every chained product here.
//
// Warps 0-3 and 4-7: softmax of the two row tiles; warps 8-11 copy K and C
// rows from the pages into the operand layout (16-byte cp.async; rows that no
// row of the CTA sees become zeros, so that nothing in them reaches a sum);
// warp 12 issues the MMAs.  While one row tile is in softmax the tensor cores
// work for the other.  Order of issue: PV(j) then S(j + 1) of a row tile, so one
// commit tells its softmax both that O(j) can be added and that S(j + 1) is there.
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
constexpr uint32_t kDtAtom = kDtKeys * 128;  // 128 rows x 128 bytes

// registers a thread: 512 x 128 at launch = 256 x 200 + 256 x 56
constexpr int kDtRegsSoftmax = 200, kDtRegsOther = 56;

template <int RMAX> constexpr int dt_cstages() { return RMAX <= 64 ? 3 : 2; }

struct DtLayout {
  uint32_t q, k, c, bar, total;
};
template <int RMAX>
__host__ __device__ constexpr DtLayout dt_layout(int d) {
  DtLayout l{};
  uint32_t o = 0;
  l.q = o; o += 2 * (uint32_t)(d / 64) * kDtAtom;
  l.k = o; o += kDtK * (uint32_t)(d / 64) * kDtAtom;
  l.c = o; o += dt_cstages<RMAX>() * (uint32_t)((RMAX + 63) / 64) * kDtAtom;
  l.bar = o; o += 256;
  l.total = o;
  return l;
}

// D += A B with A in tensor memory
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%5, %6, %7, %8}, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accum), "r"(0u), "r"(0u), "r"(0u), "r"(0u)
      : "memory");
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
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// K-step j (16 elements) of a K-major swizzled operand of 128 rows
__device__ __forceinline__ uint64_t dt_kdesc(const unsigned char* base, int j) {
  return smem_desc_sw128(base + (size_t)(j >> 2) * kDtAtom) + (uint64_t)((j & 3) * 32 >> 4);
}
// K-step j (16 keys) of the C tile: the columns of a key contiguous (MN-major), 64 of them per swizzled
// 128-byte row, 8-key groups 1024 bytes apart, 64-column atoms kDtAtom apart
__device__ __forceinline__ uint64_t dt_cdesc(const unsigned char* base, int j) {
  const uint64_t addr = smem_u32(base) + (uint32_t)j * 2048u;
  return ((addr >> 4) & 0x3fffull) | ((uint64_t)(kDtAtom >> 4) << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

template <int RMAX>
__global__ void __launch_bounds__(kDtThreads, 1) dense_tc_kernel(DenseParams p) {
  constexpr int CS = dt_cstages<RMAX>();
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint32_t s_tmem;
  __shared__ int s_last;
  __shared__ uint32_t s_pages[kDtMasks];  // bit x: page x of the tile is there
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int d = p.d, r = p.r, P = p.page;
  const DtLayout lay = dt_layout<RMAX>(d);
  unsigned char* sQ = smem + lay.q;
  const uint32_t k_stage = (uint32_t)(d / 64) * kDtAtom, c_stage = (uint32_t)((RMAX + 63) / 64) * kDtAtom;
  uint64_t* kfull = reinterpret_cast<uint64_t*>(smem + lay.bar);
  uint64_t* kempty = kfull + kDtK;
  uint64_t* cfull = kempty + kDtK;
  uint64_t* cempty = cfull + CS;
  uint64_t* sfull = cempty + CS;   // per row tile: S(j) there, O(j - 1) too
  uint64_t* pfull = sfull + 2;     // per row tile: P(j) there, O(j - 1) taken
  uint64_t* odone = pfull + 2;     // the last O of both row tiles

  // this CTA's rows and keys; the last row tiles of a prompt see the most keys and start first
  const int tiles = (int)(((long long)p.n_new * p.G + kDtRows - 1) / kDtRows);
  const int split = blockIdx.x % p.splits;
  int u = blockIdx.x / p.splits;
  const int g = u % p.Hkv;
  u /= p.Hkv;
  const int b = u % p.batch, rt = tiles - 1 - u / p.batch;
  const long long row0 = (long long)rt * kDtRows;
  const int rows = (int)min((long long)kDtRows, (long long)p.n_new * p.G - row0);
  const int mt = rows > kDtM ? 2 : 1;
  const DenseSeq sq = dense_seq(p, b, tid == 0 && g == 0);
  const int pos0 = sq.L - p.n_new;
  const int t_lo = (int)(row0 / p.G), t_hi = (int)((row0 + rows - 1) / p.G);
  KeyTiles kt{0, 0, 0};
  if (sq.L > 0) kt = key_tiles(pos0 + t_lo, pos0 + t_hi, sq.L, p.window, sq.prefix, kDtKeys);
  const int lo = (int)((long long)kt.count() * split / p.splits);
  const int n = (int)((long long)kt.count() * (split + 1) / p.splits) - lo;  // key tiles of this CTA

  if (tid == 0) {
    for (int s = 0; s < kDtK; ++s) {
      mbar_init(&kfull[s], 128);
      mbar_init(&kempty[s], 1);
    }
    for (int s = 0; s < CS; ++s) {
      mbar_init(&cfull[s], 128);
      mbar_init(&cempty[s], 1);
    }
    for (int m = 0; m < 2; ++m) {
      mbar_init(&sfull[m], 1);
      mbar_init(&pfull[m], 128);
    }
    mbar_init(odone, 1);
    fence_mbar_init();
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  {  // the rows' queries, as the A operand
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q);
    const int cpr = d / 8;
    for (int x = tid; x < mt * kDtM * cpr; x += kDtThreads) {
      const int row = x / cpr, c = x - row * cpr;
      const bool valid = row < rows;
      const long long gr = row0 + (valid ? row : 0);
      const long long t = gr / p.G;
      const size_t src = (((size_t)b * p.n_new + t) * p.Hq + (size_t)g * p.G + (gr - t * p.G)) * d + (size_t)c * 8;
      unsigned char* dst = sQ + (size_t)(row / kDtM) * k_stage + (size_t)(c >> 3) * kDtAtom + (row % kDtM) * 128 +
                           (((c & 7) ^ (row & 7)) << 4);
      cp_async16_zfill(dst, q + src, valid);
    }
    cp_async_commit_group();
    cp_async_wait_group<0>();
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  bool ok = true;

  if (warp < 8) {
    // ------------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kDtRegsSoftmax));
    const int m = warp >> 2;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + (uint32_t)m * 128, tO = tmem + lanes + 256 + (uint32_t)m * 128;
    const int row = tid & 255;  // of the CTA
    const bool active = m < mt;
    const long long grow = row0 + min(row, rows - 1);
    const int t = (int)(grow / p.G), h = g * p.G + (int)(grow - (long long)t * p.G);
    const int pos = pos0 + t;
    // positions of this row tile's first and last row
    const int i0 = pos0 + (int)((row0 + min(m * kDtM, rows - 1)) / p.G);
    const int i1 = pos0 + (int)((row0 + min(m * kDtM + kDtM - 1, rows - 1)) / p.G);
    const float slope = p.slopes ? p.slopes[h] * kLog2e : 0.f;
    const bool mod = p.cap > 0.f || p.slopes;
    const float c1 = mod ? 1.f : p.scale;
    const uint32_t all_pages = (P == 64) ? 3u : (P == 32) ? 15u : 255u;
    const int psh = 31 - __clz(P);
    float mx = -INFINITY, l = 0.f, corr = 1.f;
    float acc[RMAX];
#pragma unroll
    for (int c = 0; c < RMAX; ++c) acc[c] = 0.f;

    auto add_o = [&]() {
#pragma unroll
      for (int c0 = 0; c0 < RMAX; c0 += 16) {
        if (c0 < r) {
          float o[16];
          tc_ld16(tO + (uint32_t)c0, o);
#pragma unroll
          for (int c = 0; c < 16; ++c) acc[c0 + c] = fmaf(acc[c0 + c], corr, o[c]);
        }
      }
    };

    for (int j = 0; active && j < n; ++j) {
      if (!__all_sync(kFull, mbar_wait_bounded(&sfull[m], (uint32_t)(j & 1)))) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (j > 0) add_o();
      const int j0 = kt.tile(lo + j) * kDtKeys;
      const uint32_t pages = s_pages[j % kDtMasks];
      const bool whole = pages == all_pages &&
          (j0 + kDtKeys <= sq.prefix || (j0 + kDtKeys - 1 <= i0 && (p.window == 0 || i1 - j0 < p.window)));
      float top = -INFINITY;
      if (whole && !mod) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t s[32];
          tc_ld32(tS + 32 * c, s);
          tc_wait_ld();
#pragma unroll
          for (int x = 0; x < 32; x += 2) top = fmaxf(top, fmaxf(__uint_as_float(s[x]), __uint_as_float(s[x + 1])));
        }
      } else {
        // scores as they count, written back over S
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t s[32];
          tc_ld32(tS + 32 * c, s);
          tc_wait_ld();
#pragma unroll
          for (int x = 0; x < 32; ++x) {
            const int jj = 32 * c + x, key = j0 + jj;
            float v = __uint_as_float(s[x]);
            if (mod) v = mod_score(v, p.scale, p.cap, slope, pos, key);
            if (!whole && !(((pages >> (jj >> psh)) & 1u) && sees(pos, key, sq.L, p.window, sq.prefix))) v = -INFINITY;
            top = fmaxf(top, v);
            s[x] = __float_as_uint(v);
          }
          tc_st32(tS + 32 * c, s);
          tc_wait_st();
        }
      }
      const float mn = fmaxf(mx, top * c1);
      const float base = mn == -INFINITY ? 0.f : mn;  // nothing seen yet: scores are -inf or NaN, weights 0 or NaN
      corr = mn == -INFINITY ? 1.f : ex2(mx - mn);
      mx = mn;
      float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t s[32];
        tc_ld32(tS + 32 * c, s);
        tc_wait_ld();
        uint32_t w[32];  // 16 words of hi pairs, 16 of lo pairs
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const float a = ex2(fmaf(__uint_as_float(s[2 * x]), c1, -base));
          const float e = ex2(fmaf(__uint_as_float(s[2 * x + 1]), c1, -base));
          sum0 += a;
          sum1 += e;
          const __nv_bfloat162 hi = __floats2bfloat162_rn(a, e);
          w[x] = *reinterpret_cast<const uint32_t*>(&hi);
          const __nv_bfloat162 low = __floats2bfloat162_rn(a - bf16lo(w[x]), e - bf16hi(w[x]));
          w[16 + x] = *reinterpret_cast<const uint32_t*>(&low);
        }
        tc_st32(tS + 32 * c, w);
      }
      l = fmaf(l, corr, sum0 + sum1);
      tc_wait_st();
      tc_fence_before();
      mbar_arrive(&pfull[m]);
    }
    if (active && n > 0 && ok) {
      if (__all_sync(kFull, mbar_wait_bounded(odone, 0))) {
        tc_fence_after();
        add_o();
      } else {
        ok = false;
      }
    }
    if (!ok) l = __int_as_float(0x7fc00000);
    if (active && row < rows) {
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
            *reinterpret_cast<float4*>(p.o + at * r + c) = make_float4(acc[c] * inv, acc[c + 1] * inv, acc[c + 2] * inv, acc[c + 3] * inv);
        if (p.lse) p.lse[at] = l > 0.f ? (mx + log2f(l)) * kLn2 : (l == l ? -INFINITY : l);
      }
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------------ copies
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kDtRegsOther));
    const int ct = tid - 256;
    const __nv_bfloat16* kr = static_cast<const __nv_bfloat16*>(p.k_raw);
    const __nv_bfloat16* cl = static_cast<const __nv_bfloat16*>(p.c_lat);
    const int psh = 31 - __clz(P), np = kDtKeys >> psh;
    const int see_lo = p.window > 0 ? pos0 + t_lo - p.window + 1 : 0;
    const int see_hi = min(sq.L, max(pos0 + t_hi + 1, sq.prefix));
    auto seen = [&](int key) { return key < see_hi && (key >= see_lo || key < sq.prefix); };
    // lane x < np: physical page x of tile j (-1: nothing seen there, or a bad entry)
    auto pages_of = [&](int j) {
      int id = -1;
      if (j < n && lane < np) {
        const int first = kt.tile(lo + j) * kDtKeys + (lane << psh);
        if (first < see_hi && (first + P > see_lo || first < sq.prefix)) id = dense_page(p, b, first >> psh);
      }
      return id;
    };
    const int kc = d / 8, krow = ct / kc, kch = ct - krow * kc, kstep = 128 / kc;
    const int cc = r / 8;
    auto copy_k = [&](int j, int ids) {
      const int j0 = kt.tile(lo + j) * kDtKeys;
      unsigned char* dst = smem + lay.k + (size_t)(j % kDtK) * k_stage + (size_t)(kch >> 3) * kDtAtom + ((kch & 7) << 4);
      for (int row = krow; row < kDtKeys; row += kstep) {
        const int id = __shfl_sync(kFull, ids, row >> psh);
        const bool valid = id >= 0 && seen(j0 + row);
        const size_t src = valid ? (((size_t)id * p.Hkv + g) * P + (row & (P - 1))) * d + (size_t)kch * 8 : 0;
        cp_async16_zfill(dst + row * 128, kr + src, valid);  // stored swizzle = operand swizzle
      }
    };
    auto copy_c = [&](int j, int ids) {
      const int j0 = kt.tile(lo + j) * kDtKeys;
      unsigned char* dst = smem + lay.c + (size_t)(j % CS) * c_stage;
      const int dr = 128 / cc, dc = 128 - dr * cc;
      int row = ct / cc, ch = ct - row * cc;
      for (int x = 0; x < cc; ++x) {
        const int id = __shfl_sync(kFull, ids, row >> psh);
        const bool valid = id >= 0 && seen(j0 + row);
        const size_t src = valid ? (((size_t)id * p.Hkv + g) * P + (row & (P - 1))) * r + (size_t)ch * 8 : 0;
        const int c = ch ^ (row & p.mc);  // the chunk that is stored here
        cp_async16_zfill(dst + (size_t)(c >> 3) * kDtAtom + row * 128 + (((c & 7) ^ (row & 7)) << 4), cl + src, valid);
        row += dr;
        ch += dc;
        if (ch >= cc) {
          ch -= cc;
          ++row;
        }
      }
    };
    // groups in the order K(0), [K(1), C(0)], [K(2), C(1)] ...: a pair is told to the MMA warp when the
    // next pair has been issued, so that two tiles are always in flight
    int ids_k = pages_of(0), ids_c = -1;
    for (int j = 0; j <= n && ok; ++j) {
      const int ids_next = pages_of(j + 1);
      if (j < n) {
        if (j >= kDtK && !__all_sync(kFull, mbar_wait_bounded(&kempty[j % kDtK], (uint32_t)((j / kDtK - 1) & 1)))) {
          ok = false;
          break;
        }
        if (warp == 8) {
          const uint32_t bits = __ballot_sync(kFull, ids_k >= 0);
          if (lane == 0) s_pages[j % kDtMasks] = bits;
        }
        __syncwarp();
        copy_k(j, ids_k);
      }
      cp_async_commit_group();
      if (j > 0) {
        if (j - 1 >= CS && !__all_sync(kFull, mbar_wait_bounded(&cempty[(j - 1) % CS], (uint32_t)(((j - 1) / CS - 1) & 1)))) {
          ok = false;
          break;
        }
        copy_c(j - 1, ids_c);
      }
      cp_async_commit_group();
      cp_async_wait_group<2>();  // K(j - 1) and C(j - 2) are there
      fence_proxy_async_smem();
      if (j >= 1) mbar_arrive(&kfull[(j - 1) % kDtK]);
      if (j >= 2) mbar_arrive(&cfull[(j - 2) % CS]);
      ids_c = ids_k;
      ids_k = ids_next;
    }
    cp_async_wait_group<0>();
    if (ok && n > 0) {
      fence_proxy_async_smem();
      mbar_arrive(&cfull[(n - 1) % CS]);
    }
  } else {
    // ------------------------------------------------------------------ MMA
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kDtRegsOther));
    if (warp == 12 && lane == 0 && n > 0) {
      const uint32_t id_s = idesc_bf16(kDtM, kDtKeys);
      const uint32_t id_o = idesc_bf16(kDtM, r) | (1u << 16);  // B with its columns contiguous
      const int ks = d / 16;
      auto scores = [&](int m, int j) {
        const unsigned char* a = sQ + (size_t)m * k_stage;
        const unsigned char* bb = smem + lay.k + (size_t)(j % kDtK) * k_stage;
        for (int x = 0; x < ks; ++x)
          tc_mma(tmem + (uint32_t)m * 128, dt_kdesc(a, x), dt_kdesc(bb, x), id_s, x > 0 ? 1u : 0u);
      };
      auto values = [&](int m, int j) {
        const unsigned char* bb = smem + lay.c + (size_t)(j % CS) * c_stage;
        const uint32_t o = tmem + 256 + (uint32_t)m * 128, pa = tmem + (uint32_t)m * 128;
        for (int x = 0; x < kDtKeys / 16; ++x) {
          const uint32_t at = pa + (uint32_t)(x >> 1) * 32 + (uint32_t)(x & 1) * 8;
          tc_mma_ts(o, at, dt_cdesc(bb, x), id_o, x > 0 ? 1u : 0u);
          tc_mma_ts(o, at + 16, dt_cdesc(bb, x), id_o, 1u);
        }
      };
      for (int j = 0; j <= n && ok; ++j) {
        // S(j) once K(j) is there; before it, the products of tile j - 1
        if (j < n && !mbar_wait_bounded(&kfull[j % kDtK], (uint32_t)((j / kDtK) & 1))) {
          ok = false;
          break;
        }
        if (j > 0 && !mbar_wait_bounded(&cfull[(j - 1) % CS], (uint32_t)(((j - 1) / CS) & 1))) {
          ok = false;
          break;
        }
        for (int m = 0; m < mt; ++m) {
          if (j > 0) {
            if (!mbar_wait_bounded(&pfull[m], (uint32_t)((j - 1) & 1))) {
          ok = false;
          break;
        }
            tc_fence_after();
            values(m, j - 1);
          }
          if (j < n) {
            tc_fence_after();
            scores(m, j);
            tc_commit(&sfull[m]);
          }
        }
        if (!ok) break;
        if (j > 0) tc_commit(&cempty[(j - 1) % CS]);
        if (j < n) tc_commit(&kempty[j % kDtK]);
      }
      // with every product issued this covers the last of them; after a failed wait, what was issued
      tc_commit(odone);
      if (!mbar_wait_bounded(odone, 0)) ok = false;
    }
  }
  if (!ok) set_err(p.err, BASISKV_DEVERR_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
  if (p.splits == 1) return;
  const size_t unit = blockIdx.x / p.splits;
  if (!dense_last_split(p.cnt + unit, p.splits, p.err, &s_last)) return;
  const size_t stride = (size_t)kDtRows * (r + 2);
  for (int row = warp; row < rows; row += kDtThreads / 32) {
    const long long gr = row0 + row, t = gr / p.G;
    const size_t at = ((size_t)b * p.n_new + t) * p.Hq + (size_t)g * p.G + (gr - t * p.G);
    dense_join_row(p.part + unit * p.splits * stride + (size_t)row * (r + 2), stride, p.splits, r, p.o + at * r,
                   p.lse ? p.lse + at : nullptr, lane, false);
  }
}

void dense_plan_tc(DensePlan* pl, int batch, long long rows, int Hkv, int r, int page, int max_pages, int num_sms) {
  const long long units = (rows + kDtRows - 1) / kDtRows * Hkv * batch;
  const long long key_tiles = ((long long)max_pages * page + kDtKeys - 1) / kDtKeys;
  // where there are fewer units than SMs, each is split over its keys, four tiles to a split at least
  pl->splits = (int)std::max(1LL, std::min((long long)num_sms / units, key_tiles / 4));
  pl->cnt_off = 0;
  pl->part_off = ((size_t)units * 4 + 255) & ~(size_t)255;
  pl->bytes = pl->part_off;
  if (pl->splits > 1) pl->bytes += ((size_t)units * pl->splits * kDtRows * (r + 2) * 4 + 255) & ~(size_t)255;
}

template <int RMAX>
static cudaError_t launch_dt(const DenseParams& p, cudaStream_t st) {
  const size_t smem = dt_layout<RMAX>(p.d).total + 1024;
  cudaError_t e = ensure_smem((const void*)dense_tc_kernel<RMAX>, smem);
  if (e != cudaSuccess) return e;
  const long long units = ((long long)p.n_new * p.G + kDtRows - 1) / kDtRows * p.Hkv * p.batch;
  dense_tc_kernel<RMAX><<<(unsigned)(units * p.splits), kDtThreads, smem, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_dense_tc(const DenseParams& p, cudaStream_t st) {
  return p.r <= 64 ? launch_dt<64>(p, st) : launch_dt<128>(p, st);
}

}  // namespace bkv
