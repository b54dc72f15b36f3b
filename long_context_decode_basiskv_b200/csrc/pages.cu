// Pages of the cache for requests that grow or end: block-table entries and
// token slots from the requests' lengths, on the device.
//
//   have_b = ceil(L_b / P),  need_b = ceil((L_b + a_b) / P) - have_b,  off_b = sum_{c < b} need_c
//   new page i of all (request b, i = off_b + x)  ->  free[count - 1 - i]  at  table[b][have_b + x]
//   token t of request b                          ->  slot = page * P + (L_b + t) % P
//
// and the reverse for requests that end.  The work is a few integers per page
// or token, so the call is latency: one launch, one thread-block cluster.
// Every CTA of the cluster scans the lengths by itself (they come from L2) and
// keeps lengths and offsets in shared memory; a cluster barrier stands between
// the last read of seq_len / free_count and the first write, so the outputs
// may be the inputs (a captured graph steps in place), and carries each CTA's
// fault bits to the others, so a call that cannot be met in full changes
// nothing.
//
// Measured (64 requests, pages of 16): 3.8 us for a token each, 13.6 us for
// prompts of 2048 to 32768 tokens (69 k table entries, 2.1 M slots written; the
// first kernel takes two thirds of it), 11.2 us for the release of half of them.
// Bound by the latency of a chain of dependent loads: lengths, free count, page
// ids, then the stores.  Where entries are many, the ids are read twice (checked,
// then moved) and each entry looks for its request by bisection.  A cluster of
// 16 CTAs (beyond the portable size) took 11.3 and 8.6 us for the last two; it
// is not used, since a device partitioned for others may not offer it.
#include "kernels.cuh"

namespace bkv {

constexpr int kPageThreads = 1024;
// A cluster of 8 CTAs (the portable limit) for anything but the smallest
// calls, whose few stores one CTA issues as fast without the cluster's start.
constexpr int kPageCluster = 8;
constexpr long long kPageSmall = 8192;  // slots, or pages, that one CTA writes

// the request that page p of the flattened new (or released) pages belongs to
__device__ __forceinline__ int request_of(const int* off, int B, int p) {
  int lo = 0, hi = B;  // off[lo] <= p < off[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= p) lo = mid; else hi = mid;
  }
  return lo;
}

template <bool ASSIGN>
__global__ void __launch_bounds__(kPageThreads) pages_kernel(PagesParams p) {
  extern __shared__ int s_len[];        // [B] lengths, then [B + 1] offsets
  __shared__ int warp_tot[32];
  __shared__ uint32_t s_bad;
  const int tid = threadIdx.x, B = p.batch, P = p.page, sh = 31 - __clz(P);
  const int C = gridDim.x, rank = blockIdx.x;  // one cluster: its rank is the block index
  int* s_off = s_len + B;
  if (tid == 0) s_bad = 0;
  __syncthreads();

  // pages of each request, their exclusive sums
  const int per = (B + kPageThreads - 1) / kPageThreads;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  uint32_t bad = 0;
  int sum = 0;
  for (int b = b0; b < b1; ++b) {
    const int L = p.seq_len[b], a = p.amount[b];
    const long long end = ASSIGN ? (long long)L + a : L;
    int n = 0;
    if (L < 0 || (ASSIGN && a < 0) || end > (long long)p.max_pages * P)
      bad |= BASISKV_DEVERR_SEQ_LEN;
    else if (ASSIGN)
      n = (int)((end + P - 1) >> sh) - ((L + P - 1) >> sh);
    else if (a != 0)
      n = (L + P - 1) >> sh;
    s_len[b] = L;
    s_off[b] = n;
    sum += n;
  }
  int total;
  int at = block_exclusive_scan(sum, warp_tot, total);
  for (int b = b0; b < b1; ++b) {
    const int n = s_off[b];
    s_off[b] = at;
    at += n;
  }
  if (tid == 0) s_off[B] = total;
  const int count = *p.free_count;
  if (count < 0 || count > p.num_phys || (ASSIGN ? total > count : total > p.num_phys - count))
    bad |= BASISKV_DEVERR_PAGES;
  __syncthreads();

  // the page ids this call hands on, checked before anything is written
  const int gt = rank * kPageThreads + tid, nt = C * kPageThreads;
  if (!(bad & BASISKV_DEVERR_PAGES)) {  // the same for every thread of the cluster
#pragma unroll 4
    for (int i = gt; i < total; i += nt) {
      int id;
      if (ASSIGN) {
        id = p.free_pages[count - 1 - i];
      } else {
        const int b = request_of(s_off, B, i);
        id = p.table[(size_t)b * p.max_pages + (i - s_off[b])];
      }
      if (id < 0 || id >= p.num_phys) bad |= BASISKV_DEVERR_BLOCK_TABLE;
    }
  }
  if (ASSIGN && p.slots) {  // a partly filled page that takes the first new tokens
    for (int b = gt; b < B; b += nt) {
      const int L = s_len[b];
      if (L <= 0 || (L & (P - 1)) == 0 || L > p.max_pages * P || p.amount[b] <= 0) continue;
      const int id = p.table[(size_t)b * p.max_pages + (L >> sh)];
      if (id < 0 || id >= p.num_phys) bad |= BASISKV_DEVERR_BLOCK_TABLE;
    }
  }
  if (bad) atomicOr(&s_bad, bad);
  __syncthreads();
  bad = s_bad;
  if (C > 1) {  // the others' bits; nobody leaves while its own may still be read
    __shared__ uint32_t s_all;
    if (tid == 0) s_all = 0;
    cluster_arrive_release();
    cluster_wait_acquire();
    if (tid < C) atomicOr(&s_all, ld_shared_cluster(&s_bad, (uint32_t)tid));
    cluster_arrive_relaxed();
    __syncthreads();
    bad = s_all;
  }

  if (rank == 0) {
    for (int b = tid; b < B; b += kPageThreads) {
      const int L = s_len[b];
      p.seq_len_out[b] = bad ? L : ASSIGN ? L + p.amount[b] : p.amount[b] != 0 ? 0 : L;
    }
    if (tid == 0) {
      *p.free_count_out = bad ? count : ASSIGN ? count - total : count + total;
      if (bad) set_err(p.err, (int32_t)bad);
    }
  }
  if (!bad) {
#pragma unroll 4
    for (int i = gt; i < total; i += nt) {
      const int b = request_of(s_off, B, i);
      if (ASSIGN)
        p.table[(size_t)b * p.max_pages + ((s_len[b] + P - 1) >> sh) + (i - s_off[b])] = p.free_pages[count - 1 - i];
      else
        p.free_pages[count + i] = p.table[(size_t)b * p.max_pages + (i - s_off[b])];
    }
  }
  // slots: all of them where they are few, else each request's first (-1 after a fault), from which
  // slots_kernel goes on
  if (ASSIGN && p.slots) {
    const int cols = p.rows_later ? 1 : p.slot_cols;
    const int db = nt / cols, dc = nt - db * cols;
    int b = gt / cols, t = gt - b * cols;
    while (b < B) {
      int w = -1;
      if (!bad && t < p.amount[b]) {
        const int L = s_len[b], have = (L + P - 1) >> sh, pos = L + t, pg = pos >> sh;
        const int id = pg < have ? p.table[(size_t)b * p.max_pages + pg]
                                 : p.free_pages[count - 1 - (s_off[b] + pg - have)];
        w = (id << sh) + (pos & (P - 1));
      }
      p.slots[(size_t)b * p.slot_cols + t] = w;
      b += db;
      t += dc;
      if (t >= cols) {
        t -= cols;
        ++b;
      }
    }
  }
  if (C > 1) cluster_wait_acquire();
}

// The slots of many tokens, over the whole GPU: the kernel before it has set the table, the lengths and
// each request's first slot, which says whether the call was met.
constexpr int kSlotThreads = 256;
__global__ void __launch_bounds__(kSlotThreads) slots_kernel(PagesParams p) {
  grid_dep_wait();
  const int b = blockIdx.y, P = p.page, sh = 31 - __clz(P);
  const int t0 = (blockIdx.x * kSlotThreads + threadIdx.x) * 4;
  if (t0 >= p.slot_cols) return;
  int* row = p.slots + (size_t)b * p.slot_cols;
  const int a = __ldcg(row) < 0 ? 0 : p.amount[b], pos = p.seq_len_out[b] - a + t0;
  const int32_t* table = p.table + (size_t)b * p.max_pages;
  const int left = min(4, a - t0);
  int id0 = 0, id1 = 0;
  if (left > 0) {
    id0 = table[pos >> sh];
    id1 = table[(pos + left - 1) >> sh];  // four tokens lie on two pages at most
  }
  int w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int at = pos + j;
    w[j] = j < left ? (((at >> sh) == (pos >> sh) ? id0 : id1) << sh) + (at & (P - 1)) : -1;
  }
  if (p.slot_vec == 4) {
    *reinterpret_cast<int4*>(row + t0) = make_int4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (t0 + j < p.slot_cols) row[t0 + j] = w[j];
  }
}

template <bool ASSIGN>
static cudaError_t launch_pages_t(PagesParams p, cudaStream_t st) {
  const size_t smem = ((size_t)2 * p.batch + 1) * sizeof(int);
  cudaError_t e = ensure_smem((const void*)pages_kernel<ASSIGN>, smem);
  if (e != cudaSuccess) return e;
  // what the call may have to write: slots, or pages
  const bool with_slots = ASSIGN && p.slots;
  const long long most = (long long)p.batch * (with_slots ? p.slot_cols : p.max_pages);
  const int C = most <= kPageSmall ? 1 : kPageCluster;
  p.rows_later = with_slots && most > kPageSmall;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C);
  cfg.blockDim = dim3(kPageThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, pages_kernel<ASSIGN>, p)) != cudaSuccess || !p.rows_later) return e;
  cfg.gridDim = dim3((p.slot_cols + 4 * kSlotThreads - 1) / (4 * kSlotThreads), p.batch);
  cfg.blockDim = dim3(kSlotThreads);
  cfg.dynamicSmemBytes = 0;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  return cudaLaunchKernelEx(&cfg, slots_kernel, p);
}

cudaError_t launch_assign_pages(const PagesParams& p, cudaStream_t st) { return launch_pages_t<true>(p, st); }
cudaError_t launch_release_pages(const PagesParams& p, cudaStream_t st) { return launch_pages_t<false>(p, st); }

}  // namespace bkv
