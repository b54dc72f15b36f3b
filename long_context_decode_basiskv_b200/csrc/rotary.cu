// Rotary positions of new queries and keys: pair i of a head's rotated part,
// (u, v), of the token at position x becomes
//   (u cos - v sin, v cos + u sin) * mscale,  angle = x * inv_freq[i],
// where the pair is (i, i + rot / 2) ("half") or (2 i, 2 i + 1)
// ("interleaved").  Elements past the rotated part are copied.
//
// Bound by memory: every element is read and written once.  The angle is the
// only delicate number: x * inv_freq reaches 10^5 to 10^6 radians, where fp32
// keeps no fraction worth having, so it is formed and reduced to a fraction of
// a turn in fp64, and only sin and cos of that fraction are fp32 (sincospif).
// One angle serves all heads of a token: a CTA computes its tokens' angles
// once into shared memory, then streams the heads.  The result is rounded
// once, from fp32 to the storage type.
//
// Measured: 110 us for 32767 tokens of 32 + 8 heads of 128 (bf16, slices of a
// packed projection; 671 MB, 6.1 TB/s, 0.94 of the measured copy rate); 3.3 us
// for one token of 64 sequences, which is the launch and two dependent loads.
// Parts that are no whole vectors: 617 and 521 us for 52 and 116 of 128 elements
// and 30000 tokens (614 MB), where 128 take 101: a pair, or a copied element, at
// a time.
// Four tokens to a CTA where that still leaves four CTAs for every SM.
#include "kernels.cuh"

namespace bkv {

constexpr int kRotThreads = 256;
constexpr int kRotTokens = 4;  // tokens per CTA where there are many

template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

template <typename T>
struct alignas(16) Vec {
  static constexpr int N = 16 / sizeof(T);
  T x[N];
};

// VEC: 16-byte loads and stores, for parts and strides that are multiples of
// them; otherwise one pair (or one copied element) at a time.
template <typename T, bool HALF, bool VEC>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
  __shared__ float2 s_cs[kRotTokens][64];
  const int half = p.rot / 2, tt = p.tokens_per_cta;
  const long long tok0 = (long long)blockIdx.x * tt;
  const int ntok = (int)min((long long)tt, p.tokens - tok0);
  for (int i = threadIdx.x; i < ntok * half; i += kRotThreads) {
    const int k = i / half, j = i - k * half;
    const long long tok = tok0 + k;
    int pos;
    if (p.positions) {
      pos = p.positions[tok];
    } else {
      const int b = (int)(tok / p.n_new);
      pos = p.seq_len[b] - p.n_new + (int)(tok - (long long)b * p.n_new);
    }
    const double turns = (double)pos * (p.rope.inv_freq[j] * 0.15915494309189533577);  // 1 / (2 pi)
    float s, c;
    sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
    s_cs[k][j] = make_float2(c * p.rope.mscale, s * p.rope.mscale);
  }
  __syncthreads();

  constexpr int N = VEC ? Vec<T>::N : 1;
  // items of one head: chunks of N pairs (half) or N elements (interleaved; one pair without
  // VEC), then the chunks of N copied elements
  const int turned = HALF ? half / N : VEC ? p.rot / N : half;
  const int per_head = turned + (p.d - p.rot) / N;
  const int heads = p.hq + p.hk;
  for (int it = threadIdx.x; it < ntok * heads * per_head; it += kRotThreads) {
    const int hh = it / per_head, c = it - hh * per_head;
    const int k = hh / heads, h = hh - k * heads;
    const long long tok = tok0 + k;
    const bool isq = h < p.hq;
    const T* in = static_cast<const T*>(isq ? p.q : p.k) + tok * (isq ? p.q_stride : p.k_stride) +
                  (size_t)(isq ? h : h - p.hq) * p.d;
    T* out = static_cast<T*>(isq ? p.q_out : p.k_out) + ((size_t)tok * (isq ? p.hq : p.hk) + (isq ? h : h - p.hq)) * p.d;
    if (c >= turned) {
      const int e = p.rot + (c - turned) * N;
      if constexpr (VEC) *reinterpret_cast<Vec<T>*>(out + e) = *reinterpret_cast<const Vec<T>*>(in + e);
      else out[e] = in[e];
    } else if constexpr (HALF && VEC) {
      Vec<T> u = *reinterpret_cast<const Vec<T>*>(in + c * N), v = *reinterpret_cast<const Vec<T>*>(in + half + c * N);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float2 cs = s_cs[k][c * N + j];
        const float a = Elem<T>::to_f(u.x[j]), b = Elem<T>::to_f(v.x[j]);
        u.x[j] = from_f<T>(a * cs.x - b * cs.y);
        v.x[j] = from_f<T>(b * cs.x + a * cs.y);
      }
      *reinterpret_cast<Vec<T>*>(out + c * N) = u;
      *reinterpret_cast<Vec<T>*>(out + half + c * N) = v;
    } else if constexpr (VEC) {
      Vec<T> u = *reinterpret_cast<const Vec<T>*>(in + c * N);
#pragma unroll
      for (int j = 0; j < N; j += 2) {
        const float2 cs = s_cs[k][(c * N + j) / 2];
        const float a = Elem<T>::to_f(u.x[j]), b = Elem<T>::to_f(u.x[j + 1]);
        u.x[j] = from_f<T>(a * cs.x - b * cs.y);
        u.x[j + 1] = from_f<T>(b * cs.x + a * cs.y);
      }
      *reinterpret_cast<Vec<T>*>(out + c * N) = u;
    } else {
      const int e0 = HALF ? c : 2 * c, e1 = HALF ? c + half : 2 * c + 1;
      const float2 cs = s_cs[k][c];
      const float a = Elem<T>::to_f(in[e0]), b = Elem<T>::to_f(in[e1]);
      out[e0] = from_f<T>(a * cs.x - b * cs.y);
      out[e1] = from_f<T>(b * cs.x + a * cs.y);
    }
  }
}

template <typename T, bool HALF>
static cudaError_t launch_t(const RotaryParams& p, bool vec, cudaStream_t st) {
  const unsigned grid = (unsigned)((p.tokens + p.tokens_per_cta - 1) / p.tokens_per_cta);
  if (vec) rotary_kernel<T, HALF, true><<<grid, kRotThreads, 0, st>>>(p);
  else rotary_kernel<T, HALF, false><<<grid, kRotThreads, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_rotary(RotaryParams p, bool bf16, int num_sms, cudaStream_t st) {
  const int es = bf16 ? 2 : 4, n = 16 / es;
  const bool half = p.rope.layout == BASISKV_ROPE_HALF;
  auto al = [&](const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15u) == 0; };
  const bool vec = p.rot % (half ? 2 * n : n) == 0 && (p.q_stride * es) % 16 == 0 && (p.k_stride * es) % 16 == 0 &&
                   al(p.q) && al(p.k) && al(p.q_out) && al(p.k_out);
  // few tokens: one to a CTA, so that a decode step spreads over the SMs
  p.tokens_per_cta = p.tokens >= 4LL * kRotTokens * num_sms ? kRotTokens : 1;
  if (bf16) return half ? launch_t<__nv_bfloat16, true>(p, vec, st) : launch_t<__nv_bfloat16, false>(p, vec, st);
  return half ? launch_t<float, true>(p, vec, st) : launch_t<float, false>(p, vec, st);
}

}  // namespace bkv
