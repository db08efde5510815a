// Log probabilities of given tokens, with the entropy of each distribution, the
// token's rank and the most likely alternatives.
//
// Per row x of V logits: m = max x, Z = sum e^{x - m}, lse = m + log Z;
//   logprob = x_tok - lse;  entropy = log Z - sum e^{x - m} (x - m) / Z;
//   rank = number of entries ordered before the token;  alternatives = the first
//   K entries of that order (value descending, then index ascending).
// An entry's place in the order is one 64-bit key: the value's bits mapped to an
// ascending unsigned number, then the complement of the index, so no two keys
// are equal and ties need no rule of their own.
#include "common.cuh"

namespace mgd {
namespace {

constexpr int kLpThreads = 512;

__device__ __forceinline__ unsigned long long order_key(float x, unsigned j) {
  const unsigned b = __float_as_uint(x + 0.f);  // -0 and +0 are one value
  const unsigned o = (b & 0x80000000u) ? ~b : b | 0x80000000u;
  return (static_cast<unsigned long long>(o) << 32) | (0xFFFFFFFFu - j);
}

__device__ __forceinline__ float key_value(unsigned long long k) {
  const unsigned o = static_cast<unsigned>(k >> 32);
  return __uint_as_float((o & 0x80000000u) ? o & 0x7FFFFFFFu : ~o);
}

__device__ float block_sum(float v, float *red) {
  v = warp_sum_xor(v, 1, 16);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < kLpThreads / 32; ++w) s += red[w];
  return s;
}

__device__ unsigned long long block_max(unsigned long long v, unsigned long long *red) {
  for (int o = 16; o; o >>= 1) {
    const unsigned long long y = __shfl_xor_sync(0xffffffffu, v, o);
    v = y > v ? y : v;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  unsigned long long m = 0;
  for (int w = 0; w < kLpThreads / 32; ++w) m = red[w] > m ? red[w] : m;
  return m;
}

template <typename Tin>
__global__ void __launch_bounds__(kLpThreads)
    logprobs_kernel(const Tin *__restrict__ logits, int64_t stride, const int32_t *__restrict__ tokens, int R, int V,
                    int K, float *__restrict__ logprob, float *__restrict__ entropy, int32_t *__restrict__ rank,
                    int32_t *__restrict__ top_ids, float *__restrict__ top_lp, WsHeader *hdr) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ unsigned long long red64[kLpThreads / 32];
  __shared__ float red[kLpThreads / 32];
  if (blockIdx.x == 0) {
    // one CTA looks at every token and writes the call's error bits
    int bad = 0;
    for (int i = threadIdx.x; i < R; i += kLpThreads) bad |= tokens[i] < -1 || tokens[i] >= V;
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
      hdr->err[0] = bad ? 0x4u : 0u;
      hdr->err[1] = 0u;
    }
  }
  const int64_t row = blockIdx.x;
  const int tok = tokens[row];
  const Tin *x = logits + row * stride;
  const bool live = tok >= 0 && tok < V;
  unsigned long long best = 0;
  int none = 1;
  if (live) {
    none = 0;
    for (int j = threadIdx.x; j < V; j += kLpThreads) {
      const float f = to_f32(x[j]);
      none |= !(f < INFINITY);
      const unsigned long long key = order_key(f, j);
      best = key > best ? key : best;
    }
    none = __syncthreads_or(none);
    best = block_max(best, red64);
    none |= key_value(best) == -INFINITY;
  }
  if (none) {  // no token, or no distribution
    if (threadIdx.x == 0) {
      const float no = live ? __int_as_float(0x7FFFFFFF) : 0.f;
      logprob[row] = no;
      entropy[row] = no;
      rank[row] = -1;
    }
    for (int i = threadIdx.x; i < K; i += kLpThreads) {
      top_ids[row * K + i] = -1;
      top_lp[row * K + i] = -INFINITY;
    }
    return;
  }
  const float m = key_value(best), xt = to_f32(x[tok]);
  const unsigned long long tkey = order_key(xt, tok);
  float z = 0.f, zx = 0.f;
  int nb = 0;
  for (int j = threadIdx.x; j < V; j += kLpThreads) {
    const float f = to_f32(x[j]);
    const float d = f - m, e = expf(d);
    z += e;
    zx += e > 0.f ? e * d : 0.f;
    nb += order_key(f, j) > tkey;
  }
  z = block_sum(z, red);
  zx = block_sum(zx, red);
  __shared__ int cnt;
  if (threadIdx.x == 0) cnt = 0;
  __syncthreads();
  atomicAdd(&cnt, nb);
  __syncthreads();
  const float lz = logf(z);
  if (threadIdx.x == 0) {
    logprob[row] = (xt - m) - lz;
    entropy[row] = lz - zx / z;
    rank[row] = cnt;
  }
  unsigned long long below = ~0ull;
  for (int i = 0; i < K; ++i) {
    unsigned long long b = 0;
    for (int j = threadIdx.x; j < V; j += kLpThreads) {
      const unsigned long long key = order_key(to_f32(x[j]), j);
      if (key < below && key > b) b = key;
    }
    below = block_max(b, red64);
    if (threadIdx.x == 0) {
      const float f = key_value(below);
      const bool some = below != 0 && f > -INFINITY;
      top_ids[row * K + i] = some ? static_cast<int32_t>(0xFFFFFFFFu - static_cast<unsigned>(below)) : -1;
      top_lp[row * K + i] = some ? (f - m) - lz : -INFINITY;
    }
  }
}

template <typename Tin>
cudaError_t logprobs_one(const LogprobArgs &a) {
  return launch_pdl(logprobs_kernel<Tin>, dim3(a.R), dim3(kLpThreads), 0, a.stream, static_cast<const Tin *>(a.logits),
                    a.row_stride, a.tokens, a.R, a.V, a.K, a.logprob, a.entropy, a.rank, a.top_ids, a.top_logprobs,
                    static_cast<WsHeader *>(a.ws));
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs &a) {
  return a.in_f32 ? logprobs_one<float>(a) : logprobs_one<__nv_bfloat16>(a);
}

}  // namespace mgd
