// Rotary positions for the new rows of every sequence, and their append to the
// KV cache, in one pass.
//
// Pair i of a head (elements i and i + R/2, or 2i and 2i + 1; R = rotary_dim)
// at position pos turns by the angle 2 pi * frac(pos * f_i), f_i in turns per
// position: (x, y) -> mag * (x cos - y sin, x sin + y cos).  f_i is held as
// round(f_i * 2^64) in an unsigned 64-bit number, so pos * f_i modulo one turn is
// one wrapping integer product with an error of |pos| / 2 units of 2^-64 turns at
// any position, where a float32 angle at position 10^6 would be off by 0.03
// radians.  The cosine and sine of each (row, pair) are computed once in float32
// and shared by all heads; rotated values are rounded once, to the data's type.
//
// Bound by HBM: every element is read once and written once.
#include "common.cuh"

namespace mgd {
namespace {

constexpr int kRopeThreads = 256;

struct RopeParams {
  int T, Hq, Hkv, D, half, interleaved, kv_cap, pos_stride;
  int64_t q_stride, k_stride, v_stride;  // elements between the rows of two tokens
  int64_t kv_bstride, kv_hstride;
  float magnitude;
};

template <typename Tin>
__device__ __forceinline__ Tin from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

template <typename Tin>
__global__ void __launch_bounds__(kRopeThreads)
    rope_append_kernel(const Tin *__restrict__ q, const Tin *__restrict__ kn, const Tin *__restrict__ vn,
                       const unsigned long long *__restrict__ turns, const int32_t *__restrict__ kv_len,
                       const int32_t *__restrict__ new_len, const int32_t *__restrict__ pos_offset,
                       Tin *__restrict__ q_out, Tin *__restrict__ k, Tin *__restrict__ v, int B, RopeParams p,
                       WsHeader *hdr) {
  pdl_launch_dependents();
  pdl_wait();
  extern __shared__ float2 cs[];  // [half]
  if (blockIdx.x == 0) {
    // one CTA looks at every sequence and writes the call's error bits
    int bad = 0;
    for (int i = threadIdx.x; i < B; i += kRopeThreads) {
      const int L = kv_len[i], n = new_len ? new_len[i] : p.T;
      bad |= n < 0 || n > p.T || L < n || L > p.kv_cap;
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
      hdr->err[0] = bad ? 0x1u : 0u;
      hdr->err[1] = 0u;
    }
  }
  const int64_t token = blockIdx.x;
  const int b = static_cast<int>(token / p.T), t = static_cast<int>(token % p.T);
  const int L = kv_len[b], n = new_len ? new_len[b] : p.T;
  if (n < 0 || n > p.T || L < n || L > p.kv_cap || t >= n) return;
  const int row = L - n + t;
  const int64_t pos = static_cast<int64_t>(row) + (pos_offset ? pos_offset[b * p.pos_stride] : 0);
  for (int i = threadIdx.x; i < p.half; i += kRopeThreads) {
    const long long a = static_cast<long long>(static_cast<unsigned long long>(pos) * turns[i]);
    float sn, cn;
    sincospif(static_cast<float>(a) * 0x1p-63f, &sn, &cn);
    cs[i] = make_float2(cn * p.magnitude, sn * p.magnitude);
  }
  __syncthreads();
  const int heads = p.Hq + 2 * p.Hkv;
  const int units = p.half + (p.D - 2 * p.half);  // pairs, then the elements past the rotated part
  for (int i = threadIdx.x; i < heads * units; i += kRopeThreads) {
    const int h = i / units, u = i % units;
    const Tin *src;
    Tin *dst;
    bool turn = true;
    if (h < p.Hq) {
      src = q + token * p.q_stride + static_cast<int64_t>(h) * p.D;
      dst = q_out + (token * p.Hq + h) * p.D;
    } else if (h < p.Hq + p.Hkv) {
      const int hk = h - p.Hq;
      src = kn + token * p.k_stride + static_cast<int64_t>(hk) * p.D;
      dst = k + b * p.kv_bstride + hk * p.kv_hstride + static_cast<int64_t>(row) * p.D;
    } else {
      const int hk = h - p.Hq - p.Hkv;
      src = vn + token * p.v_stride + static_cast<int64_t>(hk) * p.D;
      dst = v + b * p.kv_bstride + hk * p.kv_hstride + static_cast<int64_t>(row) * p.D;
      turn = false;
    }
    if (u >= p.half) {
      dst[u + p.half] = src[u + p.half];
      continue;
    }
    const int i0 = p.interleaved ? 2 * u : u, i1 = p.interleaved ? 2 * u + 1 : u + p.half;
    const Tin x = src[i0], y = src[i1];
    if (!turn) {
      dst[i0] = x;
      dst[i1] = y;
      continue;
    }
    const float xf = to_f32(x), yf = to_f32(y);
    const float2 c = cs[u];
    dst[i0] = from_f32<Tin>(xf * c.x - yf * c.y);
    dst[i1] = from_f32<Tin>(xf * c.y + yf * c.x);
  }
}

template <typename Tin>
cudaError_t rope_one(const RopeArgs &a, const RopeParams &p) {
  return launch_pdl(rope_append_kernel<Tin>, dim3(static_cast<unsigned>(a.B) * a.T), dim3(kRopeThreads),
                    static_cast<size_t>(p.half) * sizeof(float2), a.stream, static_cast<const Tin *>(a.q),
                    static_cast<const Tin *>(a.k_new), static_cast<const Tin *>(a.v_new),
                    static_cast<const unsigned long long *>(a.turns), a.kv_len, a.new_len, a.pos_offset,
                    static_cast<Tin *>(a.q_out), static_cast<Tin *>(a.k), static_cast<Tin *>(a.v), a.B, p,
                    static_cast<WsHeader *>(a.ws));
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs &a) {
  RopeParams p;
  p.T = a.T;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.D = a.D;
  p.half = a.rotary_dim / 2;
  p.interleaved = a.interleaved;
  p.kv_cap = a.kv_cap;
  p.pos_stride = a.pos_stride;
  p.q_stride = a.q_stride;
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  p.kv_bstride = a.kv_batch_stride;
  p.kv_hstride = a.kv_head_stride;
  p.magnitude = a.magnitude;
  return a.in_f32 ? rope_one<float>(a, p) : rope_one<__nv_bfloat16>(a, p);
}

}  // namespace mgd
