// Attention over a prefix that every sequence of a batch shares, computed once
// for all of them: the plan, the CUDA-core kernel for float32 inputs, and the merge of
// the prefix part with the part over each sequence's own cache.
//
// With s_j = scale <q, k_j>, the softmax over prefix and own keys splits exactly:
//   (O_P, l_P), (O_b, l_b) = the two parts' outputs and log-sum-exps
//   l = log(e^{l_P} + e^{l_b}),  O = e^{l_P - l} O_P + e^{l_b - l} O_b.
// The own part is the verify attention kernel with a float32 output; the prefix part has
// B * T * G query rows a KV head instead of T * G, which turns the one
// read of the prefix into a matrix product.
#include <algorithm>

#include "common.cuh"
#include "prefix.cuh"

namespace mgd {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ---------------------------------------------------------------- CUDA cores
// Tiles of 64 rows x 64 keys, float32 throughout: 256 threads as 16 x 16, each
// with 4 x 4 scores and 4 x D/16 outputs in registers, K and V tiles in shared
// memory, the running maximum and sum of a row held by the 16 threads that share
// it.  It serves float32 inputs (the tensor cores have no float32 form).
constexpr int kSRows = 64, kSKeys = 64, kSThreads = 256;

template <int D>
struct SimtLayout {
  static constexpr int kStride = D + 4;  // floats between rows: 16 rows fall into 8 bank groups of 4
  static constexpr int kPStride = kSKeys + 4;
  static constexpr int off_k = kSRows * kStride;
  static constexpr int off_v = off_k + kSKeys * kStride;
  static constexpr int off_p = off_v + kSKeys * kStride;
  static constexpr int bytes = (off_p + kSRows * kPStride) * 4;
};

__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }

template <int D>
__global__ void __launch_bounds__(kSThreads)
    prefix_simt_kernel(const float *__restrict__ q, const float *__restrict__ k, const float *__restrict__ v,
                       const int32_t *__restrict__ prefix_len, int64_t head_stride, float sl2, PrefixGeom g,
                       float *__restrict__ part_o, float *__restrict__ part_l, WsHeader *hdr) {
  pdl_launch_dependents();
  pdl_wait();
  using Lay = SimtLayout<D>;
  constexpr int NC = D / 64;  // float4 output columns a thread holds, 64 apart
  extern __shared__ float sm[];
  float *sq = sm, *sk = sm + Lay::off_k, *sv = sm + Lay::off_v, *sp = sm + Lay::off_p;
  const int plen = prefix_len[0];
  if (plen < 0 || plen > g.prefix_cap) {
    if (blockIdx.x == 0 && threadIdx.x == 0) raise_error_sr(hdr, 0x1u);
    return;
  }
  const PrefixLine w = prefix_line(g, plen, gridDim.x);
  const int c = blockIdx.x;
  if (c >= w.n) return;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  int x = prefix_cta_begin(w, c);
  const int x1 = prefix_cta_begin(w, c + 1);
  while (x < x1) {
    const int h = x / w.head;
    const int rt = min((x - h * w.head) / w.nt, g.RT - 1);
    const int begin = prefix_pair_begin(w, h, rt);
    const int end = min(x1, begin + prefix_pair_steps(g, w, rt));
    const int row0 = rt * kSRows;
    __syncthreads();
    for (int i = threadIdx.x; i < kSRows * (D / 4); i += kSThreads) {
      const int r = i / (D / 4), d = 4 * (i % (D / 4));
      float4 val = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row0 + r < g.R) {
        const int bt = (row0 + r) / g.G, gg = (row0 + r) % g.G;
        val = load4(q + (static_cast<int64_t>(bt) * g.Hq + h * g.G + gg) * D + d);
      }
      *reinterpret_cast<float4 *>(sq + r * Lay::kStride + d) = val;
    }
    float m[4], l[4], acc[4][4 * NC];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int e = 0; e < 4 * NC; ++e) acc[i][e] = 0.f;
    }
    for (; x < end; ++x) {
      const int key0 = (x - begin) * kSKeys;
      const int nk = min(kSKeys, plen - key0);
      __syncthreads();  // the tile before has been read
      for (int i = threadIdx.x; i < kSKeys * (D / 4); i += kSThreads) {
        const int r = i / (D / 4), d = 4 * (i % (D / 4));
        float4 kk = make_float4(0.f, 0.f, 0.f, 0.f), vv = kk;  // rows past the prefix hold anything
        if (r < nk) {
          const int64_t off = h * head_stride + static_cast<int64_t>(key0 + r) * D + d;
          kk = load4(k + off);
          vv = load4(v + off);
        }
        *reinterpret_cast<float4 *>(sk + r * Lay::kStride + d) = kk;
        *reinterpret_cast<float4 *>(sv + r * Lay::kStride + d) = vv;
      }
      __syncthreads();
      float s[4][4] = {};
      for (int d = 0; d < D; d += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4 *>(sq + (4 * ty + i) * Lay::kStride + d);
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4 *>(sk + (tx + 16 * j) * Lay::kStride + d);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s[i][j] = fmaf(a[i].x, b[j].x, s[i][j]);
            s[i][j] = fmaf(a[i].y, b[j].y, s[i][j]);
            s[i][j] = fmaf(a[i].z, b[j].z, s[i][j]);
            s[i][j] = fmaf(a[i].w, b[j].w, s[i][j]);
          }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = (tx + 16 * j < nk) ? s[i][j] * sl2 : -INFINITY;
          mx = fmaxf(mx, s[i][j]);
        }
        mx = fmaxf(m[i], warp_max_xor(mx, 1, 8));
        const float mu = (mx == -INFINITY) ? 0.f : mx;
        const float alpha = exp2f(m[i] - mu);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float e = exp2f(s[i][j] - mu);
          sum += e;
          sp[(4 * ty + i) * Lay::kPStride + tx + 16 * j] = e;
        }
        l[i] = l[i] * alpha + warp_sum_xor(sum, 1, 8);
        m[i] = mx;
#pragma unroll
        for (int e = 0; e < 4 * NC; ++e) acc[i][e] *= alpha;
      }
      __syncwarp();  // a row's 64 probabilities come from the 16 threads of its own half-warp
      for (int j = 0; j < kSKeys; j += 4) {
        float4 pr[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) pr[i] = *reinterpret_cast<const float4 *>(sp + (4 * ty + i) * Lay::kPStride + j);
#pragma unroll
        for (int jj = 0; jj < 4; ++jj)
#pragma unroll
          for (int cc = 0; cc < NC; ++cc) {
            const float4 vv = *reinterpret_cast<const float4 *>(sv + (j + jj) * Lay::kStride + 64 * cc + 4 * tx);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float pe = jj == 0 ? pr[i].x : jj == 1 ? pr[i].y : jj == 2 ? pr[i].z : pr[i].w;
              acc[i][4 * cc] = fmaf(pe, vv.x, acc[i][4 * cc]);
              acc[i][4 * cc + 1] = fmaf(pe, vv.y, acc[i][4 * cc + 1]);
              acc[i][4 * cc + 2] = fmaf(pe, vv.z, acc[i][4 * cc + 2]);
              acc[i][4 * cc + 3] = fmaf(pe, vv.w, acc[i][4 * cc + 3]);
            }
          }
      }
      __syncwarp();
    }
    const int64_t slot = c + h * g.RT + rt;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * ty + i;
      if (row0 + r >= g.R) continue;
      const float inv = l[i] > 0.f ? 1.f / l[i] : 0.f;
#pragma unroll
      for (int cc = 0; cc < NC; ++cc)
        *reinterpret_cast<float4 *>(part_o + (slot * g.slot_rows + r) * D + 64 * cc + 4 * tx) =
            make_float4(acc[i][4 * cc] * inv, acc[i][4 * cc + 1] * inv, acc[i][4 * cc + 2] * inv,
                        acc[i][4 * cc + 3] * inv);
      if (tx == 0) part_l[slot * g.slot_rows + r] = l[i] > 0.f ? (m[i] + log2f(l[i])) * kLn2 : -INFINITY;
    }
  }
}

// ---------------------------------------------------------------- merge
// D / 4 lanes per query row, four columns each: the own part and the row's partial results over the
// prefix, weighted by their log-sum-exps.  Bound by L2: own part, partial results and output once each.
constexpr int kMergeThreads = 256;

template <int D>
__global__ void __launch_bounds__(kMergeThreads)
    prefix_merge_kernel(const float *__restrict__ own_o, const float *__restrict__ own_l,
                        const float *__restrict__ part_o, const float *__restrict__ part_l,
                        const int32_t *__restrict__ prefix_len, PrefixGeom g, int grid, float *__restrict__ out_f32,
                        __nv_bfloat16 *__restrict__ out_bf16, float *__restrict__ lse_out) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int kLanes = D / 4;
  const int d = 4 * (threadIdx.x % kLanes);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kMergeThreads / kLanes) + threadIdx.x / kLanes;  // (b, t, hq)
  if (row >= static_cast<int64_t>(g.B) * g.T * g.Hq) return;
  const int plen = prefix_len[0];
  float m = own_l[row], sum = 1.f;
  float4 o = *reinterpret_cast<const float4 *>(own_o + row * D + d);
  if (plen < 0 || plen > g.prefix_cap) return;  // flagged by the prefix kernel
  if (plen > 0) {
    const int hq = static_cast<int>(row % g.Hq), bt = static_cast<int>(row / g.Hq);
    const int h = hq / g.G, r = bt * g.G + hq % g.G;
    const int rt = r / g.tile_rows, lr = r % g.tile_rows;
    const PrefixLine w = prefix_line(g, plen, grid);
    const int begin = prefix_pair_begin(w, h, rt);
    const int c0 = prefix_cta_of(w, begin), c1 = prefix_cta_of(w, begin + prefix_pair_steps(g, w, rt) - 1);
    const int64_t at0 = static_cast<int64_t>(h * g.RT + rt) * g.slot_rows + lr;
    for (int c = c0; c <= c1; c += 4) {  // four partial results on their way at once
      float l[4];
      float4 x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t at = at0 + static_cast<int64_t>(min(c + i, c1)) * g.slot_rows;
        l[i] = __ldcg(part_l + at);
        x[i] = __ldcg(reinterpret_cast<const float4 *>(part_o + at * D + d));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float mn = fmaxf(m, l[i]);
        if (c + i > c1 || mn == -INFINITY) continue;  // past the last, or no finite score so far
        const float a = expf(m - mn), b = expf(l[i] - mn);
        sum = sum * a + b;
        o.x = o.x * a + x[i].x * b;
        o.y = o.y * a + x[i].y * b;
        o.z = o.z * a + x[i].z * b;
        o.w = o.w * a + x[i].w * b;
        m = mn;
      }
    }
  }
  const float inv = 1.f / sum;
  o.x *= inv;
  o.y *= inv;
  o.z *= inv;
  o.w *= inv;
  if (out_bf16)
    *reinterpret_cast<uint2 *>(out_bf16 + row * D + d) = make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
  else
    *reinterpret_cast<float4 *>(out_f32 + row * D + d) = o;
  if (lse_out && d == 0) lse_out[row] = m + logf(sum);
}

template <int D>
cudaError_t simt_one(const PrefixPlan &p, const PrefixArgs &a) {
  auto kern = prefix_simt_kernel<D>;
  constexpr int smem = SimtLayout<D>::bytes;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  unsigned char *ws = static_cast<unsigned char *>(a.ws);
  return launch_pdl(kern, dim3(p.grid), dim3(kSThreads), smem, a.stream, static_cast<const float *>(a.q),
                    static_cast<const float *>(a.k), static_cast<const float *>(a.v), a.prefix_len, a.head_stride,
                    a.sm_scale * kLog2e, p.g, reinterpret_cast<float *>(ws + p.off_part_o),
                    reinterpret_cast<float *>(ws + p.off_part_l), static_cast<WsHeader *>(a.ws));
}

}  // namespace

cudaError_t launch_prefix_simt(const PrefixPlan &p, const PrefixArgs &a) {
  return p.g.D == 128 ? simt_one<128>(p, a) : simt_one<64>(p, a);
}

cudaError_t launch_prefix_merge(const PrefixPlan &p, const PrefixArgs &a) {
  const unsigned char *ws = static_cast<const unsigned char *>(a.ws);
  const int64_t rows = static_cast<int64_t>(p.g.B) * p.g.T * p.g.Hq;
  const int per = kMergeThreads / (p.g.D / 4);
  const dim3 grid(static_cast<unsigned>((rows + per - 1) / per));
  return launch_pdl(p.g.D == 128 ? prefix_merge_kernel<128> : prefix_merge_kernel<64>, grid, dim3(kMergeThreads), 0,
                    a.stream, reinterpret_cast<const float *>(ws + p.off_own_o),
                    reinterpret_cast<const float *>(ws + p.off_own_l),
                    reinterpret_cast<const float *>(ws + p.off_part_o),
                    reinterpret_cast<const float *>(ws + p.off_part_l), a.prefix_len, p.g, p.grid,
                    a.out_bf16 ? nullptr : static_cast<float *>(a.out),
                    a.out_bf16 ? static_cast<__nv_bfloat16 *>(a.out) : nullptr, a.lse);
}

// The prefix kernel is bound by its tensor cores and their latency, the attention over the own caches by
// HBM, so the prefix kernel takes only part of the SMs and the other one runs beside it.  Its clusters
// out of `most`: the number that by these measured rates ends both first -- 1.7 us a step, 100 GB/s of
// own cache an SM, 6600 GB/s in all -- with the capacities in place of the lengths, which only the device
// knows.
int prefix_share(const PrefixPlan &p, int most, int sm_count) {
  const PrefixLine line = prefix_line(p.g, p.g.prefix_cap, most);
  const double own = 4.0 * p.g.B * p.g.Hkv * p.own_cap * p.g.D;  // bytes of K and V
  double best = 0.0;
  int share = most;
  for (int n = most; n >= (most + 1) / 2; --n) {
    const double prefix_us = 1.7 * ((line.total + n - 1) / n);
    const double beside = 0.1e6 * (sm_count - 2 * n) * prefix_us;
    const double us = prefix_us + (own > beside ? (own - beside) / 6.6e6 : 0.0);
    if (n == most || us < best) {
      best = us;
      share = n;
    }
  }
  return share;
}

PrefixPlan plan_prefix(int B, int T, int Hq, int Hkv, int D, int prefix_cap, int kv_cap, int in_f32, int sm_count) {
  PrefixPlan p{};
  PrefixGeom &g = p.g;
  g.B = B;
  g.T = T;
  g.Hq = Hq;
  g.Hkv = Hkv;
  g.D = D;
  g.G = Hq / Hkv;
  g.R = B * T * g.G;
  g.prefix_cap = prefix_cap;
  g.tile_rows = in_f32 ? kSRows : 512;
  g.key_tile = in_f32 ? kSKeys : 128;
  g.RT = (g.R + g.tile_rows - 1) / g.tile_rows;
  g.last_half = !in_f32 && g.R - (g.RT - 1) * g.tile_rows <= 256;
  g.slot_rows = std::min(g.tile_rows, g.R);
  p.own = plan_attention(B, T, Hq, Hkv, D, kv_cap, sm_count, !in_f32);
  p.own_cap = kv_cap;
  // what fits at once: two CTAs of 116 KB shared memory an SM; clusters of two CTAs of 226 KB
  p.grid = in_f32 ? 2 * sm_count : std::max(1, sm_count / 2);
  const size_t rows = static_cast<size_t>(B) * T * Hq;
  const size_t slots = static_cast<size_t>(p.grid) + static_cast<size_t>(Hkv) * g.RT;
  size_t off = align_up(p.own.ws_bytes);  // the own attention's scratch (and the header) comes first
  p.off_own_o = off;
  off = align_up(off + rows * D * sizeof(float));
  p.off_own_l = off;
  off = align_up(off + rows * sizeof(float));
  p.off_part_o = off;
  off = align_up(off + slots * g.slot_rows * D * sizeof(float));
  p.off_part_l = off;
  off = align_up(off + slots * g.slot_rows * sizeof(float));
  p.ws_bytes = off;
  return p;
}

}  // namespace mgd
