// Log probabilities of given tokens, with the entropy of each distribution, the
// token's rank and the most likely alternatives, in one pass over the logits.
//
// Per row x of V logits: m = max x, Z = sum e^{x - m}, W = sum e^{x - m} (x - m);
//   logprob = (x_tok - m) - log Z;  entropy = log Z - W / Z;
//   rank = number of entries ordered before the token;  alternatives = the first
//   K entries of that order (value descending, then index ascending).
// An entry's place in the order is one 64-bit key: the value's bits mapped to an
// ascending unsigned number, then the complement of the index, so no two keys
// are equal and ties need no rule of their own.
//
// Bound by HBM.  A cluster of up to 8 CTAs shares a row; each thread holds 32
// entries of its CTA's part in registers, folds them into its own running
// (m, Z, W), counts those before the token, and the CTA looks for alternatives only
// among entries that can be one: of the 64 groups of 4 threads, each with its
// largest value, the K-th largest of these values bounds the K-th best entry from
// below, so a handful more than K entries are left to be put in order.  (Where ties
// or sorted rows leave more than the list holds, the CTA takes the maximum K times.)
// The parts meet in the first CTA's shared memory.
#include <algorithm>

#include "common.cuh"

namespace mgd {
namespace {

constexpr int kLpThreads = 256;
constexpr int kLpCtas = 3;                        // CTAs of an SM
constexpr int kLpHeld = 32;                       // entries a thread holds at once
constexpr int kLpBlock = kLpThreads * kLpHeld;    // entries a CTA holds at once
constexpr int kLpGroups = 64;                     // groups of threads, the candidates for the bound below
constexpr int kLpList = 512;                      // entries that may be put in order at once
constexpr int kLpMaxK = 32;                       // kLpGroups bounds it
constexpr int kLpMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ unsigned long long order_key(float x, unsigned j) {
  const unsigned b = __float_as_uint(x + 0.f);  // -0 and +0 are one value
  const unsigned o = (b & 0x80000000u) ? ~b : b | 0x80000000u;
  return (static_cast<unsigned long long>(o) << 32) | (0xFFFFFFFFu - j);
}
__device__ __forceinline__ float key_value(unsigned long long k) {
  const unsigned o = static_cast<unsigned>(k >> 32);
  return __uint_as_float((o & 0x80000000u) ? o & 0x7FFFFFFFu : ~o);
}
// max(a, b, c), NaN if one of them is.
__device__ __forceinline__ float fmax3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// What a CTA knows of a row.
struct RowPart {
  float m, z, w;   // maximum, sum e^{x - m}, sum e^{x - m} (x - m)
  int before;      // entries before the token
  int none;        // a NaN or +inf was seen
  int pad[3];
};
struct LpShared {
  unsigned long long list[kLpList];             // entries that may be alternatives
  unsigned long long best[kLpMaxK];             // the best so far, in order
  unsigned long long red[kLpThreads / 32];
  unsigned long long all[kLpMaxCluster][kLpMaxK];  // of every CTA, in the first one's shared memory
  RowPart part[kLpMaxCluster];
  RowPart warp[kLpThreads / 32];
  float group[kLpGroups];
  float floor;     // no alternative is below this value
  int count;
};

// One 16-byte chunk of logits as floats.
template <typename Tin>
__device__ __forceinline__ void unpack(const uint4 &c, float *x);
template <>
__device__ __forceinline__ void unpack<float>(const uint4 &c, float *x) {
  x[0] = __uint_as_float(c.x);
  x[1] = __uint_as_float(c.y);
  x[2] = __uint_as_float(c.z);
  x[3] = __uint_as_float(c.w);
}
template <>
__device__ __forceinline__ void unpack<__nv_bfloat16>(const uint4 &c, float *x) {
  const unsigned w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ void fold(RowPart &a, const RowPart &b) {
  const float m = fmaxf(a.m, b.m);
  if (m == -INFINITY) return;
  const float da = a.m - m, db = b.m - m;  // -inf for a side without a finite entry: its sums are 0
  const float ea = da == -INFINITY ? 0.f : expf(da), eb = db == -INFINITY ? 0.f : expf(db);
  const float wa = ea > 0.f ? a.w + a.z * da : 0.f, wb = eb > 0.f ? b.w + b.z * db : 0.f;
  a.w = wa * ea + wb * eb;
  a.z = a.z * ea + b.z * eb;
  a.m = m;
}

// The n keys of `from` in descending order into `to`, at most K of them: each key's place is the number
// of larger ones.  Ends with a barrier.
__device__ __forceinline__ void put_in_order(const unsigned long long *from, int n, unsigned long long *to, int K) {
  for (int i = threadIdx.x; i < n; i += kLpThreads) {
    const unsigned long long mine = from[i];
    int place = 0;
    for (int j = 0; j < n; ++j) place += from[j] > mine;
    if (mine != 0 && place < K) to[place] = mine;
  }
  __syncthreads();
}

template <typename Tin>
__global__ void __launch_bounds__(kLpThreads, kLpCtas)
    logprobs_kernel(const Tin *__restrict__ logits, int64_t stride, const int32_t *__restrict__ tokens, int R, int V,
                    int K, float *__restrict__ logprob, float *__restrict__ entropy, int32_t *__restrict__ rank,
                    int32_t *__restrict__ top_ids, float *__restrict__ top_lp, WsHeader *hdr) {
  constexpr int VE = 16 / sizeof(Tin), NCH = kLpHeld / VE;  // entries of a chunk, chunks a thread holds
  constexpr int kPerGroup = kLpThreads / kLpGroups;
  pdl_launch_dependents();
  pdl_wait();
  __shared__ LpShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = gridDim.x, part = blockIdx.x;  // the cluster spans the grid's x
  if (part == 0 && blockIdx.y == 0) {
    // one CTA looks at every token and writes the call's error bits
    int bad = 0;
    for (int i = tid; i < R; i += kLpThreads) bad |= tokens[i] < -1 || tokens[i] >= V;
    bad = __syncthreads_or(bad);
    if (tid == 0) {
      hdr->err[0] = bad ? 0x4u : 0u;
      hdr->err[1] = 0u;
    }
  }
  for (int64_t row = blockIdx.y; row < R; row += gridDim.y) {
    const int tok = tokens[row];
    if (tok < 0 || tok >= V) {  // no token (the whole cluster sees that)
      if (part == 0) {
        if (tid == 0) {
          logprob[row] = 0.f;
          entropy[row] = 0.f;
          rank[row] = -1;
        }
        if (tid < K) {
          top_ids[row * K + tid] = -1;
          top_lp[row * K + tid] = -INFINITY;
        }
      }
      continue;
    }
    const Tin *x0 = logits + row * stride;
    const float xt = to_f32(x0[tok]);
    // entries before and after the row's whole 16-byte chunks: the first CTA's first threads hold one each
    const int head = min(V, static_cast<int>(((16u - (reinterpret_cast<uintptr_t>(x0) & 15u)) & 15u) / sizeof(Tin)));
    const int chunks = (V - head) / VE, tail = V - head - chunks * VE;
    int edge = -1;  // index of that entry
    if (part == 0 && tid < head + tail) edge = tid < head ? tid : V - tail + (tid - head);
    const int per = (chunks + C - 1) / C;
    const int c0 = min(part * per, chunks), c1 = min(c0 + per, chunks);
    if (tid == 0) sh.count = 0;
    if (tid < K) sh.best[tid] = 0;

    RowPart me;
    me.m = -INFINITY;
    me.z = me.w = 0.f;
    me.before = 0;
    me.none = 0;
    float floor = -INFINITY;  // value that an alternative of this CTA has at least
    for (int base = c0; base < c1 || base == c0; base += kLpThreads * NCH) {
      float x[kLpHeld];
      {
        uint4 raw[NCH];
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
          const int c = base + i * kLpThreads + tid;
          if (c < c1) raw[i] = __ldcs(reinterpret_cast<const uint4 *>(x0 + head) + c);
        }
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
          const int c = base + i * kLpThreads + tid;
          unpack<Tin>(raw[i], x + i * VE);
          if (c >= c1) {
#pragma unroll
            for (int e = 0; e < VE; ++e) x[i * VE + e] = -INFINITY;
          }
        }
      }
      const float ex = (edge >= 0 && base == c0) ? to_f32(x0[edge]) : -INFINITY;
      float mx[2] = {ex, -INFINITY};
#pragma unroll
      for (int e = 0; e < kLpHeld; e += 4) {
        mx[0] = fmax3_nan(mx[0], x[e], x[e + 1]);
        mx[1] = fmax3_nan(mx[1], x[e + 2], x[e + 3]);
      }
      const float top = fmax3_nan(mx[0], mx[1], mx[1]);
      me.none |= !(top < INFINITY);
      // ---- sums, relative to the thread's own maximum
      if (top > me.m) {
        const float d = me.m - top;  // -inf at first: nothing is there yet
        const float e = d == -INFINITY ? 0.f : ex2(d * kLog2e);
        me.w = e > 0.f ? (me.w + me.z * d) * e : 0.f;
        me.z *= e;
        me.m = top;
      }
      const float mu = me.m == -INFINITY ? 0.f : me.m;
      const float2 nm = make_float2(-mu, -mu), l2 = make_float2(kLog2e, kLog2e);
      float2 z = make_float2(0.f, 0.f), w = make_float2(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < kLpHeld; e += 2) {
        float2 d = __fadd2_rn(make_float2(x[e], x[e + 1]), nm);
        d.x = fmaxf(d.x, -200.f);  // its exponential is 0, and so is the product with it
        d.y = fmaxf(d.y, -200.f);
        const float2 y = __fmul2_rn(d, l2);
        const float2 p = make_float2(ex2(y.x), ex2(y.y));
        z = __fadd2_rn(z, p);
        w = __ffma2_rn(p, d, w);
      }
      me.z += z.x + z.y;
      me.w += w.x + w.y;
      if (edge >= 0 && base == c0) {
        const float d = fmaxf(ex - mu, -200.f), p = ex2(d * kLog2e);
        me.z += p;
        me.w += p * d;
        me.before += ex > xt || (ex == xt && edge < tok);
      }
      // ---- entries before the token: of equal values those with a lower index
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        const int j0 = head + (base + i * kLpThreads + tid) * VE;
        if (j0 + VE <= tok) {
#pragma unroll
          for (int e = 0; e < VE; ++e) me.before += x[i * VE + e] >= xt;
        } else {
#pragma unroll
          for (int e = 0; e < VE; ++e) me.before += x[i * VE + e] > xt;
          if (j0 < tok) {  // the token's own chunk
#pragma unroll
            for (int e = 0; e < VE; ++e) me.before += x[i * VE + e] == xt && j0 + e < tok;
          }
        }
      }
      // entries past this CTA's part are -inf: none of them counts, unless the token itself is -inf
      if (xt == -INFINITY) {
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
          const int c = base + i * kLpThreads + tid, j0 = head + c * VE;
          if (c >= c1)
#pragma unroll
            for (int e = 0; e < VE; ++e) me.before -= j0 + e < tok;
        }
      }
      if (K == 0) continue;
      // ---- alternatives
      float g = top;
#pragma unroll
      for (int o = 1; o < kPerGroup; o <<= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
      __syncthreads();  // the list of the entries before this block has been used
      if (tid % kPerGroup == 0) sh.group[tid / kPerGroup] = g;
      __syncthreads();
      if (tid < kLpGroups) {
        const float mine = sh.group[tid];
        int place = 0;
        for (int j = 0; j < kLpGroups; ++j) place += sh.group[j] > mine || (sh.group[j] == mine && j < tid);
        if (place == K - 1) sh.floor = fmaxf(mine, floor);
      }
      __syncthreads();
      floor = sh.floor;
      if (top >= floor && top > -INFINITY) {
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
          const int j0 = head + (base + i * kLpThreads + tid) * VE;
#pragma unroll
          for (int e = 0; e < VE; ++e)
            if (x[i * VE + e] >= floor && x[i * VE + e] > -INFINITY) {
              const int at = atomicAdd(&sh.count, 1);
              if (at < kLpList - kLpMaxK) sh.list[at] = order_key(x[i * VE + e], j0 + e);
            }
        }
        if (edge >= 0 && base == c0 && ex >= floor && ex > -INFINITY) {
          const int at = atomicAdd(&sh.count, 1);
          if (at < kLpList - kLpMaxK) sh.list[at] = order_key(ex, edge);
        }
      }
      __syncthreads();
      const int n = sh.count;
      if (n <= kLpList - kLpMaxK) {
        // the best so far go behind them, and all are put in order
        if (tid < K) sh.list[n + tid] = sh.best[tid];
        __syncthreads();
        if (tid < K) sh.best[tid] = 0;
        if (tid == 0) sh.count = 0;
        __syncthreads();
        put_in_order(sh.list, n + K, sh.best, K);
      } else {
        // too many are level: the largest key below the last one, K times
        if (tid < K) sh.list[tid] = sh.best[tid];
        unsigned long long below = ~0ull;
        __syncthreads();
        for (int k = 0; k < K; ++k) {
          unsigned long long b = tid < K && sh.list[tid] < below ? sh.list[tid] : 0;
#pragma unroll
          for (int i = 0; i < NCH; ++i) {
            const int j0 = head + (base + i * kLpThreads + tid) * VE;
#pragma unroll
            for (int e = 0; e < VE; ++e) {
              const unsigned long long key = x[i * VE + e] > -INFINITY ? order_key(x[i * VE + e], j0 + e) : 0;
              if (key < below && key > b) b = key;
            }
          }
          if (edge >= 0 && base == c0 && ex > -INFINITY) {
            const unsigned long long key = order_key(ex, edge);
            if (key < below && key > b) b = key;
          }
          for (int o = 16; o; o >>= 1) {
            const unsigned long long y = __shfl_xor_sync(0xffffffffu, b, o);
            b = y > b ? y : b;
          }
          if (lane == 0) sh.red[warp] = b;
          __syncthreads();
          b = 0;
          for (int i = 0; i < kLpThreads / 32; ++i) b = sh.red[i] > b ? sh.red[i] : b;
          if (tid == 0) sh.best[k] = b;
          below = b;
          __syncthreads();
        }
        if (tid == 0) sh.count = 0;
      }
      if (sh.best[K - 1] != 0) floor = fmaxf(floor, key_value(sh.best[K - 1]));
    }
    // ---- this CTA's part
    for (int o = 16; o; o >>= 1) {
      RowPart y;
      y.m = __shfl_xor_sync(0xffffffffu, me.m, o);
      y.z = __shfl_xor_sync(0xffffffffu, me.z, o);
      y.w = __shfl_xor_sync(0xffffffffu, me.w, o);
      fold(me, y);
    }
    me.before = __reduce_add_sync(0xffffffffu, me.before);
    me.none = __any_sync(0xffffffffu, me.none);
    if (lane == 0) sh.warp[warp] = me;
    __syncthreads();
    if (warp == 0) {
      me = sh.warp[lane & (kLpThreads / 32 - 1)];
      if (lane >= kLpThreads / 32) {
        me.m = -INFINITY;
        me.z = me.w = 0.f;
        me.before = me.none = 0;
      }
      for (int o = 16; o; o >>= 1) {
        RowPart y;
        y.m = __shfl_xor_sync(0xffffffffu, me.m, o);
        y.z = __shfl_xor_sync(0xffffffffu, me.z, o);
        y.w = __shfl_xor_sync(0xffffffffu, me.w, o);
        fold(me, y);
      }
      me.before = __reduce_add_sync(0xffffffffu, me.before);
      me.none = __any_sync(0xffffffffu, me.none);
      if (lane < 8) {  // to the first CTA: the part as eight words
        const float v = lane == 0 ? me.m : lane == 1 ? me.z : lane == 2 ? me.w : __int_as_float(lane == 3 ? me.before : lane == 4 ? me.none : 0);
        st_cluster_f(reinterpret_cast<float *>(&sh.part[part]) + lane, 0, v);
      }
    }
    if (tid < K) st_cluster_u64(&sh.all[part][tid], 0, sh.best[tid]);
    if (C > 1)
      cluster_sync_all();
    else
      __syncthreads();
    // ---- the first CTA joins the parts
    if (part == 0) {
      RowPart r = sh.part[0];
      for (int c = 1; c < C; ++c) {
        const RowPart o = sh.part[c];
        fold(r, o);
        r.before += o.before;
        r.none |= o.none;
      }
      const bool none = r.none || r.m == -INFINITY;
      const float lz = logf(r.z);
      if (tid == 0) {
        logprob[row] = none ? __int_as_float(0x7FFFFFFF) : (xt - r.m) - lz;
        entropy[row] = none ? __int_as_float(0x7FFFFFFF) : lz - r.w / r.z;
        rank[row] = none ? -1 : r.before;
      }
      if (K > 0) {
        if (C > 1) {
          for (int i = tid; i < C * K; i += kLpThreads) sh.list[i] = sh.all[i / K][i % K];
          __syncthreads();
          if (tid < K) sh.best[tid] = 0;
          __syncthreads();
          put_in_order(sh.list, C * K, sh.best, K);
        }
        if (tid < K) {
          const unsigned long long key = none ? 0 : sh.best[tid];
          top_ids[row * K + tid] = key ? static_cast<int32_t>(0xFFFFFFFFu - static_cast<unsigned>(key)) : -1;
          top_lp[row * K + tid] = key ? (key_value(key) - r.m) - lz : -INFINITY;
        }
      }
    }
    // the next row's parts come after this one's have been read
    if (C > 1)
      cluster_sync_all();
    else
      __syncthreads();
  }
}

template <typename Tin>
cudaError_t logprobs_one(const LogprobArgs &a) {
  // CTAs a row: as many as the row fills, up to 8, for few rows; with many rows fewer and longer parts,
  // as long as about eight waves of CTAs are left to even out the ends.
  int C = 1;
  while (C < kLpMaxCluster && a.V > C * (kLpBlock / 4)) C *= 2;
  while (C > 1 && static_cast<int64_t>(a.R) * (C / 2) >= 8LL * kLpCtas * current_sm_count()) C /= 2;
  return launch_pdl_cluster(logprobs_kernel<Tin>, dim3(C, std::min(a.R, 65535)), dim3(kLpThreads), dim3(C), 0, a.stream,
                            static_cast<const Tin *>(a.logits), a.row_stride, a.tokens, a.R, a.V, a.K, a.logprob,
                            a.entropy, a.rank, a.top_ids, a.top_logprobs, static_cast<WsHeader *>(a.ws));
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs &a) {
  return a.in_f32 ? logprobs_one<float>(a) : logprobs_one<__nv_bfloat16>(a);
}

}  // namespace mgd
