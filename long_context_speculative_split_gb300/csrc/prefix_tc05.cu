// Attention of all B * T * G query rows of a KV head over the shared prefix on
// the 5th-generation tensor cores (bf16 inputs), sm_103a.
//
// A CTA works on two blocks of 128 query rows at a time ("slots"), each with its
// own accumulators in tensor memory and its own group of four softmax warps:
//   S_w = Q_w K^T      tcgen05.mma, both operands in shared memory, 128 x 128
//   P_w = 2^(S_w * scale*log2(e) - m_w)   float16, written over S_w
//   O_w += P_w V       tcgen05.mma, P_w from tensor memory, V float16
// The MMA thread issues O_0 += P_0 V, S_0 = Q_0 K (next tile), O_1 += P_1 V,
// S_1 = Q_1 K, ..., so while one slot's softmax runs the tensor cores work for the
// other slot, and both slots use a key tile while it is in shared memory.  A head's
// last row block may have 128 rows or fewer: then both slots hold the same rows and
// take alternate key tiles, and their results are joined in tensor memory at the end.
//
// P in float16 has 11 significant bits (bfloat16: 8), which keeps the error of the
// P V product at 1.5e-4 of the result; an MMA takes A and B of one type, so four
// warps load the V tiles from global memory, convert them (exact for magnitudes in
// [2^-14, 65504]) and store them in the tensor cores' swizzled layout.  The running
// maximum m_w is only raised when a row's maximum exceeds it by more than 2^8 (P
// stays below 256, far inside float16): raising it means rescaling O_w in tensor
// memory.  The sum of exponentials is kept in float32, unrounded.
//
// Roles (16 warps, one CTA per SM): 0-3 and 4-7 softmax of slot 0 / 1, 8-11 query
// rows and V, 12 MMA issue, 13 K tiles by TMA.  Registers a thread: 192, 96 and 32 for
// the three kinds of warp group (2 * 192 + 96 + 32 = 4 * 128, the launch's own total).
#include <algorithm>

#include "common.cuh"
#include "prefix.cuh"

namespace mgd {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kPRows = 128;   // query rows of a slot
constexpr int kPKeys = 128;   // keys of a tile
constexpr int kPThreads = 512;
constexpr float kRaise = 8.f;  // log2 of how far a row's maximum may exceed the one P is scaled by

template <int D>
struct PLayout {
  static constexpr int kHalf = 128 * 128;         // 128 rows x 64 16-bit columns, 128-byte swizzled
  static constexpr int kTile = (D / 64) * kHalf;  // 128 rows of Q, K or V
  static constexpr int kKStages = D == 128 ? 3 : 4;
  static constexpr int kVStages = D == 128 ? 2 : 4;
  static constexpr int off_q = 0;
  static constexpr int off_k = 2 * kTile;
  static constexpr int off_v = off_k + kKStages * kTile;
  static constexpr int off_bar = off_v + kVStages * kTile;
  static constexpr int kBars = 2 * kKStages + 2 * kVStages + 2 + 2 + 2 + 2 + 2 + 1;
  static constexpr int off_tmem = off_bar + kBars * 8;
  static constexpr int off_abort = off_tmem + 8;
  static constexpr int off_ml = off_abort + 8;    // float2 [128]: slot 1's maximum and sum
  static constexpr int bytes = off_ml + 128 * 8;
  static constexpr int alloc = bytes + 1024;      // the base is rounded up to 1024
  static_assert(alloc <= 227 * 1024, "shared memory of one CTA");
};
constexpr uint32_t kPTmemCols = 512;  // S_0, S_1 (128 columns each), O_0, O_1 (D each)

struct PParams {
  PrefixGeom g;
  int64_t head_stride;
  float sl2;      // |scale| * log2(e); the sign goes into the query rows
  uint32_t flip;  // 0x80008000 when the scale is negative
};

// This CTA's next run of steps within one pair.
struct PSeg {
  int h, rt, first, n;  // first: step within the pair
  bool dual;            // two row blocks, one key tile a step
};
__device__ __forceinline__ PSeg next_seg(const PrefixGeom &g, const PrefixLine &w, int x, int x1) {
  PSeg s;
  s.h = x / w.head;
  s.rt = min((x - s.h * w.head) / w.nt, g.RT - 1);
  const int begin = prefix_pair_begin(w, s.h, s.rt);
  s.first = x - begin;
  s.n = min(x1, begin + prefix_pair_steps(g, w, s.rt)) - x;
  s.dual = !(g.last_half && s.rt == g.RT - 1);
  return s;
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e != 0;
}
// D[128 x N] (+)= A[128 x 16] B[16 x N] with A (float16 pairs) in tensor memory.
__device__ __forceinline__ void umma_f16_ts(uint32_t dtmem, uint32_t atmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(dtmem),
      "r"(atmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Descriptor of V as the B operand, its rows (keys) along the contraction and its columns contiguous:
// 128-byte swizzle, 64-column blocks kHalf bytes apart, groups of 8 keys 1024 bytes apart.
__device__ __forceinline__ uint64_t umma_desc_v(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>((128 * 128) >> 4) << 16;  // leading byte offset
  d |= static_cast<uint64_t>(1024u >> 4) << 32;        // stride byte offset
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}
// kind::f16 with D float32, A and B float16, A along the contraction, B across it.
__host__ __device__ constexpr uint32_t umma_idesc_f16_bt(uint32_t M, uint32_t N) {
  return (1u << 4) | (1u << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// A bounded wait that also gives up at once after any other wait of the CTA
// gave up; a failure raises the timeout bit and sets the CTA's abort flag.
__device__ __forceinline__ bool wait_or_abort(uint64_t *bar, uint32_t parity, WsHeader *hdr, volatile int *abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  if (*abort_flag) return false;
  if (mbar_wait(bar, parity)) return true;
  raise_error_sr(hdr, 0x8u);
  *abort_flag = 1;
  return false;
}

// The same for a whole warp, which goes on or gives up together.
__device__ __forceinline__ bool all_wait(uint64_t *bar, uint32_t parity, WsHeader *hdr, volatile int *abort_flag) {
  return __all_sync(0xffffffffu, wait_or_abort(bar, parity, hdr, abort_flag));
}

// P = 2^(s * s2 - mu) of one row's 128 scores into tensor memory as float16 pairs, 32 keys a store;
// returns their float32 sum.  kMask: only the first nk keys count (with a scale of 0 the product
// of a masked score is NaN, so they are left out by their place).
template <bool kMask>
__device__ __forceinline__ float weights(const uint32_t (&sv)[4][32], uint32_t p_addr, float2 s2, float mu, int nk) {
  const float2 nm = make_float2(-mu, -mu);
  float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    uint32_t pk[16];
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
      const float2 y =
          __ffma2_rn(make_float2(__uint_as_float(sv[h][c]), __uint_as_float(sv[h][c + 1])), s2, nm);
      float a = ex2(y.x), b = ex2(y.y);
      if (kMask) {
        a = 32 * h + c < nk ? a : 0.f;
        b = 32 * h + c + 1 < nk ? b : 0.f;
      }
      sum[(c >> 1) & 1] = __fadd2_rn(sum[(c >> 1) & 1], make_float2(a, b));
      pk[c >> 1] = pack_f16(a, b);
    }
    tmem_st16(p_addr + 16 * h, pk);
  }
  return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}

// 8 consecutive floats in one store.
__device__ __forceinline__ void st_f8(float *p, const float (&v)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

template <int D>
__global__ void __launch_bounds__(kPThreads, 1)
    prefix_tc05_kernel(const __grid_constant__ CUtensorMap kmap, const __nv_bfloat16 *__restrict__ q,
                       const __nv_bfloat16 *__restrict__ v, const int32_t *__restrict__ prefix_len,
                       float *__restrict__ part_o, float *__restrict__ part_l, WsHeader *hdr, PParams p) {
  using Lay = PLayout<D>;
  constexpr int KS = Lay::kKStages, VS = Lay::kVStages;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *k_full = reinterpret_cast<uint64_t *>(smem + Lay::off_bar);  // [KS] K tile landed
  uint64_t *k_empty = k_full + KS;   // [KS] its products are done
  uint64_t *v_full = k_empty + KS;   // [VS] V tile stored by the four converting warps
  uint64_t *v_empty = v_full + VS;   // [VS] its products are done
  uint64_t *q_full = v_empty + VS;   // query rows of the segment stored
  uint64_t *q_empty = q_full + 1;    // every S product of the segment done
  uint64_t *s_full = q_empty + 1;    // [2] S of a slot written (and every earlier product done)
  uint64_t *p_full = s_full + 2;     // [2] P of a slot written by its four warps
  uint64_t *o_done = p_full + 2;     // [2] a slot's last product of the segment done
  uint64_t *o_free = o_done + 2;     // [2] a slot's accumulators read
  uint64_t *mma_done = o_free + 2;   // every MMA issued has completed
  static_assert(2 * KS + 2 * VS + 11 == Lay::kBars, "mbarrier slots");
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Lay::off_tmem);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + Lay::off_abort);
  float2 *sm_ml = reinterpret_cast<float2 *>(smem + Lay::off_ml);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < KS; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < VS; ++i) {
      mbar_init(&v_full[i], 4);
      mbar_init(&v_empty[i], 1);
    }
    mbar_init(q_full, 4);
    mbar_init(q_empty, 1);
    for (int w = 0; w < 2; ++w) {
      mbar_init(&s_full[w], 1);
      mbar_init(&p_full[w], 4);
      mbar_init(&o_done[w], 1);
      mbar_init(&o_free[w], 4);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                 "r"(kPTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();

  const int plen = prefix_len[0];
  const bool valid = plen >= 0 && plen <= p.g.prefix_cap;
  if (!valid && blockIdx.x == 0 && threadIdx.x == 0) raise_error_sr(hdr, 0x1u);
  const PrefixLine line = prefix_line(p.g, valid ? plen : 0, gridDim.x);
  const int cta = blockIdx.x;
  int x = 0, x1 = 0;
  if (cta < line.n) {
    x = prefix_cta_begin(line, cta);
    x1 = prefix_cta_begin(line, cta + 1);
  }

  if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 32;");
    if (warp == 12) {
      // ------------------------------------------------------------------ MMA issue
      // The whole warp walks the steps and one elected lane issues: in a branch that the
      // compiler takes for divergent, an MMA costs about 100 clocks to issue.
      constexpr uint32_t kIdescS = umma_idesc_bf16(kPRows, kPKeys);
      constexpr uint32_t kIdescO = umma_idesc_f16_bt(kPRows, D);
      const uint64_t q_desc = umma_desc(smem_addr(smem + Lay::off_q)), k_desc = umma_desc(smem_addr(smem + Lay::off_k)),
                     v_desc = umma_desc_v(smem_addr(smem + Lay::off_v));
      uint32_t ks = 0, kph = 0, vs = 0, vph = 0;  // stage and parity of the K and V tile in use
      uint32_t ppar = 0;                          // parity of the next P tile (the same for both slots)
      uint32_t segs = 0;
      bool ok = true;
      while (x < x1 && ok) {
        const PSeg sg = next_seg(p.g, line, x, x1);
        // O_w (+)= P_w V
        auto pv = [&](int s, int w) {
          if (!all_wait(&p_full[w], ppar, hdr, abort_flag)) return false;
          if ((w == 0 || !sg.dual) && !all_wait(&v_full[vs], vph, hdr, abort_flag)) return false;
          if (s == 0 && segs > 0 && !all_wait(&o_free[w], (segs - 1) & 1u, hdr, abort_flag)) return false;
          tc_fence_after();
          const uint64_t vd = v_desc + static_cast<uint64_t>(vs * (Lay::kTile >> 4));
          const bool last_use = w == 1 || !sg.dual;
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kPKeys / 16; ++kk)
              umma_f16_ts(tmem + 256 + w * D, tmem + w * 128 + kk * 8, vd + kk * (2048 >> 4), kIdescO,
                          (s > 0 || kk > 0) ? 1u : 0u);
            if (last_use) umma_commit(&v_empty[vs]);
          }
          __syncwarp();
          if (last_use && ++vs == VS) {
            vs = 0;
            vph ^= 1u;
          }
          return true;
        };
        if (!(ok = all_wait(q_full, segs & 1u, hdr, abort_flag))) break;
        for (int s = 0; s < sg.n && ok; ++s) {
          for (int w = 0; w < 2 && ok; ++w) {
            if (s > 0 && !(ok = pv(s - 1, w))) break;
            if ((w == 0 || !sg.dual) && !(ok = all_wait(&k_full[ks], kph, hdr, abort_flag))) break;
            tc_fence_after();
            const uint64_t qd = q_desc + static_cast<uint64_t>((sg.dual ? w : 0) * (Lay::kTile >> 4));
            const uint64_t kd = k_desc + static_cast<uint64_t>(ks * (Lay::kTile >> 4));
            const bool last_use = w == 1 || !sg.dual;
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint64_t off = ((kk >> 2) * Lay::kHalf + (kk & 3) * 32) >> 4;
                umma_f16(tmem + w * 128, qd + off, kd + off, kIdescS, kk > 0 ? 1u : 0u);
              }
              if (last_use) umma_commit(&k_empty[ks]);
              umma_commit(&s_full[w]);
            }
            __syncwarp();
            if (last_use && ++ks == KS) {
              ks = 0;
              kph ^= 1u;
            }
          }
          if (s > 0) ppar ^= 1u;
        }
        if (!ok) break;
        if (elect_one()) umma_commit(q_empty);
        __syncwarp();
        for (int w = 0; w < 2 && ok; ++w) {
          ok = pv(sg.n - 1, w);
          if (ok && elect_one()) umma_commit(&o_done[w]);
          __syncwarp();
        }
        ppar ^= 1u;
        ++segs;
        x += sg.n;
      }
      if (elect_one()) umma_commit(mma_done);
      __syncwarp();
      mbar_wait(mma_done, 0);
    } else if (warp == 13 && lane == 0) {
      // ------------------------------------------------------------------ K tiles
      tma_prefetch_desc(&kmap);
      uint32_t kc = 0;
      bool ok = true;
      while (x < x1 && ok) {
        const PSeg sg = next_seg(p.g, line, x, x1);
        const int per = sg.dual ? 1 : 2;
        for (int i = 0; i < sg.n * per && ok; ++i) {
          const uint32_t st = kc % KS;
          if (!(ok = wait_or_abort(&k_empty[st], ((kc / KS) & 1u) ^ 1u, hdr, abort_flag))) break;
          mbar_arrive_expect_tx(&k_full[st], Lay::kTile);
          for (int hf = 0; hf < D / 64; ++hf)
            tma_load_4d(smem + Lay::off_k + st * Lay::kTile + hf * Lay::kHalf, &kmap, &k_full[st], 64 * hf,
                        (sg.first * per + i) * kPKeys, sg.h, 0);
          ++kc;
        }
        x += sg.n;
      }
      // every copy issued has landed before the CTA ends
      for (uint32_t i = kc > KS ? kc - KS : 0; i < kc; ++i) mbar_wait(&k_full[i % KS], (i / KS) & 1u);
    }
  } else if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    // ------------------------------------------------------------------ query rows and V tiles
    constexpr int kChunks = D / 8;               // 16-byte chunks of a row
    constexpr int kPer = 128 * kChunks / 128;    // chunks of a tile per thread
    constexpr int kRowStep = 128 / kChunks;      // rows between a thread's chunks
    const int tid = threadIdx.x - 256;
    const int ch = tid % kChunks, r0 = tid / kChunks;
    const uint32_t half_off = (ch >> 3) * Lay::kHalf;
    uint32_t vc = 0, segs = 0;
    bool ok = true;
    while (x < x1 && ok) {
      const PSeg sg = next_seg(p.g, line, x, x1);
      const int per = sg.dual ? 1 : 2, tiles = sg.n * per;
      const __nv_bfloat16 *vh = v + sg.h * p.head_stride + ch * 8;
      uint4 reg[kPer];
      auto fetch = [&](int i) {
        const int key0 = (sg.first * per + i) * kPKeys + r0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int key = key0 + j * kRowStep;  // rows past the prefix hold anything: zero
          reg[j] = key < plen ? __ldg(reinterpret_cast<const uint4 *>(vh + static_cast<int64_t>(key) * D))
                              : make_uint4(0u, 0u, 0u, 0u);
        }
      };
      // query rows, zero past the last; a negative scale turns their sign
      ok = segs == 0 || all_wait(q_empty, (segs - 1) & 1u, hdr, abort_flag);
      if (!ok) break;
      for (int w = 0; w < (sg.dual ? 2 : 1); ++w) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int r = sg.rt * 256 + w * 128 + r0 + j * kRowStep;
          reg[j] = make_uint4(0u, 0u, 0u, 0u);
          if (r < p.g.R) {
            const int bt = r / p.g.G, gg = r - bt * p.g.G;
            reg[j] = __ldg(reinterpret_cast<const uint4 *>(
                q + (static_cast<int64_t>(bt) * p.g.Hq + sg.h * p.g.G + gg) * D + ch * 8));
          }
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          uint4 y = reg[j];
          y.x ^= p.flip;
          y.y ^= p.flip;
          y.z ^= p.flip;
          y.w ^= p.flip;
          *reinterpret_cast<uint4 *>(smem + Lay::off_q + w * Lay::kTile + half_off + swz128(r0 + j * kRowStep, ch & 7)) = y;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
      fetch(0);
      for (int i = 0; i < tiles; ++i) {
        const uint32_t st = vc % VS;
        ok = all_wait(&v_empty[st], ((vc / VS) & 1u) ^ 1u, hdr, abort_flag);
        if (!ok) break;
        unsigned char *vt = smem + Lay::off_v + st * Lay::kTile + half_off;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          uint4 y;
          y.x = bf16x2_to_f16x2(reg[j].x);
          y.y = bf16x2_to_f16x2(reg[j].y);
          y.z = bf16x2_to_f16x2(reg[j].z);
          y.w = bf16x2_to_f16x2(reg[j].w);
          *reinterpret_cast<uint4 *>(vt + swz128(r0 + j * kRowStep, ch & 7)) = y;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_full[st]);
        ++vc;
        if (i + 1 < tiles) fetch(i + 1);
      }
      ++segs;
      x += sg.n;
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    // ------------------------------------------------------------------ softmax
    // Warp i of a slot reads tensor memory lanes 32 i .. 32 i + 31: one query row a thread.
    const int w = warp >> 2, qd = warp & 3;
    const int tl = qd * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(qd * 32) << 16;
    const uint32_t s_addr = tmem + lane_off + w * 128, o_addr = tmem + lane_off + 256 + w * D;
    const float2 s2 = make_float2(p.sl2, p.sl2);
    uint32_t sc = 0, segs = 0;
    while (x < x1) {
      const PSeg sg = next_seg(p.g, line, x, x1);
      float m = -INFINITY, l = 0.f;  // m: what P and O are scaled by (in units of log2)
      for (int s = 0; s < sg.n; ++s) {
        // tensor memory accesses are warp-collective: a warp skips a tile only as a whole
        if (!all_wait(&s_full[w], sc++ & 1u, hdr, abort_flag)) continue;
        tc_fence_after();
        const int tile = sg.dual ? sg.first + s : 2 * (sg.first + s) + w;
        const int nk = plen - tile * kPKeys;  // keys of this tile; zero or less: none
        uint32_t sv[4][32];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(s_addr + 32 * i, sv[i]);
        tmem_wait_ld();
        if (nk < kPKeys) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (32 * i + c >= nk) sv[i][c] = 0xFF800000u;  // -inf
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int c = 0; c < 32; c += 2)
            mx[i] = fmax3(mx[i], __uint_as_float(sv[i][c]), __uint_as_float(sv[i][c + 1]));
        const float top = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]);
        // a row whose every score is -inf so far keeps m = -inf and subtracts 0 instead
        const float mt = top == -INFINITY ? -INFINITY : top * p.sl2;
        const bool raise = mt > m + kRaise || (m == -INFINITY && mt > -INFINITY);
        if (__any_sync(0xffffffffu, raise)) {
          const float mn = raise ? mt : m;
          const float alpha = raise ? ex2(m - mn) : 1.f;  // m == -inf: 0, nothing is there yet
          m = mn;
          l *= alpha;
          if (s > 0) {  // S of this step written means that every earlier product is done
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t o[16];
              tmem_ld16(o_addr + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st16(o_addr + c, o);
            }
          }
        }
        const float mu = m == -INFINITY ? 0.f : m;
        l += nk < kPKeys ? weights<true>(sv, s_addr, s2, mu, nk) : weights<false>(sv, s_addr, s2, mu, nk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[w]);
      }
      // ---- end of the segment: this CTA's partial result of the pair
      const bool got = all_wait(&o_done[w], segs & 1u, hdr, abort_flag);
      tc_fence_after();
      if (!sg.dual) {  // both slots hold the same rows: slot 0 joins slot 1's result to its own
        if (w == 1) sm_ml[tl] = make_float2(m, l);
        tc_fence_before();
        named_bar(1, 256);
        tc_fence_after();
      }
      float f0 = 1.f, f1 = 0.f;
      if (!sg.dual && w == 0) {
        const float2 other = sm_ml[tl];
        const float mn = fmaxf(m, other.x), mu = mn == -INFINITY ? 0.f : mn;
        f0 = ex2(m - mu);
        f1 = ex2(other.x - mu);
        l = l * f0 + other.y * f1;
        m = mn;
      }
      const float inv = l > 0.f ? 1.f / l : 0.f;
      f0 *= inv;
      f1 *= inv;
      const int lr = w * 128 + tl;  // row within the pair
      const bool store = got && (sg.dual || w == 0) && sg.rt * 256 + lr < p.g.R;
      const int64_t at = static_cast<int64_t>(cta + sg.h * p.g.RT + sg.rt) * p.g.slot_rows + lr;
      if (sg.dual || w == 0) {
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32], o1[32];
          tmem_ld32(o_addr + c, o);
          if (!sg.dual) tmem_ld32(o_addr + D + c, o1);
          tmem_wait_ld();
          if (store) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              float y[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                y[e] = __uint_as_float(o[i + e]) * f0;
                if (!sg.dual) y[e] += __uint_as_float(o1[i + e]) * f1;
              }
              st_f8(part_o + at * D + c + i, y);
            }
          }
        }
        if (store) part_l[at] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&o_free[w]);
          if (!sg.dual) mbar_arrive(&o_free[1]);
        }
      }
      ++segs;
      x += sg.n;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kPTmemCols) : "memory");
  }
}

template <int D>
cudaError_t launch_one(const PrefixPlan &pl, const PrefixArgs &a, const CUtensorMap &kmap) {
  auto kern = prefix_tc05_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, PLayout<D>::alloc);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (e != cudaSuccess) return e;
  PParams kp;
  kp.g = pl.g;
  kp.head_stride = a.head_stride;
  kp.sl2 = fabsf(a.sm_scale) * kLog2e;
  kp.flip = a.sm_scale < 0.f ? 0x80008000u : 0u;
  unsigned char *ws = static_cast<unsigned char *>(a.ws);
  return launch_pdl(kern, dim3(pl.grid), dim3(kPThreads), PLayout<D>::alloc, a.stream, kmap,
                    static_cast<const __nv_bfloat16 *>(a.q), static_cast<const __nv_bfloat16 *>(a.v), a.prefix_len,
                    reinterpret_cast<float *>(ws + pl.off_part_o), reinterpret_cast<float *>(ws + pl.off_part_l),
                    static_cast<WsHeader *>(a.ws), kp);
}

}  // namespace

cudaError_t launch_prefix_tc05(const PrefixPlan &p, const PrefixArgs &a, const CUtensorMap &kmap) {
  return p.g.D == 128 ? launch_one<128>(p, a, kmap) : launch_one<64>(p, a, kmap);
}

}  // namespace mgd
