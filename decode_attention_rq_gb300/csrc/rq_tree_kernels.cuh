// The tensor-core path of rq_tree_attention (shared-anchor caches): query prep, the
// streaming kernel, the merge.  rq_tree.cu has the mathematics and the choice of path.
//
// Work unit: the queries of one (row, KV head) -- T nodes times the Hq / H query heads
// that share the head, consecutive rows of q -- in blocks of NB = 16, 32 or 64, times
// the head's cached tokens in steps of 128.  The steps of all units are dealt out evenly
// to a persistent grid of one CTA per SM; a CTA leaves one partial softmax state
// (m, l, O) per unit it touched, and the merge joins them.
//
// Per step, transposed products keep the padding off the queries' side: the 128-row
// operand is made of cache data, the N side is the NB queries.
//   scores  S^T [128 tokens x NB] = K' Q'^T     (anchor and residual part apart:
//                                                s = c Sa + Sr, c in the token's lane)
//   values  O^T [channels x NB] += V'^T P^T     (anchor and residual part apart)
// K' and V'^T are dequantized into registers and stored to tensor memory as the A operand
// (f16, one token or channel per lane): dequantized data never touches shared memory.
// Roles (24 warps, in groups of four, one per 32 lanes): K, softmax, two for V of the anchor (64
// queries: one, and a second for softmax, 32 queries each), V of the residual (idle in the anchor
// loop), and a group with the copy warp and one warp for each kind of product.
//
// Dequantization: an f16 whose bits are an integer n < 1024 has the value n 2^-24, so masking a
// code word leaves codes times 2^(p - 24), p the field's first bit; one fused multiply-add with
// (s 2^(24 - p - k), o 2^-k) gives (s code + o) 2^-k.  k = 15: every E4M3 s and o stays in f16's
// range and, being a multiple of 2^-9, exact; s code + o, below 4 exact, too, is rounded to 11 bits above.  (Logic
// and shift instructions run at half rate here and bound this kernel: 7 of them a word of 8 codes, 11 of 16.)
//
// Softmax: a token's scores sit in one lane, a query's across the lanes.  The running
// reference of a query therefore moves only when some score exceeds it by 2^8 (the first
// step, then rarely): weights stay below 2^14, in f16 range, and O is rescaled in
// tensor memory then.  Sums stay in the lanes' registers until the unit ends.
//
// Measured (GB300; the three launches of a call, inputs cold): 16 heads of 128, residual loop, 8192 tokens,
// 4 rows of 16 nodes 54 us, of which the streaming kernel 44 (120 MB: 2.7 TB/s in it, 2.2 TB/s over the call); 16384
// tokens paged, 2 rows of 61 nodes 73 us; 8 rows of 13 nodes, 4 query heads a KV head 121 us; anchor loop, 55 heads
// of 96, 4096 tokens, 2 rows of 25 nodes 36 us.  Not bound by memory: dequantizing 256 channels x 128 tokens of K and
// V a step, with the softmax, keeps the schedulers at 0.66 instructions a clock (0.60 with 64 queries)
// and each role's chain of waits at about 2600 clocks a step; the tensor pipe is 9 to 25 % busy.
#pragma once

#include <atomic>
#include <type_traits>

#include <cuda_fp8.h>

#include "rq_internal.cuh"

namespace rq {

struct TreeArgs {
  Geom g;
  const uint8_t* base;
  const float* R;
  const __nv_bfloat16 *q, *k_new, *v_new;
  const unsigned long long* mask;
  const int32_t *counts, *seq_lens;
  __nv_bfloat16* out;
  int32_t* status;
  int layer, group, batch, T, words, loop, nres;
  float qscale;                    // softmax_scale * log2(e)
  // tensor-core path
  int M, nqb;                      // queries per (row, KV head); blocks of NB of them
  float* partials;                 // [num CTAs + units][pstride]
  uint8_t* packs;                  // [units][image]: query operands
  float* q_scale;                  // [units][NB]: factor from a score product to log2 units
  int64_t pstride;
};

cudaError_t launch_tree_mma(const TreeArgs& a, int nb, int num_sms, cudaStream_t stream);
cudaError_t launch_tree_mma_96(const TreeArgs& a, int nb, int num_sms, cudaStream_t stream);

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTreeStep = 128;               // tokens per step: two layout tiles
constexpr int kTreeThreads = 24 * 32;
constexpr int kTreeRows = RQ_MAX_DECODE_BATCH;
constexpr float kHead = 6.f;                 // a row maximum's weight is 2^kHead
constexpr float kTop = 14.f;                 // largest log2 weight before the reference moves

__device__ __forceinline__ int clamp_len(int n, int nmax) { return n < 0 ? 0 : (n > nmax ? nmax : n); }
__device__ __forceinline__ bool sees(const TreeArgs& a, int b, int t, int j) {
  if (!a.mask) return j <= t;
  return (__ldg(a.mask + ((size_t)b * a.T + t) * a.words + (j >> 6)) >> (j & 63)) & 1u;
}

struct TreeSplit {
  int q, rem;
  __device__ __forceinline__ int start(int c) const { return c * q + min(c, rem); }
  __device__ __forceinline__ int owner(int u) const {
    const int big = (q + 1) * rem;
    return u < big ? u / (q + 1) : rem + (u - big) / q;
  }
};

// ---- tcgen05 ---------------------------------------------------------------------
__device__ __forceinline__ void tc_alloc(uint32_t* slot, int cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols)
               : "memory");
}
__device__ __forceinline__ void tc_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tc_dealloc(uint32_t addr, int cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
// D[128 x N] (+)= A[128 x 16] B[16 x N]: A in tensor memory, B in shared memory
template <bool ACC>
__device__ __forceinline__ void tc_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "n"(ACC ? 1 : 0)
      : "memory");
}
// One lane of a converged warp.  The compiler then knows that a single thread issues what
// follows and keeps the operands in uniform registers: 12 to 16 clocks a product of 16
// columns, against 50 behind a test of the lane number.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// N products, one behind the other.  A loop: unrolled it saves 30 clocks a product and costs instruction cache
// (54.7 -> 54.2 us at 8k, 36.4 -> 37.3 in the anchor loop).
template <int N>
__device__ __forceinline__ void tc_chain(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t b_step,
                                         uint32_t idesc, bool fresh) {
  const uint64_t b0 = (uint64_t)b_hi << 32 | b_lo;
  if (fresh) tc_mma<false>(d, a, b0, idesc); else tc_mma<true>(d, a, b0, idesc);
#pragma unroll 1
  for (int k = 1; k < N; ++k) {
    a += 8;
    b_lo += b_step;
    tc_mma<true>(d, a, (uint64_t)b_hi << 32 | b_lo, idesc);
  }
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 16 lanes x 32 columns: lane l of the warp holds, of rows l / 4 and l / 4 + 8 (registers + 2), the
// columns 8 j + 2 (l % 4) and the next (registers 4 j, 4 j + 1)
__device__ __forceinline__ void tc_st_frag(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tc_ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
// f16 x f16 -> f32 products of 128 rows and n columns; b_mn: B's columns contiguous
constexpr uint32_t tc_idesc(int n, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(n / 8) << 17) | ((128u / 16) << 24);
}
// Shared-memory operands.  Queries: 16 channels of a row make 32 bytes, 8 rows 256 (32-byte
// swizzle), so that the products of a plane step through blocks of NB * 32 bytes.  Weights: a
// token's 64 queries make 128 bytes, 8 tokens 1024 (128-byte swizzle).
constexpr uint32_t kDescHiQ = (256u >> 4) | 1u << 14 | 6u << 29, kDescHiP = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr) { return (addr & 0x3FFFF) >> 4 | (1024u >> 4) << 16; }
// Named barrier of one warpgroup; wg_any: true when any thread's predicate holds.
__device__ __forceinline__ void wg_sync(int id) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(id) : "memory"); }
// the same of two warpgroups
__device__ __forceinline__ void wg_sync2(int id) { asm volatile("barrier.cta.sync %0, 256;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool wg_any(int id, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"((uint32_t)p)
      : "memory");
  return r != 0;
}
template <int N>
__device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Waits for a phase: kTries - `from` tries at most, false when none found it complete.  A failing
// try lasts up to about 1.4 us, so that all of them take some seconds.  One short instruction
// sequence with nothing to jump over when the first try succeeds: with all SMs fetching, the
// streaming kernel is bound by instruction fetch as soon as the code of its roles' steps exceeds
// the 32 KB instruction cache of an SM (1.2 -> 3.2 clocks an instruction).
constexpr uint32_t kTries = 1u << 21;
__device__ __forceinline__ bool tree_try(uint64_t* bar, uint32_t parity, uint32_t from) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\tmov.u32 n, %3;\n\t"
      "TRY:\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tadd.u32 n, n, 1;\n\t"
      "setp.lt.and.u32 q, n, %4, !p;\n\t@q bra TRY;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(from), "n"(kTries)
      : "memory");
  return ok != 0;
}

// ---- f16 pairs ---------------------------------------------------------------------
__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 u2h(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
__device__ __forceinline__ __half2 e4m3_pair(uint16_t v) {   // (scale, offset), exact
  uint32_t h2;
  asm("{\n\t.reg .b16 t;\n\tmov.b16 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h2) : "h"(v));
  return u2h(h2);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
// two f32 -> f16x2, lo in the low half; no saturation: infinities stay
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// INT4 word: r[s] = 2^-20 times the codes at bits 4 s and 4 s + 16
__device__ __forceinline__ void codes4(uint32_t w, uint32_t (&r)[4]) {
  r[0] = (w << 4) & 0x00F000F0u;
  r[1] = w & 0x00F000F0u;
  r[2] = (w >> 4) & 0x00F000F0u;
  r[3] = (w >> 8) & 0x00F000F0u;
}
// INT2 word: r[4 i + m] = 2^-22, 2^-22, 2^-20, 2^-18 (m = 0 .. 3) times the codes at bits 8 i + 2 m
// and 16 further, i = 0, 1
__device__ __forceinline__ void codes2(uint32_t w, uint32_t (&r)[8]) {
  r[0] = (w << 2) & 0x000C000Cu;
  r[1] = w & 0x000C000Cu;
  r[2] = w & 0x00300030u;
  r[3] = w & 0x00C000C0u;
  r[4] = (w >> 6) & 0x000C000Cu;
  r[5] = (w >> 8) & 0x000C000Cu;
  r[6] = (w >> 8) & 0x00300030u;
  r[7] = (w >> 8) & 0x00C000C0u;
}
// f16 2^e, -14 <= e <= 15
__device__ __forceinline__ __half half_pow2(int e) { return __ushort_as_half((unsigned short)((e + 15) << 10)); }
constexpr int kScaleK = 15;    // dequantized operands carry 2^-15 (V's anchor under a coefficient: 2^-7)

// Channel in the low half of column col of a K' row (the other half: 4 further in the anchor's
// part, 8 in the residual's): the order in which the dequantizers leave them.
template <int D>
__device__ __forceinline__ int k_channel(int col, bool res) {
  if (D != 128) return res ? (col >> 3) * 16 + (col & 7) : (col >> 2) * 8 + (col & 3);
  const int j = col >> 3, t = (col >> 1) & 3, e = col & 1;   // thread t of four holds channels 32 t ..
  return 32 * t + (res ? (j >> 2) * 16 + 2 * (j & 3) + e : (j >> 1) * 8 + 2 * (j & 1) + e);
}
// Row of token tau's weights in P, that is the place of its column half in V'^T
__device__ __forceinline__ int v_slot(int tau) {
  return 16 * ((tau & 31) >> 2) + 4 * (tau >> 5) + 2 * (tau & 1) + ((tau >> 1) & 1);
}

// Per-CTA view of the call's work, in shared memory: steps before row b, steps of a unit of row b
struct TreeRowsShared {
  int pre[kTreeRows + 1];
  int len[kTreeRows];
};
// Fills it (first warp; every thread of the CTA then synchronizes); units_per_row = H * nqb.
__device__ __forceinline__ void tree_rows(const TreeArgs& a, TreeRowsShared* s) {
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x, per = a.g.H * a.nqb;
    int run = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
      const int b = b0 + lane;
      const int n = b < a.batch ? clamp_len(a.seq_lens[b], a.g.Nmax) : 0;
      if (b < a.batch) s->len[b] = n;
      int x = (n + kTreeStep - 1) / kTreeStep * per;
      const int own = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (b < a.batch) s->pre[b] = run + x - own;
      run += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) s->pre[a.batch] = run;
  }
}

// A position in the sequence of steps
struct TreeCursor {
  int b, in_row, step, steps;       // row, unit within the row, step of the unit, its steps
  __device__ __forceinline__ void seek(const TreeRowsShared& s, int batch, int u) {
    int lo = 0, hi = batch - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s.pre[mid] <= u) lo = mid; else hi = mid - 1;
    }
    b = lo;
    steps = (s.len[b] + kTreeStep - 1) / kTreeStep;
    const int rem = u - s.pre[b];
    in_row = rem / steps;
    step = rem % steps;
  }
  // to the next step (there is one); per: units per row
  __device__ __forceinline__ void next(const TreeRowsShared& s, int per) {
    if (++step < steps) return;
    step = 0;
    if (++in_row < per) return;
    in_row = 0;
    do {
      ++b;
      steps = (s.len[b] + kTreeStep - 1) / kTreeStep;
    } while (steps == 0);
  }
};

template <int D, int GS, int NRES, int NB>
struct TreeCfg {
  static constexpr int NG = D / GS;
  static constexpr int A_CODES = kTile * D / 2, R_CODES = kTile * D / 4, META = kTile * NG * 2;
  static constexpr int A_TILE = A_CODES + META, R_TILE = R_CODES + META + kTile * 2;
  // stage: K anchor, V anchor, K residual, V residual, two tiles each
  static constexpr int AV = 2 * A_TILE, RK = 4 * A_TILE, RV = 4 * A_TILE + 2 * R_TILE;
  static constexpr int STAGE = 4 * A_TILE + NRES * 4 * R_TILE;
  static constexpr int PL = 1 + NRES;
  static constexpr int QSTEP = NB * 32;                    // 16 channels of all queries
  static constexpr int IMG = PL * (D / 16) * QSTEP;        // query operand of a unit
  static constexpr int PBUF = kTreeStep * 128;             // weights: 128-byte row per token
  static constexpr int TAB = PL * NG * 64 * 8 + NRES * 256; // V constants
  // tables of V constants: two (one barrier a step less) where they leave room for four stages
  static constexpr int TABS = 2 * IMG + PBUF + 2 * TAB + 4 * STAGE + 6144 <= 226 * 1024 ? 2 : 1;
  static constexpr int FIX = 2 * IMG + PBUF + TABS * TAB;
  static constexpr int STAGES = FIX + 4 * STAGE + 6144 <= 226 * 1024 ? 4 : 3;
  static constexpr int SMEM = FIX + STAGES * STAGE + 1024;
  // tensor memory columns
  static constexpr int KA = 0, KR = 64, VA = 128, VR = 192, OA = 256, OR = 256 + NB, S0 = 256 + 2 * NB;
  // scores: two buffers where they fit and the softmax is the longer for its coefficients (57.6 ->
  // 56.2 us at 8k, batch 4, 16 queries; the anchor loop is not faster with two)
  static constexpr int SBUF = NRES && NB <= 32 ? 2 : 1;
  static constexpr int SCOLS = SBUF * PL * NB;             // Sa, Sr
  static_assert(S0 + SCOLS <= 512, "tensor memory");
  static_assert(SMEM <= 227 * 1024 - 5120, "shared memory");
  static constexpr int NS = NB / 32 > 1 ? 2 : 1, NQ = NB / NS;   // softmax groups, queries of each
  static constexpr int NVA = 3 - NS;                             // groups of V's anchor
  // registers a thread: 80 at launch (6 groups: 480), then softmax, the dequantizers, the others
  static constexpr int REGS = NS == 2 ? 112 : 136;
  static constexpr int REGD = NS == 2 ? 64 : 72;
  static constexpr int REGP = 56;
  static_assert(NS * REGS + (5 - NS) * REGD + REGP <= 480, "registers");
  // floats of a partial: m[NB], l[NB], O as [plane][NB/4][D][4]
  static constexpr int PSTRIDE = 2 * NB + PL * NB * D;
};

// ---- query prep --------------------------------------------------------------------
// One CTA per QP queries of a unit: x and R x as f16 times a power of two of the query's own (its largest
// component to 2^10 .. 2^11: R keeps norms, so both stay below 2^15), in the layout of the B
// operand.  x is BF16 and so exact; R x is a product on the 16-bit tensor cores with R as two
// BF16 pieces (16 bits, against the 11 of its result), summed in float32: 8 warps with 16 rows
// of R each in registers, one pass over the queries.
// Bound by latency: R, the queries and the barriers in turn, 9 us cold at 64 units of 16 queries (6 in the
// anchor loop); the loads of R come ahead of the wait for the kernel before.
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// two floats as BF16 pairs: the rounded values and the rounded remainders
__device__ __forceinline__ void bf16_pieces(float2 x, uint32_t& hi, uint32_t& lo) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
  const float2 f = __bfloat1622float2(h);
  const __nv_bfloat162 l = __floats2bfloat162_rn(x.x - f.x, x.y - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

template <int D, int NRES, int NB, int QP>
__global__ void __launch_bounds__(256) tree_prep_kernel(TreeArgs a) {
  constexpr int PL = 1 + NRES;
  constexpr int IMG = PL * (D / 16) * NB * 32;
  constexpr int PITCH = D + 8;             // BF16 elements: rows 4 banks apart
  constexpr int RPITCH = D + 4;
  __shared__ __align__(16) __nv_bfloat16 q_s[QP][PITCH];
  __shared__ __align__(16) float r_s[NRES ? QP : 1][RPITCH];
  __shared__ float up_s[QP];               // the query's power of two
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
  const int unit = blockIdx.x / (NB / QP), q0 = blockIdx.x % (NB / QP) * QP;
  const int qb = unit % a.nqb, bh = unit / a.nqb, b = bh / a.g.H;
  const bool hadamard = (a.g.mode & RQ_MODE_HADAMARD) != 0;
  uint32_t hi[NRES ? D / 16 : 1][4], lo[NRES ? D / 16 : 1][4];
  if (NRES && !hadamard && warp < D / 16) {   // R does not change while the cache is used: before the wait
    const float* rp = a.R + (size_t)(16 * warp + g) * D + 2 * t4;
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)   // rows g, g + 8; columns 2 t4, 2 t4 + 8
        bf16_pieces(__ldg(reinterpret_cast<const float2*>(rp + (i & 1) * 8 * D + 16 * k + (i >> 1) * 8)), hi[k][i],
                    lo[k][i]);
  }
  pdl_wait();
  pdl_launch_dependents();   // what ran before the call is complete: the next kernel may read the cache
  const int cnt = a.counts ? clamp_len(a.counts[b], a.T) : a.T;
  const int at = qb * NB + q0, rows = min(QP, a.M - at);   // may be negative: no query here
  const __nv_bfloat16* qu = a.q + ((size_t)bh * a.M + at) * D;
  // one warp per query: its values (zeros for a node not in use), its power of two; a query that
  // is not finite keeps the scale 1 and stays so
#pragma unroll
  for (int r = warp; r < QP; r += 8) {
    const bool on = r < rows && (at + r) % a.T < cnt;
    uint2 v = make_uint2(0u, 0u);
    if (on && lane < D / 4) v = __ldg(reinterpret_cast<const uint2*>(qu + (size_t)r * D) + lane);
    if (lane < D / 4) *reinterpret_cast<uint2*>(&q_s[r][4 * lane]) = v;
    // magnitudes of BF16 numbers compare as integers
    uint32_t big = max(max(v.x & 0x7FFFu, (v.x >> 16) & 0x7FFFu), max(v.y & 0x7FFFu, (v.y >> 16) & 0x7FFFu));
    big = __reduce_max_sync(0xffffffffu, big);
    int e = 11;
    if (big > 0 && big < 0x7F80u) frexpf(__uint_as_float(big << 16), &e);   // f 2^e, f in [0.5, 1)
    e = max(e, -115);                                                       // 2^(11 - e) stays finite
    if (lane == 0) {
      up_s[r] = ldexpf(1.f, 11 - e);
      a.q_scale[(size_t)unit * NB + q0 + r] = ldexpf(a.qscale, e - 11 + kScaleK);
    }
  }
  __syncthreads();
  if (NRES && hadamard) {
    // one warp per query: lane holds channels lane, lane + 32, ...; stages h = 1 .. 64
    for (int r = warp; r < QP; r += 8) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __bfloat162float(q_s[r][(lane + 32 * i) % D]);
#pragma unroll
      for (int h = 1; h < 32; h <<= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = __shfl_xor_sync(0xffffffffu, v[i], h);
          v[i] = (lane & h) ? p - v[i] : v[i] + p;
        }
      const float s0 = v[0] + v[1], s1 = v[0] - v[1], s2 = v[2] + v[3], s3 = v[2] - v[3];
      if (D == 128) {
        r_s[r][lane] = (s0 + s2) * kInvSqrt128;
        r_s[r][lane + 32] = (s1 + s3) * kInvSqrt128;
        r_s[r][(lane + 64) % D] = (s0 - s2) * kInvSqrt128;
        r_s[r][(lane + 96) % D] = (s1 - s3) * kInvSqrt128;
      }
    }
    __syncthreads();
  } else if (NRES) {
    if (warp < D / 16) {
#pragma unroll
      for (int n = 0; n < QP; n += 8) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t* bp = reinterpret_cast<const uint32_t*>(&q_s[n + g][16 * k + 2 * t4]);
          const uint32_t b0 = bp[0], b1 = bp[4];
          mma_bf16(d, hi[k], b0, b1);
          mma_bf16(d, lo[k], b0, b1);
        }
        const int c = 16 * warp + g, q = n + 2 * t4;
        r_s[q][c] = d[0];
        r_s[q + 1][c] = d[1];
        r_s[q][c + 8] = d[2];
        r_s[q + 1][c + 8] = d[3];
      }
    }
    __syncthreads();
  }
  // the operand: 8 channels (16 bytes) a thread, 16 to a block of 32 bytes a query, swizzled
  uint8_t* img = a.packs + (size_t)unit * IMG;
  for (int i = tid; i < PL * QP * (D / 8); i += 256) {
    const int c = i % (D / 8), r = i / (D / 8) % QP, pl = i / (D / 8 * QP), row = q0 + r;
    const float up = up_s[r];
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int ch = k_channel<D>(4 * c + j, pl != 0);
      const float x0 = pl ? r_s[NRES ? r : 0][ch] : __bfloat162float(q_s[r][ch]);
      const float x1 = pl ? r_s[NRES ? r : 0][ch + 8] : __bfloat162float(q_s[r][ch + 4]);
      w[j] = f16x2(x0 * up, x1 * up);
    }
    *reinterpret_cast<uint4*>(img + ((pl * (D / 16) + (c >> 1)) * NB + row) * 32 + (((c & 1) ^ ((row >> 2) & 1)) << 4)) =
        make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Every query's maximum or sum over the warp's lanes, to row: a reduce-scatter, each step halving
// what a lane holds (31 exchanges for 32 queries, against 160)
template <int NQ, bool MAX>
__device__ __forceinline__ void tree_spread(float (&x)[NQ], float* row, int lane) {
#pragma unroll
  for (int o = 16, n = NQ / 2; o >= 1; o >>= 1) {
    if (n >= 1) {
      const bool up = (lane & o) != 0;
#pragma unroll
      for (int i = 0; i < NQ / 2; ++i)
        if (i < n) {
          const float send = up ? x[i] : x[i + n], keep = up ? x[i + n] : x[i];
          const float y = __shfl_xor_sync(0xffffffffu, send, o);
          x[i] = MAX ? fmaxf(keep, y) : keep + y;
        }
      n >>= 1;
    } else {
      const float y = __shfl_xor_sync(0xffffffffu, x[0], o);
      x[0] = MAX ? fmaxf(x[0], y) : x[0] + y;
    }
  }
  // 32 queries: one a lane; 16: one for two lanes
  if (NQ == 32)
    row[lane] = x[0];
  else if ((lane & 1) == 0)
    row[lane >> 1] = x[0];
}

// ---- the streaming kernel --------------------------------------------------------
template <int D, int GS, int NRES, int NB>
__global__ void __launch_bounds__(kTreeThreads, 1) tree_mma_kernel(TreeArgs a) {
  using C = TreeCfg<D, GS, NRES, NB>;
  constexpr int ST = C::STAGES, NG = C::NG, PL = C::PL;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full_bar[ST], empty_bar[ST], qfull_bar[2], qempty_bar[2], kfull_bar[2], kempty_bar[2],
      vfull_bar[2], vempty_bar[2], sfull_bar[2], sempty_bar[2], pfull_bar, pempty_bar, drain_bar[2];
  __shared__ TreeRowsShared rows_s;
  __shared__ __align__(16) float qm_s[NB / 2][4];   // two queries: their scales, minus their references
  __shared__ __align__(16) float f_s[NB];
  __shared__ float wred_s[4][NB];
  __shared__ uint32_t tmem_s;
  // per step (eight in flight at most): tokens in use | first, last of its unit << 8, 9; the unit
  __shared__ int2 info_s[8];

  // aligned by an offset, not by a cast: the compiler keeps the address space (shared, not generic, loads)
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* q_img = smem;                                  // two query operands
  uint8_t* p_buf = q_img + 2 * C::IMG;                    // weights
  uint8_t* stages = p_buf + C::PBUF;
  uint8_t* tabs = stages + ST * C::STAGE;                 // V constants

  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int per = a.g.H * a.nqb;

  tree_rows(a, &rows_s);
  if (tid == 32) {
    for (int i = 0; i < ST; ++i) { mbar_init(&full_bar[i], 1); mbar_init(&empty_bar[i], NRES ? 20 : 4 + 4 * C::NVA); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&qfull_bar[i], 1); mbar_init(&qempty_bar[i], 1);
      mbar_init(&kfull_bar[i], 4); mbar_init(&kempty_bar[i], 1);
      mbar_init(&vfull_bar[i], i ? 4 : 4 * C::NVA); mbar_init(&vempty_bar[i], 1);
      mbar_init(&sfull_bar[i], 1); mbar_init(&sempty_bar[i], 4 * C::NS);
    }
    mbar_init(&pfull_bar, 4 * C::NS); mbar_init(&pempty_bar, 1);
    mbar_init(&drain_bar[0], 1); mbar_init(&drain_bar[1], 1);
    fence_mbar_init();
  }
  __syncthreads();
  const int U = rows_s.pre[a.batch];
  const TreeSplit split{U / (int)gridDim.x, U % (int)gridDim.x};
  const int u0 = split.start(blockIdx.x), n_it = split.start(blockIdx.x + 1) - u0;
  if (n_it <= 0) {
    pdl_launch_dependents();
    pdl_wait();
    return;
  }
  if (warp == 21) {
    tc_alloc(&tmem_s, 512);
    tc_relinquish();
    tc_before();
  }
  __syncthreads();
  tc_after();
  constexpr uint32_t tmem = 0;   // all 512 columns are this CTA's, from column 0 (tc_alloc wrote tmem_s = 0)
  pdl_launch_dependents();

  // Waits are bounded.  A warp that gave up sets the status word; the copy warp then stops, the
  // other roles run on to their end, one try a wait (their warps share named barriers, so none
  // may leave alone).  What they compute is lost, every address stays as planned.
  uint32_t from = 0;
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (tree_try(bar, parity, from)) return true;
    from = kTries - 1;
    a.status[0] = 1;
    return false;
  };
  // buffer and phase of step `it`'s scores
  auto s_buf = [](int it) { return C::SBUF == 2 ? it & 1 : 0; };
  auto s_par = [](int it) { return (uint32_t)(C::SBUF == 2 ? it >> 1 : it) & 1; };
  // the same by a whole warp, which goes on together (the tcgen05 loads and stores are warp-wide)
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
    (void)wait(bar, parity);
    __syncwarp();
  };
  // ================= V: rows of channels, plane pl =================
  auto v_role = [&](auto plane, int part) {
    constexpr int pl = decltype(plane)::value;
    const int w4 = warp & 3, lt = tid & 127;
    auto v_sync = [&]() {   // the groups that share constants
      if (pl) wg_sync(3); else if (C::NVA == 1) wg_sync(2); else wg_sync2(2);
    };
    const uint32_t lanes = tmem + ((uint32_t)(w4 * 32) << 16);
    const int col = v_slot(lt) >> 1, hf = v_slot(lt) & 1;   // the token's place among the constants
    const int t4 = lane & 3;                                // the lane's 32 tokens: 32 t4 ..
    const int tok = lt & 63, tau = lt >> 6;
    // the field of this token in residual words starts at bit 2, 2, 4, 6 (as codes2 leaves it); its
    // multiplier is that many powers of two below the one of bit 4
    const int quad = (lt & 31) >> 2;
    const __half2 field = __halves2half2(half_pow2((quad & 3) < 2 ? 2 : ((quad & 3) == 2 ? 0 : -2)), half_pow2(0));
    const __half2 to_k = __halves2half2(half_pow2(24 - 4 - kScaleK), __ushort_as_half(0x0200));     // 2^5, 2^-15
    int st = 0;
    uint32_t par = 0;
#pragma unroll 1
    for (int it = 0; it < n_it; ++it) {
      wait_warp(&full_bar[st], par);
      const uint8_t* s = stages + st * C::STAGE;
      const bool on = lt < (info_s[it & 7].x & 255);
      // the step's table: the one before is still in use; with a single one, wait until it is not
      uint8_t* tab = tabs + (C::TABS == 2 ? (it & 1) * C::TAB : 0);
      if (C::TABS == 1) v_sync();
      // Constants of this lane's token.  The anchor's coefficient c = m f, f a power of two: f goes into the
      // constants, where powers of two are exact, and m multiplies the finished f (s code + o), so that a value is
      // rounded relative to itself and not to its group's range.  That product carries 2^-7: its operands 2^-13 and m
      // 2^6.  The multiplier s 2^7 f has to stay below 2^16, and s goes to 448: f <= 1, so that 1 <= |m| < 2 only for
      // |c| < 2, and m takes the larger powers of two, up to |m| < 2^10.  Beyond that f grows again: V is finite
      // while s f < 2^9, that is while |c| s < 2^18.  Scales and offsets are multiples of 2^-9, so with f >= 1/4
      // subnormal operands stay exact, too; with a smaller f a value below 1/2 may be off by 2^-10: its own half step and
      // its group's offset's, 2^-25 each against 2^-13 and |m| < 2 (1.25 * 2^-10 where f is two factors: the offset rounds
      // twice).
      __half2 f1 = __half2half2(half_pow2(0)), f2 = f1;
      if (NRES && pl == 0) {
        uint16_t cb =
            *reinterpret_cast<const uint16_t*>(s + C::RV + tau * C::R_TILE + C::R_CODES + C::META + tok * 2);
        if ((cb & 0x7F80) == 0 || !on) cb = 0;                          // a subnormal c counts as zero
        const int e = (cb >> 7) & 0xFF;
        const bool plain = e != 0 && e != 255;                          // infinite and NaN c keep f = 1
        const int up = plain ? min(max(e - 127, 0), 9) : 0;             // m = 2^up times c's sign and significand
        // 4 f = 2^x as two factors of f16 range
        const int x = plain ? e - 125 - up : 2, x1 = min(max(x, -14), 15), x2 = min(max(x - x1, -14), 15);
        f1 = __half2half2(half_pow2(x1));
        f2 = __half2half2(half_pow2(x2));
        const uint32_t m = plain ? (cb & 0x807Fu) | (uint32_t)(127 + up) << 7 : cb;
        *reinterpret_cast<__half*>(tab + PL * NG * 512 + col * 4 + hf * 2) =
            __float2half_rn(bf16_bits_to_f32(m) * 64.f);
      }
      {
        const uint8_t* tile = pl ? s + C::RV + tau * C::R_TILE : s + C::AV + tau * C::A_TILE;
        const uint16_t* meta = reinterpret_cast<const uint16_t*>(tile + (pl ? C::R_CODES : C::A_CODES)) + tok * NG;
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) {
          if (pl == 0 && C::NVA == 2 && (gi & 1) != part) continue;
          __half2 so = __hmul2(e4m3_pair(on ? meta[gi] : (uint16_t)0), to_k);
          if (pl) so = __hmul2(so, field);
          else if (NRES) so = __hmul2(__hmul2(so, f1), f2);
          uint8_t* e = tab + ((pl * NG + gi) * 64 + col) * 8 + hf * 2;
          *reinterpret_cast<__half*>(e) = __low2half(so);
          *reinterpret_cast<__half*>(e + 4) = __high2half(so);
        }
      }
      v_sync();
      {
        wait_warp(&vempty_bar[pl], (it & 1) ^ 1);
        tc_after();
        if (D == 128 || w4 < 3) {
          // four lanes share a channel, 32 tokens each; a lane has four channels (l / 4 + 8 k), so that
          // a constant read from shared memory serves four (groups of 16 channels: two)
          const uint8_t* row = (pl ? s + C::RV + (t4 >> 1) * C::R_TILE : s + C::AV + (t4 >> 1) * C::A_TILE) +
                               (w4 * 32 + (lane >> 2)) * (pl ? 16 : 32) + (t4 & 1) * (pl ? 8 : 16);
          const uint4* tb = reinterpret_cast<const uint4*>(tab + (pl * NG + w4 * (32 / GS)) * 512) + t4;
          const uint2* cm = reinterpret_cast<const uint2*>(tab + PL * NG * 512) + t4;   // significands of c
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {        // 16 of the lane's tokens: four pairs of columns
            uint4 kq[4];
            uint2 mq[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (GS == 32) kq[j] = tb[16 * c + 4 * j];
              if (NRES && pl == 0) mq[j] = cm[16 * c + 4 * j];
            }
#pragma unroll 1
            for (int hh = pl || C::NVA == 1 ? 0 : part; hh < (pl || C::NVA == 1 ? 2 : part + 1); ++hh) {
              if (GS == 16) {
#pragma unroll
                for (int j = 0; j < 4; ++j) kq[j] = tb[hh * 32 + 16 * c + 4 * j];
              }
              uint32_t r[16];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint8_t* p = row + (16 * hh + 8 * k) * (pl ? 16 : 32) + c * (pl ? 4 : 8);
                if (pl == 0) {
                  const uint2 w = *reinterpret_cast<const uint2*>(p);
                  const uint32_t ww[2] = {w.x, w.y};
#pragma unroll
                  for (int i = 0; i < 2; ++i) {
                    uint32_t v[4];
                    codes4(ww[i], v);          // v[x]: tokens (0, 2) of quad x & 1 from token x >> 1
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                      const int j = 2 * i + (x & 1), e = x >> 1;
                      __half2 z = __hfma2(u2h(v[x]), u2h(e ? kq[j].z : kq[j].x), u2h(e ? kq[j].w : kq[j].y));
                      if (NRES) z = __hmul2(z, u2h(e ? mq[j].y : mq[j].x));
                      r[4 * j + 2 * k + e] = h2u(z);
                    }
                  }
                } else {
                  uint32_t v[8];
                  codes2(*reinterpret_cast<const uint32_t*>(p), v);   // v[4 e + j]: quad j from token e
#pragma unroll
                  for (int x = 0; x < 8; ++x) {
                    const int j = x & 3, e = x >> 2;
                    r[4 * j + 2 * k + e] =
                        h2u(__hfma2(u2h(v[x]), u2h(e ? kq[j].z : kq[j].x), u2h(e ? kq[j].w : kq[j].y)));
                  }
                }
              }
              tc_st_frag(lanes + ((uint32_t)(16 * hh) << 16) + (pl ? C::VR : C::VA) + 32 * c, r);
            }
          }
          tc_wait_st();
        }
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&vfull_bar[pl]);
      }
      if (lane == 0) mbar_arrive(&empty_bar[st]);
      if (++st == ST) { st = 0; par ^= 1; }
    }
  };

  if (warp >= 20) {
    reg_dec<C::REGP>();
  if (warp == 20) {
    // ================= copies =================
    if (lane == 0) {
      const uint64_t pol = l2_evict_first_policy();
      TreeCursor cur;
      cur.seek(rows_s, a.batch, u0);
      int st = 0, seg = 0, q_unit = -1;          // q_unit: a unit whose query operand is still to be fetched
      uint32_t par = 1;                          // parity of the stage's empty barrier
      bool ok = true;
      const uint8_t *pa = nullptr, *pr = nullptr;   // next K tile of the anchor, of the residual
      int it = 0;
#pragma unroll 1
      for (; it < n_it; ++it) {
        if (!(ok = wait(&empty_bar[st], par))) break;
        const int left = rows_s.len[cur.b] - cur.step * kTreeStep, tiles = left > kTile ? 2 : 1, t0 = cur.step * 2;
        const bool first = it == 0 || cur.step == 0, last = it + 1 == n_it || cur.step + 1 == cur.steps;
        const int unit = cur.b * per + cur.in_row;
        info_s[it & 7] = make_int2(min(left, kTreeStep) | (first ? 256 : 0) | (last ? 512 : 0), unit);
        uint8_t* dst = stages + st * C::STAGE;
        uint64_t* bar = &full_bar[st];
        mbar_arrive_expect_tx(bar, tiles * (2 * C::A_TILE + NRES * 2 * C::R_TILE));
        if (first) {
          const int h = cur.in_row / a.nqb, t = a.g.paged ? 0 : t0;   // paged: page 0; a page adds page_bytes
          pa = a.base + a.g.tile_offset(a.layer, a.group, cur.b, h, true, 0, 0, t, 0);
          if (NRES) pr = a.base + a.g.tile_offset(a.layer, a.group, cur.b, h, false, a.loop, 0, t, 0);
          q_unit = unit;
        }
        // contiguous: the two tiles of a plane are neighbours, one copy; paged: one a tile
        int64_t off = 0, va = a.g.plane_a, vr = a.g.plane_r;
        int n = a.g.paged ? 1 : tiles, i = 0;
#pragma unroll 1
        do {
          if (a.g.paged) {
            const int page = checked_page(a.g, raw_page(a.g, cur.b, t0 + i), a.status);
            off = (int64_t)max(page, 0) * a.g.page_bytes;
            va = C::A_TILE;
            vr = C::R_TILE;
          }
          bulk_g2s_hint(dst, pa + off, n * C::A_TILE, bar, pol);
          bulk_g2s_hint(dst + C::AV, pa + off + va, n * C::A_TILE, bar, pol);
          if (NRES) {
            bulk_g2s_hint(dst + C::RK - i * (C::A_TILE - C::R_TILE), pr + off, n * C::R_TILE, bar, pol);
            bulk_g2s_hint(dst + C::RV - i * (C::A_TILE - C::R_TILE), pr + off + vr, n * C::R_TILE, bar, pol);
          }
          dst += C::A_TILE;
          i += n;
        } while (i < tiles);
        if (!a.g.paged) {
          pa += 2 * C::A_TILE;
          if (NRES) pr += 2 * C::R_TILE;
        }
        if (++st == ST) { st = 0; par ^= 1; }
        // the query operand; the call's first one a step late, as the prep kernel may still run
        if (q_unit >= 0 && (it > 0 || last)) {
          if (seg == 0) pdl_wait();
          if (!(ok = wait(&qempty_bar[seg & 1], ((seg >> 1) & 1) ^ 1))) break;
          uint64_t* qb = &qfull_bar[seg & 1];
          mbar_arrive_expect_tx(qb, C::IMG);
          bulk_g2s(q_img + (seg & 1) * C::IMG, a.packs + (size_t)q_unit * C::IMG, C::IMG, qb);
          ++seg;
          q_unit = -1;
        }
        if (it + 1 < n_it) cur.next(rows_s, per);
      }
      if (!ok) {   // copies in flight land before the CTA leaves
        for (int i = max(0, it - ST); i < it; ++i) (void)mbar_wait_bounded(&full_bar[i % ST], (i / ST) & 1);
        for (int i = max(0, seg - 2); i < seg; ++i) (void)mbar_wait_bounded(&qfull_bar[i & 1], (i >> 1) & 1);
      }
    }
    __syncwarp();
  } else if (warp == 21) {
    // ================= products: scores =================
    const uint32_t q_lo = desc_lo(smem_u32(q_img));
    int seg = -1;
#pragma unroll 1
    for (int it = 0; it < n_it; ++it) {
      wait(&kfull_bar[0], it & 1);
      const int flags = info_s[it & 7].x;
      if (flags & 256) {
        ++seg;
        wait(&qfull_bar[seg & 1], (seg >> 1) & 1);
      }
      wait(&sempty_bar[s_buf(it)], s_par(it) ^ 1);
#pragma unroll
      for (int pl = 0; pl < PL; ++pl) {
        if (pl) wait(&kfull_bar[pl], it & 1);
        tc_after();
        __syncwarp();
        if (elect_one()) {
          tc_chain<D / 16>(tmem + C::S0 + (s_buf(it) * PL + pl) * NB, tmem + (pl ? C::KR : C::KA),
                           q_lo + (((seg & 1) * C::IMG + pl * (D / 16) * C::QSTEP) >> 4), kDescHiQ, C::QSTEP >> 4,
                           tc_idesc(NB, false), true);
          tc_commit(&kempty_bar[pl]);
          if (pl == PL - 1) {
            tc_commit(&sfull_bar[s_buf(it)]);
            if (flags & 512) tc_commit(&qempty_bar[seg & 1]);
          }
        }
        __syncwarp();
      }
    }
    // every product has ended before tensor memory is given back
    if (elect_one()) tc_commit(&drain_bar[0]);
    wait(&drain_bar[0], 0);
    __syncwarp();
  } else if (warp == 22) {
    // ================= products: values =================
    const uint32_t p_lo = desc_lo(smem_u32(p_buf));
#pragma unroll 1
    for (int it = 0; it < n_it; ++it) {
#pragma unroll
      for (int pl = 0; pl < PL; ++pl) {
        wait(&vfull_bar[pl], it & 1);
        if (pl == 0) wait(&pfull_bar, it & 1);
        tc_after();
        __syncwarp();
        const bool first = (info_s[it & 7].x & 256) != 0;
        if (elect_one()) {
          tc_chain<kTreeStep / 16>(tmem + (pl ? C::OR : C::OA), tmem + (pl ? C::VR : C::VA), p_lo, kDescHiP, 2048 >> 4,
                                   tc_idesc(NB, true), first);
          tc_commit(&vempty_bar[pl]);
          if (pl == PL - 1) tc_commit(&pempty_bar);
        }
        __syncwarp();
      }
    }
    if (elect_one()) tc_commit(&drain_bar[1]);
    wait(&drain_bar[1], 0);
    __syncwarp();
  }
  } else if (warp >> 2 == 1 || (C::NS == 2 && warp >> 2 == 3)) {
    reg_inc<C::REGS>();
    // ================= softmax: one token a lane =================
    const int lt = tid & 127, tok = lt & 63, tau = lt >> 6, w4 = warp & 3;
    // this group's queries: NQ from q_at; its named barrier
    constexpr int NQ = C::NQ;
    const int q_at = C::NS == 2 && warp >= 12 ? NQ : 0, my_bar = q_at ? 4 : 1;
    float(*qm)[4] = qm_s + q_at / 2;
    float* f_q = f_s + q_at;
    const uint32_t lanes = tmem + ((uint32_t)(w4 * 32) << 16);
    const int slot = v_slot(lt);
    float l[NQ];
    pdl_wait();
    int st = 0;
    uint32_t par = 0;
#pragma unroll 1
    for (int it = 0; it < n_it; ++it) {
      if (NRES) wait_warp(&full_bar[st], par); else wait_warp(&sfull_bar[s_buf(it)], s_par(it));
      const int2 info = info_s[it & 7];
      const bool first = (info.x & 256) != 0, on = lt < (info.x & 255);
      const int unit = info.y;
      if (first) {
#pragma unroll
        for (int i = 0; i < NQ; ++i) l[i] = 0.f;
        if (lt < NQ) {
          qm[lt >> 1][lt & 1] = __ldcg(a.q_scale + (size_t)unit * NB + q_at + lt);
          qm[lt >> 1][2 + (lt & 1)] = INFINITY;
        }
        wg_sync(my_bar);
      }
      float c = 0.f;
      if (NRES) {
        const uint16_t cb = *reinterpret_cast<const uint16_t*>(stages + st * C::STAGE + C::RK + tau * C::R_TILE +
                                                               C::R_CODES + C::META + tok * 2);
        c = on ? bf16_bits_to_f32(cb) : 0.f;
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty_bar[st]);
        if (++st == ST) { st = 0; par ^= 1; }
        wait_warp(&sfull_bar[s_buf(it)], s_par(it));
      }
      const float2 c2 = make_float2(c, c);
      tc_after();
      const uint32_t s0 = lanes + C::S0 + s_buf(it) * PL * NB + q_at;
      // score products of 16 queries with this lane's token
      auto scores = [&](int ch, float2 (&y)[8]) {
        uint32_t ra[16], rr[16];
        tc_ld16(s0 + 16 * ch, ra);
        if (NRES) tc_ld16(s0 + NB + 16 * ch, rr);
        tc_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          y[i] = make_float2(__uint_as_float(ra[2 * i]), __uint_as_float(ra[2 * i + 1]));
          if (NRES)
            y[i] = fma2(y[i], c2, make_float2(__uint_as_float(rr[2 * i]), __uint_as_float(rr[2 * i + 1])));
        }
      };
      // ... in log2 units, relative to the query's reference
      auto relative = [&](int ch, float2 (&y)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 k = *reinterpret_cast<const float4*>(qm[8 * ch + i]);
          y[i] = fma2(y[i], make_float2(k.x, k.y), make_float2(k.z, k.w));
        }
      };
      float top = -INFINITY;
      float2 kept[NQ / 2];     // relative scores
#pragma unroll
      for (int ch = 0; ch < NQ / 16; ++ch) {
        float2 y[8];
        scores(ch, y);
        relative(ch, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          top = fmaxf(top, fmaxf(y[i].x, y[i].y));
          kept[8 * ch + i] = y[i];
        }
      }
      if (__builtin_expect(wg_any(my_bar, on && top > kTop), 0)) {
        // move the references to this step's maxima where those are higher
        float top_q[NQ];
#pragma unroll
        for (int ch = 0; ch < NQ / 16; ++ch) {
          float2 y[8];
          scores(ch, y);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            top_q[16 * ch + i] = on ? (i & 1 ? y[i / 2].y : y[i / 2].x) * qm[8 * ch + i / 2][i & 1] : -INFINITY;
        }
        tree_spread<NQ, true>(top_q, wred_s[w4] + q_at, lane);
        wg_sync(my_bar);
        if (lt < NQ) {
          const float old = -qm[lt >> 1][2 + (lt & 1)];
          const float(*wr)[NB] = wred_s;
          const int q = q_at + lt;
          const float mx = fmaxf(fmaxf(wr[0][q], wr[1][q]), fmaxf(wr[2][q], wr[3][q])) - kHead;
          const float now = fmaxf(old, mx);
          f_q[lt] = old == now ? 1.f : exp2f(old - now);
          qm[lt >> 1][2 + (lt & 1)] = -now;
        }
        wg_sync(my_bar);
#pragma unroll
        for (int i = 0; i < NQ; ++i) l[i] *= f_q[i];
        if (!first) {   // O holds products of the steps before: all of them done, then scaled
          wait_warp(&pempty_bar, (it - 1) & 1);
          tc_after();
#pragma unroll
          for (int ch = 0; ch < PL * NQ / 16; ++ch) {
            uint32_t r[16];
            const uint32_t at = lanes + C::OA + (16 * ch / NQ) * NB + q_at + 16 * ch % NQ;
            tc_ld16(at, r);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f_q[(16 * ch + i) % NQ]);
            tc_st16(at, r);
          }
          tc_wait_st();
        }
#pragma unroll
        for (int ch = 0; ch < NQ / 16; ++ch) {
          float2 y[8];
          scores(ch, y);
          relative(ch, y);
#pragma unroll
          for (int i = 0; i < 8; ++i) kept[8 * ch + i] = y[i];
        }
      }
      // weights
      // the scores are in registers: their place in tensor memory is free
      tc_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sempty_bar[s_buf(it)]);
      wait_warp(&pempty_bar, (it & 1) ^ 1);
      uint8_t* prow = p_buf + slot * 128;
#pragma unroll
      for (int ch = 0; ch < NQ / 16; ++ch) {
        float2 y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = kept[8 * ch + i];
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          y[i].x = on ? ex2_fast(y[i].x) : 0.f;
          y[i].y = on ? ex2_fast(y[i].y) : 0.f;
          l[16 * ch + 2 * i] += y[i].x;
          l[16 * ch + 2 * i + 1] += y[i].y;
          w[i] = f16x2(y[i].x, y[i].y);
        }
        *reinterpret_cast<uint4*>(prow + (((q_at / 8 + 2 * ch) ^ (slot & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(prow + (((q_at / 8 + 2 * ch + 1) ^ (slot & 7)) << 4)) =
            make_uint4(w[4], w[5], w[6], w[7]);
      }
      fence_async_smem();
      tc_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&pfull_bar);
      if (__builtin_expect((info.x & 512) != 0, 0)) {
        // the unit's state out
        wait_warp(&pempty_bar, it & 1);
        tc_after();
        float* part = a.partials + (size_t)(blockIdx.x + unit) * a.pstride;
        if (lt < D) {
#pragma unroll
          for (int c = 0; c < PL * NQ / 16; ++c) {
            uint32_t r[16];
            const int q0 = (16 * c / NQ) * NB + q_at + 16 * c % NQ;   // plane and query
            if (D == 128 || w4 < 3) {
              tc_ld16(lanes + C::OA + q0, r);
              tc_wait_ld();
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(part + 2 * NB + ((size_t)(q0 / 4 + i) * D + lt) * 4) =
                  make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
          }
        }
        tc_before();
        tree_spread<NQ, false>(l, wred_s[w4] + q_at, lane);   // then over the warps in order
        wg_sync(my_bar);
        if (lt < NQ) {
          const int q = q_at + lt;
          part[q] = -qm[lt >> 1][2 + (lt & 1)];
          part[NB + q] = wred_s[0][q] + wred_s[1][q] + wred_s[2][q] + wred_s[3][q];
        }
        wg_sync(my_bar);
      }
    }
  } else {
    reg_dec<C::REGD>();
    if (warp < 4) {
    // ================= K: rows of tokens =================
    const int tau = warp >> 1;                              // the warp's tile of the step
    const int t4 = lane & 3, base = warp * 32;
    const uint32_t lanes = tmem + ((uint32_t)base << 16);
    int st = 0;
    uint32_t par = 0;
#pragma unroll 1
    for (int it = 0; it < n_it; ++it) {
      wait_warp(&full_bar[st], par);
      const uint8_t* s = stages + st * C::STAGE;
      const int nv = info_s[it & 7].x & 255;
#pragma unroll
      for (int pl = 0; pl < PL; ++pl) {
        const uint8_t* tile = pl ? s + C::RK + tau * C::R_TILE : s + tau * C::A_TILE;
        const uint16_t* meta = reinterpret_cast<const uint16_t*>(tile + (pl ? C::R_CODES : C::A_CODES));
        // the multiplier (residual: of the fields at bit 2, 4, 6) and the addend of group gi of the
        // tile's token `tok`; behind the row's end zeros, so that what lies there stays finite
        struct Consts { __half2 m[3], o; };
        auto consts = [&](int tok, int gi) {
          __half2 so = e4m3_pair(tau * kTile + tok < nv ? meta[tok * NG + gi] : (uint16_t)0);
          so = __hmul2(so, __halves2half2(half_pow2(24 - 4 - kScaleK), __ushort_as_half(0x0200)));   // 2^5, 2^-15
          Consts c;
          const __half2 m = __low2half2(so);
          c.o = __high2half2(so);
          c.m[0] = pl ? __hmul2(m, __half2half2(half_pow2(2))) : m;
          c.m[1] = m;
          c.m[2] = pl ? __hmul2(m, __half2half2(half_pow2(-2))) : m;
          return c;
        };
        wait_warp(&kempty_bar[pl], (it & 1) ^ 1);
        tc_after();
        if (D == 128) {
          // four lanes share a token, 32 channels each: contiguous shared-memory reads
#pragma unroll 1   // straight-line code for every part would stream through the instruction caches
          for (int hh = 0; hh < 2; ++hh) {
            uint32_t w[2][4];
            Consts k2[2][32 / GS];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int tok = (base & 63) + 16 * hh + 8 * k + (lane >> 2);
              if (pl == 0) {
                const uint4 v = *reinterpret_cast<const uint4*>(tile + tok * (D / 2) + t4 * 16);
                w[k][0] = v.x; w[k][1] = v.y; w[k][2] = v.z; w[k][3] = v.w;
              } else {
                const uint2 v = *reinterpret_cast<const uint2*>(tile + tok * (D / 4) + t4 * 8);
                w[k][0] = v.x; w[k][1] = v.y;
              }
#pragma unroll
              for (int c = 0; c < 32 / GS; ++c) k2[k][c] = consts(tok, t4 * (32 / GS) + c);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              constexpr int G1 = 32 / GS - 1;
              uint32_t r[16];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const Consts& q = k2[k][c & G1];
                if (pl == 0) {
#pragma unroll
                  for (int i = 0; i < 2; ++i) {
                    uint32_t v[4];
                    codes4(w[k][2 * c + i], v);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                      r[4 * (2 * i + (j >> 1)) + 2 * k + (j & 1)] = h2u(__hfma2(u2h(v[j]), q.m[1], q.o));
                  }
                } else {
                  uint32_t v[8];
                  codes2(w[k][c], v);
#pragma unroll
                  for (int j = 0; j < 8; ++j)
                    r[4 * (j >> 1) + 2 * k + (j & 1)] =
                        h2u(__hfma2(u2h(v[j]), q.m[(j & 3) < 2 ? 0 : (j & 3) - 1], q.o));
                }
              }
              tc_st_frag(lanes + ((uint32_t)(16 * hh) << 16) + (pl ? C::KR : C::KA) + 32 * c, r);
            }
          }
        } else {
          // width 96 does not split into four; one token a lane (rows of 48 bytes: no bank conflicts)
          const int tok = tid & 63;
          const uint8_t* row = tile + tok * (pl ? D / 4 : D / 2);
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {   // 32 channels: 16 columns
            uint32_t r[16];
            Consts q;
            if (pl == 0) {
              const uint4 w = reinterpret_cast<const uint4*>(row)[c];
              const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (i * 8 % GS == 0) q = consts(tok, c * (32 / GS) + i * 8 / GS);
                uint32_t v[4];
                codes4(ww[i], v);
#pragma unroll
                for (int j = 0; j < 4; ++j) r[4 * i + j] = h2u(__hfma2(u2h(v[j]), q.m[1], q.o));
              }
            } else {
              const uint2 w = reinterpret_cast<const uint2*>(row)[c];
              const uint32_t ww[2] = {w.x, w.y};
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                if (i * 16 % GS == 0) q = consts(tok, c * (32 / GS) + i * 16 / GS);
                uint32_t v[8];
                codes2(ww[i], v);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  r[8 * i + j] = h2u(__hfma2(u2h(v[j]), q.m[(j & 3) < 2 ? 0 : (j & 3) - 1], q.o));
              }
            }
            tc_st16(lanes + (pl ? C::KR : C::KA) + 16 * c, r);
          }
        }
        tc_wait_st();
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&kfull_bar[pl]);
      }
      if (lane == 0) mbar_arrive(&empty_bar[st]);
      if (++st == ST) { st = 0; par ^= 1; }
    }
    } else if (warp < 16) {   // 8 .. 11; with one softmax group 12 .. 15, too
      v_role(std::integral_constant<int, 0>{}, warp >= 12);
    } else if (NRES) {
      v_role(std::integral_constant<int, NRES>{}, 0);
    }
  }
  tc_before();
  __syncthreads();
  if (warp == 21) {
    tc_after();
    tc_dealloc(tmem, 512);
  }
}

// ---- merge -------------------------------------------------------------------------
// One CTA per MQ queries of a (row, KV head).  The drafted tokens first (before the wait:
// nothing of it depends on the streaming kernel), then the partial states, R^T, the quotient.
// Scores of the draft are products of BF16 numbers, exact on the 16-bit tensor cores with
// float32 sums; its values are added in float32, as a hidden one may be infinite or NaN and must
// not enter.  R^T is a product with both sides as two BF16 pieces (2^-16 against the result's
// 2^-9).  The kernel is a chain of latencies: what a part needs is loaded together, ahead of it
// (16 to 17 us cold and alone at 128 or 440 CTAs, of which a call sees what comes behind the wait).
// The 16-query instances do not fit their 64 registers: 44 to 144 bytes a thread are spilled and 268 to 416 reloaded (the
// 8-query ones 8 to 32 of each).
constexpr int kMergeThreads = 256;
constexpr int kDraftPitch = 272;       // bytes of a staged row: rows 4 banks apart
constexpr int kMergeChunk = 32;        // partial states whose weights are held at a time

template <int D, int NRES, int NB, int MQ>
__global__ void __launch_bounds__(kMergeThreads, NRES && MQ == 8 ? 2 : 4) tree_merge_kernel(TreeArgs a, int ctas) {
  constexpr int NT = MQ / 8, PARTS = kMergeThreads / MQ;
  // R^T loaded ahead in 64 registers, or, where many CTAs share an SM, when it is needed (4 CTAs an SM, not
  // 2: grouped-query batch 8 129 -> 124 us; 128 CTAs of 8 queries are 3 us slower that way)
  constexpr bool AHEAD = NRES && MQ == 8;
  __shared__ TreeRowsShared rows_s;
  __shared__ __align__(16) uint8_t kv_s[128 * kDraftPitch];   // drafted keys, then values
  __shared__ __align__(16) __nv_bfloat16 q_s[MQ][D + 8];
  __shared__ __align__(16) float p_s[128][MQ];                // [key][query], then R^T's operand [channel][query]
  __shared__ __align__(16) float w_s[kMergeChunk][MQ];        // weights of partial states
  __shared__ unsigned long long vis_s[MQ][RQ_MAX_TREE_NODES / 64];
  __shared__ float red_s[kMergeThreads / 32][MQ], m_s[MQ], l_s[MQ], f_s[MQ];
  __shared__ int range_s[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, half = tid >> 7, ch = tid & 127;
  const int g = lane >> 2, t4 = lane & 3, my_q = tid % MQ, part = tid / MQ;
  const int per_bh = (a.M + MQ - 1) / MQ;
  const int bh = blockIdx.x / per_bh, r0 = blockIdx.x % per_bh * MQ, b = bh / a.g.H;
  const int nq = min(MQ, a.M - r0);
  const bool hadamard = (a.g.mode & RQ_MODE_HADAMARD) != 0, dense = NRES && !hadamard && warp < D / 16;
  const int cnt = a.counts ? clamp_len(a.counts[b], a.T) : a.T;
  const uint4* kp = reinterpret_cast<const uint4*>(a.k_new + (size_t)bh * a.T * D);
  const uint4* vp = reinterpret_cast<const uint4*>(a.v_new + (size_t)bh * a.T * D);
  constexpr int RC = D / 8;              // 16-byte pieces of a row
  // rows j0 .. of the draft into shared memory
  auto stage = [&](const uint4* src, int j0) {
    const int n = min(128, cnt - j0) * RC;
#pragma unroll 4
    for (int i = tid; i < n; i += kMergeThreads)
      *reinterpret_cast<uint4*>(kv_s + (i / RC) * kDraftPitch + (i % RC) * 16) = __ldg(src + (size_t)j0 * RC + i);
  };
  // every query's value over all threads' (of one query: PARTS threads), in a fixed order
  auto reduce = [&](float v, bool sum) {
#pragma unroll
    for (int o = MQ; o < 32; o <<= 1) {
      const float y = __shfl_xor_sync(0xffffffffu, v, o);
      v = sum ? v + y : fmaxf(v, y);
    }
    __syncthreads();
    if (lane < MQ) red_s[warp][lane] = v;
    __syncthreads();
    v = red_s[0][my_q];
#pragma unroll
    for (int w = 1; w < kMergeThreads / 32; ++w) v = sum ? v + red_s[w][my_q] : fmaxf(v, red_s[w][my_q]);
    return v;
  };
  const uint4* qp = reinterpret_cast<const uint4*>(a.q + ((size_t)bh * a.M + r0) * D);
  for (int i = tid; i < MQ * RC; i += kMergeThreads)
    *reinterpret_cast<uint4*>(&q_s[i / RC][(i % RC) * 8]) = i / RC < nq ? __ldg(qp + i) : make_uint4(0u, 0u, 0u, 0u);
  if (cnt > 0) stage(kp, 0);
  // R^T, rows (output channels) 16 warp + g, + 8, columns 16 k .., as two pieces
  auto r_pieces = [&](int k, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float* rp = a.R + (size_t)(16 * k + 2 * t4 + (i >> 1) * 8) * D + 16 * warp + g + (i & 1) * 8;
      bf16_pieces(make_float2(__ldg(rp), __ldg(rp + D)), hi[i], lo[i]);
    }
  };
  uint32_t rhi[AHEAD ? D / 16 : 1][4], rlo[AHEAD ? D / 16 : 1][4];
  if (AHEAD && dense) {
#pragma unroll
    for (int k = 0; k < D / 16; ++k) r_pieces(k, rhi[AHEAD ? k : 0], rlo[AHEAD ? k : 0]);
  }
  for (int i = tid; i < MQ * (RQ_MAX_TREE_NODES / 64); i += kMergeThreads) {
    const int qi = i % MQ, w = i / MQ, t = (r0 + qi) % a.T;
    unsigned long long v = 0;
    if (qi < nq && t < cnt && w * 64 < cnt) {
      v = a.mask ? __ldg(a.mask + ((size_t)b * a.T + t) * a.words + w)
                 : (t >= w * 64 + 63 ? ~0ull : (t < w * 64 ? 0ull : (2ull << (t - w * 64)) - 1ull));
      if (cnt - w * 64 < 64) v &= (1ull << (cnt - w * 64)) - 1ull;
    }
    vis_s[qi][w] = v;
  }
  if (tid < MQ) {
    m_s[tid] = -INFINITY;
    l_s[tid] = 0.f;
  }
  tree_rows(a, &rows_s);
  __syncthreads();
  if (tid == 0) {   // the CTAs that hold a partial state of this unit
    const int U = rows_s.pre[a.batch];
    const int steps = (rows_s.len[b] + kTreeStep - 1) / kTreeStep;
    range_s[0] = 0;
    range_s[1] = -1;
    if (steps) {
      const TreeSplit split{U / ctas, U % ctas};
      const int s0 = rows_s.pre[b] + (bh * a.nqb + r0 / NB - b * a.g.H * a.nqb) * steps;
      range_s[0] = split.owner(s0);
      range_s[1] = split.owner(s0 + steps - 1);
    }
  }

  float o[MQ];            // this thread's channel: drafted values of its half of the tokens
#pragma unroll
  for (int i = 0; i < MQ; ++i) o[i] = 0.f;
#pragma unroll 1
  for (int j0 = 0; j0 < cnt; j0 += 128) {
    const int nk = min(128, cnt - j0);
    if (j0) {
      __syncthreads();
      stage(kp, j0);
      __syncthreads();
    }
    if (16 * warp < nk) {   // scores of 16 keys a warp
      float d[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) d[n][0] = d[n][1] = d[n][2] = d[n][3] = 0.f;
      const uint32_t* k0 = reinterpret_cast<const uint32_t*>(kv_s + (16 * warp + g) * kDraftPitch) + t4;
      const uint32_t* k1 = k0 + 8 * kDraftPitch / 4;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t ak[4] = {k0[8 * k], k1[8 * k], k0[8 * k + 4], k1[8 * k + 4]};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint32_t* bp = reinterpret_cast<const uint32_t*>(&q_s[8 * n + g][16 * k + 2 * t4]);
          mma_bf16(d[n], ak, bp[0], bp[4]);
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        *reinterpret_cast<float2*>(&p_s[16 * warp + g][8 * n + 2 * t4]) = make_float2(d[n][0], d[n][1]);
        *reinterpret_cast<float2*>(&p_s[16 * warp + g + 8][8 * n + 2 * t4]) = make_float2(d[n][2], d[n][3]);
      }
    }
    __syncthreads();
    stage(vp, j0);     // the keys are used up
    auto seen = [&](int k) { return (vis_s[my_q][(j0 + k) >> 6] >> ((j0 + k) & 63)) & 1; };
    float mx = -INFINITY;
    for (int k = part; k < nk; k += PARTS)
      if (seen(k)) mx = fmaxf(mx, p_s[k][my_q] * a.qscale);
    const float old = m_s[my_q], now = fmaxf(old, reduce(mx, false));   // its barriers: staged, m_s read
    const float ref = now == -INFINITY ? 0.f : now;
    float sum = 0.f;
    for (int k = part; k < nk; k += PARTS) {
      const float p = seen(k) ? exp2f(p_s[k][my_q] * a.qscale - ref) : 0.f;   // a NaN score stays
      p_s[k][my_q] = p;
      sum += p;
    }
    sum = reduce(sum, true);
    if (tid < MQ) {
      f_s[tid] = exp2f(old - ref);
      m_s[tid] = now;
      l_s[tid] = l_s[tid] * f_s[tid] + sum;
    }
    __syncthreads();
    if (ch < D) {
#pragma unroll
      for (int i = 0; i < MQ; ++i) o[i] *= f_s[i];
#pragma unroll 2
      for (int k = half; k < nk; k += 2) {
        const float v = bf16_bits_to_f32(*reinterpret_cast<const uint16_t*>(kv_s + k * kDraftPitch + ch * 2));
        const float4* pp = reinterpret_cast<const float4*>(p_s[k]);
        if (__builtin_expect(isfinite(v), 1)) {
#pragma unroll
          for (int i = 0; i < MQ / 4; ++i) {
            const float4 x = pp[i];
            o[4 * i] = fmaf(x.x, v, o[4 * i]);
            o[4 * i + 1] = fmaf(x.y, v, o[4 * i + 1]);
            o[4 * i + 2] = fmaf(x.z, v, o[4 * i + 2]);
            o[4 * i + 3] = fmaf(x.w, v, o[4 * i + 3]);
          }
        } else {   // enters only where it is seen
#pragma unroll
          for (int i = 0; i < MQ; ++i)
            if ((vis_s[i][(j0 + k) >> 6] >> ((j0 + k) & 63)) & 1) o[i] = fmaf(p_s[k][i], v, o[i]);
        }
      }
    }
  }

  // the cached tokens' partial states: the lower half takes the anchor's part, the upper the residual's
  pdl_wait();
  __syncthreads();
  const int c_lo = range_s[0], c_hi = range_s[1], qo = r0 % NB;
  const float* unit = a.partials + (size_t)(bh * a.nqb + r0 / NB) * a.pstride;
  float mx = -INFINITY;
  for (int c = c_lo + part; c <= c_hi; c += PARTS) mx = fmaxf(mx, __ldcg(unit + (size_t)c * a.pstride + qo + my_q));
  const float old = m_s[my_q];
  float ref = fmaxf(old, reduce(mx, false));     // common reference
  if (ref == -INFINITY) ref = 0.f;
  const float fd = exp2f(old - ref);             // the draft's weight
  float oc[MQ], lsum = 0.f;                      // this thread's plane of the cached tokens; their sums
#pragma unroll
  for (int i = 0; i < MQ; ++i) oc[i] = 0.f;
  const bool mine = ch < D && (NRES || !half);
#pragma unroll 1
  for (int c0 = c_lo; c0 <= c_hi; c0 += kMergeChunk) {
    const int nc = min(kMergeChunk, c_hi - c0 + 1);
    if (c0 != c_lo) __syncthreads();
    for (int c = part; c < nc; c += PARTS) {
      const float* p = unit + (size_t)(c0 + c) * a.pstride + qo + my_q;
      const float w = exp2f(__ldcg(p) - ref);
      w_s[c][my_q] = w;
      lsum = fmaf(w, __ldcg(p + NB), lsum);
    }
    __syncthreads();
    if (mine) {
#pragma unroll 4
      for (int c = 0; c < nc; ++c) {
        const float4* xp = reinterpret_cast<const float4*>(unit + (size_t)(c0 + c) * a.pstride + 2 * NB) +
                           (size_t)(half * (NB / 4) + qo / 4) * D + ch;
        const float4* wp = reinterpret_cast<const float4*>(w_s[c]);
#pragma unroll
        for (int i = 0; i < MQ / 4; ++i) {
          const float4 x = __ldcg(xp + i * D), w = wp[i];
          oc[4 * i] = fmaf(w.x, x.x, oc[4 * i]);
          oc[4 * i + 1] = fmaf(w.y, x.y, oc[4 * i + 1]);
          oc[4 * i + 2] = fmaf(w.z, x.z, oc[4 * i + 2]);
          oc[4 * i + 3] = fmaf(w.w, x.w, oc[4 * i + 3]);
        }
      }
    }
  }
  lsum = reduce(lsum, true);                     // its barriers also free p_s
  if (tid < MQ) {
    l_s[tid] = l_s[tid] * fd + lsum;
    f_s[tid] = fd;
  }
  // the operands' powers of two: V's anchor under a coefficient 2^-7, else 2^-15
  const float up = NRES && !half ? 128.f : 32768.f;
#pragma unroll
  for (int i = 0; i < MQ; ++i) oc[i] *= up;
  if (NRES && half) {
#pragma unroll
    for (int i = 0; i < MQ; ++i) p_s[ch][i] = oc[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < MQ; ++i) o[i] = o[i] * f_s[i] + (half ? 0.f : oc[i]);
  float* h_s = reinterpret_cast<float*>(kv_s);   // [query][channel + pad]: what joins the lower half's sum
  constexpr int HP = 132;
  if (NRES && hadamard) {
    float t[MQ];
#pragma unroll
    for (int i = 0; i < MQ; ++i) t[i] = half ? 0.f : p_s[ch][i];
    __syncthreads();
    hadamard128<MQ>(t, tid, h_s);   // threads >= 128 only take part in its barriers
    __syncthreads();
    if (!half) {
#pragma unroll
      for (int i = 0; i < MQ; ++i) o[i] += t[i];
    }
  }
  if (half) {
#pragma unroll
    for (int i = 0; i < MQ; ++i) h_s[i * HP + ch] = o[i];
  }
  __syncthreads();
  if (dense) {
    float d[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) d[n][0] = d[n][1] = d[n][2] = d[n][3] = 0.f;
#pragma unroll(AHEAD ? D / 16 : 2)
    for (int k = 0; k < D / 16; ++k) {
      if (!AHEAD) r_pieces(k, rhi[0], rlo[0]);
      const uint32_t(&hi)[4] = rhi[AHEAD ? k : 0], (&lo)[4] = rlo[AHEAD ? k : 0];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint32_t bh2[2], bl2[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int kk = 16 * k + 2 * t4 + 8 * i;
          bf16_pieces(make_float2(p_s[kk][8 * n + g], p_s[kk + 1][8 * n + g]), bh2[i], bl2[i]);
        }
        mma_bf16(d[n], hi, bh2[0], bh2[1]);
        mma_bf16(d[n], lo, bh2[0], bh2[1]);
        mma_bf16(d[n], hi, bl2[0], bl2[1]);
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float* h = h_s + (8 * n + 2 * t4) * HP + 16 * warp + g;
      h[0] += d[n][0];
      h[HP] += d[n][1];
      h[8] += d[n][2];
      h[HP + 8] += d[n][3];
    }
  }
  __syncthreads();
  if (!half && ch < D) {
    __nv_bfloat16* op = a.out + ((size_t)bh * a.M + r0) * D + ch;
#pragma unroll
    for (int i = 0; i < MQ; ++i) {
      const float l = l_s[i];
      if (i < nq && (r0 + i) % a.T < cnt)   // no key seen: zero; NaN stays
        op[(size_t)i * D] = __float2bfloat16_rn(l != 0.f ? (o[i] + h_s[i * HP + ch]) / l : 0.f);
    }
  }
}

template <int D, int GS, int NRES, int NB>
cudaError_t launch_tree_t(const TreeArgs& args, int num_sms, cudaStream_t stream) {
  using C = TreeCfg<D, GS, NRES, NB>;
  TreeArgs a = args;
  a.pstride = C::PSTRIDE;
  auto* kern = tree_mma_kernel<D, GS, NRES, NB>;
  static std::atomic<int> ready[kMaxDevices];   // shared-memory limit set on this device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    ready[dev].store(1, std::memory_order_release);
  }
  const int units = a.batch * a.g.H * a.nqb;
  // queries a prep CTA: 16, or 32 once 16 make more CTAs than are resident at a time (R is then read half as
  // often; 512 CTAs of 16: the call takes 123.6 us, 256 of 32: 121.3; the other way 220 CTAs 36.6 and 110 37.3 us)
  constexpr int QP2 = NB < 32 ? NB : 32;
  if (units * (NB / 16) > 2 * num_sms)
    e = launch_dependent(tree_prep_kernel<D, NRES, NB, QP2>, dim3(units * (NB / QP2)), dim3(256), 0, stream, a);
  else
    e = launch_dependent(tree_prep_kernel<D, NRES, NB, 16>, dim3(units * (NB / 16)), dim3(256), 0, stream, a);
  if (e != cudaSuccess) return e;
  e = launch_dependent(kern, dim3(num_sms), dim3(kTreeThreads), (size_t)C::SMEM, stream, a);
  if (e != cudaSuccess) return e;
  // queries a merge CTA: 8, or 16 once that still leaves every SM several CTAs (R^T and the draft are
  // then read half as often: 512 CTAs 121 us a call, against 130 with 1024 of 8; but 64 CTAs of 16 take 66 us, 128 of
  // 8 54 us)
  const int bh = a.batch * a.g.H;
  if (bh * ((a.M + 15) / 16) >= 2 * num_sms)
    return launch_dependent(tree_merge_kernel<D, NRES, NB, 16>, dim3(bh * ((a.M + 15) / 16)), dim3(kMergeThreads), 0,
                            stream, a, num_sms);
  return launch_dependent(tree_merge_kernel<D, NRES, NB, 8>, dim3(bh * ((a.M + 7) / 8)), dim3(kMergeThreads), 0, stream,
                          a, num_sms);
}

template <int D, int GS, int NRES>
cudaError_t launch_tree_nb(const TreeArgs& a, int nb, int num_sms, cudaStream_t stream) {
  if (nb == 16) return launch_tree_t<D, GS, NRES, 16>(a, num_sms, stream);
  if (nb == 32) return launch_tree_t<D, GS, NRES, 32>(a, num_sms, stream);
  return launch_tree_t<D, GS, NRES, 64>(a, num_sms, stream);
}

template <int D>
cudaError_t launch_tree_d(const TreeArgs& a, int nb, int num_sms, cudaStream_t stream) {
  if (a.g.g == 32)
    return a.nres ? launch_tree_nb<D, 32, 1>(a, nb, num_sms, stream) : launch_tree_nb<D, 32, 0>(a, nb, num_sms, stream);
  return a.nres ? launch_tree_nb<D, 16, 1>(a, nb, num_sms, stream) : launch_tree_nb<D, 16, 0>(a, nb, num_sms, stream);
}

}  // namespace
}  // namespace rq
