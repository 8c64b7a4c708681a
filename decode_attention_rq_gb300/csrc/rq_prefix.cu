// rq_prefix_plan, rq_prefix_attention: decode attention of rows that share pages.
//
// Rows of a family (a prompt's samples or beams) name the same pages in their first tiles.  With S such
// tiles, row b's attention over its n cached tokens and the current one splits by tokens,
//   out = (sum_{k < 64 S} e^(s_k - m) v_k + sum_{64 S <= k < n} ... + e^(s_now - m) v_now) / (the same without v),
// and in the first sum every row of the family meets the same keys: a matrix product of all their queries.
//
// Plan (once a step, for all layers and loops): the tiles that every family shares, found by comparing its rows' table
// entries; each row's rest as a table and a length of its own; the split of the work.  Then a call is four launches,
// each but the first started early by the one before:
//   1. prefix_prep_kernel: q and R q as operands of both streaming kernels.
//   2. the tensor-core streaming kernel of rq_tree_kernels.cuh over the shared tiles: its "rows" are blocks of NB queries
//      of a family, so that the shared tiles are read and dequantized once for NB rows.
//   3. each row's own tiles: the decode streaming kernel (rq_decode_kernels.cuh, rq_decode_gqa.cu), or, for 3 to 16 query heads a
//      KV head, the tensor-core one again, the query heads making its N side.
//   4. prefix_merge_kernel: both kinds of partial states, the current token, R^T, the quotient.
//
// Measured with 16 heads of 128, 32 rows of one 8192-token prompt and up to 512 tokens of their own (60 MB to read, 9 us at
// the memory's rate), a residual loop: 48 us a call; every row alone 219.  Bound by latencies: the streaming kernel's 7 steps
// a CTA with their start take 22 us, the rows' own tiles 10 to 14 more, the merge 6 behind them, the prep 6 ahead; the first
// steps of each overlap the end of the one before.  64 rows of eight prompts, four query heads a KV head, groups of 16: 161 us against 41 at
// the memory's rate, bound by dequantizing, as rq_tree_attention (0.67 and 0.58 instructions a clock of each scheduler).
// Two rows and one shared tile already make a family, whatever it costs: with 16 heads of 128 the call is faster than
// rq_decode_attention from 4 rows of 8192 shared tokens (34 us for 37) or 32 rows of 512 (28 for 35) on, with four query
// heads a KV head from 2 rows of 2048 (22 for 23) or 8 of 64 (20.6 for 21.2).  The plan takes 6.5 us, once a step.
#include "rq_tree_kernels.cuh"
#include "rq_decode_kernels.cuh"

namespace rq {
namespace {

constexpr int kPlanMagic = 0x52515031;
constexpr int kPlanRows = RQ_MAX_DECODE_BATCH;
constexpr int kPlanThreads = 256;         // >= kPlanRows: a thread a row, a family, a block of queries
constexpr int kPrepQ = 16;                // queries of a prep CTA
constexpr int kOwnNB = 16;                // queries of a block where a row's own tiles take the tensor-core kernel
constexpr int kShareRows = 2;             // rows that have to share a tile for it to be read once for all

// Where a plan keeps what (offsets in int32 words).
struct PlanLayout {
  int batch, n, nb, ntiles, max_blocks, max_merges, max_preps;
  int mq;                                 // queries of a merge CTA
  int row;                                // per row: length, shared tiles, length of the rest, units before it
  int rest;                               // lengths of the rests again, as the streaming kernel reads them
  int common, lead, family;               // per row: scratch of the first step
  int b_len, b_family;                    // per block of NB queries: length, family (-1: none)
  int f_row;                              // per family: first row
  // per merge CTA of a KV head: first row of its family (-1: nothing to do), first query, queries, block of queries (-1: nothing
  // shared); steps of the block, steps before it, all steps, all units of the rows' rests
  int merge;
  int prep;                               // per prep CTA of a KV head: first row, first query, queries of the family, first block
  int rest_table, block_table;            // [batch][ntiles], [max_blocks][ntiles]
  int r_image, rt_image;                  // R and R^T as tensor-core operands, two BF16 pieces
  size_t words;
};
enum PlanHead { H_MAGIC, H_BATCH, H_N, H_NB, H_HEADS, H_QPK, H_TILES, H_ROT, H_TABLE, H_R = 10, H_WORDS = 12 };

int plan_nb(const Geom& g, int batch, int n) {   // the average family's queries a KV head (see tree_nb's figures)
  const int64_t m = ((int64_t)batch * g.qpk + n - 1) / n;
  return m <= 16 ? 16 : (m <= 32 ? 32 : 64);
}

// A row's own tiles go through the tensor-core kernel from three query heads a KV head on: a step of 128 tokens takes it the same
// time for up to 16 of them.  Measured with 16 KV heads of 128, 32 rows of four 2048-token prompts, a call: four query heads
// and tails of up to 1024 tokens 72 us (the decode kernel 83), up to 300 tokens in groups of 16 channels 51 (71); three
// query heads and up to 300 tokens 49 (65), two 44.8 (44.5).
bool own_tree(const Geom& g) { return g.qpk >= 3 && g.qpk <= kOwnNB; }

// width and kind of the rotation
__host__ __device__ constexpr int plan_rotation(const Geom& g) { return g.d << 8 | (g.mode & RQ_MODE_HADAMARD); }

// where the plan's tables and rotation came from: two words each
__device__ __forceinline__ int4 plan_origin(const Geom& g, const float* R) {
  const uint64_t t = reinterpret_cast<uint64_t>(g.table), r = g.mode & RQ_MODE_HADAMARD ? 0 : reinterpret_cast<uint64_t>(R);
  return make_int4((int)(uint32_t)t, (int)(t >> 32), (int)(uint32_t)r, (int)(r >> 32));
}

constexpr int image_words(int d) { return d * d; }   // two BF16 pieces of d x d

PlanLayout plan_layout(const Geom& g, int batch, int n) {
  PlanLayout l = {};
  l.batch = batch;
  l.n = n;
  l.nb = plan_nb(g, batch, n);
  l.ntiles = g.ntiles;
  const int64_t queries = (int64_t)batch * g.qpk;
  const int64_t blocks = (queries + l.nb - 1) / l.nb + (n < batch / 2 ? n : batch / 2);   // a family that shares has two rows
  l.max_blocks = (int)(blocks < kPlanRows ? blocks : kPlanRows);
  // queries a merge CTA: 8, or 16 where that still makes two CTAs on each of 152 SMs (R^T is then read half as often).  64
  // query and 16 KV heads, 128 rows: 103 us with 16, 106 with 8 (512 CTAs); 55 heads of 96, 256 rows: 226 and 233; 80 rows
  // in families of ten, whose last CTA of 16 is half empty: 83 and 79 (320); 64 rows: 62 and 64 (256)
  l.mq = g.H * ((queries + 15) / 16) >= 304 ? 16 : 8;
  l.max_merges = (int)((queries + l.mq - 1) / l.mq + n);
  l.max_preps = (int)((queries + kPrepQ - 1) / kPrepQ + n);
  size_t at = H_WORDS;
  auto take = [&](size_t words) {
    const size_t p = at;
    at += (words + 3) / 4 * 4;
    return (int)p;
  };
  l.row = take(4 * (size_t)batch);
  for (int* p : {&l.rest, &l.common, &l.lead, &l.family}) *p = take(batch);
  for (int* p : {&l.b_len, &l.b_family}) *p = take(l.max_blocks);
  l.f_row = take(n);
  l.merge = take(8 * (size_t)l.max_merges);
  l.prep = take(4 * (size_t)l.max_preps);
  for (int* p : {&l.r_image, &l.rt_image}) *p = take(image_words(g.d));
  l.rest_table = take((size_t)batch * l.ntiles);
  l.block_table = take((size_t)l.max_blocks * l.ntiles);
  l.words = at;
  return l;
}

struct PlanArgs {
  Geom g;
  PlanLayout l;
  const int32_t *starts, *seq_lens;
  const float* R;
  int32_t* plan;
  int per_unit;                           // units of a row that cover the same tokens, one per KV head or group of query heads
};

// First rows of the families in shared memory: taken into 0 .. batch, never falling, 0 for the first, batch behind the
// last.  Every thread of the CTA (kPlanThreads) calls it.
__device__ __forceinline__ void plan_starts(const PlanArgs& a, int (&s)[kPlanRows + 1]) {
  const int t = threadIdx.x;
  int v = t > 0 && t < a.l.n ? min(max(a.starts[t], 0), a.l.batch) : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, o);
    if ((t & 31) >= o) v = max(v, y);
  }
  s[t] = v;
  __syncthreads();
  for (int w = 0; w < t >> 5; ++w) v = max(v, s[32 * w + 31]);
  __syncthreads();
  s[t] = t < a.l.n ? v : a.l.batch;
  if (t == 0) s[kPlanRows] = a.l.batch;
  __syncthreads();
}

// One CTA per row: its family, and how many leading tiles it has in common with the family's first row that is not
// empty (whole tiles, pages of the pool).
__global__ void __launch_bounds__(kPlanThreads) plan_rows_kernel(PlanArgs a) {
  __shared__ int starts_s[kPlanRows + 1];
  __shared__ int lead_s, diff_s;
  const int t = threadIdx.x, b = blockIdx.x;
  pdl_launch_dependents();
  plan_starts(a, starts_s);
  const int f = __syncthreads_count(t < a.l.n && starts_s[t] <= b) - 1;
  const int r0 = starts_s[f], r1 = starts_s[f + 1];
  if (t == 0) {
    lead_s = r1;
    diff_s = 0x7fffffff;
  }
  __syncthreads();
  if (r0 + t < r1 && a.seq_lens[r0 + t] > 0) atomicMin(&lead_s, r0 + t);
  __syncthreads();
  const int lead = lead_s, len = clamp_len(a.seq_lens[b], a.g.Nmax);
  const int most = lead < r1 ? min(len, clamp_len(a.seq_lens[lead], a.g.Nmax)) / kTile : 0;
  const int32_t *mine = a.g.table + (size_t)b * a.g.max_tiles, *first = a.g.table + (size_t)lead * a.g.max_tiles;
  for (int i = t; i < most; i += kPlanThreads) {
    const int p = mine[i];
    if (p < 0 || p >= a.g.num_pages || p != first[i]) {
      atomicMin(&diff_s, i);
      break;
    }
  }
  __syncthreads();
  if (t == 0) {
    a.plan[a.l.row + 4 * b] = len;
    a.plan[a.l.family + b] = f;
    a.plan[a.l.lead + b] = lead;
    a.plan[a.l.common + b] = min(most, diff_s);
  }
}

// Exclusive prefix sum over the CTA's kPlanThreads threads; *total: the sum.
__device__ __forceinline__ int plan_scan(int v, int* total) {
  __shared__ int warp_s[kPlanThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();   // a previous call's readers
  if (lane == 31) warp_s[warp] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) before += warp_s[w];
    all += warp_s[w];
  }
  *total = all;
  return before + x - v;
}

// One CTA: the families' shared tiles, the blocks of their queries, the split of the work.
__global__ void __launch_bounds__(kPlanThreads) plan_families_kernel(PlanArgs a) {
  __shared__ int starts_s[kPlanRows + 1];
  __shared__ int tiles_s[kPlanRows], rows_s[kPlanRows], block_s[kPlanRows], steps_s[kPlanRows], first_s[kPlanRows];
  __shared__ int merge_s[kPlanRows], prep_s[kPlanRows];
  const int t = threadIdx.x;
  const PlanLayout& l = a.l;
  pdl_launch_dependents();
  plan_starts(a, starts_s);
  pdl_wait();
  tiles_s[t] = 0x7fffffff;
  rows_s[t] = 0;
  __syncthreads();
  const int len = t < l.batch ? __ldcg(a.plan + l.row + 4 * t) : 0, fam = t < l.batch ? __ldcg(a.plan + l.family + t) : 0;
  if (len > 0) {
    atomicMin(&tiles_s[fam], __ldcg(a.plan + l.common + t));
    atomicAdd(&rows_s[fam], 1);
  }
  __syncthreads();
  // family t: its blocks of queries, its steps, its merge CTAs
  const int queries = t < l.n ? (starts_s[t + 1] - starts_s[t]) * a.g.qpk : 0;
  int tiles = t < l.n && rows_s[t] >= kShareRows ? tiles_s[t] : 0;
  int blocks = tiles ? (queries + l.nb - 1) / l.nb : 0, total = 0;
  const int block0 = plan_scan(blocks, &total);
  if (block0 + blocks > l.max_blocks) tiles = blocks = 0;    // no room: its rows attend alone
  const int steps = (tiles + 1) / 2 * a.g.H;
  const int steps0 = plan_scan(blocks * steps, &total);
  const int all_steps = total;
  const int merges = (queries + l.mq - 1) / l.mq;
  const int merge0 = plan_scan(merges, &total);
  const int all_merges = total;
  const int preps = (queries + kPrepQ - 1) / kPrepQ;
  const int prep0 = plan_scan(preps, &total);
  const int all_preps = total;
  __syncthreads();
  tiles_s[t] = tiles;
  block_s[t] = blocks ? block0 : 0x7fffffff;
  steps_s[t] = steps0;
  first_s[t] = blocks;
  merge_s[t] = merge0;
  prep_s[t] = prep0;
  if (t < l.n) a.plan[l.f_row + t] = starts_s[t];
  __syncthreads();
  // row t
  const int share = len > 0 ? tiles_s[fam] : 0;
  const int rest = len - share * kTile, units = (rest + 2 * kTile - 1) / (2 * kTile) * a.per_unit;
  const int units0 = plan_scan(t < l.batch ? units : 0, &total);
  const int all_units = total;
  if (t < l.batch) {
    a.plan[l.row + 4 * t + 1] = share;
    a.plan[l.row + 4 * t + 2] = a.plan[l.rest + t] = rest;
    a.plan[l.row + 4 * t + 3] = units0;
  }
  // block t
  if (t < l.max_blocks) {
    int f = -1;
    for (int i = 0; i < l.n; ++i)
      if (block_s[i] <= t && t < block_s[i] + first_s[i]) f = i;
    a.plan[l.b_len + t] = f >= 0 ? tiles_s[f] * kTile : 0;
    a.plan[l.b_family + t] = f;
  }
  // CTA m of families in a row: its family, `start` holding the first CTA of each
  auto family = [&](const int (&start)[kPlanRows], int m) {
    int lo = 0, hi = l.n - 1;                     // the last family that starts at or before m
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (start[mid] <= m) lo = mid; else hi = mid - 1;
    }
    return lo;
  };
  auto queries_of = [&](int f) { return (starts_s[f + 1] - starts_s[f]) * a.g.qpk; };
  for (int m = t; m < l.max_merges; m += kPlanThreads) {
    int4 x = make_int4(-1, 0, 0, -1), y = make_int4(0, 0, 0, 0);
    if (m < all_merges) {
      const int f = family(merge_s, m), i0 = (m - merge_s[f]) * l.mq;
      x = make_int4(starts_s[f], i0, min(l.mq, queries_of(f) - i0), -1);
      if (first_s[f]) {
        const int each = (tiles_s[f] + 1) / 2, b = i0 / l.nb;
        x.w = block_s[f] + b;
        y = make_int4(each, steps_s[f] + b * each * a.g.H, 0, 0);
      }
      y.z = all_steps;
      y.w = all_units;
    }
    reinterpret_cast<int4*>(a.plan + l.merge)[2 * m] = x;
    reinterpret_cast<int4*>(a.plan + l.merge)[2 * m + 1] = y;
  }
  for (int m = t; m < l.max_preps; m += kPlanThreads) {
    int4 x = make_int4(-1, 0, 0, -1);
    if (m < all_preps) {
      const int f = family(prep_s, m);
      x = make_int4(starts_s[f], (m - prep_s[f]) * kPrepQ, queries_of(f), first_s[f] ? block_s[f] : -1);
    }
    reinterpret_cast<int4*>(a.plan + l.prep)[m] = x;
  }
  if (t == 0) {
    a.plan[H_BATCH] = l.batch;
    a.plan[H_N] = l.n;
    a.plan[H_NB] = l.nb;
    a.plan[H_HEADS] = a.g.H;
    a.plan[H_QPK] = a.g.qpk;
    a.plan[H_TILES] = l.ntiles;
    a.plan[H_ROT] = plan_rotation(a.g);
    *reinterpret_cast<int4*>(a.plan + H_TABLE) = plan_origin(a.g, a.R);
    a.plan[H_MAGIC] = kPlanMagic;
  }
}

// The tables: one CTA per row (its tiles behind the shared ones) and per block (the shared ones); then two per 16 rows of
// R: rows of R and of R^T as the A operands of 16-bit products, hi[4] and lo[4] of a lane together.
__global__ void __launch_bounds__(kPlanThreads) plan_tables_kernel(PlanArgs a) {
  const PlanLayout& l = a.l;
  const int i = blockIdx.x;
  int from, n;
  int32_t* to;
  const int32_t* row;
  if (i >= l.batch + l.max_blocks) {
    const int part = i - l.batch - l.max_blocks, d = a.g.d, w = part >> 1;
    const bool turned = part & 1;
    const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    for (int k = threadIdx.x >> 5; k < d / 16; k += kPlanThreads / 32) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {               // rows g, g + 8; columns 2 t4, 2 t4 + 8
        const int r = 16 * w + g + (x & 1) * 8, c = 16 * k + 2 * t4 + (x >> 1) * 8;
        const float2 v = turned ? make_float2(a.R[(size_t)c * d + r], a.R[(size_t)(c + 1) * d + r])
                                : make_float2(a.R[(size_t)r * d + c], a.R[(size_t)r * d + c + 1]);
        bf16_pieces(v, hi[x], lo[x]);
      }
      uint4* out = reinterpret_cast<uint4*>(a.plan + (turned ? l.rt_image : l.r_image)) + ((w * (d / 16) + k) * 32 + lane) * 2;
      out[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      out[1] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    pdl_wait();
    return;
  }
  pdl_wait();
  if (i < l.batch) {
    from = __ldcg(a.plan + l.row + 4 * i + 1);
    n = (__ldcg(a.plan + l.rest + i) + kTile - 1) / kTile;
    row = a.g.table + (size_t)i * a.g.max_tiles;
    to = a.plan + l.rest_table + (size_t)i * l.ntiles;
  } else {
    const int v = i - l.batch, f = __ldcg(a.plan + l.b_family + v);
    if (f < 0) return;
    from = 0;
    n = __ldcg(a.plan + l.b_len + v) / kTile;
    row = a.g.table + (size_t)__ldcg(a.plan + l.lead + __ldcg(a.plan + l.f_row + f)) * a.g.max_tiles;
    to = a.plan + l.block_table + (size_t)v * l.ntiles;
  }
  for (int t = threadIdx.x; t < n; t += kPlanThreads) to[t] = row[from + t];
}

// ---- one call -------------------------------------------------------------------

struct PrefixArgs {
  Geom g;
  PlanLayout l;
  const int32_t* plan;
  const float* R;
  const __nv_bfloat16 *q, *k_cur, *v_cur;
  const int32_t* seq_lens;
  __nv_bfloat16* out;
  int32_t* status;
  float qscale;                    // softmax_scale * log2(e)
  // shared tiles: the tensor-core streaming kernel's operands and partial states
  uint8_t* packs;
  float *scales, *partials;
  int64_t pstride;
  int ctas;
  // the rows' own tiles: the same of the kernel that reads them
  uint8_t* o_packs;
  float *o_scales, *o_partials;
  int64_t o_pstride;
  int o_ctas, qh;                  // qh: query heads of a decode unit
};

// Whether the plan is one of this shape, table and rotation (uniform over the grid).
__device__ __forceinline__ bool plan_fits(const PrefixArgs& a) {
  const int4 x = __ldg(reinterpret_cast<const int4*>(a.plan)), y = __ldg(reinterpret_cast<const int4*>(a.plan) + 1);
  const int4 z = __ldg(reinterpret_cast<const int4*>(a.plan) + 2), w = plan_origin(a.g, a.R);
  return x.x == kPlanMagic && x.y == a.l.batch && x.z == a.l.n && x.w == a.l.nb && y.x == a.g.H && y.y == a.g.qpk &&
         y.z == a.l.ntiles && y.w == plan_rotation(a.g) && z.x == w.x && z.y == w.y && z.z == w.z && z.w == w.w;
}

// 16 queries a CTA, neighbours in their family and of one KV head: as operands of the tensor-core kernel for the shared
// tiles (their place in a block of NB), and for the row's own (OWN: their place among its query heads) or as packs of
// the decode kernel.  x is BF16 and so exact; R x is a product on the 16-bit tensor cores, R as two BF16 pieces
// (2^-16) from the plan.  Only the plan is read ahead of the wait (its last kernel releases no dependents early): the
// kernel before the call may release its own early and write queries, tokens or the cache.  The call's other kernels start
// behind this wait and may read them at once.
template <int D, int GS, int NRES, int NB, bool OWN>
__global__ void __launch_bounds__(256) prefix_prep_kernel(PrefixArgs a) {
  using C = Cfg<D, GS, NRES>;
  constexpr int PL = 1 + NRES, NG = C::NG, NIMG = C::NIMG, NMA = C::NMA;
  constexpr int IMG = PL * (D / 16) * NB * 32, OIMG = PL * (D / 16) * kOwnNB * 32;
  constexpr int PITCH = D + 8, RPITCH = D + 4;
  constexpr int WORDS = kPackHeader + 8 * NIMG;             // words of a decode pack in use
  __shared__ __align__(16) __nv_bfloat16 q_s[kPrepQ][PITCH];
  __shared__ __align__(16) float r_s[NRES ? kPrepQ : 1][RPITCH];
  __shared__ __align__(16) uint4 img_s[PL * (D / 8)][kPrepQ];    // 8 channels of a query
  __shared__ __align__(16) uint32_t out_s[OWN ? 4 : kPrepQ * WORDS];
  __shared__ float up_s[kPrepQ][3], scale_s[kPrepQ];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
  const bool hadamard = (a.g.mode & RQ_MODE_HADAMARD) != 0;
  const int part = blockIdx.x / a.g.H, h = blockIdx.x % a.g.H;
  const bool fits = plan_fits(a);
  const int4 rec = __ldg(reinterpret_cast<const int4*>(a.plan + a.l.prep) + part);
  const int row0 = rec.x, first = rec.y, queries = rec.z, block0 = rec.w, valid = min(kPrepQ, queries - first);
  uint4 rf[NRES ? D / 16 : 1][2];
  if (NRES && !hadamard && warp < D / 16) {
    const uint4* rp = reinterpret_cast<const uint4*>(a.plan + a.l.r_image) + (warp * (D / 16) * 32 + lane) * 2;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      rf[NRES ? k : 0][0] = __ldg(rp + k * 64);
      rf[NRES ? k : 0][1] = __ldg(rp + k * 64 + 1);
    }
  }
  pdl_wait();
  pdl_launch_dependents();
  if (!fits || row0 < 0) return;
  // one warp per query: its values (zeros where there is none), its power of two
#pragma unroll
  for (int r = warp; r < kPrepQ; r += 8) {
    uint2 v = make_uint2(0u, 0u);
    if (r < valid && lane < D / 4) {
      const int i = first + r;
      const size_t row = (size_t)(row0 + i / a.g.qpk) * a.g.Hq + h * a.g.qpk + i % a.g.qpk;
      v = __ldg(reinterpret_cast<const uint2*>(a.q + row * D) + lane);
    }
    if (lane < D / 4) *reinterpret_cast<uint2*>(&q_s[r][4 * lane]) = v;
    uint32_t big = max(max(v.x & 0x7FFFu, (v.x >> 16) & 0x7FFFu), max(v.y & 0x7FFFu, (v.y >> 16) & 0x7FFFu));
    big = __reduce_max_sync(0xffffffffu, big);   // magnitudes of BF16 numbers compare as integers
    int e = 11;
    if (big > 0 && big < 0x7F80u) frexpf(__uint_as_float(big << 16), &e);   // f 2^e, f in [0.5, 1)
    e = max(e, -115);                                                       // 2^(11 - e) stays finite
    if (lane == 0) {
      up_s[r][2] = ldexpf(1.f, 11 - e);
      scale_s[r] = ldexpf(a.qscale, e - 11 + kScaleK);
    }
  }
  __syncthreads();
  if (NRES && hadamard) {
    for (int r = warp; r < kPrepQ; r += 8) {   // lane holds channels lane, lane + 32, ...; stages h = 1 .. 64
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __bfloat162float(q_s[r][(lane + 32 * i) % D]);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = __shfl_xor_sync(0xffffffffu, v[i], o);
          v[i] = (lane & o) ? p - v[i] : v[i] + p;
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
      for (int n = 0; n < kPrepQ; n += 8) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t* bp = reinterpret_cast<const uint32_t*>(&q_s[n + g][16 * k + 2 * t4]);
          const uint32_t b0 = bp[0], b1 = bp[4];
          const uint4 x = rf[NRES ? k : 0][0], y = rf[NRES ? k : 0][1];
          const uint32_t hi[4] = {x.x, x.y, x.z, x.w}, lo[4] = {y.x, y.y, y.z, y.w};
          mma_bf16(d, hi, b0, b1);
          mma_bf16(d, lo, b0, b1);
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
  // the tensor-core operand: 8 channels (16 bytes) a thread
  if (OWN || block0 >= 0)
    for (int i = tid; i < PL * kPrepQ * (D / 8); i += 256) {
      const int r = i % kPrepQ, c = i / kPrepQ % (D / 8), pl = i / (D / 8 * kPrepQ);
      const float up = up_s[r][2];
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int ch = k_channel<D>(4 * c + j, pl != 0);
        const float x0 = pl ? r_s[NRES ? r : 0][ch] : __bfloat162float(q_s[r][ch]);
        const float x1 = pl ? r_s[NRES ? r : 0][ch + 8] : __bfloat162float(q_s[r][ch + 4]);
        w[j] = f16x2(x0 * up, x1 * up);
      }
      img_s[pl * (D / 8) + c][r] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  if (!OWN) {
    // decode packs: a warp per query's header (scales, the groups' sums) ...
    for (int r = warp; r < kPrepQ; r += 8) {
      uint32_t* pack = out_s + r * WORDS;
      pack[lane] = 0u;                               // kPackHeader = 32
      __syncwarp();
#pragma unroll
      for (int p = 0; p < PL; ++p) {
        float s = 0.f, mx = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int ch = 4 * lane + i;
          const float x = ch < D ? (p ? r_s[NRES ? r : 0][ch] : __bfloat162float(q_s[r][ch])) * a.qscale : 0.f;
          s += x;
          mx = fmaxf(mx, fabsf(x));
        }
#pragma unroll
        for (int o = 1; o < GS / 4; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (4 * lane < D && lane % (GS / 4) == 0) pack[4 + p * NG + lane / (GS / 4)] = __float_as_uint(s);
#pragma unroll
        for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        int e = 0;
        (void)frexpf(mx, &e);                        // mx = f 2^e, f in [0.5, 1)
        const int k = mx > 0.f ? 15 - e : 0;
        if (lane == 0) {
          up_s[r][p] = ldexpf(1.f, k);
          pack[p] = __float_as_uint(ldexpf(1.f, 24 - k));   // sum(code x) = D 2^(24 - k)
        }
      }
    }
    __syncthreads();
    // ... then the images, a thread per (query, piece, lane, register), as qprep_kernel lays them out
    for (int i = tid; i < kPrepQ * 8 * NIMG; i += 256) {
      const int r = i / (8 * NIMG), w = i % (8 * NIMG), piece = w / (4 * NIMG), t = (w / NIMG) % 4, rho = w % NIMG;
      uint32_t v = 0u;
      int c0 = -1, c1 = 0, pl = 0;
      float sc = 1.f;
      if (rho < 2 * NMA) {                           // anchor: word rho / 4 of the lane, register k
        const int k = rho & 3, wd = t * C::WA + (rho >> 2);
        c0 = 8 * wd + k;
        c1 = c0 + 4;
        sc = (k & 1) ? 0.0625f : 1.f;
      } else if (t < C::TR) {                        // residual: word (rho - 2 NMA) / 8 of the lane, register 2m + hb
        const int k = rho - 2 * NMA, wd = 2 * t + (k >> 3), m = (k & 7) >> 1, hb = k & 1;
        c0 = 16 * wd + 4 * hb + m;
        c1 = c0 + 8;
        sc = m == 0 ? 1.f : (m == 1 ? 0.25f : (m == 2 ? 0.0625f : 0.015625f));
        pl = 1;
      }
      if (c0 >= 0) {
        const float f2 = up_s[r][pl] * sc;
        const float x0 = (pl ? r_s[NRES ? r : 0][c0] : __bfloat162float(q_s[r][c0])) * a.qscale;
        const float x1 = (pl ? r_s[NRES ? r : 0][c1] : __bfloat162float(q_s[r][c1])) * a.qscale;
        __half h0, l0, h1, l1;
        f16_pieces(x0 * f2, h0, l0);
        f16_pieces(x1 * f2, h1, l1);
        v = piece == 0 ? pack_f16x2(h0, h1) : pack_f16x2(l0, l1);
      }
      out_s[r * WORDS + kPackHeader + w] = v;
    }
  }
  __syncthreads();
  // 16 channels make a block of 32 bytes a query, swizzled by the query's place
  auto at = [](int row, int c, int nb) { return ((c >> 1) * nb + row) * 32 + (((c & 1) ^ ((row >> 2) & 1)) << 4); };
  if (block0 >= 0) {
    const int q0 = first % NB, unit = (block0 + first / NB) * a.g.H + h;
    uint8_t* img = a.packs + (size_t)unit * IMG;
    for (int i = tid; i < PL * (D / 8) * valid; i += 256) {
      const int r = i % valid, c = i / valid;
      *reinterpret_cast<uint4*>(img + at(q0 + r, c, NB)) = img_s[c][r];
    }
    // Places without a query keep what they hold: with the scale zero its scores are zero or NaN, which moves no
    // reference, and its weights stay in its own column.
    const int rows = first + kPrepQ >= queries ? NB - q0 : kPrepQ;
    if (tid < rows) a.scales[(size_t)unit * NB + q0 + tid] = tid < valid ? scale_s[tid] : 0.f;
  }
  if (OWN) {
    for (int x = tid; x < PL * (D / 8) * valid; x += 256) {
      const int r = x % valid, c = x / valid, i = first + r, unit = (row0 + i / a.g.qpk) * a.g.H + h;
      *reinterpret_cast<uint4*>(a.o_packs + (size_t)unit * OIMG + at(i % a.g.qpk, c, kOwnNB)) = img_s[c][r];
    }
    // a row's last query head also has the places behind it
    for (int x = tid; x < valid * kOwnNB; x += 256) {
      const int r = x / kOwnNB, k = x % kOwnNB, i = first + r, slot = i % a.g.qpk;
      if (k == slot || (slot + 1 == a.g.qpk && k > slot))
        a.o_scales[(size_t)((row0 + i / a.g.qpk) * a.g.H + h) * kOwnNB + k] = k == slot ? scale_s[r] : 0.f;
    }
  } else {
    static_assert(WORDS % 4 == 0 && kPackWords % 4 == 0, "16-byte pieces");
    for (int x = tid; x < valid * (WORDS / 4); x += 256) {
      const int i = first + x / (WORDS / 4);
      const size_t row = (size_t)(row0 + i / a.g.qpk) * a.g.Hq + h * a.g.qpk + i % a.g.qpk;
      reinterpret_cast<uint4*>(reinterpret_cast<uint32_t*>(a.o_packs) + row * kPackWords)[x % (WORDS / 4)] =
          reinterpret_cast<const uint4*>(out_s)[x];
    }
  }
}

// One CTA per MQ queries of a family and KV head: neighbours in the block, so that the shared tiles' partial states (four
// queries to 16 bytes) are read whole.  256 threads: a channel's anchor part below, its residual part above; a warp takes a
// query's (MQ = 16: two queries') score, maxima and weights.  R^T comes into shared memory by one bulk copy, ahead of
// the wait.  Dependents are not released early: a decode call, which reads its queries ahead of its wait, may take `out`
// for them.  A chain of latencies: states' references, weights, accumulators, R^T: 6.3 us behind the wait in the header's
// case (9 with addresses computed in its loops and R^T read from the L2 by each warp).
constexpr int kWeights = 32;              // states whose weights are held at a time
template <int D, int NRES, int NB, int MQ, bool OWN>
__global__ void __launch_bounds__(256, 2) prefix_merge_kernel(PrefixArgs a) {
  constexpr int HP = 132, NT = MQ / 8;
  extern __shared__ __align__(128) uint4 rt_s[];            // R^T's operand (dense rotations, residual loops)
  __shared__ __align__(16) float wp_s[kWeights][MQ];        // weights of the first partial states of the shared tiles
  __shared__ float wd_s[MQ][kWeights + 1];                  // and of the rows' own
  __shared__ __align__(16) float p_s[128][MQ];              // R^T's other operand [channel][query]
  __shared__ __align__(16) float h_s[MQ * HP];
  __shared__ float wn_s[MQ], l_s[MQ], top_s[MQ];
  __shared__ int row_s[MQ], n_s[MQ], share_s[MQ];
  __shared__ size_t own_s[MQ], out_s[MQ];                   // a query's first own state, its result
  __shared__ uint64_t r_bar;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, half = tid >> 7, ch = tid & 127;
  const int g = lane >> 2, t4 = lane & 3;
  const int m = blockIdx.x / a.g.H, h = blockIdx.x % a.g.H;
  const bool hadamard = (a.g.mode & RQ_MODE_HADAMARD) != 0, dense = NRES && !hadamard;
  const bool fits = plan_fits(a);
  const int4 rec = __ldg(reinterpret_cast<const int4*>(a.plan + a.l.merge) + 2 * m);
  const int4 work = __ldg(reinterpret_cast<const int4*>(a.plan + a.l.merge) + 2 * m + 1);
  const int row0 = rec.x, i0 = rec.y, nq = rec.z, block = max(rec.w, 0);
  if (!fits || row0 < 0) {
    if (!fits && tid == 0) a.status[3] = 1;
    pdl_wait();
    return;
  }
  if (dense && tid == 0) {
    mbar_init(&r_bar, 1);
    fence_mbar_init();
    mbar_arrive_expect_tx(&r_bar, image_words(D) * 4);
    bulk_g2s(rt_s, a.plan + a.l.rt_image, image_words(D) * 4, &r_bar);
  }
  if (tid < MQ) {
    const int i = i0 + min(tid, nq - 1), b = row0 + i / a.g.qpk, hq = h * a.g.qpk + i % a.g.qpk;
    const int4 row = __ldg(reinterpret_cast<const int4*>(a.plan + a.l.row) + b);   // length, shared tiles, rest, units before
    row_s[tid] = b;
    out_s[tid] = ((size_t)b * a.g.Hq + hq) * D;
    share_s[tid] = row.y;
    if (clamp_len(__ldg(a.seq_lens + b), a.g.Nmax) != row.x) a.status[3] = 1;      // the plan is of other lengths
    // the CTAs that hold the units of the row's own tiles
    const int nt = (row.z + 2 * kTile - 1) / (2 * kTile);
    int from = 0, n = 0;
    if (nt > 0) {
      const Split split{work.w / a.o_ctas, work.w % a.o_ctas};
      const int s0 = row.w + (OWN ? h : hq / a.qh) * nt;
      from = split.owner(s0);
      n = split.owner(s0 + nt - 1) - from + 1;
    }
    n_s[tid] = n;
    own_s[tid] = OWN ? (size_t)(from + b * a.g.H + h) * a.o_pstride + i % a.g.qpk
                     : ((size_t)(from + b * (a.g.Hq / a.qh) + hq / a.qh) * a.qh + hq % a.qh) * a.o_pstride;
  }
  // the tensor-core CTAs that hold this block's steps
  int c_lo = 0, n_c = 0;
  const int qo = i0 % NB;
  if (rec.w >= 0) {
    const TreeSplit split{work.z / a.ctas, work.z % a.ctas};
    const int s0 = work.y + h * work.x;
    c_lo = split.owner(s0);
    n_c = split.owner(s0 + work.x - 1) - c_lo + 1;
  }
  __syncthreads();
  // warp w: the scores of queries w, w + 8 with the current token
  float now[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int row = row_s[warp + 8 * n];
    now[n] = 0.f;
    if (lane < D / 4) {
      const uint2 x = __ldg(reinterpret_cast<const uint2*>(a.q + out_s[warp + 8 * n]) + lane);
      const uint2 y = __ldg(reinterpret_cast<const uint2*>(a.k_cur + ((size_t)row * a.g.H + h) * D) + lane);
      now[n] = bf16_bits_to_f32(x.x & 0xFFFF) * bf16_bits_to_f32(y.x & 0xFFFF) +
               bf16_bits_to_f32(x.x >> 16) * bf16_bits_to_f32(y.x >> 16) +
               bf16_bits_to_f32(x.y & 0xFFFF) * bf16_bits_to_f32(y.y & 0xFFFF) +
               bf16_bits_to_f32(x.y >> 16) * bf16_bits_to_f32(y.y >> 16);
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int o = 16; o; o >>= 1) now[n] += __shfl_xor_sync(0xffffffffu, now[n], o);
    now[n] *= a.qscale;
  }
  float o[MQ];                                   // this thread's channel: the current token's value (lower half)
#pragma unroll
  for (int i = 0; i < MQ; ++i)
    o[i] = !half && ch < D ? __bfloat162float(__ldg(a.v_cur + ((size_t)row_s[i] * a.g.H + h) * D + ch)) : 0.f;
  // a query's first state of its own row's tiles: reference, sum (O_SUM further) and, this thread's, accumulator (from
  // O_ACC; OWN: four query heads to 16 bytes), and from one CTA to the next
  const size_t o_step = OWN ? (size_t)a.o_pstride : (size_t)a.qh * a.o_pstride;
  constexpr int O_SUM = OWN ? kOwnNB : 1, O_ACC = OWN ? 2 * kOwnNB : 2;
  const int o_at = O_ACC + (OWN ? half * kOwnNB * D + ch * 4 : half * D + ch);

  pdl_wait();
  // the first accumulators are on their way while the weights are made
  const bool mine = ch < D && (NRES || !half);
  constexpr int PF = MQ == 8 ? 4 : 2;
  float4 ahead[PF][MQ / 4];
  const float4* x0 = reinterpret_cast<const float4*>(a.partials + (size_t)(c_lo + block * a.g.H + h) * a.pstride + 2 * NB) +
                     (size_t)(half * (NB / 4) + qo / 4) * D + ch;
#pragma unroll
  for (int c = 0; c < PF; ++c)
#pragma unroll
    for (int i = 0; i < MQ / 4; ++i)
      ahead[c][i] = mine && c < n_c ? __ldcg(x0 + (size_t)c * (a.pstride / 4) + i * D) : make_float4(0.f, 0.f, 0.f, 0.f);
  // weights, relative to the largest reference of the query's states and the current token
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int qi = warp + 8 * n, nd = n_s[qi];
    const bool sharing = share_s[qi] > 0;
    const float *pp = a.partials + (size_t)(c_lo + block * a.g.H + h) * a.pstride + qo + qi, *dp = a.o_partials + own_s[qi];
    float top = now[n], sum = 0.f;
    // the first of each kind, one a lane
    const float mp = sharing && lane < n_c ? __ldcg(pp + (size_t)lane * a.pstride) : -INFINITY;
    const float lp = sharing && lane < n_c ? __ldcg(pp + (size_t)lane * a.pstride + NB) : 0.f;
    const float md = lane < nd ? __ldcg(dp + lane * o_step) : -INFINITY;
    const float ld = lane < nd ? __ldcg(dp + lane * o_step + O_SUM) : 0.f;
    top = fmaxf(top, fmaxf(mp, md));
    for (int c = lane + kWeights; c < n_c; c += 32) top = sharing ? fmaxf(top, __ldcg(pp + (size_t)c * a.pstride)) : top;
    for (int c = lane + kWeights; c < nd; c += 32) top = fmaxf(top, __ldcg(dp + c * o_step));
#pragma unroll
    for (int s = 16; s; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
    if (top == -INFINITY) top = 0.f;
    auto weight = [&](float x) { return x == -INFINITY ? 0.f : exp2f(x - top); };
    if (lane < n_c) wp_s[lane][qi] = weight(mp);
    if (lane < nd) wd_s[qi][lane] = weight(md);
    sum = fmaf(weight(mp), lp, weight(md) * ld);
    if (sharing)
      for (int c = lane + kWeights; c < n_c; c += 32)
        sum = fmaf(weight(__ldcg(pp + (size_t)c * a.pstride)), __ldcg(pp + (size_t)c * a.pstride + NB), sum);
    for (int c = lane + kWeights; c < nd; c += 32) sum = fmaf(weight(__ldcg(dp + c * o_step)), __ldcg(dp + c * o_step + O_SUM), sum);
#pragma unroll
    for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
    if (lane == 0) {
      const float w = exp2f(now[n] - top);
      wn_s[qi] = w;
      l_s[qi] = sum + w;
      top_s[qi] = top;
    }
  }
  __syncthreads();
  float oc[MQ];                                  // this thread's plane of the cached tokens
#pragma unroll
  for (int i = 0; i < MQ; ++i) oc[i] = 0.f;
  // the operands' powers of two: V's anchor under a coefficient 2^-7, else 2^-15
  const float up = NRES && !half ? 128.f : 32768.f;
  if (mine) {
    auto add = [&](const float4* wp, const float4 (&x)[MQ / 4]) {
#pragma unroll
      for (int i = 0; i < MQ / 4; ++i) {
        const float4 w = wp[i];
        oc[4 * i] = fmaf(w.x, x[i].x, oc[4 * i]);
        oc[4 * i + 1] = fmaf(w.y, x[i].y, oc[4 * i + 1]);
        oc[4 * i + 2] = fmaf(w.z, x[i].z, oc[4 * i + 2]);
        oc[4 * i + 3] = fmaf(w.w, x[i].w, oc[4 * i + 3]);
      }
    };
    auto weights = [&](int c) { return reinterpret_cast<const float4*>(wp_s[c]); };
#pragma unroll
    for (int c = 0; c < PF; ++c)
      if (c < n_c) add(weights(c), ahead[c]);
#pragma unroll 4
    for (int c = PF; c < min(n_c, kWeights); ++c) {
      float4 x[MQ / 4];
#pragma unroll
      for (int i = 0; i < MQ / 4; ++i) x[i] = __ldcg(x0 + (size_t)c * (a.pstride / 4) + i * D);
      add(weights(c), x);
    }
  }
  // the shared tiles' further states, a chunk at a time
  for (int c0 = kWeights; c0 < n_c; c0 += kWeights) {
    const int n = min(kWeights, n_c - c0);
    __syncthreads();
    for (int i = tid; i < n * MQ; i += 256) {
      const int c = i / MQ, qi = i % MQ;
      const float x = __ldcg(a.partials + (size_t)(c_lo + c0 + c + block * a.g.H + h) * a.pstride + qo + qi);
      wp_s[c][qi] = share_s[qi] > 0 ? exp2f(x - top_s[qi]) : 0.f;
    }
    __syncthreads();
    if (mine)
#pragma unroll 4
      for (int c = 0; c < n; ++c) {
        float4 x[MQ / 4];
#pragma unroll
        for (int i = 0; i < MQ / 4; ++i) x[i] = __ldcg(x0 + (size_t)(c0 + c) * (a.pstride / 4) + i * D);
        const float4* wp = reinterpret_cast<const float4*>(wp_s[c]);
#pragma unroll
        for (int i = 0; i < MQ / 4; ++i) {
          oc[4 * i] = fmaf(wp[i].x, x[i].x, oc[4 * i]);
          oc[4 * i + 1] = fmaf(wp[i].y, x[i].y, oc[4 * i + 1]);
          oc[4 * i + 2] = fmaf(wp[i].z, x[i].z, oc[4 * i + 2]);
          oc[4 * i + 3] = fmaf(wp[i].w, x[i].w, oc[4 * i + 3]);
        }
      }
  }
  int most = 0;
#pragma unroll
  for (int i = 0; i < MQ; ++i) {
    if (!OWN) oc[i] *= up;
    most = max(most, n_s[i]);
  }
  for (int c0 = 0; c0 < most; c0 += kWeights) {
    if (c0) {
      __syncthreads();
      for (int i = tid; i < kWeights * MQ; i += 256) {
        const int c = i % kWeights, qi = i / kWeights;
        if (c0 + c < n_s[qi]) wd_s[qi][c] = exp2f(__ldcg(a.o_partials + own_s[qi] + (c0 + c) * o_step) - top_s[qi]);
      }
      __syncthreads();
    }
    if (mine) {
      const float* st[MQ];
      int left[MQ];
#pragma unroll
      for (int i = 0; i < MQ; ++i) {
        const int slot = OWN ? (i0 + min(i, nq - 1)) % a.g.qpk : 0;
        st[i] = a.o_partials + own_s[i] + (OWN ? (slot / 4) * (4 * D) + slot % 4 - slot : 0) + c0 * o_step + o_at;
        left[i] = n_s[i] - c0;
      }
#pragma unroll 2
      for (int c = 0; c < min(kWeights, most - c0); ++c) {
        float x[MQ];
#pragma unroll
        for (int i = 0; i < MQ; ++i) x[i] = c < left[i] ? __ldcg(st[i] + c * o_step) : 0.f;
#pragma unroll
        for (int i = 0; i < MQ; ++i) oc[i] = fmaf(c < left[i] ? wd_s[i][c] : 0.f, x[i], oc[i]);
      }
    }
  }
  if (OWN)
#pragma unroll
    for (int i = 0; i < MQ; ++i) oc[i] *= up;
  if (NRES && half) {
#pragma unroll
    for (int i = 0; i < MQ; ++i) p_s[ch][i] = oc[i];
  } else {
#pragma unroll
    for (int i = 0; i < MQ; ++i) o[i] = fmaf(o[i], wn_s[i], oc[i]);
  }
  if (dense) {
    const bool ok = mbar_wait_bounded(&r_bar, 0);
    if (__syncthreads_or(!ok)) {
      if (tid == 0) a.status[0] = 1;
      return;
    }
  } else {
    __syncthreads();
  }
  if (NRES && hadamard) {
    float t[MQ];
#pragma unroll
    for (int i = 0; i < MQ; ++i) t[i] = half ? 0.f : p_s[ch][i];
    __syncthreads();
    hadamard128<MQ>(t, tid, h_s);                // threads >= 128 only take part in its barriers
    __syncthreads();
    if (!half) {
#pragma unroll
      for (int i = 0; i < MQ; ++i) o[i] += t[i];
    }
  }
  if (dense) {
    if (warp < D / 16) {
      float d[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) d[n][0] = d[n][1] = d[n][2] = d[n][3] = 0.f;
      const uint4* rp = rt_s + (warp * (D / 16) * 32 + lane) * 2;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint4 x = rp[k * 64], y = rp[k * 64 + 1];
        const uint32_t hi[4] = {x.x, x.y, x.z, x.w}, lo[4] = {y.x, y.y, y.z, y.w};
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
        float* y = h_s + (8 * n + 2 * t4) * HP + 16 * warp + g;
        y[0] = d[n][0];
        y[HP] = d[n][1];
        y[8] = d[n][2];
        y[HP + 8] = d[n][3];
      }
    }
    __syncthreads();
  }
  if (!half && ch < D) {
#pragma unroll
    for (int i = 0; i < MQ; ++i)
      if (i < nq)
        a.out[out_s[i] + ch] =
            __float2bfloat16_rn((o[i] + (dense ? h_s[i * HP + ch] : 0.f)) / l_s[i]);
  }
}

template <int D, int GS, int NRES, int NB, bool OWN>
cudaError_t launch_prep(const PrefixArgs& a, cudaStream_t stream) {
  return launch_dependent(prefix_prep_kernel<D, GS, NRES, NB, OWN>, dim3((unsigned)(a.l.max_preps * a.g.H)), dim3(256), 0,
                          stream, a);
}
template <int D, int NRES, int NB, int MQ, bool OWN>
cudaError_t launch_merge(const PrefixArgs& a, cudaStream_t stream) {
  auto* kern = prefix_merge_kernel<D, NRES, NB, MQ, OWN>;
  constexpr int kSmem = NRES ? image_words(D) * 4 : 0;
  static std::atomic<int> ready[kMaxDevices];   // shared-memory limit set on this device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (e != cudaSuccess) return e;
    ready[dev].store(1, std::memory_order_release);
  }
  const size_t smem = a.g.mode & RQ_MODE_HADAMARD ? 0 : kSmem;
  return launch_dependent(kern, dim3((unsigned)(a.l.max_merges * a.g.H)), dim3(256), smem, stream, a);
}

template <int D, int NRES, int NB, bool OWN>
cudaError_t launch_prefix_t(PrefixArgs a, const TreeArgs& t, const TreeArgs& own, const DecodeArgs& d, int num_sms,
                            cudaStream_t stream) {
  auto tree = [&](const TreeArgs& x, int nb) {
    return D == 128 ? launch_tree_mma(x, nb, num_sms, stream, true) : launch_tree_mma_96(x, nb, num_sms, stream, true);
  };
  a.pstride = 2 * NB + (1 + NRES) * NB * D;      // the tensor-core kernel's
  cudaError_t e = a.g.g == 32 ? launch_prep<D, 32, NRES, NB, OWN>(a, stream) : launch_prep<D, 16, NRES, NB, OWN>(a, stream);
  if (e != cudaSuccess) return e;
  e = tree(t, NB);
  if (e != cudaSuccess) return e;
  if (OWN) {
    a.o_pstride = 2 * kOwnNB + (1 + NRES) * kOwnNB * D;
    a.o_ctas = num_sms;
    e = tree(own, kOwnNB);
  } else {
    e = launch_decode_stream(d, num_sms, NRES, stream, &a.o_ctas);
  }
  if (e != cudaSuccess) return e;
  return a.l.mq == 8 ? launch_merge<D, NRES, NB, 8, OWN>(a, stream) : launch_merge<D, NRES, NB, 16, OWN>(a, stream);
}
template <int D, int NRES, bool OWN>
cudaError_t launch_prefix_nb(const PrefixArgs& a, const TreeArgs& t, const TreeArgs& own, const DecodeArgs& d, int num_sms,
                             cudaStream_t stream) {
  if (a.l.nb == 16) return launch_prefix_t<D, NRES, 16, OWN>(a, t, own, d, num_sms, stream);
  if (a.l.nb == 32) return launch_prefix_t<D, NRES, 32, OWN>(a, t, own, d, num_sms, stream);
  return launch_prefix_t<D, NRES, 64, OWN>(a, t, own, d, num_sms, stream);
}
template <int D, int NRES>
cudaError_t launch_prefix_own(const PrefixArgs& a, const TreeArgs& t, const TreeArgs& own, const DecodeArgs& d, int num_sms,
                              cudaStream_t stream) {
  return own_tree(a.g) ? launch_prefix_nb<D, NRES, true>(a, t, own, d, num_sms, stream)
                       : launch_prefix_nb<D, NRES, false>(a, t, own, d, num_sms, stream);
}

struct PrefixSpace {
  size_t partials, scales, packs, o_partials, o_scales, o_packs, total;   // byte offsets
};
PrefixSpace prefix_space(const Geom& g, const PlanLayout& l, int num_sms) {
  PrefixSpace s;
  size_t at = 256;
  auto take = [&](size_t bytes) {
    const size_t p = at;
    at += (bytes + 255) / 256 * 256;
    return p;
  };
  const size_t planes = g.P > 1 ? 2 : 1;
  auto states = [&](size_t units, size_t nb) { return (units + num_sms) * (2 * nb + planes * nb * g.d) * sizeof(float); };
  const size_t units = (size_t)l.max_blocks * g.H, rows = (size_t)l.batch * g.H;
  s.partials = take(states(units, l.nb));
  s.scales = take(units * l.nb * sizeof(float));
  s.packs = take(units * planes * 2 * l.nb * g.d);
  if (own_tree(g)) {
    s.o_partials = take(states(rows, kOwnNB));
    s.o_scales = take(rows * kOwnNB * sizeof(float));
    s.o_packs = take(rows * planes * 2 * kOwnNB * g.d);
  } else {
    s.o_partials = take(decode_partials(g, l.batch, num_sms).bytes);
    s.o_scales = at;
    s.o_packs = take((size_t)l.batch * g.Hq * kPackWords * sizeof(uint32_t));
  }
  s.total = at;
  return s;
}

}  // namespace

size_t prefix_plan_bytes(const Geom& g, int batch, int n) { return plan_layout(g, batch, n).words * sizeof(int32_t); }

size_t prefix_workspace_bytes(const Geom& g, int batch, int n, int num_sms) {
  return prefix_space(g, plan_layout(g, batch, n), num_sms).total;
}

// Whether a call's steps and CTAs stay within int32.
static bool prefix_fits(const Geom& g, const PlanLayout& l) {
  const int64_t most = 0x7fffffff, units = ((int64_t)g.Nmax + 2 * kTile - 1) / (2 * kTile);
  return l.words <= (size_t)most && (int64_t)l.max_blocks * g.H * units <= most && (int64_t)l.batch * g.Hq * units <= most &&
         (int64_t)l.max_merges * g.H <= most && (int64_t)l.max_preps * g.H <= most;
}

cudaError_t launch_prefix_plan(const rq_cache& c, int batch, int n, const int32_t* starts, const int32_t* seq_lens,
                               void* plan, cudaStream_t stream) {
  PlanArgs a = {};
  a.g = c.geom;
  a.l = plan_layout(c.geom, batch, n);
  if (!prefix_fits(c.geom, a.l)) return cudaErrorNotSupported;
  a.starts = starts;
  a.seq_lens = seq_lens;
  a.plan = static_cast<int32_t*>(plan);
  a.R = c.R;
  a.per_unit = own_tree(c.geom) ? c.geom.H : c.geom.Hq / decode_partials(c.geom, batch, c.num_sms).qh;
  const int images = c.geom.mode & RQ_MODE_HADAMARD ? 0 : 2 * (c.geom.d / 16);
  plan_rows_kernel<<<batch, kPlanThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = launch_dependent(plan_families_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a);
  if (e == cudaSuccess)   // releases its dependents only when it ends: what follows finds the plan complete
    e = launch_dependent(plan_tables_kernel, dim3(batch + a.l.max_blocks + images), dim3(kPlanThreads), 0, stream, a);
  return e;
}

cudaError_t launch_prefix(const rq_cache& c, int layer, int group, int loop, int batch, int n, const void* plan,
                          const __nv_bfloat16* q, const __nv_bfloat16* k_cur, const __nv_bfloat16* v_cur,
                          const int32_t* seq_lens, float scale, __nv_bfloat16* out, void* workspace,
                          cudaStream_t stream) {
  const Geom& g = c.geom;
  const PlanLayout l = plan_layout(g, batch, n);
  if (!prefix_fits(g, l)) return cudaErrorNotSupported;
  const PrefixSpace s = prefix_space(g, l, c.num_sms);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const int nres = loop == g.P - 1 ? 0 : 1;
  const DecodePartials dp = decode_partials(g, batch, c.num_sms);
  PrefixArgs a = {};
  a.g = g;
  a.l = l;
  a.plan = static_cast<const int32_t*>(plan);
  a.R = c.R;
  a.q = q;
  a.k_cur = k_cur;
  a.v_cur = v_cur;
  a.seq_lens = seq_lens;
  a.out = out;
  a.status = reinterpret_cast<int32_t*>(ws);
  a.qscale = scale * kLog2e;
  a.packs = ws + s.packs;
  a.scales = reinterpret_cast<float*>(ws + s.scales);
  a.partials = reinterpret_cast<float*>(ws + s.partials);
  a.ctas = c.num_sms;
  a.o_packs = ws + s.o_packs;
  a.o_scales = reinterpret_cast<float*>(ws + s.o_scales);
  a.o_partials = reinterpret_cast<float*>(ws + s.o_partials);
  a.o_pstride = dp.pstride;
  a.qh = dp.qh;
  // the shared tiles: blocks of queries as rows
  TreeArgs t = {};
  t.g = g;
  t.g.table = a.plan + l.block_table;
  t.g.max_tiles = l.ntiles;
  t.base = c.base;
  t.R = c.R;
  t.seq_lens = a.plan + l.b_len;
  t.status = a.status;
  t.layer = layer;
  t.group = group;
  t.batch = l.max_blocks;
  t.loop = loop;
  t.nres = nres;
  t.qscale = a.qscale;
  t.nqb = 1;
  t.M = t.T = l.nb;
  t.partials = a.partials;
  t.packs = a.packs;
  t.q_scale = a.scales;
  // the rows' own tiles
  TreeArgs own = t;
  own.g.table = a.plan + l.rest_table;
  own.seq_lens = a.plan + l.rest;
  own.batch = batch;
  own.M = own.T = g.qpk;
  own.partials = a.o_partials;
  own.packs = a.o_packs;
  own.q_scale = a.o_scales;
  DecodeArgs d = {};
  d.g = own.g;
  d.base = c.base;
  d.R = c.R;
  d.q = q;
  d.seq_lens = own.seq_lens;
  d.status = a.status;
  d.partials = a.o_partials;
  d.packs = reinterpret_cast<uint32_t*>(a.o_packs);
  d.pstride = dp.pstride;
  d.layer = layer;
  d.group = group;
  d.batch = batch;
  d.res0 = loop;
  d.qh = dp.qh;
  d.qscale = a.qscale;
  if (g.d == 128)
    return nres ? launch_prefix_own<128, 1>(a, t, own, d, c.num_sms, stream)
                : launch_prefix_own<128, 0>(a, t, own, d, c.num_sms, stream);
  return nres ? launch_prefix_own<96, 1>(a, t, own, d, c.num_sms, stream)
              : launch_prefix_own<96, 0>(a, t, own, d, c.num_sms, stream);
}

}  // namespace rq
