// Page bookkeeping of a paged cache: rq_pages_copy, _fork, _reserve, _free, _compact.
//
// The state is the cache's block table and refs[page] = number of table entries
// that name the page (0: free).  Everything runs on the device in stream order:
// a short planning kernel decides (deterministically: lowest page, row order)
// which pages move, then a copy kernel moves their bytes.  A page spans every
// layer and group: L * G blocks of page_bytes, num_pages * page_bytes apart.
//
// Planning is one CTA's latency (5 to 7 us for 32 rows or 256 pages), copying is bound by memory: 24
// pages of 9.7 MB copied on write 68 us with the plan (467 MB read and written, 6.9 TB/s, a page that several rows
// share being read from L2); 5 listed pages 57 us (338 MB, 5.9 TB/s); 50 pages packed to the front 166 us
// (973 MB, 5.9 TB/s).
#include "rq_internal.cuh"

namespace rq {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kCopyThreads = 512;
constexpr int kCopyCtasPerSm = 4;
constexpr int kForkCols = 32;
constexpr int kMaxForkPairs = 6144;

__device__ __forceinline__ void flag(int32_t* status, int word) {
  if (status) atomicExch(&status[word], 1);
}
__device__ __forceinline__ bool in_pool(int p, int num_pages) { return p >= 0 && p < num_pages; }

// Exclusive prefix sum over the CTA (kPlanThreads threads); *total: the sum.
// Every thread of the CTA calls it.
__device__ __forceinline__ int block_scan(int v, int* total) {
  __shared__ int warp_s[kPlanThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();   // a previous call's readers of warp_s
  if (lane == 31) warp_s[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = warp_s[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    warp_s[lane] = w;
  }
  __syncthreads();
  *total = warp_s[kPlanThreads / 32 - 1];
  return x - v + (warp ? warp_s[warp - 1] : 0);
}

// ---- moving bytes --------------------------------------------------------------

struct CopyArgs {
  uint8_t* base;
  int64_t page_bytes;
  int num_pages, planes;          // planes: L * G
  const int32_t *src, *dst;       // pairs; src < 0: nothing to copy
  const int32_t* count;           // device count of pairs, or NULL: n
  int n;
  int check;                      // caller's list: skip pairs that collide
  int32_t* status;
  // compaction: table entries follow the moved pages
  int32_t* table;
  int64_t entries;
  const int32_t* map;
};

// Pair i of a caller's list may be copied: its pages exist, its target is no
// other pair's source and no earlier pair's target.
__device__ bool pair_ok(const CopyArgs& a, int n, int i) {
  const int s = a.src[i], t = a.dst[i];
  bool bad = !in_pool(s, a.num_pages) || !in_pool(t, a.num_pages);
  for (int j = threadIdx.x; j < n; j += blockDim.x)
    if (j != i && (a.src[j] == t || (j < i && a.dst[j] == t))) bad = true;
  return !__syncthreads_or(bad);
}

// The (pair, plane) blocks, cut into pieces of kPiece bytes, in one row; CTA c
// takes a contiguous share, so that it walks along few pages.  Four loads in flight a thread; at 45 registers two of
// the grid's four CTAs an SM run at a time, 1024 threads.  256 threads with eight loads take 72, 58 and 169 us in
// the three cases above; two loads 82, 64 and 182.
constexpr int kUnroll = 4;
constexpr int kPiece = kCopyThreads * kUnroll * 16;

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(CopyArgs a) {
  const int n = a.count ? *a.count : a.n;
  if (a.table) {
    for (int64_t i = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x; i < a.entries;
         i += (int64_t)gridDim.x * kCopyThreads) {
      const int e = a.table[i];
      if (in_pool(e, a.num_pages) && a.map[e] != e) a.table[i] = a.map[e];
    }
  }
  const int64_t per = (a.page_bytes + kPiece - 1) / kPiece;
  const int64_t items = per * a.planes * n;
  const int64_t q = items / gridDim.x, rem = items % gridDim.x, c = blockIdx.x;
  int64_t i0 = c * q + (c < rem ? c : rem);
  const int64_t i1 = i0 + q + (c < rem ? 1 : 0);
  int known = -1;
  bool ok = true;
  for (; i0 < i1; ++i0) {
    const int pair = (int)(i0 / (per * a.planes));
    const int64_t in_pair = i0 % (per * a.planes);
    if (a.check && pair != known) {
      ok = pair_ok(a, n, pair);
      known = pair;
      if (!ok && threadIdx.x == 0) flag(a.status, 2);
    }
    const int s = a.src[pair], t = a.dst[pair];
    if (!ok || s < 0 || s == t) continue;
    const int64_t plane = in_pair / per, at = (in_pair % per) * kPiece;
    const uint8_t* from = a.base + (plane * a.num_pages + s) * a.page_bytes + at;
    uint8_t* to = a.base + (plane * a.num_pages + t) * a.page_bytes + at;
    const int64_t left = a.page_bytes - at;
    uint4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int off = (u * kCopyThreads + threadIdx.x) * 16;
      if (off < left) v[u] = __ldcs(reinterpret_cast<const uint4*>(from + off));
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int off = (u * kCopyThreads + threadIdx.x) * 16;
      if (off < left) __stcs(reinterpret_cast<uint4*>(to + off), v[u]);
    }
  }
}

cudaError_t launch_copy(const CopyArgs& a, int num_sms, cudaStream_t stream) {
  copy_kernel<<<num_sms * kCopyCtasPerSm, kCopyThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

// ---- fork ------------------------------------------------------------------------
// Columns of the table are independent: a CTA loads its columns of every pair's
// two rows, then writes.  A later pair with the same target wins.  Latency: 11 us at 64 pairs of 256 tiles.
struct ForkArgs {
  int32_t* table;
  int max_tiles, rows, num_pages, n, cols;
  const int32_t *src, *dst;
  int32_t *refs, *status;
};

__global__ void __launch_bounds__(1024) fork_kernel(ForkArgs a) {
  extern __shared__ int32_t fresh_s[];          // [n][cols]: the sources' entries
  int32_t* take_s = fresh_s + (size_t)a.n * a.cols;   // [n]: the pair applies
  const int c0 = blockIdx.x * a.cols;
  for (int i = threadIdx.x; i < a.n; i += blockDim.x) {
    const int s = a.src[i], t = a.dst[i];
    bool ok = s >= 0 && s < a.rows && t >= 0 && t < a.rows;
    if (!ok && blockIdx.x == 0) flag(a.status, 1);
    for (int j = i + 1; ok && j < a.n; ++j)     // a later valid pair takes this target
      if (a.dst[j] == t && a.src[j] >= 0 && a.src[j] < a.rows) ok = false;
    take_s[i] = ok;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.n * a.cols; e += blockDim.x) {
    const int i = e / a.cols, col = c0 + e % a.cols;
    if (take_s[i] && col < a.max_tiles) fresh_s[e] = a.table[(size_t)a.src[i] * a.max_tiles + col];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.n * a.cols; e += blockDim.x) {
    const int i = e / a.cols, col = c0 + e % a.cols;
    if (!take_s[i] || col >= a.max_tiles) continue;
    int32_t* at = a.table + (size_t)a.dst[i] * a.max_tiles + col;
    const int old = *at, now = fresh_s[e];
    if (old == now) continue;
    *at = now;
    if (in_pool(now, a.num_pages)) atomicAdd(&a.refs[now], 1);
    if (in_pool(old, a.num_pages)) atomicSub(&a.refs[old], 1);
  }
}

// ---- free ------------------------------------------------------------------------
__global__ void __launch_bounds__(256) free_kernel(int32_t* table, int max_tiles, int rows, int num_pages, int n,
                                                   const int32_t* which, const int32_t* keep, int32_t* refs,
                                                   int32_t* status) {
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < (int64_t)n * max_tiles;
       e += (int64_t)gridDim.x * 256) {
    const int i = (int)(e / max_tiles), col = (int)(e % max_tiles), r = which[i];
    if (r < 0 || r >= rows) {
      if (col == 0) flag(status, 1);
      continue;
    }
    const int k = keep ? max(keep[i], 0) : 0;
    if (col < k / kTile + (k % kTile != 0)) continue;
    const int old = atomicExch(&table[(size_t)r * max_tiles + col], -1);   // once, if a row is named twice
    if (in_pool(old, num_pages)) atomicSub(&refs[old], 1);
  }
}

// ---- reserve ----------------------------------------------------------------------
// Workspace (int32): count[4] | asks[num_pages] | last[num_pages] | free[num_pages] |
// src[num_pages] | dst[num_pages] | map[num_pages].  At most num_pages requests can
// be served, so the lists hold num_pages pairs.
struct PlanArgs {
  int32_t* table;
  int max_tiles, num_pages, nmax, batch, n_tokens;
  const int32_t* seq_lens;
  int32_t *refs, *status, *count, *asks, *last, *free, *src, *dst;
  int32_t *map, *used;            // compaction
};

// First table entry and number of entries of row b's request; 0 when skipped.
__device__ __forceinline__ int row_tiles(const PlanArgs& a, int b, int* t0, int* len) {
  const int n = a.seq_lens[b];
  *len = n;
  if (n < 0 || n > a.nmax - a.n_tokens) return 0;
  *t0 = n / kTile;
  return (n + a.n_tokens - 1) / kTile - n / kTile + 1;
}

__global__ void __launch_bounds__(kPlanThreads) reserve_kernel(PlanArgs a) {
  const int tid = threadIdx.x;
  const int width = (a.n_tokens + kTile - 2) / kTile + 1;   // entries a row can ask for
  const int64_t slots = (int64_t)a.batch * width;
  // the entry of slot s: false when there is none
  auto entry_of = [&](int64_t s, int32_t** at, bool* holds) {
    const int b = (int)(s / width), k = (int)(s % width);
    int t0 = 0, len = 0;
    const int cnt = row_tiles(a, b, &t0, &len);
    if (cnt == 0 && k == 0) flag(a.status, 1);
    if (k >= cnt) return false;
    *at = a.table + (size_t)b * a.max_tiles + t0 + k;
    *holds = k == 0 && len % kTile != 0;                    // the tile holds tokens of the row
    return true;
  };
  int32_t* at = nullptr;
  bool holds = false;
  // how often each shared page is asked for, and by which slot last
  for (int64_t s = tid; s < slots; s += kPlanThreads)
    if (entry_of(s, &at, &holds) && in_pool(*at, a.num_pages)) { a.asks[*at] = 0; a.last[*at] = -1; }
  __syncthreads();
  for (int64_t s = tid; s < slots; s += kPlanThreads)
    if (entry_of(s, &at, &holds) && in_pool(*at, a.num_pages)) {
      atomicAdd(&a.asks[*at], 1);
      atomicMax(&a.last[*at], (int)s);
    }
  __syncthreads();
  // the free pages, ascending: each warp lists its share of the pool
  const int lane = tid & 31, warp = tid >> 5;
  const int share = ((a.num_pages + 31) / 32 + 31) / 32 * 32;   // pages a warp, a multiple of 32
  const int p0 = min(warp * share, a.num_pages), p1 = min(p0 + share, a.num_pages);
  int mine = 0;
  for (int p = p0 + lane; p < p1; p += 32) mine += a.refs[p] <= 0;
  int nfree;
  const int before = block_scan(mine, &nfree);
  int at_free = __shfl_sync(0xffffffffu, before, 0);             // free pages before the warp's share
  for (int p = p0; p < p1; p += 32) {
    const bool is = p + lane < p1 && a.refs[p + lane] <= 0;
    const unsigned m = __ballot_sync(0xffffffffu, is);
    if (is) a.free[at_free + __popc(m & ((1u << lane) - 1u))] = p + lane;
    at_free += __popc(m);
  }
  __syncthreads();
  // requests in slot order take the free pages in order
  int served = 0;
  for (int64_t s0 = 0; s0 < slots; s0 += kPlanThreads) {
    const int64_t s = s0 + tid;
    bool want = false, shared = false, copy = false;
    int old = -1;
    if (s < slots && entry_of(s, &at, &holds)) {
      old = *at;
      const bool page = in_pool(old, a.num_pages);
      // every holder of a page asks: the last one keeps it
      shared = page && a.refs[old] > 1 &&
               !(__ldcg(&a.asks[old]) >= a.refs[old] && __ldcg(&a.last[old]) == (int)s);
      want = !page || shared;
      copy = shared && holds;
    }
    int total;
    const int k = served + block_scan(want ? 1 : 0, &total);   // barriers: every read of refs is done
    if (want) {
      if (k < nfree) {
        const int p = a.free[k];
        a.src[k] = copy ? old : -1;
        a.dst[k] = p;
        a.free[k] = shared ? old : -1;   // the page that loses a holder
        *at = p;
      } else {
        flag(a.status, 3);
      }
    }
    served += total;
  }
  __syncthreads();
  served = min(served, nfree);
  for (int k = tid; k < served; k += kPlanThreads) {   // the counts, once nothing reads them any more
    a.refs[a.dst[k]] = 1;
    if (a.free[k] >= 0) atomicSub(&a.refs[a.free[k]], 1);
  }
  if (tid == 0) a.count[0] = served;
}

// ---- compact ----------------------------------------------------------------------
__global__ void __launch_bounds__(kPlanThreads) compact_kernel(PlanArgs a) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int share = ((a.num_pages + 31) / 32 + 31) / 32 * 32;
  const int p0 = min(warp * share, a.num_pages), p1 = min(p0 + share, a.num_pages);
  int live = 0;
  for (int p = p0 + lane; p < p1; p += 32) live += a.refs[p] > 0;
  int used;
  block_scan(live, &used);
  int holes = 0, high = 0;     // free pages below `used`, used pages at or above it: equally many
  for (int p = p0 + lane; p < p1; p += 32) {
    const bool on = a.refs[p] > 0;
    a.map[p] = p;
    if (p < used) holes += !on; else high += on;
  }
  int n, moves;
  int at_hole = __shfl_sync(0xffffffffu, block_scan(holes, &n), 0);
  int at_high = __shfl_sync(0xffffffffu, block_scan(high, &moves), 0);
  for (int p = p0; p < p1; p += 32) {
    const int i = p + lane;
    const bool on = i < p1 && a.refs[i] > 0;
    const bool hole = i < p1 && i < used && !on, up = on && i >= used;
    const unsigned mh = __ballot_sync(0xffffffffu, hole), mu = __ballot_sync(0xffffffffu, up);
    const unsigned below = (1u << lane) - 1u;
    if (hole) a.dst[at_hole + __popc(mh & below)] = i;
    if (up) a.src[at_high + __popc(mu & below)] = i;
    at_hole += __popc(mh);
    at_high += __popc(mu);
  }
  __syncthreads();
  for (int k = tid; k < moves; k += kPlanThreads) {
    const int s = a.src[k], t = a.dst[k];
    a.map[s] = t;
    a.refs[t] = a.refs[s];
    a.refs[s] = 0;
  }
  if (tid == 0) {
    a.count[0] = moves;
    *a.used = used;
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The block table given at creation; these calls own its contents with the caller.
int32_t* table_of(const rq_cache& c) { return const_cast<int32_t*>(c.geom.table); }

rq_status check_cache(const rq_cache* c) {
  if (!c || !on_cache_device(*c) || !c->geom.paged) return RQ_ERR_INVALID_ARG;
  return RQ_OK;
}
rq_status done(cudaError_t e) { return e == cudaSuccess ? RQ_OK : RQ_ERR_CUDA; }

CopyArgs copy_args(const rq_cache& c, const int32_t* src, const int32_t* dst) {
  CopyArgs a = {};
  a.base = c.base;
  a.page_bytes = c.geom.page_bytes;
  a.num_pages = c.geom.num_pages;
  a.planes = c.geom.L * c.geom.G;
  a.src = src;
  a.dst = dst;
  return a;
}

size_t plan_bytes(int num_pages) { return 256 + 6 * (((size_t)num_pages * 4 + 255) / 256 * 256); }

PlanArgs plan_args(const rq_cache& c, int32_t* refs, int32_t* status, void* workspace) {
  PlanArgs a = {};
  a.table = table_of(c);
  a.max_tiles = c.geom.max_tiles;
  a.num_pages = c.geom.num_pages;
  a.nmax = c.geom.Nmax;
  a.refs = refs;
  a.status = status;
  const size_t step = ((size_t)a.num_pages * 4 + 255) / 256 * 256;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  a.count = reinterpret_cast<int32_t*>(w);
  int32_t** lists[6] = {&a.asks, &a.last, &a.free, &a.src, &a.dst, &a.map};
  for (int i = 0; i < 6; ++i) *lists[i] = reinterpret_cast<int32_t*>(w + 256 + i * step);
  return a;
}

}  // namespace
}  // namespace rq

using namespace rq;

extern "C" {

size_t rq_pages_workspace_bytes(const rq_config* cfg, int32_t num_pages) {
  return rq_cache_paged_bytes(cfg, num_pages) ? plan_bytes(num_pages) : 0;
}

rq_status rq_pages_copy(rq_cache* cache, int32_t n, const int32_t* src, const int32_t* dst, int32_t* status,
                        void* stream) {
  if (check_cache(cache) != RQ_OK || !src || !dst || n < 0) return RQ_ERR_INVALID_ARG;
  if (n > cache->geom.num_pages) return RQ_ERR_CAPACITY;
  if (!aligned16(src) || !aligned16(dst) || !aligned16(status)) return RQ_ERR_ALIGNMENT;
  if (n == 0) return RQ_OK;
  CopyArgs a = copy_args(*cache, src, dst);
  a.n = n;
  a.check = 1;
  a.status = status;
  return done(launch_copy(a, cache->num_sms, static_cast<cudaStream_t>(stream)));
}

rq_status rq_pages_fork(rq_cache* cache, int32_t n, const int32_t* src_rows, const int32_t* dst_rows, int32_t* refs,
                        int32_t* status, void* stream) {
  if (check_cache(cache) != RQ_OK || !src_rows || !dst_rows || !refs || n < 0) return RQ_ERR_INVALID_ARG;
  const Geom& g = cache->geom;
  if (n > g.Bmax) return RQ_ERR_CAPACITY;
  if (n > kMaxForkPairs) return RQ_ERR_UNSUPPORTED;
  if (!aligned16(src_rows) || !aligned16(dst_rows) || !aligned16(refs) || !aligned16(status)) return RQ_ERR_ALIGNMENT;
  if (n == 0) return RQ_OK;
  ForkArgs a = {table_of(*cache), g.max_tiles, g.Bmax, g.num_pages, n, kForkCols, src_rows, dst_rows, refs, status};
  // shared memory holds the columns of every pair: 32 columns (whole 128-byte
  // lines) up to 1440 pairs, fewer beyond
  while (a.cols > 1 && (size_t)n * (a.cols + 1) * 4 > 190 * 1024) a.cols /= 2;
  const size_t smem = (size_t)n * (a.cols + 1) * 4;
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 190 * 1024);
    if (e != cudaSuccess) return RQ_ERR_CUDA;
  }
  fork_kernel<<<(g.max_tiles + a.cols - 1) / a.cols, 1024, smem, static_cast<cudaStream_t>(stream)>>>(a);
  return done(cudaGetLastError());
}

rq_status rq_pages_reserve(rq_cache* cache, int32_t batch, const int32_t* seq_lens, int32_t n_tokens, int32_t* refs,
                           int32_t* status, void* workspace, size_t workspace_bytes, void* stream) {
  if (check_cache(cache) != RQ_OK || !seq_lens || !refs || !workspace || batch <= 0 || n_tokens < 0)
    return RQ_ERR_INVALID_ARG;
  const Geom& g = cache->geom;
  if (batch > g.Bmax || n_tokens > g.Nmax) return RQ_ERR_CAPACITY;
  if (workspace_bytes < plan_bytes(g.num_pages)) return RQ_ERR_WORKSPACE;
  if (!aligned16(seq_lens) || !aligned16(refs) || !aligned16(status) || !aligned16(workspace))
    return RQ_ERR_ALIGNMENT;
  if (n_tokens == 0) return RQ_OK;
  if ((int64_t)batch * (n_tokens / kTile + 2) > 0x7fffffff) return RQ_ERR_UNSUPPORTED;   // slots are int32
  PlanArgs p = plan_args(*cache, refs, status, workspace);
  p.batch = batch;
  p.n_tokens = n_tokens;
  p.seq_lens = seq_lens;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  reserve_kernel<<<1, kPlanThreads, 0, st>>>(p);
  if (cudaGetLastError() != cudaSuccess) return RQ_ERR_CUDA;
  CopyArgs a = copy_args(*cache, p.src, p.dst);
  a.count = p.count;
  return done(launch_copy(a, cache->num_sms, st));
}

rq_status rq_pages_free(rq_cache* cache, int32_t n, const int32_t* rows, const int32_t* keep, int32_t* refs,
                        int32_t* status, void* stream) {
  if (check_cache(cache) != RQ_OK || !rows || !refs || n < 0) return RQ_ERR_INVALID_ARG;
  const Geom& g = cache->geom;
  if (n > g.Bmax) return RQ_ERR_CAPACITY;
  if (!aligned16(rows) || !aligned16(keep) || !aligned16(refs) || !aligned16(status)) return RQ_ERR_ALIGNMENT;
  if (n == 0) return RQ_OK;
  const int64_t blocks = ((int64_t)n * g.max_tiles + 255) / 256;
  const int grid = (int)(blocks < cache->num_sms * 8 ? blocks : cache->num_sms * 8);
  free_kernel<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(table_of(*cache), g.max_tiles, g.Bmax,
                                                                   g.num_pages, n, rows, keep, refs, status);
  return done(cudaGetLastError());
}

rq_status rq_pages_compact(rq_cache* cache, int32_t* refs, int32_t* used, int32_t* status, void* workspace,
                           size_t workspace_bytes, void* stream) {
  if (check_cache(cache) != RQ_OK || !refs || !used || !workspace) return RQ_ERR_INVALID_ARG;
  const Geom& g = cache->geom;
  if (workspace_bytes < plan_bytes(g.num_pages)) return RQ_ERR_WORKSPACE;
  if (!aligned16(refs) || !aligned16(used) || !aligned16(status) || !aligned16(workspace)) return RQ_ERR_ALIGNMENT;
  PlanArgs p = plan_args(*cache, refs, status, workspace);
  p.used = used;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  compact_kernel<<<1, kPlanThreads, 0, st>>>(p);
  if (cudaGetLastError() != cudaSuccess) return RQ_ERR_CUDA;
  CopyArgs a = copy_args(*cache, p.src, p.dst);
  a.count = p.count;
  a.table = table_of(*cache);
  a.entries = (int64_t)g.Bmax * g.max_tiles;
  a.map = p.map;
  return done(launch_copy(a, cache->num_sms, st));
}

}  // extern "C"
