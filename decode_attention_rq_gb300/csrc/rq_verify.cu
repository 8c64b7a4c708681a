// rq_verify: which drafted tokens of a row's tree stand, and the token after them.
//
// At node cur, with target probabilities p and the draft's q after it, r = p and z = 1.  cur's children in
// order: child c of token x stands if u_c z q(x) < r(x), and the walk goes on from it; else r <- max(r - z q, 0) and
// z <- sum r (without a draft distribution q is 1 at x and r(x) becomes 0).  r / z is then the distribution that
// the next sibling, or the row's last token, has to follow: with siblings drawn from q, every token that comes out
// is distributed as if drawn from p.  r is kept unnormalized: one rounding of z q and one of the difference.
// The last token is the first v with sum_{i <= v} r(i) > w sum r.
//
// A cluster of up to 8 CTAs per row, each with a slice of the vocabulary: r stays in shared memory, every warp's sum goes
// to all CTAs' shared memory, all take the same decisions.  A child that stands costs no pass over the vocabulary: p and q at
// every node's token are fetched at the start, and what is left of r at a sibling's token is followed beside.  A pass is
// made for every child that does not stand, and one for the last token.  Without a draft distribution only r(x) goes: it
// is taken off its segment's sum, and a pass follows only the first child refused (16 rows of 33 nodes, 65537 values: 22 -> 10 us).
// A warp's positions are neighbours, so the sums of a pass are the search's first level; 32 parts of a segment and its values
// are the other two.
// Sums: two-float (the rounding of every addition is kept), to about 2^-44, 2^-40 where much of them was taken off: a
// border between two tokens of the inverse CDF is then met as in 64 bits.  With doubles for the sums of CTAs and the search, an
// addition of which is some 0.2 us, 4 rows of 32000 values took 12.2 us where this takes 7.0; 64 rows of 131072, three
// CTAs an SM in place of two, 45 -> 28.6.
// Bound by latency: the tokens' probabilities (two loads in turn, 0.8 us), each pass (load 1.2, sums and cluster barrier 1), the
// search (1); at 64 rows of 131072 values by a first pass over 34 MB and by the rows with most children refused.
// Greedy: largest values of all nodes at once where that is little to read, a warp a row then walks; else node after node.
#include <atomic>
#include <cfloat>
#include <cstring>

#include <cuda_fp16.h>

#include "rq_internal.cuh"

namespace rq {
namespace {

// 256 threads of at most 80 registers: three CTAs with 64 KB of r each fit an SM
constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kRoom = 32 * kVerifyWarps;     // r's room is a multiple of this: equal parts for the lanes of all warps
constexpr int kMaxVocab = 262144;            // 8 slices of 32768: 129 KB of shared memory

// Greedy: up to this many bytes of target rows all nodes' largest values are found at once, for reading them costs no more
// than two or three nodes of a walk, some 3 us each (32 rows, 8 nodes, 50257 BF16 values: 9.3 us; walking 24).
constexpr int64_t kAllNodesBytes = 32 << 20;
constexpr int kFewCtas = 304;                // a node is split until two CTAs are at work on each of 152 SMs

struct VerifyArgs {
  const void *target, *draft;
  int64_t target_row, target_node, draft_row, draft_node;
  const int32_t *tokens, *parents, *counts;
  const float *u, *w;
  int32_t *path, *n_path, *next;
  int T, V, slice, room, greedy;   // slice: values a CTA, a multiple of 8; room: floats of r, slice + 8 and more
};

// A sum and the roundings of its additions: h is the float32 nearest to h + l once a pair was added.
struct Sum2 {
  float h = 0.f, l = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float s = __fadd_rn(h, x), b = __fsub_rn(s, h);
    l = __fadd_rn(l, __fadd_rn(__fsub_rn(h, __fsub_rn(s, b)), __fsub_rn(x, b)));
    h = s;
  }
  // in either order the same to the bit
  __device__ __forceinline__ void add(Sum2 o) {
    const float s = __fadd_rn(h, o.h), b = __fsub_rn(s, h);
    l = __fadd_rn(__fadd_rn(l, o.l), __fadd_rn(__fsub_rn(h, __fsub_rn(s, b)), __fsub_rn(o.h, b)));
    h = s;
    settle();
  }
  __device__ __forceinline__ void settle() {
    const float s = __fadd_rn(h, l);
    l = __fsub_rn(l, __fsub_rn(s, h));
    h = s;
  }
  __device__ __forceinline__ bool operator<(Sum2 o) const { return __fadd_rn(__fsub_rn(o.h, h), __fsub_rn(o.l, l)) > 0.f; }
  __device__ __forceinline__ unsigned long long word() const {
    return (unsigned long long)__float_as_uint(h) << 32 | __float_as_uint(l);
  }
};
__device__ __forceinline__ Sum2 sum_of(unsigned long long w) {
  Sum2 s;
  s.h = __uint_as_float((uint32_t)(w >> 32));
  s.l = __uint_as_float((uint32_t)w);
  return s;
}
// w times a sum
__device__ __forceinline__ Sum2 scaled(Sum2 s, float w) {
  Sum2 p;
  p.h = __fmul_rn(w, s.h);
  p.l = fmaf(w, s.l, fmaf(w, s.h, -p.h));
  p.settle();
  return p;
}
__device__ __forceinline__ Sum2 warp_sum(Sum2 s) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    Sum2 y;
    y.h = __shfl_xor_sync(0xffffffffu, s.h, o);
    y.l = __shfl_xor_sync(0xffffffffu, s.l, o);
    s.add(y);
  }
  return s;
}
// The first lane whose sum `at` + own_0 + .. + own_lane lies beyond thr; where rounding leaves none, the last one with
// something, and -1 where all are empty.  at: receives the sum before that lane, or, if none is beyond, behind the last one.
__device__ __forceinline__ int warp_find(Sum2 own, Sum2 thr, Sum2& at, bool* beyond) {
  const int lane = threadIdx.x & 31;
  Sum2 run = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    Sum2 y;
    y.h = __shfl_up_sync(0xffffffffu, run.h, o);
    y.l = __shfl_up_sync(0xffffffffu, run.l, o);
    if (lane >= o) run.add(y);
  }
  run.add(at);
  const unsigned some = __ballot_sync(0xffffffffu, own.h > 0.f);
  const unsigned past = __ballot_sync(0xffffffffu, own.h > 0.f && thr < run);
  const int l = past ? __ffs(past) - 1 : (some ? 31 - __clz(some) : -1);
  *beyond = past != 0;
  // the sum before lane l is the one behind lane l - 1
  const int from = past ? l - 1 : 31;
  const float h = __shfl_sync(0xffffffffu, run.h, from & 31), lo = __shfl_sync(0xffffffffu, run.l, from & 31);
  if (from >= 0) {
    at.h = h;
    at.l = lo;
  }
  return l;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// v to this shared-memory address of CTA `rank`
__device__ __forceinline__ void cluster_put(void* p, uint32_t rank, unsigned long long v) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

template <typename T> __device__ __forceinline__ float value_of(T v);
template <> __device__ __forceinline__ float value_of(float v) { return v; }
template <> __device__ __forceinline__ float value_of(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float value_of(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T of_value(float v);
template <> __device__ __forceinline__ float of_value(float v) { return v; }
template <> __device__ __forceinline__ __half of_value(float v) { return __float2half(v); }
template <> __device__ __forceinline__ __nv_bfloat16 of_value(float v) { return __float2bfloat16(v); }
// a probability: in [0, 1], NaN counts as 0
__device__ __forceinline__ float prob(float v) { return fminf(fmaxf(v, 0.f), 1.f); }
// larger for a larger value, for equal values for a lower index; NaN counts as -infinity, -0 as 0
__device__ __forceinline__ unsigned long long rank_key(float v, int i) {
  v = v == v ? v + 0.f : -INFINITY;
  const uint32_t b = __float_as_uint(v);
  return (unsigned long long)(b & 0x80000000u ? ~b : b | 0x80000000u) << 32 | (0xffffffffu - (uint32_t)i);
}

// Eight values from p + j on, j a multiple of 8: whole where `vec` (p is on a 16-byte boundary) and all lie in [lo, hi), else
// one by one, `fill` outside.  Raw, so that several can be on their way.
template <typename T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p, int j, int lo, int hi, bool vec, float fill) {
    if (vec && j >= lo && j + 8 <= hi) {
#pragma unroll
      for (int k = 0; k < (int)sizeof(T) / 2; ++k) w[k] = __ldg(reinterpret_cast<const uint4*>(p + j) + k);
    } else if (j < hi) {
      T t[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) t[k] = j + k >= lo && j + k < hi ? __ldg(p + j + k) : of_value<T>(fill);
      memcpy(w, t, sizeof(w));
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    T t[8];
    memcpy(t, w, sizeof(w));
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = value_of(t[k]);
  }
};

// A warp's part of the largest of p[0 .. nv), the values of tokens v0 on: as rank_key.  A thread notes the piece of eight
// with its largest value, keys are made for that one alone (for every value: 15.2 us where this takes 9.3, 32 rows of 8 nodes).
template <typename T>
__device__ __forceinline__ unsigned long long best_key(const T* p, int v0, int nv) {
  constexpr int kAhead = 16 / sizeof(T);
  const int lo = (reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T), end = lo + nv;   // whole pieces on 16-byte boundaries
  p -= lo;
  float most = -INFINITY;
  Raw8<T> best;
  int at = threadIdx.x * 8;
  if (at < end) best.load(p, at, lo, end, true, -INFINITY);
  for (int j0 = at; j0 < end; j0 += kVerifyThreads * 8 * kAhead) {
    Raw8<T> raw[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) raw[u].load(p, j0 + u * kVerifyThreads * 8, lo, end, true, -INFINITY);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int j = j0 + u * kVerifyThreads * 8;
      if (j >= end) break;
      float v[8];
      raw[u].get(v);
      float m = v[0];
#pragma unroll
      for (int k = 1; k < 8; ++k) m = fmaxf(m, v[k]);       // passes over NaN
      if (m > most) {
        most = m;
        best = raw[u];
        at = j;
      }
    }
  }
  unsigned long long key = 0;
  if (at < end) {
    float v[8];
    best.get(v);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (at + k >= lo && at + k < end) key = max(key, rank_key(v[k], v0 - lo + at + k));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, o));
  return key;
}

// A word of every warp of a cluster, in the order of ranks and warps, in each CTA's shared memory.  Two buffers: the other
// CTAs may still read one until they arrive at the next barrier.
struct Meeting {
  unsigned long long (*words)[kMaxCluster * kVerifyWarps];
  uint32_t ranks, rank;
  int phase = 0;
  __device__ __forceinline__ unsigned long long* met() const { return words[phase ^ 1]; }
  // the same word in all lanes of a warp; a barrier
  __device__ __forceinline__ void meet(unsigned long long word) {
    const int lane = threadIdx.x & 31, at = rank * kVerifyWarps + (threadIdx.x >> 5);
    if (ranks == 1) {
      words[phase][at] = word;
      __syncthreads();
    } else {
      if (lane < (int)ranks) cluster_put(&words[phase][at], lane, word);
      cluster_sync();
    }
    phase ^= 1;
  }
  // a lane's two of them; 0: none
  __device__ __forceinline__ unsigned long long mine(int i) const {
    const int at = (threadIdx.x & 31) * 2 + i;
    return at < (int)ranks * kVerifyWarps ? met()[at] : 0ull;
  }
  __device__ __forceinline__ Sum2 sum() const {
    Sum2 s = sum_of(mine(0));
    s.add(sum_of(mine(1)));
    return warp_sum(s);
  }
  __device__ __forceinline__ int best() const {   // of rank_keys: the token
    unsigned long long key = max(mine(0), mine(1));
#pragma unroll
    for (int o = 16; o; o >>= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, o));
    return (int)(0xffffffffu - (uint32_t)key);
  }
};
static_assert(kMaxCluster * kVerifyWarps == 64, "two words a lane");

template <typename T>
__global__ void __launch_bounds__(kVerifyThreads, 3) verify_kernel(VerifyArgs a) {
  extern __shared__ __align__(16) float r_s[];              // what is left of the target's probabilities, this slice
  __shared__ int token_s[RQ_MAX_TREE_NODES], parent_s[RQ_MAX_TREE_NODES], path_s[RQ_MAX_TREE_NODES];
  __shared__ float left_s[RQ_MAX_TREE_NODES], q_s[RQ_MAX_TREE_NODES], u_s[RQ_MAX_TREE_NODES];   // r and q at the node's token
  __shared__ unsigned long long words_s[2][kMaxCluster * kVerifyWarps];
  __shared__ float base_s[kMaxCluster * kVerifyWarps];      // segments' sums when last added up
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t ranks = cluster_size(), rank = cluster_rank();
  const int b = blockIdx.x / ranks, T_ = a.T;
  const int v0 = rank * a.slice, nv = max(0, min(a.V - v0, a.slice));   // this CTA's part of the vocabulary
  const T* target = static_cast<const T*>(a.target) + (int64_t)b * a.target_row;
  const T* draft = static_cast<const T*>(a.draft) + (int64_t)b * a.draft_row;
  const int n = a.counts ? min(max(__ldg(a.counts + b), 0), T_) : T_;
  // a CTA's shared memory may be written once it has started: awaited behind the first loads
  if (ranks > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");

  for (int t = tid; t < n; t += kVerifyThreads) {
    const int x = __ldg(a.tokens + (int64_t)b * T_ + t);
    int par = t == 0 ? -1 : (a.parents ? __ldg(a.parents + (int64_t)b * T_ + t) : t - 1);
    if (par >= t || x < 0 || x >= a.V) par = -1;           // hangs under nothing, or is no token: never stands
    token_s[t] = x;
    parent_s[t] = par;
    if (!a.greedy && par >= 0) {
      left_s[t] = prob(value_of(__ldg(target + par * a.target_node + x)));
      q_s[t] = a.draft ? prob(value_of(__ldg(draft + par * a.draft_node + x))) : 1.f;
      u_s[t] = __ldg(a.u + (int64_t)b * T_ + t);
    }
  }
  __syncthreads();
  if (ranks > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");

  Meeting m{words_s, ranks, rank};
  // node's first child behind t; n: none
  auto child = [&](int t, int node) {
    for (int s = t + 1; s < n; s += 32) {
      const unsigned hit = __ballot_sync(0xffffffffu, s + lane < n && parent_s[s + lane] == node);
      if (hit) return s + __ffs(hit) - 1;
    }
    return n;
  };
  const int seg = a.room / kVerifyWarps;                    // r's positions a warp takes, neighbours
  int skew = 0;                                             // r(v0 + i) is r_s[skew + i], zeros before and behind
  Sum2 total;                                               // of r
  // r <- p (fresh) or r_s, less z q or with r(x) = 0, and its sum.  Pieces start on 16-byte boundaries of p's row.
  auto pass = [&](int node, bool fresh, bool subtract, float z, int x) {
    constexpr int kAhead = 8 / sizeof(T);                   // pieces of eight values on their way to a thread
    const T* p = target + node * a.target_node + v0;
    skew = (reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T);
    p -= skew;
    const T* q = draft + node * a.draft_node + v0 - skew;
    const bool q_vec = (reinterpret_cast<uintptr_t>(q) & 15) == 0;
    const int end = skew + nv, stop = min(end, (warp + 1) * seg);
    x += skew - v0;
    Sum2 s;
    for (int j0 = warp * seg + lane * 8; j0 < stop; j0 += 256 * kAhead) {
      Raw8<T> pr[kAhead], qr[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (j0 + u * 256 < stop) {
          if (fresh) pr[u].load(p, j0 + u * 256, skew, end, true, 0.f);
          if (subtract) qr[u].load(q, j0 + u * 256, skew, end, q_vec, 0.f);
        }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int j = j0 + u * 256;
        if (j >= stop) break;
        float r[8], d[8];
        if (fresh) {
          pr[u].get(r);
        } else {
          const float4 lo = *reinterpret_cast<const float4*>(r_s + j), hi = *reinterpret_cast<const float4*>(r_s + j + 4);
          r[0] = lo.x; r[1] = lo.y; r[2] = lo.z; r[3] = lo.w; r[4] = hi.x; r[5] = hi.y; r[6] = hi.z; r[7] = hi.w;
        }
        if (subtract) qr[u].get(d);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (fresh) r[k] = prob(r[k]);
          if (subtract) r[k] = fmaxf(__fsub_rn(r[k], __fmul_rn(z, prob(d[k]))), 0.f);
          if (j + k == x) r[k] = 0.f;
          s.add(r[k]);
        }
        s.settle();
        *reinterpret_cast<float4*>(r_s + j) = make_float4(r[0], r[1], r[2], r[3]);
        *reinterpret_cast<float4*>(r_s + j + 4) = make_float4(r[4], r[5], r[6], r[7]);
      }
    }
    m.meet(warp_sum(s).word());
    total = m.sum();
    if (tid < kMaxCluster * kVerifyWarps) base_s[tid] = sum_of(m.met()[tid]).h;   // read behind a barrier
  };
  // Segment `at` summed as in a pass, from r_s; every warp's word goes round again.
  auto resum = [&](int at) {
    unsigned long long word = m.met()[rank * kVerifyWarps + warp];
    if (at == (int)rank * kVerifyWarps + warp) {
      const int stop = min(skew + nv, (warp + 1) * seg);
      Sum2 s;
      for (int j = warp * seg + lane * 8; j < stop; j += 256) {
        for (int k = 0; k < 8; ++k) s.add(r_s[j + k]);
        s.settle();
      }
      word = warp_sum(s).word();
    }
    m.meet(word);
    if (tid == 0) base_s[at] = sum_of(m.met()[at]).h;
  };

  int cur = 0, count = n ? 1 : 0, pick = -1;
  if (a.greedy) {
    auto best = [&](int node) {
      m.meet(best_key(target + node * a.target_node + v0, v0, nv));
      return m.best();
    };
    if (n) pick = best(0);
    for (int t = child(0, cur); t < n; t = child(t, cur))
      if (token_s[t] == pick) {
        if (tid == 0) path_s[count] = t;
        ++count;
        cur = t;
        pick = best(cur);
      }
  } else if (n) {
    float z = 1.f, whole = 0.f;         // z; the sum that the last pass found
    bool fresh = true;
    for (int t = child(0, cur); t < n; t = child(t, cur)) {
      const int x = token_s[t];
      const float rx = left_s[t];
      if (__fmul_rn(u_s[t], __fmul_rn(z, q_s[t])) < rx) {
        if (tid == 0) path_s[count] = t;
        ++count;
        cur = t;
        z = 1.f;
        fresh = true;
        continue;
      }
      __syncthreads();    // left_s is read
      // what is left at the siblings' tokens behind this one
      for (int s = t + 1 + tid; s < n; s += kVerifyThreads)
        if (parent_s[s] == cur)
          left_s[s] = a.draft ? fmaxf(__fsub_rn(left_s[s], __fmul_rn(z, q_s[s])), 0.f)
                              : (token_s[s] == x ? 0.f : left_s[s]);
      if (a.draft || fresh) {
        pass(cur, fresh, a.draft != nullptr, z, a.draft ? -1 : x);
        whole = total.h;
      } else {
        // only r(x) goes: off its segment's sum.  All is summed anew once little is left, for what cancels is 2^-44 of
        // `whole`; one segment once 2^-20 of its own sum is left, or an empty one could seem to hold something.
        const int owner = x / a.slice, j = skew + x - owner * a.slice, at = owner * kVerifyWarps + j / seg;
        if (tid == 0) {
          Sum2 s = sum_of(m.met()[at]), y;
          y.h = -rx;
          s.add(y);
          m.met()[at] = s.word();
          if (owner == (int)rank) r_s[j] = 0.f;
        }
        __syncthreads();
        if (rx > 0.f && !(sum_of(m.met()[at]).h > 0x1p-20f * base_s[at])) resum(at);
        total = m.sum();
        if (!(total.h > 0.0625f * whole)) {
          pass(cur, false, false, z, -1);
          whole = total.h;
        }
      }
      fresh = false;
      z = total.h;
    }
    if (fresh) pass(cur, true, false, 1.f, -1);
    if (!(total.h > 0.f) && !fresh) pass(cur, true, false, 1.f, -1);   // nothing is left: the target itself
    if (!(total.h > 0.f)) {
      if (rank == 0 && tid == 0) a.next[b] = -1;   // no probability anywhere
    } else if (warp == 0) {
      // which segment of which CTA (two a lane), which of its 32 parts (a lane each), which value.  thr < total: where the
      // order of additions hides what lies beyond it, the last value with something is taken.
      Sum2 thr = scaled(total, fminf(fmaxf(__ldg(a.w + b), 0.f), 0x1.fffffep-1f)), at, s = sum_of(m.mine(0));
      bool beyond;
      s.add(sum_of(m.mine(1)));
      const int l = max(warp_find(s, thr, at, &beyond), 0);
      if (!beyond) thr.h = FLT_MAX;
      const Sum2 first = sum_of(m.met()[2 * l]), second = sum_of(m.met()[2 * l + 1]);
      Sum2 mid = at;
      mid.add(first);
      int g = 2 * l;
      if (!(first.h > 0.f && (thr < mid || !(second.h > 0.f)))) {
        ++g;
        at = mid;
      }
      if (g / kVerifyWarps == (int)rank) {
        const int part = seg / 32, end = skew + nv, from = g % kVerifyWarps * seg;
        s = Sum2();
        for (int k = 0, j = lane % part; k < part; ++k, j = j + 1 < part ? j + 1 : 0) {   // not all in the same banks
          const int i = from + lane * part + j;
          if (i < end) s.add(r_s[i]);
        }
        s.settle();
        const int c = max(warp_find(s, thr, at, &beyond), 0);
        if (!beyond) thr.h = FLT_MAX;
        int found = 0;
        beyond = false;
        for (int j = 0; j < part && !beyond; j += 32) {
          const int i = from + c * part + j + lane;
          Sum2 one;
          if (j + lane < part && i < end) one.h = r_s[i];
          const int k = warp_find(one, thr, at, &beyond);
          if (k >= 0) found = i - lane + k;
        }
        if (lane == 0) a.next[b] = v0 + min(max(found, skew), end - 1) - skew;
      }
    }
  }
  if (rank == 0) {
    if (tid == 0) {
      path_s[0] = 0;
      a.n_path[b] = count;
      if (a.greedy || !n) a.next[b] = pick;
    }
    __syncthreads();
    for (int t = tid; t < T_; t += kVerifyThreads) a.path[(int64_t)b * T_ + t] = t < count ? path_s[t] : -1;
  }
  // what was written into other CTAs' shared memory was awaited at a barrier: nothing is under way
}

// Greedy, every node at once: a cluster a node leaves the token with the largest value in path[row][node].
template <typename T>
__global__ void __launch_bounds__(kVerifyThreads, 3) verify_best_kernel(VerifyArgs a) {
  __shared__ unsigned long long words_s[2][kMaxCluster * kVerifyWarps];
  const uint32_t ranks = cluster_size(), rank = cluster_rank();
  const int node = blockIdx.x / ranks, b = node / a.T, t = node % a.T;
  const int v0 = rank * a.slice, nv = max(0, min(a.V - v0, a.slice));
  if (ranks > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_launch_dependents();
  const int n = a.counts ? min(max(__ldg(a.counts + b), 0), a.T) : a.T;
  const bool used = t < n;             // the same for the cluster
  unsigned long long key = 0;
  if (used) key = best_key(static_cast<const T*>(a.target) + (int64_t)b * a.target_row + t * a.target_node + v0, v0, nv);
  if (ranks > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (!used) return;
  Meeting m{words_s, ranks, rank};
  m.meet(key);
  const int pick = m.best();
  if (rank == 0 && threadIdx.x == 0) a.path[node] = pick;
}

// The walk over them: a warp a row.  Children follow their parents: one way through the nodes, 32 at a time.
__global__ void __launch_bounds__(32) verify_walk_kernel(VerifyArgs a) {
  __shared__ int path_s[RQ_MAX_TREE_NODES];
  const int b = blockIdx.x, lane = threadIdx.x;
  const int64_t row = (int64_t)b * a.T;
  const int n = a.counts ? min(max(__ldg(a.counts + b), 0), a.T) : a.T;
  pdl_wait();
  int cur = 0, count = n ? 1 : 0, pick = n ? a.path[row] : -1;
  for (int t0 = 0; t0 < n; t0 += 32) {
    const int t = t0 + lane;
    int par = -1, x = -1, own = -1;
    if (t > 0 && t < n) {
      x = __ldg(a.tokens + row + t);
      par = a.parents ? __ldg(a.parents + row + t) : t - 1;
      if (par >= t) par = -1;
      own = a.path[row + t];
    }
    for (;;) {
      const unsigned hit = __ballot_sync(0xffffffffu, par == cur && x == pick);
      if (!hit) break;
      const int l = __ffs(hit) - 1;
      pick = __shfl_sync(0xffffffffu, own, l);
      cur = t0 + l;
      if (lane == 0) path_s[count] = cur;
      ++count;
    }
  }
  if (lane == 0) {
    path_s[0] = 0;
    a.n_path[b] = count;
    a.next[b] = pick;
  }
  __syncwarp();
  for (int t = lane; t < a.T; t += 32) a.path[row + t] = t < count ? path_s[t] : -1;
}

cudaError_t launch_clusters(void (*kern)(VerifyArgs), const VerifyArgs& a, unsigned grid, int ranks, size_t smem,
                            cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

template <typename T>
cudaError_t launch_verify(VerifyArgs& a, int batch, cudaStream_t stream) {
  auto share = [&](int ranks) { a.slice = (a.V + ranks * 8 - 1) / (ranks * 8) * 8; };
  int ranks = 1;
  if (a.greedy && (int64_t)batch * a.T * a.V * (int64_t)sizeof(T) <= kAllNodesBytes) {
    while (ranks < kMaxCluster && a.V > ranks * 4096 && batch * a.T * ranks < kFewCtas) ranks *= 2;
    share(ranks);
    const cudaError_t e = launch_clusters(verify_best_kernel<T>, a, (unsigned)(batch * a.T * ranks), ranks, 0, stream);
    return e == cudaSuccess ? launch_dependent(verify_walk_kernel, dim3((unsigned)batch), dim3(32), 0, stream, a) : e;
  }
  // as many CTAs a row as have 4096 values each: a pass is then one load of a thread
  while (ranks < kMaxCluster && a.V > ranks * 4096) ranks *= 2;
  share(ranks);
  a.room = (a.slice + 8 + kRoom - 1) / kRoom * kRoom;
  auto* kern = verify_kernel<T>;
  static std::atomic<int> ready[kMaxDevices];   // shared-memory limit set on this device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (kMaxVocab / kMaxCluster + kRoom) * (int)sizeof(float));
    if (e != cudaSuccess) return e;
    ready[dev].store(1, std::memory_order_release);
  }
  return launch_clusters(kern, a, (unsigned)batch * ranks, ranks, a.greedy ? 0 : (size_t)a.room * sizeof(float), stream);
}

bool on4(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

}  // namespace
}  // namespace rq

using namespace rq;

extern "C" rq_status rq_verify(int32_t rule, int32_t dtype, int32_t batch, int32_t n_nodes, int32_t vocab,
                               const void* target, int64_t target_row, int64_t target_node, const void* draft,
                               int64_t draft_row, int64_t draft_node, const int32_t* tokens, const int32_t* parents,
                               const int32_t* node_counts, const float* accept, const float* sample, int32_t* path,
                               int32_t* counts, int32_t* next, void* stream) {
  if (rule != RQ_VERIFY_SAMPLE && rule != RQ_VERIFY_GREEDY) return RQ_ERR_INVALID_ARG;
  if (dtype != RQ_BF16 && dtype != RQ_F16 && dtype != RQ_F32) return RQ_ERR_INVALID_ARG;
  if (batch < 0 || n_nodes < 1 || vocab < 1) return RQ_ERR_INVALID_ARG;
  if (n_nodes > RQ_MAX_TREE_NODES || vocab > kMaxVocab || batch > (1 << 24)) return RQ_ERR_UNSUPPORTED;
  if (batch == 0) return RQ_OK;
  const bool greedy = rule == RQ_VERIFY_GREEDY;
  if (!target || !tokens || !path || !counts || !next || (!greedy && (!accept || !sample))) return RQ_ERR_INVALID_ARG;
  const size_t es = dtype == RQ_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(target) % es || reinterpret_cast<uintptr_t>(draft) % es || !on4(tokens) ||
      !on4(parents) || !on4(node_counts) || !on4(accept) || !on4(sample) || !on4(path) || !on4(counts) || !on4(next))
    return RQ_ERR_ALIGNMENT;
  VerifyArgs a = {};
  a.target = target;
  a.draft = greedy ? nullptr : draft;
  a.target_row = target_row;
  a.target_node = target_node;
  a.draft_row = draft_row;
  a.draft_node = draft_node;
  a.tokens = tokens;
  a.parents = parents;
  a.counts = node_counts;
  a.u = accept;
  a.w = sample;
  a.path = path;
  a.n_path = counts;
  a.next = next;
  a.T = n_nodes;
  a.V = vocab;
  a.greedy = greedy;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == RQ_BF16  ? launch_verify<__nv_bfloat16>(a, batch, st)
                        : dtype == RQ_F16 ? launch_verify<__half>(a, batch, st)
                                          : launch_verify<float>(a, batch, st);
  return e == cudaSuccess ? RQ_OK : RQ_ERR_CUDA;
}
