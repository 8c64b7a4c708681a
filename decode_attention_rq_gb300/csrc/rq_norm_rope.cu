// rq_norm_rope, rq_norm_rope_backward: the norm of queries and keys for each head with
// the rotation by their positions, in one pass.
//
//   y = Rot(p) (w x rstd),  rstd = 1 / sqrt(mean x^2 + eps)  (means over the head's d channels)
// and with g the gradient of y, h = Rot(p)^T g, t = w h:
//   dw = sum over tokens and heads of h x rstd,   dx = rstd (t - x rstd^2 mean(t x)).
// rstd is computed again from x, which the backward pass reads in any case.
//
// Memory-bound: every element is read and written once (backward: x and g read, dx written).  A group of G lanes holds
// a head's vector in registers, 16-byte pieces; it walks along the heads of one token, so that sines and cosines are
// computed once for all of them; mean squares by shuffles within the group.  335 MB (8192 tokens, 2 rows, 40 heads of 128,
// BF16) take 60 us, 5.6 TB/s; the gradients of 4096 tokens (252 MB) 47 us, 5.3 TB/s; of 1021 tokens, 110 heads of 96 in
// float32 (259 MB) 45 us, 5.7 TB/s.  A token's call (n = 1) is a launch's latency, 3.6 us.
#include <atomic>
#include <cstring>
#include <type_traits>

#include "rq_rope.cuh"

namespace rq {
namespace {

constexpr int kNormThreads = 128;
constexpr int kMaxPartials = 1024;      // rows of weight gradients that one backward call leaves to be summed

struct NormTensor {
  const void *in, *grad, *weight;
  void* out;
  float* dweight;
  int heads;
  int64_t in_row, in_head, in_token, out_row, out_head, out_token, grad_row, grad_head, grad_token;
};

struct NormArgs {
  NormTensor x[2];
  unsigned long long turn[kMaxPairs];   // turns per position, as a fraction of 2^64
  const int32_t *start, *offsets;
  float* partials;                      // [CTAs][d]
  int batch, n, d, r, inter, wtype, aligned;
  int split;                            // CTAs of the first tensor; the others work on the second
  float mag, eps;
};

__device__ __forceinline__ float weight_at(const NormArgs& a, const void* w, int c) {
  if (!w) return 1.f;
  if (a.wtype == RQ_F32) return __ldg(static_cast<const float*>(w) + c);
  const uint16_t v = __ldg(static_cast<const uint16_t*>(w) + c);
  return a.wtype == RQ_BF16 ? __uint_as_float((uint32_t)v << 16) : __half2float(__ushort_as_half(v));
}

// Two float32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 swapped(float2 x) { return make_float2(x.y, x.x); }

// Sum over the group's G lanes (aligned within the warp), the same in each.
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The CTA's share of its tensor: items (block of GROUPS tokens, head or pack of heads), a token a group, heads innermost, so that
// sines are kept along a token's heads and neighbouring groups touch neighbouring tokens.  Shares differ by one item.
struct NormShare {
  int64_t items;                        // left
  int block, head;                      // the next item
  __device__ __forceinline__ NormShare(const NormArgs& a, int which, int groups, int heads) {
    const int64_t blocks = ((int64_t)a.batch * a.n + groups - 1) / groups, all = blocks * heads;
    const int ctas = which ? (int)gridDim.x - a.split : a.split, cta = blockIdx.x - (which ? a.split : 0);
    const int64_t each = all / ctas, more = all % ctas, from = cta * each + (cta < more ? cta : more);
    items = each + (cta < more ? 1 : 0);
    block = (int)(from / heads);
    head = (int)(from % heads);
  }
  __device__ __forceinline__ void next(int heads) {
    --items;
    if (++head == heads) {
      head = 0;
      ++block;
    }
  }
};

// The block's sums of weight gradients: every lane's dw, whose channels are c0 + i and c1 + i, over the
// groups in order, to the block's row of partials.
template <int V, int S, int GROUPS>
__device__ __forceinline__ void block_weights(const NormArgs& a, int grp, const int (&c0)[S], const int (&c1)[S],
                                              const float (&dw)[S][2 * V], float* red) {
  __syncthreads();
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (c0[s] + i < a.d) red[grp * a.d + c0[s] + i] = dw[s][i];
      if (c1[s] + i < a.d) red[grp * a.d + c1[s] + i] = dw[s][V + i];
    }
  __syncthreads();
  float* row = a.partials + (size_t)blockIdx.x * a.d;
  for (int c = threadIdx.x; c < a.d; c += kNormThreads) {
    float v = 0.f;
#pragma unroll 8
    for (int g = 0; g < GROUPS; ++g) v += red[g * a.d + c];
    row[c] = v;
  }
}

// 16 bytes of global memory to this thread's place in shared memory, asynchronously; zeros where `on` does not hold.
__device__ __forceinline__ void fetch16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void fetch_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void fetch_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Everything on 16-byte boundaries: a lane's slot is two pieces of V channels that turn with one another (c and c + r / 2;
// neighbours turn within a piece), or that do not turn (cos 1, sin 0); neighbouring lanes have neighbouring
// pieces, so that whole sectors are touched (halves of them: the float32 gradient takes 72 us, whole 45).  S slots a
// lane: two for a float32 head of more than 256.  Each thread fetches its pieces of the next items into its own places
// of a ring in shared memory (nothing to synchronize, no registers held meanwhile), across tokens without a pause.
// (Loads into registers, two heads at a time: that gradient 131 us, the BF16 one of 4096 tokens 88 where this takes 47.)
// An item is KH heads: forward two, whose chains (sum, square root, products) overlap.
template <typename T, int S, bool BACK>
struct VecRing {
  static constexpr int KH = BACK || S > 1 ? 1 : 2;
  static constexpr int PIECES = S * KH * (BACK ? 4 : 2);            // 16-byte pieces of an item
  // more in flight is slower: forward 60 us with two stages, 64 with three, 65 with four (the 8192-token prompt);
  // backward 52, 47 and 49 (4096 tokens)
  static constexpr int STAGES = BACK && S == 1 ? 3 : 2;
  static constexpr int BYTES = STAGES * PIECES * kNormThreads * 16;
};
template <typename T, bool INTER, int G, int S, bool BACK>
__global__ void __launch_bounds__(kNormThreads, BACK && S == 1 ? 4 : 1) norm_vec_kernel(NormArgs a) {
  using Ring = VecRing<T, S, BACK>;
  constexpr int V = Vec<T>::V, GROUPS = kNormThreads / G, ST = Ring::STAGES, KH = Ring::KH;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ __align__(16) float w_s[G * S * 2 * V];                // the weight
  const int lane = threadIdx.x % G, grp = threadIdx.x / G;
  const int turns = a.r / (2 * V), which = (int)blockIdx.x >= a.split;
  const NormTensor& x = a.x[which];
  int c0[S], c1[S];
  bool turn[S];                                     // halves: whether the slot turns
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int u = lane + G * s;
    if (INTER) {                                    // neighbours turn within a piece
      c0[s] = V * (lane + 2 * G * s);
      c1[s] = c0[s] + V * G;
      turn[s] = true;
    } else {
      // the first slots turn, the next `stay` do not, the rest are empty
      const int stay = (a.d - a.r + 2 * V - 1) / (2 * V);
      turn[s] = u < turns;
      c0[s] = u < turns ? V * u : (u < turns + stay ? a.r + V * (u - turns) : a.d);
      c1[s] = c0[s] + (u < turns ? a.r / 2 : V * stay);
    }
  }
  const float inv_d = 1.f / (float)a.d;
  const int tokens = a.batch * a.n, packs = (x.heads + KH - 1) / KH;
  const uint8_t* mine = ring + threadIdx.x * 16;                    // piece i of stage k: + (k PIECES + i) 16 threads
  const uint32_t mine_u = smem_u32(mine);
  constexpr int PITCH = kNormThreads * 16;
  NormShare share(a, which, GROUPS, packs), ahead = share;

  int f_stage = 0;
  bool f_on = false;
  const T *f_in = nullptr, *f_grad = nullptr;
  auto f_seek = [&]() {                             // the group's vectors of item `ahead`
    const int token = ahead.block * GROUPS + grp;
    f_on = token < tokens;
    const int b = f_on ? token / a.n : 0, t = f_on ? token - b * a.n : 0;
    f_in = static_cast<const T*>(x.in) + b * x.in_row + t * x.in_token + (int64_t)(ahead.head * KH) * x.in_head;
    if (BACK)
      f_grad = static_cast<const T*>(x.grad) + b * x.grad_row + t * x.grad_token + (int64_t)(ahead.head * KH) * x.grad_head;
  };
  auto fetch = [&]() {
    if (ahead.items > 0) {
      const uint32_t at = mine_u + f_stage * (Ring::PIECES * PITCH);
#pragma unroll
      for (int k = 0; k < KH; ++k)
#pragma unroll
        for (int s = 0; s < S; ++s) {
          const bool have = f_on && (k == 0 || ahead.head * KH + k < x.heads);
          const bool on0 = have && c0[s] < a.d, on1 = have && c1[s] < a.d;
          const int piece = (k * S + s) * 2;
          fetch16(at + piece * PITCH, f_in + (on0 ? k * x.in_head + c0[s] : 0), on0);
          fetch16(at + (piece + 1) * PITCH, f_in + (on1 ? k * x.in_head + c1[s] : 0), on1);
          if (BACK) {
            fetch16(at + (2 * S * KH + piece) * PITCH, f_grad + (on0 ? k * x.grad_head + c0[s] : 0), on0);
            fetch16(at + (2 * S * KH + piece + 1) * PITCH, f_grad + (on1 ? k * x.grad_head + c1[s] : 0), on1);
          }
        }
      ahead.next(packs);
      if (ahead.head == 0) {
        f_seek();
      } else {
        f_in += KH * x.in_head;
        if (BACK) f_grad += KH * x.grad_head;
      }
    }
    fetch_commit();
    if (++f_stage == ST) f_stage = 0;
  };
  f_seek();
#pragma unroll
  for (int k = 0; k < ST - 1; ++k) fetch();
  for (int c = threadIdx.x; c < G * S * 2 * V; c += kNormThreads) w_s[c] = c < a.d ? weight_at(a, x.weight, c) : 0.f;
  __syncthreads();

  // Pairs of floats: V / 2 of the first piece and V / 2 of the second (INTER: V pairs that turn with themselves).
  // Forward: p = (w cos) and q = (w' sin) of the partner's weight, so that y = rstd (x p + x' q).
  // Backward: p = cos, q = sin (its sign included), h = g p + g' q.
  constexpr int H = V / 2;
  float2 p[S][V], q[S][V], w[S][V], dw[S][V];
  auto weights = [&](int s, float (&f)[2 * V]) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const int z = a.d - 4;                        // pieces behind the head's end: any of it
      *reinterpret_cast<float4*>(f + i) = *reinterpret_cast<const float4*>(w_s + min(c0[s] + i, z));
      *reinterpret_cast<float4*>(f + V + i) = *reinterpret_cast<const float4*>(w_s + min(c1[s] + i, z));
    }
  };
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int i = 0; i < V; ++i) dw[s][i] = both(0.f);
  if (BACK) {
#pragma unroll
    for (int s = 0; s < S; ++s) {
      float f[2 * V];
      weights(s, f);
#pragma unroll
      for (int i = 0; i < V; ++i) w[s][i] = make_float2(f[2 * i], f[2 * i + 1]);
    }
  }
  // x of a pair and its partner: the same pair turned round (INTER), or the other piece's
  auto partner = [&](const float2 (&v)[V], int i) { return INTER ? swapped(v[i]) : v[i < H ? i + H : i - H]; };
  int stage = 0;
  T* o = nullptr;
  bool on = false, fresh = true;
  for (; share.items > 0; share.next(packs), o += KH * x.out_head) {
    if (fresh || share.head == 0) {                 // another token
      fresh = false;
      const int token = share.block * GROUPS + grp;
      on = token < tokens;
      const int b = on ? token / a.n : 0, t = on ? token - b * a.n : 0;
      const int pos = position(a, b * a.n + t, b, t);
#pragma unroll
      for (int s = 0; s < S; ++s) {
        float cs[V], sn[V], f[2 * V];
        if (!BACK) weights(s, f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int pair = INTER ? (i < H ? c0[s] / 2 + i : c1[s] / 2 + i - H) : V * (lane + G * s) + i;
          const float2 z = (INTER ? 2 * pair < a.r : turn[s]) ? turn_of(a, pair, pos) : make_float2(1.f, 0.f);
          cs[i] = z.x;
          sn[i] = BACK ? -z.y : z.y;
        }
        // element k of a slot (k < V: the first piece): cos, and what its partner is multiplied with
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float c2[2], s2[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int e = 2 * i + k, pair = INTER ? i : e % V, other = INTER ? e ^ 1 : (e < V ? e + V : e - V);
            const bool first = INTER ? k == 0 : e < V;
            c2[k] = cs[pair] * (BACK ? 1.f : f[e]);
            s2[k] = (first ? -sn[pair] : sn[pair]) * (BACK ? 1.f : f[other]);
          }
          p[s][i] = make_float2(c2[0], c2[1]);
          q[s][i] = make_float2(s2[0], s2[1]);
        }
      }
      o = static_cast<T*>(x.out) + b * x.out_row + t * x.out_token + (int64_t)(share.head * KH) * x.out_head;
    }
    fetch_wait<ST - 2>();
    const uint8_t* at = mine + stage * (Ring::PIECES * PITCH);
    if (++stage == ST) stage = 0;
    float2 v[KH][S][V], g[S][V];
    auto pairs = [&](int piece, float2 (&z)[V], int i0) {
      float f[V];
      Vec<T>::load(*reinterpret_cast<const uint4*>(at + piece * PITCH), f);
#pragma unroll
      for (int i = 0; i < H; ++i) z[i0 + i] = make_float2(f[2 * i], f[2 * i + 1]);
    };
    auto put = [&](T* to, int s, const float2 (&y)[V]) {
      float f[2 * V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        f[2 * i] = y[i].x;
        f[2 * i + 1] = y[i].y;
      }
      if (c0[s] < a.d) *reinterpret_cast<uint4*>(to + c0[s]) = Vec<T>::store(f);
      if (c1[s] < a.d) *reinterpret_cast<uint4*>(to + c1[s]) = Vec<T>::store(f + V);
    };
#pragma unroll
    for (int k = 0; k < KH; ++k)
#pragma unroll
      for (int s = 0; s < S; ++s) {
        pairs((k * S + s) * 2, v[k][s], 0);
        pairs((k * S + s) * 2 + 1, v[k][s], H);
        if (BACK) {
          pairs(2 * S * KH + 2 * s, g[s], 0);
          pairs(2 * S * KH + 2 * s + 1, g[s], H);
        }
      }
    fetch();                                        // into the stage before this one
    float sum[KH];
#pragma unroll
    for (int k = 0; k < KH; ++k) {
      float2 ss = both(0.f);
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < V; ++i) ss = fma2(v[k][s][i], v[k][s][i], ss);
      sum[k] = (ss.x + ss.y) * inv_d;   // a lane's share of the mean: 512 squares of 2^60 would not fit a sum
    }
#pragma unroll
    for (int k = 0; k < KH; ++k) sum[k] = group_sum<G>(sum[k]);
    if (!BACK) {
#pragma unroll
      for (int k = 0; k < KH; ++k) {
        const float2 rstd = both(rsqrtf(sum[k] + a.eps));
        const bool have = on && (k == 0 || share.head * KH + k < x.heads);
#pragma unroll
        for (int s = 0; s < S; ++s) {
          float2 y[V];
#pragma unroll
          for (int i = 0; i < V; ++i) y[i] = mul2(rstd, fma2(v[k][s][i], p[s][i], mul2(partner(v[k][s], i), q[s][i])));
          if (have) put(o + k * x.out_head, s, y);
        }
      }
    } else {
      float2 dot = both(0.f), h[S][V];
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          h[s][i] = fma2(g[s][i], p[s][i], mul2(partner(g[s], i), q[s][i]));
          dot = fma2(mul2(h[s][i], w[s][i]), v[0][s][i], dot);
        }
      const float td = group_sum<G>(dot.x + dot.y);
      // a group without a token has zeros: eps = 0 must not make its weights' sums NaN
      const float r = on ? rsqrtf(sum[0] + a.eps) : 0.f;
      const float2 rstd = both(r), c = both(-td * inv_d * r * r);
#pragma unroll
      for (int s = 0; s < S; ++s) {
        float2 y[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          dw[s][i] = fma2(h[s][i], mul2(v[0][s][i], rstd), dw[s][i]);
          y[i] = mul2(rstd, fma2(c, v[0][s][i], mul2(h[s][i], w[s][i])));
        }
        if (on) put(o, s, y);
      }
    }
  }
  fetch_wait<0>();
  if (BACK && x.dweight) {   // a slot's registers are in the order of its channels; the ring is free
    float f[S][2 * V];
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        f[s][2 * i] = dw[s][i].x;
        f[s][2 * i + 1] = dw[s][i].y;
      }
    block_weights<V, S, GROUPS>(a, grp, c0, c1, f, reinterpret_cast<float*>(ring));
  }
}

// Any widths, strides and alignment: a lane's slot is the pieces u and u + G of the head; what turns with one another
// meets in shared memory (x w forward, g backward).  Pieces are loaded whole where all is on 16-byte boundaries
// (`aligned`: only r does not fit then), else channel by channel; an item's while the one before is worked on.
// 6452 tokens, 2 rows, 20 heads of 128, 58 channels as halves, BF16: 43 us (132 MB, 3.1 TB/s; without the item ahead 76), their
// gradient 73; the vector kernel takes 28 and 41 with 64 of the channels.  Bound by loads on their way: 12 warps an SM.
template <typename T>
__device__ __forceinline__ uint4 raw_piece(const T* p, int c, int d, bool aligned) {
  constexpr int V = Vec<T>::V;
  uint4 w = make_uint4(0u, 0u, 0u, 0u);
  if (aligned) {
    if (c < d) w = *reinterpret_cast<const uint4*>(p + c);
  } else {
    T t[V];
#pragma unroll
    for (int i = 0; i < V; ++i) t[i] = c + i < d ? p[c + i] : from_f<T>(0.f);
    memcpy(&w, t, sizeof(w));
  }
  return w;
}
template <typename T>
__device__ __forceinline__ void store_piece(T* p, int c, int d, bool aligned, const float* f) {
  constexpr int V = Vec<T>::V;
  if (aligned) {
    if (c < d) *reinterpret_cast<uint4*>(p + c) = Vec<T>::store(f);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (c + i < d) p[c + i] = from_f<T>(f[i]);
  }
}

template <typename T, int G, bool BACK>
__global__ void __launch_bounds__(kNormThreads) norm_any_kernel(NormArgs a) {
  constexpr int V = Vec<T>::V, GROUPS = kNormThreads / G, S = G == 32 && V == 4 ? 2 : 1;
  constexpr int ROW = G * S * 2 * V;       // channels a group can hold
  __shared__ float z_s[2][GROUPS][ROW];
  __shared__ float2 turn_s[GROUPS][ROW / 2];        // cos and sin of the group's token
  __shared__ float red[BACK ? GROUPS * ROW : 1];
  const int lane = threadIdx.x % G, grp = threadIdx.x / G, half = a.r / 2, which = (int)blockIdx.x >= a.split;
  const NormTensor& x = a.x[which];
  int c0[S], c1[S];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    c0[s] = V * (lane + 2 * G * s);
    c1[s] = c0[s] + V * G;
  }
  auto channel = [&](int s, int i) { return i < V ? c0[s] + i : c1[s] + i - V; };
  const float inv_d = 1.f / (float)a.d;
  const int tokens = a.batch * a.n;
  const bool aligned = a.aligned != 0;
  float w[S][2 * V], dw[S][2 * V], cs[S][2 * V], sn[S][2 * V];
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int i = 0; i < 2 * V; ++i) {
      w[s][i] = channel(s, i) < a.d ? weight_at(a, x.weight, channel(s, i)) : 0.f;
      dw[s][i] = 0.f;
    }
  T* o = nullptr;
  bool on = false, fresh = true;
  int buf = 0;
  NormShare share(a, which, GROUPS, x.heads), ahead = share;
  // the next item's pieces are on their way while this one is worked on
  uint4 next[S][BACK ? 4 : 2];
  bool f_on = false;
  const T *f_in = nullptr, *f_grad = nullptr;
  auto f_seek = [&]() {
    const int token = ahead.block * GROUPS + grp;
    f_on = token < tokens;
    const int b = f_on ? token / a.n : 0, t = f_on ? token - b * a.n : 0;
    f_in = static_cast<const T*>(x.in) + b * x.in_row + t * x.in_token + ahead.head * x.in_head;
    if (BACK) f_grad = static_cast<const T*>(x.grad) + b * x.grad_row + t * x.grad_token + ahead.head * x.grad_head;
  };
  auto fetch = [&]() {
    if (ahead.items <= 0) return;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int at0 = f_on ? c0[s] : a.d, at1 = f_on ? c1[s] : a.d;
      next[s][0] = raw_piece(f_in, at0, a.d, aligned);
      next[s][1] = raw_piece(f_in, at1, a.d, aligned);
      if (BACK) {
        next[s][BACK ? 2 : 0] = raw_piece(f_grad, at0, a.d, aligned);
        next[s][BACK ? 3 : 0] = raw_piece(f_grad, at1, a.d, aligned);
      }
    }
    ahead.next(x.heads);
    if (ahead.head == 0) {
      f_seek();
    } else {
      f_in += x.in_head;
      if (BACK) f_grad += x.grad_head;
    }
  };
  f_seek();
  fetch();
  for (; share.items > 0; share.next(x.heads), o += x.out_head) {
    if (fresh || share.head == 0) {                 // another token
      fresh = false;
      const int token = share.block * GROUPS + grp;
      on = token < tokens;
      const int b = on ? token / a.n : 0, t = on ? token - b * a.n : 0;
      // this lane's channels: cos, and the sine that the partner's value takes (its sign included)
      const int pos = position(a, b * a.n + t, b, t);
      __syncwarp();
      for (int i = lane; i < half; i += G) turn_s[grp][i] = turn_of(a, i, pos);
      __syncwarp();
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < 2 * V; ++i) {
          const int c = channel(s, i);
          float2 z = make_float2(1.f, 0.f);
          if (c < a.r) {
            z = turn_s[grp][a.inter ? c >> 1 : (c < half ? c : c - half)];
            const bool first = a.inter ? (c & 1) == 0 : c < half;
            if (first != BACK) z.y = -z.y;          // forward: a cos - b sin, b cos + a sin
          }
          cs[s][i] = z.x;
          sn[s][i] = z.y;
        }
      o = static_cast<T*>(x.out) + b * x.out_row + t * x.out_token + share.head * x.out_head;
    }
    float* z = z_s[buf][grp];                       // two in turn: one barrier an item
    buf ^= 1;
    float v[S][2 * V], ss = 0.f;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      Vec<T>::load(next[s][0], v[s]);
      Vec<T>::load(next[s][1], v[s] + V);
      if (BACK) {
        float g[2 * V];
        Vec<T>::load(next[s][BACK ? 2 : 0], g);
        Vec<T>::load(next[s][BACK ? 3 : 0], g + V);
#pragma unroll
        for (int i = 0; i < 2 * V; ++i) z[channel(s, i)] = g[i];
      }
#pragma unroll
      for (int i = 0; i < 2 * V; ++i) ss = fmaf(v[s][i], v[s][i], ss);
    }
    fetch();
    ss = group_sum<G>(ss * inv_d);
    const float rstd = on ? rsqrtf(ss + a.eps) : 0.f;
    if (!BACK)
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < 2 * V; ++i) {
          v[s][i] *= rstd * w[s][i];
          z[channel(s, i)] = v[s][i];
        }
    __syncwarp();
    float y[S][2 * V], dot = 0.f;
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int i = 0; i < 2 * V; ++i) {
        const int c = channel(s, i);
        const int partner = a.inter ? c ^ 1 : (c < half ? c + half : c - half);
        const float own = BACK ? z[c] : v[s][i];
        y[s][i] = c < a.r ? own * cs[s][i] + z[partner] * sn[s][i] : own;
        if (BACK) {
          dw[s][i] = fmaf(y[s][i], v[s][i] * rstd, dw[s][i]);
          y[s][i] *= w[s][i];
          dot = fmaf(y[s][i], v[s][i], dot);
        }
      }
    if (BACK) {
      const float c = group_sum<G>(dot) * inv_d * rstd * rstd;
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < 2 * V; ++i) y[s][i] = rstd * fmaf(-c, v[s][i], y[s][i]);
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
      store_piece(o, on ? c0[s] : a.d, a.d, aligned, y[s]);
      store_piece(o, on ? c1[s] : a.d, a.d, aligned, y[s] + V);
    }
  }
  if (BACK && x.dweight) block_weights<V, S, GROUPS>(a, grp, c0, c1, dw, red);
}

// Weight gradients: the partial rows, in a fixed order.  One block per 32 channels of a tensor, 32 shares of the rows.
__global__ void __launch_bounds__(1024) norm_weights_kernel(NormArgs a, int rows) {
  __shared__ float red[32][33];
  pdl_wait();
  const int which = blockIdx.y, col = threadIdx.x % 32, part = threadIdx.x / 32, c = blockIdx.x * 32 + col;
  float* out = a.x[which].dweight;
  float v = 0.f;
  if (out && c < a.d) {
#pragma unroll 8
    for (int i = (which ? a.split : 0) + part; i < (which ? rows : a.split); i += 32) v += __ldcg(a.partials + (size_t)i * a.d + c);
  }
  red[part][col] = v;
  __syncthreads();
  v = red[col][part];                      // channel `part`, share `col`
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (out && col == 0 && blockIdx.x * 32 + part < a.d) out[blockIdx.x * 32 + part] = v;
}

// Whether every 16-byte piece that is touched starts on a 16-byte boundary.
template <typename T>
bool pieces_fit(const NormArgs& a, bool back) {
  constexpr int V = Vec<T>::V;
  if (a.d % V) return false;
  for (const NormTensor& x : a.x) {
    if (!x.heads) continue;
    if (!aligned_to(x.in, 16) || !aligned_to(x.out, 16) || (back && !aligned_to(x.grad, 16))) return false;
    for (int64_t s : {x.in_row, x.in_head, x.in_token, x.out_row, x.out_head, x.out_token})
      if (s % V) return false;
    if (back)
      for (int64_t s : {x.grad_row, x.grad_head, x.grad_token})
        if (s % V) return false;
  }
  return true;
}

// A CTA for every place on the GPU (fewer where there are fewer items), shared out between the tensors by their items.
// (The template arguments name the kernel: each has its own occupancy; S = 0: the kernel for any alignment.)
template <typename T, bool INTER, int G, int S, bool BACK, typename K>
cudaError_t launch_shares(K kern, size_t smem, int groups, NormArgs& a, int num_sms, cudaStream_t stream, int* rows) {
  static std::atomic<int> per_sm_dev[kMaxDevices];     // one per kernel
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  int per_sm = per_sm_dev[dev].load(std::memory_order_acquire);
  if (per_sm == 0) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (e != cudaSuccess) return e;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kNormThreads, smem);
    if (e != cudaSuccess) return e;
    if (per_sm < 1) return cudaErrorNotSupported;
    per_sm_dev[dev].store(per_sm, std::memory_order_release);
  }
  const int64_t blocks = ((int64_t)a.batch * a.n + groups - 1) / groups;
  const int kh = S > 0 ? VecRing<T, S, BACK>::KH : 1;
  const int64_t first = blocks * ((a.x[0].heads + kh - 1) / kh), second = blocks * ((a.x[1].heads + kh - 1) / kh), places = (int64_t)num_sms * per_sm;
  int64_t most = places < kMaxPartials ? places : kMaxPartials;
  if (most > first + second) most = first + second;
  int64_t split = most;
  if (second) {
    split = (int64_t)((double)most * first / (first + second) + 0.5);
    split = split < 1 ? 1 : (split > most - 1 ? most - 1 : split);
  }
  a.split = (int)split;
  *rows = (int)most;
  kern<<<(unsigned)most, kNormThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

template <typename T, bool INTER, int G, int S, bool BACK>
cudaError_t launch_vec(NormArgs& a, int num_sms, cudaStream_t stream, int* rows) {
  return launch_shares<T, INTER, G, S, BACK>(norm_vec_kernel<T, INTER, G, S, BACK>, VecRing<T, S, BACK>::BYTES,
                                             kNormThreads / G, a, num_sms, stream, rows);
}
template <typename T, int G, bool BACK>
cudaError_t launch_any(NormArgs& a, int num_sms, cudaStream_t stream, int* rows) {
  return launch_shares<T, false, G, 0, BACK>(norm_any_kernel<T, G, BACK>, 0, kNormThreads / G, a, num_sms, stream, rows);
}

template <typename T, bool BACK>
cudaError_t launch_norm(NormArgs& a, int num_sms, cudaStream_t stream) {
  constexpr int V = Vec<T>::V;
  a.aligned = pieces_fit<T>(a, BACK);
  int rows = 0;
  cudaError_t e;
  // neighbours turn within a piece, so that r needs no alignment
  if (a.aligned && (a.inter || a.r % (2 * V) == 0)) {
    const int slots = a.inter ? (a.d + 2 * V - 1) / (2 * V) : a.r / (2 * V) + (a.d - a.r + 2 * V - 1) / (2 * V);
    auto go = [&](auto inter) {
      constexpr bool I = decltype(inter)::value;
      if (slots <= 4) return launch_vec<T, I, 4, 1, BACK>(a, num_sms, stream, &rows);
      if (slots <= 8) return launch_vec<T, I, 8, 1, BACK>(a, num_sms, stream, &rows);
      if (slots <= 16) return launch_vec<T, I, 16, 1, BACK>(a, num_sms, stream, &rows);
      if (V == 8 || slots <= 32) return launch_vec<T, I, 32, 1, BACK>(a, num_sms, stream, &rows);
      return launch_vec<T, I, 32, V == 4 ? 2 : 1, BACK>(a, num_sms, stream, &rows);
    };
    e = a.inter ? go(std::true_type()) : go(std::false_type());
  } else {
    const int slots = (a.d + 2 * V - 1) / (2 * V);
    e = slots <= 4    ? launch_any<T, 4, BACK>(a, num_sms, stream, &rows)
        : slots <= 8  ? launch_any<T, 8, BACK>(a, num_sms, stream, &rows)
        : slots <= 16 ? launch_any<T, 16, BACK>(a, num_sms, stream, &rows)
                      : launch_any<T, 32, BACK>(a, num_sms, stream, &rows);
  }
  if (e != cudaSuccess || !BACK || (!a.x[0].dweight && !a.x[1].dweight)) return e;
  return launch_dependent(norm_weights_kernel, dim3((a.d + 31) / 32, 2), dim3(1024), 0, stream, a, rows);
}

rq_status norm_rope(const rq_rope_config* cfg, int dtype, int weight_dtype, int batch, int n, const rq_norm_tensor* q,
                    const rq_norm_tensor* k, double eps, const int32_t* start, const int32_t* offsets, bool back,
                    void* workspace, size_t workspace_bytes, void* stream) {
  if (!cfg || (!q && !k) || batch < 0 || n < 0) return RQ_ERR_INVALID_ARG;
  for (int t : {dtype, weight_dtype})
    if (t != RQ_BF16 && t != RQ_F16 && t != RQ_F32) return RQ_ERR_INVALID_ARG;
  if (!(eps >= 0.0) || !std::isfinite((float)eps)) return RQ_ERR_INVALID_ARG;
  const rq_status st_c = rope_check(*cfg);
  if (st_c != RQ_OK) return st_c;
  NormArgs a = {};
  const rq_status st_f = rope_turns(*cfg, a.turn);
  if (st_f != RQ_OK) return st_f;
  const size_t es = dtype == RQ_F32 ? 4 : 2, ws = weight_dtype == RQ_F32 ? 4 : 2;
  const bool empty = batch == 0 || n == 0;
  int64_t heads = 0;
  bool weights = false;
  for (const rq_norm_tensor* x : {q, k}) {
    if (!x) continue;
    if (x->x.heads <= 0 || ((!x->x.in || !x->x.out || (back && !x->grad)) && !empty)) return RQ_ERR_INVALID_ARG;
    if (!aligned_to(x->x.in, es) || !aligned_to(x->x.out, es) || !aligned_to(x->weight, ws)) return RQ_ERR_ALIGNMENT;
    if (back && (!aligned_to(x->grad, es) || !aligned_to(x->weight_grad, 4))) return RQ_ERR_ALIGNMENT;
    heads += x->x.heads;
    weights = weights || (back && x->weight_grad);
  }
  if (back && q && k && q->weight_grad && k->weight_grad) {   // two sums in one place
    const uintptr_t x = reinterpret_cast<uintptr_t>(q->weight_grad), y = reinterpret_cast<uintptr_t>(k->weight_grad);
    if ((x < y ? y - x : x - y) < cfg->head_dim * sizeof(float)) return RQ_ERR_INVALID_ARG;
  }
  if (heads * (batch > 0 ? batch : 1) > (1 << 30) || (int64_t)batch * n > (1 << 30)) return RQ_ERR_UNSUPPORTED;
  for (const rq_norm_tensor* x : {q, k})
    if (x && !empty && results_overlap({batch, x->x.heads, n}, {x->x.out_row, x->x.out_head, x->x.out_token}, cfg->head_dim))
      return RQ_ERR_INVALID_ARG;
  if (!aligned_to(start, 4) || !aligned_to(offsets, 4)) return RQ_ERR_ALIGNMENT;
  if (weights) {
    if (!workspace) return RQ_ERR_INVALID_ARG;
    if (!aligned_to(workspace, 16)) return RQ_ERR_ALIGNMENT;
    if (workspace_bytes < rq_norm_rope_workspace_bytes(cfg->head_dim)) return RQ_ERR_WORKSPACE;
  }
  if (empty && !weights) return RQ_OK;

  int i = 0;
  for (const rq_norm_tensor* x : {q, k}) {
    if (!x) continue;
    const rq_rope_tensor& t = x->x;
    a.x[i++] = {t.in, back ? x->grad : nullptr, x->weight, t.out, back ? x->weight_grad : nullptr, t.heads,
                t.in_row, t.in_head, t.in_token, t.out_row, t.out_head, t.out_token,
                x->grad_row, x->grad_head, x->grad_token};
  }
  a.start = start;
  a.offsets = offsets;
  a.partials = static_cast<float*>(workspace);
  a.batch = batch;
  a.n = n;
  a.d = cfg->head_dim;
  a.r = cfg->rotary_dim;
  a.inter = cfg->interleaved != 0;
  a.wtype = weight_dtype;
  a.mag = cfg->magnitude == 0.0 ? 1.f : (float)cfg->magnitude;
  a.eps = (float)eps;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (empty) {   // no rows: the weight gradients are zero
    norm_weights_kernel<<<dim3((a.d + 31) / 32, 2), 1024, 0, st>>>(a, 0);
    e = cudaGetLastError();
    return e == cudaSuccess ? RQ_OK : RQ_ERR_CUDA;
  }
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return RQ_ERR_CUDA;
  if (back)
    e = dtype == RQ_BF16  ? launch_norm<__nv_bfloat16, true>(a, sms, st)
        : dtype == RQ_F16 ? launch_norm<__half, true>(a, sms, st)
                          : launch_norm<float, true>(a, sms, st);
  else
    e = dtype == RQ_BF16  ? launch_norm<__nv_bfloat16, false>(a, sms, st)
        : dtype == RQ_F16 ? launch_norm<__half, false>(a, sms, st)
                          : launch_norm<float, false>(a, sms, st);
  return e == cudaSuccess ? RQ_OK : RQ_ERR_CUDA;
}

}  // namespace
}  // namespace rq

using namespace rq;

extern "C" {

size_t rq_norm_rope_workspace_bytes(int32_t head_dim) {
  if (head_dim < 2 || head_dim > 512) return 0;
  return (size_t)kMaxPartials * head_dim * sizeof(float);
}

rq_status rq_norm_rope(const rq_rope_config* cfg, int32_t dtype, int32_t weight_dtype, int32_t batch, int32_t n,
                       const rq_norm_tensor* q, const rq_norm_tensor* k, double eps, const int32_t* start,
                       const int32_t* offsets, void* stream) {
  return norm_rope(cfg, dtype, weight_dtype, batch, n, q, k, eps, start, offsets, false, nullptr, 0, stream);
}

rq_status rq_norm_rope_backward(const rq_rope_config* cfg, int32_t dtype, int32_t weight_dtype, int32_t batch,
                                int32_t n, const rq_norm_tensor* q, const rq_norm_tensor* k, double eps,
                                const int32_t* start, const int32_t* offsets, void* workspace,
                                size_t workspace_bytes, void* stream) {
  return norm_rope(cfg, dtype, weight_dtype, batch, n, q, k, eps, start, offsets, true, workspace, workspace_bytes,
                   stream);
}

}  // extern "C"
