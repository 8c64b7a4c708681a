// rq_rope: rotary positions of queries and keys.
//
// Pair (a, b) at frequency f turns by the angle position * f:
//   (a', b') = m (a cos - b sin, b cos + a sin);
// the inverse call negates the angle, which is the transposed map and so the
// gradient.  The fraction of a turn of position p is p * F mod 1 with F = f / 2 pi
// as a 64-bit binary fraction: one wrapping integer product, exact but for F itself,
// which is taken in float64.  f_i is a product of i equal ratios, each off by at most
// 2^-52 of itself with its rounding; i f_i <= r / (2 e ln theta), 5.2 at r = 256 and theta =
// 10^4, so that F is off by less than 2^-51 (2^-20 of a turn at the farthest position).
// sin and cos are then taken of a reduced float32 argument.
//
// Memory-bound: every element is read and written once.  537 MB (8192 tokens, 4 rows, 32 heads of 128, BF16)
// take 85 us, 6.3 TB/s; 172 MB of float32 (1021 tokens, 2 rows, 110 heads of 96) 33 us, 5.2 TB/s, of which some
// 6 us are a launch's start and end.  A token's call (n = 1) is a launch's latency.
#include <algorithm>
#include <cmath>
#include <utility>

#include <cuda_fp16.h>

#include "rq_internal.cuh"

namespace rq {
namespace {

constexpr int kMaxPairs = 128;
constexpr int kThreads = 128;

struct RopeTensor {
  const void* in;
  void* out;
  int heads;
  int64_t in_row, in_head, in_token, out_row, out_head, out_token;
};

struct RopeArgs {
  RopeTensor x[2];
  unsigned long long turn[kMaxPairs];   // turns per position, as a fraction of 2^64
  const int32_t *start, *offsets;
  int batch, n, d, r, inter;
  float mag;
};

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f(float v) { return v; }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ float from_f(float v) { return v; }

// magnitude * (cos, sin) of pair i at position p.  The fraction of a turn is split in
// integers into the nearest quarter and a rest of at most an eighth, |y| <= pi / 4 in radians,
// where the Taylor series to y^9 and y^10 are off by less than 2^-28 (of sin y / y: its next term, y^10 / 11!, is
// 2^-28.7) and 2^-32.
__device__ __forceinline__ float2 turn_of(const RopeArgs& a, int i, int p) {
  const unsigned long long frac = (unsigned long long)(long long)p * a.turn[i];   // mod one turn
  const unsigned q = (unsigned)((frac + (1ull << 61)) >> 62);
  const int rest = (int)((long long)(frac - ((unsigned long long)q << 62)) >> 32);   // 2^-32 turns
  const float y = (float)rest * 1.46291807926715968e-9f;                             // 2 pi / 2^32
  const float z = y * y;
  const float s = y * fmaf(z, fmaf(z, fmaf(z, fmaf(z, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), 1.f);
  const float c =
      fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f), -0.5f), 1.f);
  const float cc = q & 1 ? -s : c, ss = q & 1 ? c : s;   // a quarter turn: (cos, sin) -> (-sin, cos)
  const float sign = q & 2 ? -a.mag : a.mag;
  return make_float2(cc * sign, ss * sign);
}
__device__ __forceinline__ int position(const RopeArgs& a, int64_t token, int b, int t) {
  return (int)((unsigned)(a.start ? a.start[b] : 0) + (unsigned)(a.offsets ? a.offsets[token] : t));
}

// 16 bytes as V floats and back
template <typename T> struct Vec;
template <> struct Vec<float> {
  static constexpr int V = 4;
  static __device__ __forceinline__ void load(const uint4& u, float* f) {
    f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y); f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 store(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};
template <> struct Vec<__nv_bfloat16> {
  static constexpr int V = 8;
  static __device__ __forceinline__ void load(const uint4& u, float* f) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 store(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Vec<__half> {
  static constexpr int V = 8;
  static __device__ __forceinline__ void load(const uint4& u, float* f) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = x.x;
      f[2 * i + 1] = x.y;
    }
  }
  static __device__ __forceinline__ uint4 store(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// The vector path: everything on 16-byte boundaries.  A thread takes V pairs of one token --
// two 16-byte pieces, c and c + r / 2 (halves) or neighbours (interleaved) -- and walks along
// heads with the same sines and cosines, kHeads of them in flight at a time; further threads of
// the token copy the channels that do not turn.  (One thread a pair and head: 293 us where this takes 85.)
constexpr int kHeads = 4;
template <typename T, bool INTER>
__global__ void __launch_bounds__(kThreads) rope_vec_kernel(RopeArgs a) {
  constexpr int V = Vec<T>::V;
  const int turns = a.r / (2 * V), work = turns + (a.d - a.r) / V;    // threads a token
  const unsigned idx = blockIdx.x * (unsigned)kThreads + threadIdx.x;
  const unsigned token = idx / (unsigned)work;
  if (token >= (unsigned)a.batch * (unsigned)a.n) return;
  const int u = (int)(idx % (unsigned)work), b = (int)(token / (unsigned)a.n), t = (int)(token % (unsigned)a.n);
  const int heads = a.x[0].heads + a.x[1].heads;
  const bool turn = u < turns;
  const int c0 = turn ? (INTER ? 2 * V * u : V * u) : a.r + V * (u - turns), step = INTER ? V : a.r / 2;
  float cs[V], sn[V];
  if (turn) {
    const int pos = position(a, token, b, t);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float2 x = turn_of(a, V * u + i, pos);
      cs[i] = x.x;
      sn[i] = x.y;
    }
  }
  const T *in0 = static_cast<const T*>(a.x[0].in) + b * a.x[0].in_row + t * a.x[0].in_token + c0,
          *in1 = static_cast<const T*>(a.x[1].in) + b * a.x[1].in_row + t * a.x[1].in_token + c0;
  T *out0 = static_cast<T*>(a.x[0].out) + b * a.x[0].out_row + t * a.x[0].out_token + c0,
    *out1 = static_cast<T*>(a.x[1].out) + b * a.x[1].out_row + t * a.x[1].out_token + c0;
  const int per = (heads + gridDim.y - 1) / gridDim.y, h0 = blockIdx.y * per, h1 = min(heads, h0 + per);
  for (int h = h0; h < h1; h += kHeads) {
    uint4 lo[kHeads], hi[kHeads];
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      if (h + k >= h1) break;
      const int hh = h + k - a.x[0].heads;
      const T* p = hh < 0 ? in0 + (h + k) * a.x[0].in_head : in1 + hh * a.x[1].in_head;
      lo[k] = *reinterpret_cast<const uint4*>(p);
      if (turn) hi[k] = *reinterpret_cast<const uint4*>(p + step);
    }
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      if (h + k >= h1) break;
      const int hh = h + k - a.x[0].heads;
      T* p = hh < 0 ? out0 + (h + k) * a.x[0].out_head : out1 + hh * a.x[1].out_head;
      if (turn) {
        float x[2 * V], y[2 * V];
        Vec<T>::load(lo[k], x);
        Vec<T>::load(hi[k], x + V);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int e = INTER ? 2 * i : i, f = INTER ? 2 * i + 1 : i + V;
          y[e] = x[e] * cs[i] - x[f] * sn[i];
          y[f] = x[f] * cs[i] + x[e] * sn[i];
        }
        *reinterpret_cast<uint4*>(p) = Vec<T>::store(y);
        *reinterpret_cast<uint4*>(p + step) = Vec<T>::store(y + V);
      } else {
        *reinterpret_cast<uint4*>(p) = lo[k];
      }
    }
  }
}

// Whatever is not on 16-byte boundaries: one thread per (token, pair or copied channel), looping over its heads.  Bound by
// its small loads and stores: the BF16 prompt above with 122 of 128 channels rotated takes 304 us (1.8 TB/s).
template <typename T>
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeArgs a) {
  const int half = a.r / 2, work = half + (a.d - a.r);
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= (int64_t)a.batch * a.n * work) return;
  const int64_t token = i / work;
  const int u = (int)(i % work), b = (int)(token / a.n), t = (int)(token % a.n);
  const int heads = a.x[0].heads + a.x[1].heads;
  float2 cs = make_float2(1.f, 0.f);
  int c0, c1 = -1;
  if (u < half) {
    cs = turn_of(a, u, position(a, token, b, t));
    c0 = a.inter ? 2 * u : u;
    c1 = a.inter ? 2 * u + 1 : u + half;
  } else {
    c0 = a.r + u - half;
  }
  for (int h = blockIdx.y; h < heads; h += gridDim.y) {
    const RopeTensor& x = a.x[h < a.x[0].heads ? 0 : 1];
    const int hh = h < a.x[0].heads ? h : h - a.x[0].heads;
    const T* in = static_cast<const T*>(x.in) + b * x.in_row + hh * x.in_head + t * x.in_token;
    T* out = static_cast<T*>(x.out) + b * x.out_row + hh * x.out_head + t * x.out_token;
    if (c1 < 0) {
      out[c0] = in[c0];
    } else {
      const float p = to_f(in[c0]), q = to_f(in[c1]);
      out[c0] = from_f<T>(p * cs.x - q * cs.y);
      out[c1] = from_f<T>(q * cs.x + p * cs.y);
    }
  }
}

// Whether every vector of 16 bytes that the vector path touches starts on a 16-byte boundary.
template <typename T>
bool vectors_fit(const RopeArgs& a) {
  constexpr int V = Vec<T>::V;
  if (a.d % V || a.r % (2 * V)) return false;
  for (const RopeTensor& x : a.x) {
    if (!x.heads) continue;
    if (reinterpret_cast<uintptr_t>(x.in) % 16 || reinterpret_cast<uintptr_t>(x.out) % 16) return false;
    for (int64_t s : {x.in_row, x.in_head, x.in_token, x.out_row, x.out_head, x.out_token})
      if (s % V) return false;
  }
  return true;
}

template <typename T>
cudaError_t launch_rope(const RopeArgs& a, int num_sms, cudaStream_t stream) {
  const int heads = a.x[0].heads + a.x[1].heads;
  if (vectors_fit<T>(a)) {
    constexpr int V = Vec<T>::V;
    const int64_t threads = (int64_t)a.batch * a.n * (a.r / (2 * V) + (a.d - a.r) / V);
    if (threads <= 0x7fffff00) {   // 32-bit thread numbers
      const int blocks = (int)((threads + kThreads - 1) / kThreads);
      // heads split over gridDim.y only as far as the tokens alone do not fill the GPU (a split
      // repeats the sines): some 8 blocks an SM
      int split = num_sms * 8 / blocks;
      split = split < 1 ? 1 : (split > heads ? heads : split);
      if (a.inter)
        rope_vec_kernel<T, true><<<dim3(blocks, split), kThreads, 0, stream>>>(a);
      else
        rope_vec_kernel<T, false><<<dim3(blocks, split), kThreads, 0, stream>>>(a);
      return cudaGetLastError();
    }
  }
  const int64_t work = (int64_t)a.batch * a.n * (a.r / 2 + a.d - a.r);
  const int64_t blocks = (work + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffff) return cudaErrorNotSupported;
  rope_kernel<T><<<dim3((unsigned)blocks, heads < 8 ? heads : 8), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

// Whether two of the tensor's results, of d channels each, share an element: whether some step (i, j, k), not
// all zero, along its axes leads less than d elements away.  Axes sorted by stride: where each one steps
// over all that lies inside it, as in ordinary layouts, none does.  Otherwise (axes that interlock) the steps along
// the two longer strides are tried as far as the shortest axis could lead back from them.
bool results_overlap(const int64_t (&size)[3], const int64_t (&stride)[3], int d) {
  using wide = __int128;
  wide n[3] = {0, 0, 0}, s[3] = {1, 1, 1};     // last steps (0: an axis not in use), lengths of a step
  for (int i = 0; i < 3; ++i)
    if (size[i] > 1) {
      n[i] = size[i] - 1;
      s[i] = stride[i] < 0 ? -(wide)stride[i] : (wide)stride[i];
    }
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if ((n[j] ? s[j] : 0) > (n[j + 1] ? s[j + 1] : 0)) {
        std::swap(n[j], n[j + 1]);
        std::swap(s[j], s[j + 1]);
      }
  wide inside = d;
  bool nested = true;
  for (int i = 0; i < 3; ++i)
    if (n[i]) {
      nested = nested && s[i] >= inside;
      inside += n[i] * s[i];
    }
  if (nested) return false;
  for (wide k = 0; k <= n[2] && k * s[2] < n[1] * s[1] + n[0] * s[0] + d; ++k) {
    // j s1 within reach of -k s2: n0 s0 + d away at most
    const wide reach = n[0] * s[0] + d;
    const wide j0 = std::max((-k * s[2] - reach) / s[1], -n[1]), j1 = std::min((reach - k * s[2]) / s[1], n[1]);
    for (wide j = k ? j0 : 0; j <= j1; ++j) {   // k = 0: a step and its opposite are alike
      // the steps along the shortest axis that lead nearest
      const wide at = k * s[2] + j * s[1], back = std::clamp(-at / s[0], -n[0], n[0]);
      for (wide i = std::max(back - 1, -n[0]); i <= std::min(back + 1, n[0]); ++i) {
        const wide gap = at + i * s[0];
        if ((i || j || k) && gap < d && gap > -(wide)d) return true;
      }
    }
  }
  return false;
}

bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace
}  // namespace rq

using namespace rq;

extern "C" rq_status rq_rope(const rq_rope_config* cfg, int32_t dtype, int32_t batch, int32_t n,
                             const rq_rope_tensor* q, const rq_rope_tensor* k, const int32_t* start,
                             const int32_t* offsets, void* stream) {
  if (!cfg || (!q && !k) || batch < 0 || n < 0) return RQ_ERR_INVALID_ARG;
  if (dtype != RQ_BF16 && dtype != RQ_F16 && dtype != RQ_F32) return RQ_ERR_INVALID_ARG;
  const int d = cfg->head_dim, r = cfg->rotary_dim;
  if (d < 2 || d > 512 || r < 2 || r > 2 * kMaxPairs || r > d || (r & 1)) return RQ_ERR_UNSUPPORTED;
  if (cfg->scaling < RQ_ROPE_PLAIN || cfg->scaling > RQ_ROPE_PARTS) return RQ_ERR_INVALID_ARG;
  if (!(cfg->theta > 1.0) || !std::isfinite(cfg->theta) || !std::isfinite((float)cfg->magnitude))
    return RQ_ERR_INVALID_ARG;
  if (cfg->scaling != RQ_ROPE_PLAIN && !(cfg->factor > 0.0 && std::isfinite(cfg->factor))) return RQ_ERR_INVALID_ARG;
  if (cfg->scaling == RQ_ROPE_BASE && r == 2) return RQ_ERR_INVALID_ARG;   // r / (r - 2)
  if (cfg->scaling == RQ_ROPE_PARTS && !(cfg->original_len > 0 && cfg->low_turns < cfg->high_turns &&
                                         std::isfinite(cfg->low_turns) && std::isfinite(cfg->high_turns)))
    return RQ_ERR_INVALID_ARG;
  const size_t es = dtype == RQ_F32 ? 4 : 2;
  int64_t heads = 0;
  for (const rq_rope_tensor* x : {q, k}) {
    if (!x) continue;
    if (x->heads <= 0 || ((!x->in || !x->out) && batch > 0 && n > 0)) return RQ_ERR_INVALID_ARG;   // empty: any pointer
    if (!aligned_to(x->in, es) || !aligned_to(x->out, es)) return RQ_ERR_ALIGNMENT;
    // two results in one place
    if ((batch > 1 && x->out_row == 0) || (x->heads > 1 && x->out_head == 0) || (n > 1 && x->out_token == 0))
      return RQ_ERR_INVALID_ARG;
    heads += x->heads;
  }
  if (heads * (batch > 0 ? batch : 1) > (1 << 30)) return RQ_ERR_UNSUPPORTED;
  for (const rq_rope_tensor* x : {q, k})
    if (x && batch > 0 && n > 0 && results_overlap({batch, x->heads, n}, {x->out_row, x->out_head, x->out_token}, d))
      return RQ_ERR_INVALID_ARG;
  if (!aligned_to(start, 4) || !aligned_to(offsets, 4)) return RQ_ERR_ALIGNMENT;
  if (batch == 0 || n == 0) return RQ_OK;

  RopeArgs a = {};
  int i = 0;
  for (const rq_rope_tensor* x : {q, k}) {
    if (!x) continue;
    a.x[i++] = {x->in, x->out, x->heads, x->in_row, x->in_head, x->in_token, x->out_row, x->out_head, x->out_token};
  }
  // frequencies in float64: f_i = theta^(-2i/r) by repeated products (relative
  // error about i * 2^-53), then turns per position modulo one, to 64 bits
  const double kTwoPi = 6.283185307179586476925;
  double theta = cfg->theta;
  if (cfg->scaling == RQ_ROPE_BASE) theta *= std::pow(cfg->factor, (double)r / (r - 2));
  if (!std::isfinite(theta)) return RQ_ERR_INVALID_ARG;   // every pair but the first would stand still
  const double ratio = std::pow(theta, -2.0 / r);
  double f = 1.0;
  for (int j = 0; j < r / 2; ++j, f *= ratio) {
    double s = f;
    if (cfg->scaling == RQ_ROPE_LINEAR) s = f / cfg->factor;
    if (cfg->scaling == RQ_ROPE_PARTS) {
      double keep = (cfg->original_len * f / kTwoPi - cfg->low_turns) / (cfg->high_turns - cfg->low_turns);
      keep = keep < 0 ? 0 : (keep > 1 ? 1 : keep);
      s = f * (keep + (1 - keep) / cfg->factor);
    }
    if (!std::isfinite(s)) return RQ_ERR_INVALID_ARG;   // a factor near zero
    double turns = s / kTwoPi;
    turns -= std::floor(turns);
    unsigned long long u = (unsigned long long)(turns * 0x1p63) << 1;   // turns < 1: below 2^63
    a.turn[j] = cfg->inverse ? 0ull - u : u;
  }
  a.start = start;
  a.offsets = offsets;
  a.batch = batch;
  a.n = n;
  a.d = d;
  a.r = r;
  a.inter = cfg->interleaved != 0;
  a.mag = cfg->magnitude == 0.0 ? 1.f : (float)cfg->magnitude;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return RQ_ERR_CUDA;
  const cudaError_t e = dtype == RQ_BF16  ? launch_rope<__nv_bfloat16>(a, sms, st)
                        : dtype == RQ_F16 ? launch_rope<__half>(a, sms, st)
                                          : launch_rope<float>(a, sms, st);
  return e == cudaSuccess ? RQ_OK : (e == cudaErrorNotSupported ? RQ_ERR_UNSUPPORTED : RQ_ERR_CUDA);
}
