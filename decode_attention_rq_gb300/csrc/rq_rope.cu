// rq_rope: rotary positions of queries and keys.
//
// Pair (a, b) at frequency f turns by the angle position * f:
//   (a', b') = m (a cos - b sin, b cos + a sin);
// the inverse call negates the angle, which is the transposed map and so the
// gradient.  The fraction of a turn of position p is p * F mod 1 with F = f / 2 pi
// as a 64-bit binary fraction: one wrapping integer product, exact for every
// int32 position up to the rounding of F (2^-65 of a turn a position, 2^-34 at
// the farthest).  sin and cos are then taken of a reduced float32 argument.
//
// Memory-bound: every element is read and written once.
#include <cmath>

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

// magnitude * (cos, sin) of pair i at position p
__device__ __forceinline__ float2 turn_of(const RopeArgs& a, int i, int p) {
  const long long frac = (long long)((unsigned long long)(long long)p * a.turn[i]);   // mod one turn
  float s, c;
  sincospif((float)(int)(frac >> 32) * 0x1p-31f, &s, &c);   // top 32 bits: half turns / 2^31
  return make_float2(c * a.mag, s * a.mag);
}

// One thread per (token, pair or copied channel), looping over its heads.
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
    const int pos = (int)((unsigned)(a.start ? a.start[b] : 0) + (unsigned)(a.offsets ? a.offsets[token] : t));
    cs = turn_of(a, u, pos);
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

template <typename T>
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t stream) {
  const int64_t work = (int64_t)a.batch * a.n * (a.r / 2 + a.d - a.r);
  const int64_t blocks = (work + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffff) return cudaErrorNotSupported;
  const int heads = a.x[0].heads + a.x[1].heads;
  rope_kernel<T><<<dim3((unsigned)blocks, heads < 8 ? heads : 8), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
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
  if (!(cfg->theta > 1.0) || !std::isfinite(cfg->theta) || !std::isfinite(cfg->magnitude)) return RQ_ERR_INVALID_ARG;
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
    heads += x->heads;
  }
  if (!aligned_to(start, 4) || !aligned_to(offsets, 4)) return RQ_ERR_ALIGNMENT;
  if (heads * (batch > 0 ? batch : 1) > (1 << 30)) return RQ_ERR_UNSUPPORTED;
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
  const cudaError_t e = dtype == RQ_BF16 ? launch_rope<__nv_bfloat16>(a, st)
                                         : (dtype == RQ_F16 ? launch_rope<__half>(a, st) : launch_rope<float>(a, st));
  return e == cudaSuccess ? RQ_OK : (e == cudaErrorNotSupported ? RQ_ERR_UNSUPPORTED : RQ_ERR_CUDA);
}
