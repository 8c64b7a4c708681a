// rq_tree_attention: attention of drafted tokens (a tree per row) over the
// compressed cache and the row's own draft.
//
// Node t of row b, query head hq (KV head h = hq / (Hq / H)) attends the row's n
// cached tokens and the drafted tokens that its mask names:
//   s_k = scale * q . k,   out = sum_k exp(s_k - m) v_k / sum_k exp(s_k - m).
// A cached key of a residual loop is k = c a + R^T r (a: dequantized anchor, r:
// dequantized residual), so with R applied once to the query and once to the sum
//   q . k = c (q . a) + (R q) . r,    sum p v = sum (p c) a + R^T sum p r;
// chained caches fold the planes from the anchor down: x <- c_j x + (R q) . r_j.
#include "rq_tree_kernels.cuh"

namespace rq {
namespace {

__device__ __forceinline__ float2 meta2(const uint8_t* p) {   // (scale, offset)
  return e4m3x2_to_f32x2(*reinterpret_cast<const uint16_t*>(p));
}
// ---- one CTA per (node, query head, row) -------------------------------------
// The path of chained caches, whose planes fold into one another and so do not make a matrix product of
// two parts.  Dequantizes every key and value for its one query: the CTAs of one KV head read the same tiles
// from L2.  Bound by that arithmetic, not by memory: 16 heads of 128, 8192 tokens, 4 rows of 16 nodes take 5206 us with one
// residual plane to read and 9619 with three (one node a row: 4746); the tensor-core path takes 54 on a
// shared-anchor cache.
constexpr int kRowThreads = 128;
constexpr int kMaxPlanes = kMaxLoops;      // anchor + residual planes a call reads

__global__ void __launch_bounds__(kRowThreads) tree_row_kernel(TreeArgs a) {
  const int t = blockIdx.x, hq = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int d = a.g.d, gs = a.g.g, ng = a.g.ng, h = hq / a.g.qpk;
  const int cnt = a.counts ? clamp_len(a.counts[b], a.T) : a.T;
  if (t >= cnt) return;
  const int n = clamp_len(a.seq_lens[b], a.g.Nmax);
  const bool hadamard = (a.g.mode & RQ_MODE_HADAMARD) != 0;

  __shared__ __align__(16) float q_s[128], rq_s[128];
  __shared__ float dot_s[2][kMaxPlanes][64];    // half-row dot products per plane
  __shared__ float w_s[kMaxPlanes][64];         // value weights per plane
  __shared__ float red_s[8];
  __shared__ int page_s;

  const size_t qoff = (((size_t)b * a.g.Hq + hq) * a.T + t) * d;
  q_s[tid] = tid < d ? __bfloat162float(a.q[qoff + tid]) : 0.f;
  __syncthreads();
  if (hadamard) {
    float v[1] = {q_s[tid]};
    hadamard128<1>(v, tid, rq_s);
    rq_s[tid] = v[0];
  } else if (a.nres && tid < d) {
    float s = 0.f;
    for (int k = 0; k < d; ++k) s = fmaf(__ldg(a.R + (size_t)tid * d + k), q_s[k], s);
    rq_s[tid] = s;
  }
  __syncthreads();

  float m = -INFINITY, l = 0.f, oa = 0.f, orr = 0.f;
  const int tok = tid & 63, half = tid >> 6;

  // score of slot `tok` (threads 0..63) -> its softmax weight, the running state updated
  auto weigh = [&](float s, bool on) -> float {
    float mx = on ? s : -INFINITY;
    if (tid < 64) {
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      if ((tid & 31) == 0) red_s[tid >> 5] = mx;
    }
    __syncthreads();
    const float mn = fmaxf(m, fmaxf(red_s[0], red_s[1]));
    const float ref = mn == -INFINITY ? 0.f : mn;
    const float alpha = exp2f(m - ref);
    const float p = on ? exp2f(s - ref) : 0.f;
    if (tid < 64) {
      float sum = p;
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if ((tid & 31) == 0) red_s[2 + (tid >> 5)] = sum;
    }
    __syncthreads();
    l = l * alpha + red_s[2] + red_s[3];
    oa *= alpha;
    orr *= alpha;
    m = mn;
    return p;
  };

  for (int tile = 0; tile * kTile < n; ++tile) {
    const int nv = min(kTile, n - tile * kTile);
    if (a.g.paged && tid == 0) {
      const int pg = checked_page(a.g, raw_page(a.g, b, tile), a.status);
      page_s = pg < 0 ? 0 : pg;
    }
    __syncthreads();
    const int page = a.g.paged ? page_s : 0;
    auto tile_ptr = [&](int plane, int kv) {   // plane 0: anchor; i >= 1: residual P-1-i (shared: this loop)
      const int j = a.nres == 1 ? a.loop : a.g.P - 1 - plane;
      return a.base + a.g.tile_offset(a.layer, a.group, b, h, plane == 0, j, kv, tile, page);
    };
    for (int pl = 0; pl <= a.nres; ++pl) {
      const int bits = pl ? 2 : 4, per = 8 / bits, row = d / per;
      const uint8_t* tp = tile_ptr(pl, 0);
      const uint8_t* meta = tp + (pl ? a.g.r_codes : a.g.a_codes) + (size_t)tok * ng * 2;
      const float* qv = pl ? rq_s : q_s;
      float dot = 0.f;
      if (tok < nv) {
        for (int gi = 0; gi < ng; ++gi) {
          const float2 so = meta2(meta + 2 * gi);
          float sc = 0.f, sq = 0.f;
          for (int ch = gi * gs + half * gs / 2; ch < gi * gs + (half + 1) * gs / 2; ++ch) {
            const int code = (tp[tok * row + ch / per] >> (bits * (ch % per))) & ((1 << bits) - 1);
            sc = fmaf((float)code, qv[ch], sc);
            sq += qv[ch];
          }
          dot = fmaf(so.x, sc, fmaf(so.y, sq, dot));
        }
      }
      dot_s[half][pl][tok] = dot;
    }
    __syncthreads();
    float s = 0.f;
    const bool on = tid < nv;
    if (on) {
      s = dot_s[0][0][tid] + dot_s[1][0][tid];
      for (int pl = 1; pl <= a.nres; ++pl) {
        const uint8_t* tp = tile_ptr(pl, 0) + a.g.r_codes + a.g.meta;
        const float c = bf16_bits_to_f32(*reinterpret_cast<const uint16_t*>(tp + 2 * tid));
        s = fmaf(c, s, dot_s[0][pl][tid] + dot_s[1][pl][tid]);
      }
      s *= a.qscale;
    }
    const float p = weigh(s, on);
    if (tid < 64) {   // weight of plane pl: p times the coefficients of the planes behind it
      float w = p;
      for (int pl = a.nres; pl >= 0; --pl) {
        w_s[pl][tid] = w;
        if (pl && on) {
          const uint8_t* tp = tile_ptr(pl, 1) + a.g.r_codes + a.g.meta;
          w *= bf16_bits_to_f32(*reinterpret_cast<const uint16_t*>(tp + 2 * tid));
        }
      }
    }
    __syncthreads();
    if (tid < d) {
      for (int pl = 0; pl <= a.nres; ++pl) {
        const int bits = pl ? 2 : 4, run = 32 / bits;
        const uint8_t* tp = tile_ptr(pl, 1);
        const uint8_t* meta = tp + (pl ? a.g.r_codes : a.g.a_codes) + (tid / gs) * 2;
        float acc = 0.f;
        for (int k = 0; k < nv; ++k) {
          const int code = (tp[tid * 8 * bits + 4 * (k / run) + (k & 3)] >> (bits * ((k % run) >> 2))) &
                           ((1 << bits) - 1);
          const float2 so = meta2(meta + k * ng * 2);
          acc = fmaf(w_s[pl][k], fmaf(so.x, (float)code, so.y), acc);
        }
        if (pl) orr += acc; else oa += acc;
      }
    }
    __syncthreads();
  }

  // the drafted tokens this node sees
  const size_t kvoff = ((size_t)b * a.g.H + h) * a.T * d;
  for (int j0 = 0; j0 < cnt; j0 += 64) {
    const int j = j0 + tok;
    const bool vis = j < cnt && sees(a, b, t, j);
    float dot = 0.f;
    if (vis)
      for (int ch = half * d / 2; ch < (half + 1) * d / 2; ++ch)
        dot = fmaf(q_s[ch], __bfloat162float(a.k_new[kvoff + (size_t)j * d + ch]), dot);
    dot_s[half][0][tok] = dot;
    __syncthreads();
    const bool on = tid < 64 && vis;
    const float p = weigh(on ? (dot_s[0][0][tid] + dot_s[1][0][tid]) * a.qscale : 0.f, on);
    if (tid < 64) w_s[0][tid] = p;
    __syncthreads();
    if (tid < d)
      for (int k = 0; k < 64 && j0 + k < cnt; ++k)
        if (sees(a, b, t, j0 + k))
          oa = fmaf(w_s[0][k], __bfloat162float(a.v_new[kvoff + (size_t)(j0 + k) * d + tid]), oa);
    __syncthreads();
  }

  float o = oa;
  if (a.nres) {
    q_s[tid] = tid < d ? orr : 0.f;
    __syncthreads();
    if (hadamard) {
      float v[1] = {q_s[tid]};
      hadamard128<1>(v, tid, rq_s);
      o += v[0];
    } else if (tid < d) {
      for (int k = 0; k < d; ++k) o = fmaf(__ldg(a.R + (size_t)k * d + tid), q_s[k], o);
    }
  }
  if (tid < d) a.out[qoff + tid] = __float2bfloat16_rn(l != 0.f ? o / l : 0.f);   // no key seen: zero; NaN stays
}

}  // namespace

// Queries per block: the smallest operand width that holds a KV head's M queries, 64 at most.  A block
// dequantizes its unit's cache once, whatever its width: 61 queries in one block of 64 take 73 us (16384
// tokens, 2 rows), in two of 32 102 us; 16 in a block of 16 54 us (8192 tokens, 4 rows), of 64 69 us.
static int tree_nb(int M) { return M <= 16 ? 16 : (M <= 32 ? 32 : 64); }

namespace {
struct TreeSpace {
  size_t partials, scales, packs, total;   // byte offsets
};
TreeSpace tree_space(const Geom& g, int batch, int n_nodes, int num_sms) {
  TreeSpace w = {256, 256, 256, 256};
  if (g.mode & RQ_MODE_CHAINED) return w;
  const int M = g.qpk * n_nodes, nb = tree_nb(M), planes = g.P > 1 ? 2 : 1;
  const size_t units = (size_t)batch * g.H * ((M + nb - 1) / nb);
  w.scales = w.partials + (units + num_sms) * (size_t)(2 * nb + planes * nb * g.d) * sizeof(float);
  w.packs = (w.scales + units * nb * sizeof(float) + 255) / 256 * 256;
  w.total = w.packs + units * planes * 2 * nb * 128;
  return w;
}
}  // namespace

size_t tree_workspace_bytes(const Geom& g, int batch, int n_nodes, int num_sms) {
  return tree_space(g, batch, n_nodes, num_sms).total;
}

cudaError_t launch_tree(const rq_cache& c, int layer, int group, int loop, int batch, int n_nodes,
                        const __nv_bfloat16* q, const __nv_bfloat16* k_new, const __nv_bfloat16* v_new,
                        const uint64_t* mask, const int32_t* counts, const int32_t* seq_lens, float scale,
                        __nv_bfloat16* out, void* workspace, cudaStream_t stream) {
  TreeArgs a = {};
  a.g = c.geom;
  a.base = c.base;
  a.R = c.R;
  a.q = q;
  a.k_new = k_new;
  a.v_new = v_new;
  a.mask = reinterpret_cast<const unsigned long long*>(mask);
  a.counts = counts;
  a.seq_lens = seq_lens;
  a.out = out;
  a.status = static_cast<int32_t*>(workspace);
  a.layer = layer;
  a.group = group;
  a.batch = batch;
  a.T = n_nodes;
  a.words = (n_nodes + 63) / 64;
  a.loop = loop;
  const bool chained = (c.geom.mode & RQ_MODE_CHAINED) != 0;
  a.nres = loop == c.geom.P - 1 ? 0 : (chained ? c.geom.P - 1 - loop : 1);
  a.qscale = scale * kLog2e;
  if ((int64_t)batch * c.geom.Hq * n_nodes > (1 << 30)) return cudaErrorNotSupported;   // blocks are int32
  if (!chained) {
    const int nb = tree_nb(c.geom.qpk * n_nodes);
    const int64_t units = (int64_t)batch * c.geom.H * ((c.geom.qpk * n_nodes + nb - 1) / nb);
    if (units * ((c.geom.Nmax + kTreeStep - 1) / kTreeStep) > 0x7fffffff) return cudaErrorNotSupported;   // steps, too
    const TreeSpace w = tree_space(c.geom, batch, n_nodes, c.num_sms);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.M = c.geom.qpk * n_nodes;
    a.nqb = (a.M + nb - 1) / nb;
    a.partials = reinterpret_cast<float*>(ws + w.partials);
    a.q_scale = reinterpret_cast<float*>(ws + w.scales);
    a.packs = ws + w.packs;
    return c.geom.d == 128 ? launch_tree_mma(a, nb, c.num_sms, stream) : launch_tree_mma_96(a, nb, c.num_sms, stream);
  }
  if (c.geom.Hq > 65535) return cudaErrorNotSupported;   // grid.y
  tree_row_kernel<<<dim3(n_nodes, c.geom.Hq, batch), kRowThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_tree_mma(const TreeArgs& a, int nb, int num_sms, cudaStream_t stream) {
  return launch_tree_d<128>(a, nb, num_sms, stream);
}

}  // namespace rq
