"""GPU: tree attention over values of the whole range that the library states -- rebuilt V up to 65504 in
magnitude, from wide groups under small coefficients to narrow ones under large coefficients.

Bar, from the kernel's roundings, all of them relative: the value product takes its operands with 11 significant
bits, half a step 2^-11 each.  A product p (c a + R^T r) is p, a = s code + o and c a rounded (3 * 2^-11 of p |c a|), p and r
rounded (2 * 2^-11 of p |R^T| |r|); float32 sums of at most 400 such terms and R^T in 16-bit pieces add less than 2^-14 of
both.  A score is off by at most e = scale * 2^-11 (sum |q| |c a| + 2 sum |R q| |r|), and by 2^-14 of the same sums in
float32; weights then change by a factor within exp(+-2e), the result by at most (exp(2e) - 1) sum p |v - out|.
Last the result's own BF16 rounding, 2^-8.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from rq_harness import Case, GpuCache, rotation32
from test_gpu_tree import bf16, call, mask_words, tree_masks

pytestmark = pytest.mark.gpu


def parts(buf, geom, b, h, kv, loop, n):
    """c a and r of the cached vectors, float64: the anchor's part and the rotated residual."""
    g = geom.group_size
    x = oracle.dequantize(*oracle.read_plane_tokens(buf, geom, 0, 0, b, h, kv, "anchor", 0, n), g)
    if loop == geom.loops_per_group - 1:
        return x, np.zeros_like(x)
    *codes, c = oracle.read_plane_tokens(buf, geom, 0, 0, b, h, kv, "res", loop, n)
    return oracle.bf16_decode(c)[:, None] * x, oracle.dequantize(*codes, g)


def expected(buf, geom, R, Hq, loop, q, kn, vn, see, lens, scale):
    """Float64 results and the bar of each element."""
    B, _, T, d = q.shape
    H = geom.num_heads
    out, bar = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(B):
        for hq in range(Hq):
            h = hq * H // Hq
            ka, kr = parts(buf, geom, b, h, 0, loop, lens[b])
            va, vr = parts(buf, geom, b, h, 1, loop, lens[b])
            K, V = np.concatenate([ka + kr @ R, kn[b, h]]), np.concatenate([va + vr @ R, vn[b, h]])
            size = np.concatenate([3 * np.abs(va) + 2 * np.abs(vr) @ np.abs(R), 3 * np.abs(vn[b, h])])
            for t in range(T):
                vis = np.concatenate([np.ones(lens[b], dtype=bool), see[b, t]])
                x = q[b, hq, t]
                s = K[vis] @ x * scale
                p = np.exp(s - s.max())
                p /= p.sum()
                o = p @ V[vis]
                e = scale * (2.0 ** -11 + 2.0 ** -14) * (
                    np.abs(ka) @ np.abs(x) + 2 * np.abs(kr) @ np.abs(R @ x)).max()
                out[b, hq, t] = o
                bar[b, hq, t] = (2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2.0 ** -14) * (p @ size[vis])
                                 + math.expm1(2 * e) * (p @ np.abs(V[vis] - o)))
    return out, bar


def cache_of(case, n, v_loops, seed):
    """K of ordinary size, V as given ([loop][1][H][n][d]; the last is the anchor): the library's cache, and the oracle's bytes,
    which it holds."""
    rng = np.random.default_rng(seed)
    base = rng.standard_normal((case.B, case.H, n, case.d))
    k = [a * base + 0.2 * rng.standard_normal(base.shape) for a in (0.8, -0.9)] + [base]
    kvb = torch.from_numpy(np.stack([np.stack(x) for x in zip(k, v_loops)]).astype(np.float32)).to(torch.bfloat16)
    R32, R = rotation32(case.d, kind=case.rotation)
    gpu = GpuCache(case, R32)
    geom = oracle.Geometry(case.L, case.P, case.G, case.H, case.d, case.g, case.B, case.Nmax)
    buf = np.zeros(geom.total_bytes, dtype=np.uint8)
    gpu.append(0, 0, kvb, [0] * case.B)
    oracle.append(buf, geom, R, 0, 0, kvb.double().numpy(), np.zeros(case.B, dtype=np.int64), rotation=case.rotation)
    assert np.array_equal(gpu.bytes_host(), buf)
    return gpu, geom, R, buf


# range of the anchor's groups (a scale is a 15th of it), coefficients of the two coded loops.  The product of scale and
# coefficient: 256 and 512; 1024 and 1800; 853 and 3600; 2000 and 5400; then narrow groups, 1000 to 17000
@pytest.mark.parametrize("width,alphas", [
    (1920.0, (2.0, 4.0)), (3840.0, (4.0, -7.0)), (6400.0, (2.0, 8.5)), (6720.0, (-4.5, 12.0)),
    (120.0, (130.0, -500.0)), (30.0, (700.0, 1020.0)), (16.0, (1030.0, -4000.0)), (1.0, (17000.0, 60000.0))])
@pytest.mark.parametrize("d,g,T,Hq,rotation", [(128, 32, 5, 2, "dense"), (96, 16, 21, 2, "dense"),
                                               (128, 16, 13, 8, "hadamard")])
def test_large_values_match_float64(width, alphas, d, g, T, Hq, rotation):
    n, H = 150, 2
    case = Case(L=1, P=3, G=1, H=H, d=d, g=g, B=1, Nmax=200, Hq=Hq, rotation=rotation)
    rng = np.random.default_rng(int(width))
    # an offset is an E4M3 number of at most 448 in magnitude
    base = -min(400.0, width / 2) + width * rng.random((1, H, n, d))
    top = np.abs(base).max()
    # least squares of a multiple of the anchor and some noise; V itself stays below 60000
    v = [np.clip(a * base, -60000, 60000) + 0.05 * min(abs(a) * top, 60000) * rng.standard_normal(base.shape) for a in alphas]
    gpu, geom, R, buf = cache_of(case, n, [np.clip(x, -65000, 65000) for x in v] + [base], 3)
    see, scale = tree_masks(T, 1, T), 1 / math.sqrt(d)
    for loop in range(3):
        qb, q = bf16(rng, 1, Hq, T, d)
        kb, kn = bf16(rng, 1, H, T, d)
        vb, vn = bf16(rng, 1, H, T, d)
        out = call(gpu, 0, 0, loop, qb, kb, vb, mask_words(see), None, [n], scale)
        ref, bar = expected(buf, geom, R, Hq, loop, q, kn, vn, see, [n], scale)
        got = out.double().cpu().numpy()
        assert np.isfinite(got).all(), f"loop {loop}"
        ratio = np.abs(got - ref) / bar
        assert ratio.max() <= 1, f"loop {loop}: {ratio.max():.2f} times the bar"
    gpu.close()
