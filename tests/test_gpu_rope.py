"""GPU: rotary positions (rq_rope) against float64.

Bars.  A result is one rounding to the tensors' type (half a step: 2^-8 BF16,
2^-11 FP16, 2^-24 FP32 of the value) of a float32 sum a cos -+ b sin: two products and
one sum (3 * 2^-24 of |a| + |b|), and cos, sin to within 2^-22 (float32 series of an
argument of at most pi / 4, rounded twice: 2 * 2^-24 * pi / 4, plus two units of the series).
|gpu - float64| <= step * |x| + magnitude * (|a| + |b|) * 2^-21.  FP16 values below the
normal range add half their step, 2^-25.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def config(rq, **kw):
    base = dict(head_dim=128, rotary_dim=128, interleaved=0, inverse=0, scaling=rq.RQ_ROPE_PLAIN, original_len=8192,
                theta=10000.0, factor=4.0, low_turns=1.0, high_turns=32.0, magnitude=0.0)
    base.update(kw)
    return rq.rq_rope_config(**base)


def angles(rq, cfg, pos):
    """float64 angles [..., r / 2] of integer positions, and the magnitude."""
    r = cfg.rotary_dim
    theta = cfg.theta * (cfg.factor ** (r / (r - 2)) if cfg.scaling == rq.RQ_ROPE_BASE else 1.0)
    f = np.array([theta ** (-2.0 * i / r) for i in range(r // 2)])
    if cfg.scaling == rq.RQ_ROPE_LINEAR:
        f = f / cfg.factor
    if cfg.scaling == rq.RQ_ROPE_PARTS:
        k = np.clip((cfg.original_len * f / (2 * math.pi) - cfg.low_turns) / (cfg.high_turns - cfg.low_turns), 0, 1)
        f = f * (k + (1 - k) / cfg.factor)
    sign = -1.0 if cfg.inverse else 1.0
    return sign * np.asarray(pos, dtype=np.float64)[..., None] * f, cfg.magnitude or 1.0


def turned(rq, cfg, x, pos):
    """float64 result and the size |a| + |b| of each element's pair; x [B, H, n, d], pos [B, n]."""
    r = cfg.rotary_dim
    ang, mag = angles(rq, cfg, pos)
    c, s = mag * np.cos(ang)[:, None], mag * np.sin(ang)[:, None]
    first, second = (slice(0, r, 2), slice(1, r, 2)) if cfg.interleaved else (slice(0, r // 2), slice(r // 2, r))
    y, size = x.copy(), np.zeros_like(x)
    a, b = x[..., first], x[..., second]
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    size[..., first] = size[..., second] = mag * (np.abs(a) + np.abs(b))
    return y, size


def close(got, ref, size, dtype):
    ref16 = ref
    err = np.abs(got.double().cpu().numpy() - ref16)
    tol = STEP[dtype] * np.abs(ref) + size * 2.0 ** -21 + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    assert (err <= tol).all(), f"{(err - tol).max():.3e} beyond the bar"


def positions(start, n, offsets=None):
    s = np.asarray(start, dtype=np.int64)[:, None]
    return s + (np.arange(n)[None] if offsets is None else offsets)


CASES = [
    # dtype, d, r, inter, inverse, scaling, B, Hq, H, n, start, tree
    (torch.bfloat16, 128, 128, 0, 0, 0, 4, 16, 16, 1, [0, 77, 8191, 16383], False),
    (torch.bfloat16, 128, 128, 1, 0, 3, 2, 4, 2, 300, [0, 50000], False),
    (torch.float32, 96, 64, 1, 1, 1, 2, 5, 5, 61, [100000, 3], False),
    (torch.float16, 96, 96, 0, 0, 2, 3, 3, 1, 17, [1, 2, 3], True),
    (torch.float32, 64, 64, 0, 0, 0, 1, 2, 1, 9, [2147483600], False),
    (torch.float32, 128, 122, 0, 0, 3, 1, 2, 2, 33, [1000000], False),
    (torch.bfloat16, 128, 64, 0, 1, 0, 2, 6, 2, 65, [5, 9], True),
    (torch.float32, 7, 6, 1, 0, 0, 2, 3, 1, 5, [5, 9], False),
    (torch.bfloat16, 2, 2, 0, 0, 0, 1, 1, 1, 130, [0], False),
    (torch.float32, 512, 256, 0, 0, 1, 1, 2, 1, 12, [44], False),
    (torch.float16, 80, 20, 0, 0, 0, 2, 2, 2, 40, [44, 0], False),
    (torch.float32, 128, 128, 0, 0, 0, 1, 40, 8, 3, [-20], False),
]


@pytest.mark.parametrize("dtype,d,r,inter,inverse,scaling,B,Hq,H,n,start,tree", CASES)
def test_rope_matches_float64(dtype, d, r, inter, inverse, scaling, B, Hq, H, n, start, tree):
    import decode_attention_rq_gb300 as rq
    rng = np.random.default_rng(d + n)
    cfg = config(rq, head_dim=d, rotary_dim=r, interleaved=inter, inverse=inverse, scaling=scaling,
                 magnitude=1.25 if scaling == rq.RQ_ROPE_PARTS else 0.0)
    q = torch.from_numpy(rng.standard_normal((B, Hq, n, d)).astype(np.float32)).to(dtype).cuda()
    k = torch.from_numpy(rng.standard_normal((B, H, n, d)).astype(np.float32)).to(dtype).cuda()
    off = rng.integers(0, 9, (B, n)) if tree else None
    st = torch.tensor(start, dtype=torch.int32, device="cuda")
    offs = None if off is None else torch.from_numpy(off.astype(np.int32)).cuda()
    pos = positions(start, n, off)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    rq.rq_rope(cfg, q, k, st, offs, qo, ko)
    torch.cuda.synchronize()
    for x, y in ((q, qo), (k, ko)):
        ref, size = turned(rq, cfg, x.double().cpu().numpy(), pos)
        close(y, ref, size, dtype)
        assert torch.equal(y[..., r:], x[..., r:])
    # in place, and one tensor alone, give the same bits
    q2 = q.clone()
    rq.rq_rope(cfg, q2, None, st, offs)
    k2 = k.clone()
    rq.rq_rope(cfg, None, k2, st, offs)
    torch.cuda.synchronize()
    assert torch.equal(q2, qo) and torch.equal(k2, ko)


@pytest.mark.parametrize("dtype,d,pad", [(torch.bfloat16, 128, 0), (torch.bfloat16, 128, 3), (torch.float32, 96, 1),
                                         (torch.bfloat16, 96, 8)])
def test_strided_views_and_the_elements_between_them(dtype, d, pad):
    """q and k as views of one [row, token, head, channel] buffer with padding; the
    result into head-major buffers and in place; nothing between the views changes."""
    import decode_attention_rq_gb300 as rq
    rng = np.random.default_rng(pad)
    B, n, Hq, H = 2, 37, 4, 2
    buf = torch.from_numpy(rng.standard_normal((B, n, Hq + H, d + pad)).astype(np.float32)).to(dtype).cuda()
    q, k = buf[:, :, :Hq, :d].transpose(1, 2), buf[:, :, Hq:, :d].transpose(1, 2)
    cfg = config(rq, head_dim=d, rotary_dim=d)
    st = torch.tensor([10, 4000], dtype=torch.int32, device="cuda")
    qo = torch.empty((B, Hq, n, d), dtype=dtype, device="cuda")
    ko = torch.empty((B, H, n, d), dtype=dtype, device="cuda")
    before = buf.clone()
    rq.rq_rope(cfg, q, k, st, None, qo, ko)
    torch.cuda.synchronize()
    assert torch.equal(buf, before)
    pos = positions([10, 4000], n)
    for x, y in ((q, qo), (k, ko)):
        close(y, *turned(rq, cfg, x.double().cpu().numpy(), pos), dtype)
    rq.rq_rope(cfg, q, k, st)
    torch.cuda.synchronize()
    assert torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(buf[..., d:], before[..., d:])


def test_inverse_is_the_transpose_and_the_gradient():
    """<w, rope(x)> = <inverse(w), x>, and the inverse equals the difference quotient
    of x -> <w, rope(x)> (the map is linear: the quotient is exact up to rounding)."""
    import decode_attention_rq_gb300 as rq
    rng = np.random.default_rng(5)
    for inter, scaling in ((0, 3), (1, 0)):
        kw = dict(head_dim=32, rotary_dim=24, interleaved=inter, scaling=scaling, magnitude=1.1)
        fwd, inv = config(rq, **kw), config(rq, inverse=1, **kw)
        x, w = (torch.from_numpy(rng.standard_normal((1, 2, 6, 32)).astype(np.float32)).cuda() for _ in range(2))
        st = torch.tensor([123], dtype=torch.int32, device="cuda")

        def apply(cfg, t):
            y = torch.empty_like(t)
            rq.rq_rope(cfg, t, None, st, None, y)
            return y.double()

        g = apply(inv, w)
        # 384 products, each rounded as in the module's bar: 2^-21 of at most |x| |w| (1.1 * sqrt 2)
        bar = 2.0 ** -20 * float(x.double().norm() * w.double().norm())
        assert abs(float((w.double() * apply(fwd, x)).sum() - (g * x.double()).sum())) <= bar
        # w itself is the tensor whose gradient passes through forward: central differences in x
        for at in ((0, 0, 1, 3), (0, 1, 4, 20), (0, 1, 5, 31)):
            e = torch.zeros_like(x)
            e[at] = 0.5
            quotient = float((w.double() * (apply(fwd, x + e) - apply(fwd, x - e))).sum())
            # two evaluations' rounding over the pair's two elements
            assert abs(quotient - float(g[at])) <= 2.0 ** -18 * float(w.abs().max() * (x.abs().max() + 1))


def test_start_null_and_empty():
    import decode_attention_rq_gb300 as rq
    cfg = config(rq)
    q = torch.randn((2, 3, 5, 128), device="cuda")
    y, z = torch.empty_like(q), torch.empty_like(q)
    rq.rq_rope(cfg, q, None, None, None, y)
    rq.rq_rope(cfg, q, None, torch.zeros(2, dtype=torch.int32, device="cuda"), None, z)
    torch.cuda.synchronize()
    assert torch.equal(y, z) and torch.equal(y[:, :, 0], q[:, :, 0])
    empty = torch.empty((2, 3, 0, 128), device="cuda")
    rq.rq_rope(cfg, empty, None, None)


def test_captured_on_a_stream_of_its_own():
    import decode_attention_rq_gb300 as rq
    cfg = config(rq)
    q = torch.randn((2, 4, 1, 128), device="cuda").to(torch.bfloat16)
    st = torch.tensor([5, 6], dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        rq.rq_rope(cfg, q, None, st, None, out)
    for s in (5, 900):
        st.fill_(s)
        graph.replay()
        torch.cuda.synchronize()
        close(out, *turned(rq, cfg, q.double().cpu().numpy(), positions([s, s], 1)), torch.bfloat16)


def test_refusals():
    import decode_attention_rq_gb300 as rq
    q = torch.zeros((1, 2, 3, 128), device="cuda")

    def fails(status, cfg, *a):
        with pytest.raises(rq.RqError) as e:
            rq.rq_rope(cfg, *a)
        assert e.value.status == status, e.value

    for bad in (dict(rotary_dim=0), dict(rotary_dim=3), dict(rotary_dim=130)):
        fails(6, config(rq, **bad), q, None, None)
    for bad in (dict(theta=1.0), dict(theta=float("nan")), dict(scaling=4), dict(scaling=1, factor=0.0),
                dict(scaling=3, low_turns=5.0, high_turns=5.0), dict(scaling=3, original_len=0),
                dict(scaling=2, rotary_dim=2), dict(magnitude=float("inf"))):
        fails(1, config(rq, **bad), q, None, None)
    cfg = config(rq)
    fails(1, cfg, None, None, None)
    fails(1, cfg, q.cpu(), None, None)
    fails(1, cfg, q[..., ::2], None, None)
    fails(1, cfg, q.double(), None, None)
    fails(1, cfg, q[:, :, :, :64], None, None)
    fails(1, cfg, q, q.to(torch.bfloat16), None)
    fails(1, cfg, q, q[:, :, :2], None)
    fails(1, cfg, q, None, torch.zeros(0, dtype=torch.int32, device="cuda"))
    fails(1, cfg, q, None, None, torch.zeros(2, dtype=torch.int32, device="cuda"))
