"""GPU: norm of every head with the rotation (rq_norm_rope, rq_norm_rope_backward) against float64.

Bars.  rstd = 1 / sqrt(mean x^2 + eps): the squares are summed by up to 32 fused additions in a lane and 5 across lanes,
at most 37 * 2^-24 relative, half of which reaches rstd, with the two roundings of the mean and rsqrt's two units:
less than 2^-19.  Forward: y = rstd (a w_a cos -+ b w_b sin), cos and sin within 2^-22 (test_gpu_rope), four
roundings: |gpu - float64| <= step |y| + rstd m (|a w_a| + |b w_b|) 2^-18, step half a unit of the type.  FP16 values below
the normal range add half their step, 2^-25.  Backward: the same of t = w Rot^T g with its sum of up to 37 products, so
|gpu - float64| <= step |dx| + rstd (s + |x^| mean(s |x^|)) 2^-18, s = |w| m (|g_a| + |g_b|); a weight's gradient is a
float32 sum of M terms in some order, each within 2^-18: (2^-18 + M 2^-24) sum m (|g_a| + |g_b|) |x^|."""
import numpy as np
import pytest
import torch

from test_gpu_rope import STEP, angles, config, positions

pytestmark = pytest.mark.gpu
BF, HF, F = torch.bfloat16, torch.float16, torch.float32


def spin(rq, cfg, x, pos, back=False):
    """Rot x (back: Rot^T x) and |a| + |b| of each element's pair times the magnitude, float64."""
    r = cfg.rotary_dim
    ang, mag = angles(rq, cfg, pos)
    c, s = mag * np.cos(ang)[:, None], mag * np.sin(ang)[:, None]
    if back:
        s = -s
    i, j = (slice(0, r, 2), slice(1, r, 2)) if cfg.interleaved else (slice(0, r // 2), slice(r // 2, r))
    y, size = x.copy(), np.abs(x)
    a, b = x[..., i], x[..., j]
    y[..., i], y[..., j] = a * c - b * s, b * c + a * s
    size[..., i] = size[..., j] = mag * (np.abs(a) + np.abs(b))
    return y, size


def forward(rq, cfg, x, w, eps, pos):
    rstd = 1 / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    y, size = spin(rq, cfg, x * rstd * w, pos)
    return y, size


def backward(rq, cfg, x, w, eps, pos, g):
    """dx, dw and the sizes of their bars."""
    rstd = 1 / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    z = x * rstd
    h, size = spin(rq, cfg, g, pos, back=True)
    t, s = h * w, size * np.abs(w)
    dx = rstd * (t - z * (t * z).mean(-1, keepdims=True))
    bar = rstd * (s + np.abs(z) * (s * np.abs(z)).mean(-1, keepdims=True))
    return dx, (h * z).sum((0, 1, 2)), bar, (size * np.abs(z)).sum((0, 1, 2))


def close(got, ref, bar, dtype, label=""):
    err = np.abs(got.double().cpu().numpy() - ref)
    tol = STEP[dtype] * np.abs(ref) + bar + (2.0 ** -25 if dtype == HF else 0.0)
    assert (err <= tol).all(), f"{label} {(err - tol).max():.3e} beyond the bar"


CASES = [
    # dtype, weight dtype, d, r, inter, inverse, scaling, B, Hq, H, n, start, offsets
    (BF, BF, 128, 128, 0, 0, 0, 4, 16, 16, 1, [0, 77, 8191, 16383], False),
    (BF, F, 128, 128, 0, 0, 3, 2, 8, 2, 300, [0, 50000], False),
    (F, F, 96, 64, 1, 0, 1, 2, 5, 5, 61, [100000, 3], False),
    (HF, HF, 96, 96, 0, 0, 2, 3, 3, 1, 17, [1, 2, 3], True),
    (HF, BF, 64, 64, 1, 1, 0, 2, 7, 3, 33, [1, 2], True),
    (F, BF, 64, 64, 0, 0, 0, 1, 2, 1, 9, [2147483600], False),
    (BF, BF, 256, 128, 1, 0, 0, 2, 3, 2, 21, [5, 6], False),
    (BF, F, 512, 256, 0, 0, 0, 1, 2, 1, 19, [9], False),
    (F, F, 512, 256, 0, 1, 1, 1, 2, 1, 12, [44], False),
    (F, F, 512, 64, 1, 0, 0, 1, 1, 2, 5, [4], False),
    (BF, BF, 120, 16, 0, 0, 0, 2, 2, 2, 13, [5, 9], False),      # an odd number of pieces
    # off 16-byte boundaries in r, d or both
    (BF, F, 64, 58, 0, 0, 0, 2, 4, 2, 65, [5, 900], False),
    (F, F, 128, 122, 0, 0, 3, 1, 2, 2, 33, [1000000], False),
    (HF, F, 256, 58, 1, 0, 0, 2, 2, 1, 30, [5, 9], True),
    (F, HF, 7, 6, 1, 0, 0, 2, 3, 1, 5, [5, 9], False),
    (BF, BF, 2, 2, 0, 0, 0, 1, 1, 1, 130, [0], False),
    (BF, F, 511, 254, 0, 0, 0, 1, 2, 1, 7, [3], False),
    (F, F, 511, 256, 1, 0, 0, 1, 1, 1, 6, [3], False),
    (HF, F, 80, 20, 0, 0, 0, 2, 2, 2, 40, [44, 0], False),
    (F, F, 33, 2, 0, 0, 0, 1, 2, 3, 4, [8], False),
]


def inputs(case, seed=0):
    dtype, wt, d, r, inter, inverse, scaling, B, Hq, H, n, start, tree = case
    import decode_attention_rq_gb300 as rq
    cfg = config(rq, head_dim=d, rotary_dim=r, interleaved=inter, inverse=inverse, scaling=scaling,
                 magnitude=1.25 if scaling == 3 else 0.0)
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((B, n, Hq + H, d), generator=gen)
    x[..., d // 3] *= 8
    x = x.to(dtype)
    w = (1 + 0.3 * torch.randn((2, d), generator=gen)).to(wt)
    g = torch.randn((B, n, Hq + H, d), generator=gen).to(dtype)
    offs = torch.randint(0, 30, (B, n), generator=gen, dtype=torch.int32) if tree else None
    pos = positions(start, n, None if offs is None else offs.numpy())
    return rq, cfg, x, w, g, offs, pos


def heads(x, a, b):
    return x[:, :, a:b].transpose(1, 2)


def f64(x):
    return x.double().cpu().numpy()


@pytest.mark.parametrize("layout", ["views", "contiguous", "in place"])
@pytest.mark.parametrize("case", CASES, ids=[f"{i}" for i in range(len(CASES))])
def test_forward(case, layout):
    rq, cfg, x, w, _, offs, pos = inputs(case)
    Hq, eps = case[8], 1e-6
    dev = x.cuda()
    q, k = heads(dev, 0, Hq), heads(dev, Hq, None)
    if layout == "contiguous":
        q, k = q.contiguous(), k.contiguous()
    qo, ko = (None, None) if layout == "in place" else (torch.full_like(q.contiguous(), 99), torch.full_like(k.contiguous(), 99))
    qref, kref = (forward(rq, cfg, f64(z), f64(v), eps, pos) for z, v in ((q, w[0]), (k, w[1])))
    start = torch.tensor(case[11], dtype=torch.int32).cuda()
    rq.rq_norm_rope(cfg, q, k, w[0].cuda(), w[1].cuda(), eps, start, None if offs is None else offs.cuda(), qo, ko)
    for got, (ref, size) in ((q if qo is None else qo, qref), (k if ko is None else ko, kref)):
        close(got, ref, size * 2.0 ** -18, case[0])


@pytest.mark.parametrize("layout", ["views", "over x", "over the gradient"])
@pytest.mark.parametrize("case", CASES, ids=[f"{i}" for i in range(len(CASES))])
def test_backward(case, layout):
    rq, cfg, x, w, g, offs, pos = inputs(case, 1)
    dtype, Hq, eps = case[0], case[8], 1e-5
    B, n = case[7], case[10]
    dev, dg = x.cuda(), g.cuda()
    q, k, qg, kg = heads(dev, 0, Hq), heads(dev, Hq, None), heads(dg, 0, Hq), heads(dg, Hq, None)
    refs = [backward(rq, cfg, f64(z), f64(v), eps, pos, f64(y)) for z, v, y in ((q, w[0], qg), (k, w[1], kg))]
    qo, ko = {"views": (torch.full_like(q.contiguous(), 99), torch.full_like(k.contiguous(), 99)), "over x": (None, None),
              "over the gradient": (qg, kg)}[layout]
    d = case[2]
    dw = torch.full((2, d), 7.0, device="cuda")
    ws = torch.full((rq.rq_norm_rope_workspace_bytes(d),), 255, dtype=torch.uint8, device="cuda")
    start = torch.tensor(case[11], dtype=torch.int32).cuda()
    rq.rq_norm_rope_backward(cfg, q, k, qg, kg, w[0].cuda(), w[1].cuda(), eps, start,
                             None if offs is None else offs.cuda(), qo, ko, dw[0], dw[1], ws, ws.numel())
    for got, gw, nh, (dx, dwr, bar, wbar) in ((q if qo is None else qo, dw[0], Hq, refs[0]),
                                              (k if ko is None else ko, dw[1], case[9], refs[1])):
        close(got, dx, bar * 2.0 ** -18, dtype, "dx")
        close(gw, dwr, wbar * (2.0 ** -18 + B * n * nh * 2.0 ** -24), F, "dw")


def test_one_tensor_no_weights():
    """Only k, no weights, no weight gradients (no workspace), then only q with its weight's gradient alone."""
    rq, cfg, x, w, g, _, pos = inputs(CASES[1])
    start = torch.tensor(CASES[1][11], dtype=torch.int32).cuda()
    z, gr = x[:, :, :3].transpose(1, 2).cuda(), g[:, :, :3].transpose(1, 2).cuda()
    out = torch.empty_like(z.contiguous())
    rq.rq_norm_rope(cfg, None, z, None, None, 1e-6, start, None, None, out)
    ref, size = forward(rq, cfg, f64(z), 1.0, 1e-6, pos)
    close(out, ref, size * 2.0 ** -18, BF)
    rq.rq_norm_rope_backward(cfg, None, z, None, gr, None, None, 1e-6, start, None, None, out, None, None, None, 0)
    dx, dwr, bar, wbar = backward(rq, cfg, f64(z), np.ones(128), 1e-6, pos, f64(gr))
    close(out, dx, bar * 2.0 ** -18, BF)
    dw = torch.full((128,), 7.0, device="cuda")
    ws = torch.empty(rq.rq_norm_rope_workspace_bytes(128), dtype=torch.uint8, device="cuda")
    rq.rq_norm_rope_backward(cfg, z, None, gr, None, None, None, 1e-6, start, None, out, None, dw, None, ws, ws.numel())
    close(dw, dwr, wbar * (2.0 ** -18 + 1800 * 2.0 ** -24), F)
    close(out, dx, bar * 2.0 ** -18, BF)


def test_gradient_against_differences():
    """The loss sum y g along random directions of x and w: central differences of the float64 formula.  Their error is the
    third derivative's, about 1e-10 of the sums here; the kernel's that of test_backward."""
    for case in (CASES[2], CASES[12]):
        rq, cfg, x, w, g, _, pos = inputs(case, 3)
        start = torch.tensor(case[11], dtype=torch.int32).cuda()
        z, gr = x[:, :, :2].transpose(1, 2).contiguous(), g[:, :, :2].transpose(1, 2).contiguous()
        rng = np.random.default_rng(0)
        vx, vw = rng.standard_normal(z.shape), rng.standard_normal(case[2])
        X, W, G, e = f64(z), f64(w[0]), f64(gr), 1e-5
        loss = lambda a: (forward(rq, cfg, X + a * vx, W + a * vw, 1e-5, pos)[0] * G).sum()
        want = (loss(e) - loss(-e)) / (2 * e)
        dw = torch.empty(case[2], device="cuda")
        ws = torch.empty(rq.rq_norm_rope_workspace_bytes(case[2]), dtype=torch.uint8, device="cuda")
        dx = torch.empty_like(z, device="cuda")
        rq.rq_norm_rope_backward(cfg, z.cuda(), None, gr.cuda(), None, w[0].cuda(), None, 1e-5, start, None, dx, None,
                                 dw, None, ws, ws.numel())
        got = (f64(dx) * vx).sum() + (f64(dw) * vw).sum()
        _, _, bar, wbar = backward(rq, cfg, X, W, 1e-5, pos, G)
        scale = (bar * np.abs(vx)).sum() + (wbar * np.abs(vw)).sum()
        assert abs(got - want) <= scale * 2.0 ** -17


def test_repeats_and_graphs_give_equal_bits():
    """Two graphs of the backward pass with a workspace each, replayed in turn and beside an eager call."""
    rq, cfg, x, w, g, _, _ = inputs(CASES[1], 5)
    start = torch.tensor(CASES[1][11], dtype=torch.int32).cuda()
    q, qg, wq = x[:, :, :8].transpose(1, 2).cuda(), g[:, :, :8].transpose(1, 2).cuda(), w[0].cuda()
    sets = []
    for _ in range(3):
        sets.append((torch.empty_like(q.contiguous()), torch.empty(128, device="cuda"),
                     torch.empty(rq.rq_norm_rope_workspace_bytes(128), dtype=torch.uint8, device="cuda")))

    def call(s):
        rq.rq_norm_rope_backward(cfg, q, None, qg, None, wq, None, 1e-6, start, None, s[0], None, s[1], None, s[2],
                                 s[2].numel())

    call(sets[0])
    torch.cuda.synchronize()
    graphs = []
    for s in sets[1:]:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(s)
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        call(sets[0])
    torch.cuda.synchronize()
    for s in sets[1:]:
        assert torch.equal(s[0], sets[0][0]) and torch.equal(s[1], sets[0][1])


def test_empty_and_degenerate():
    """No tokens: zero weight gradients, nothing else written.  A vector of zeros: zeros for eps > 0; its gradient is
    w Rot^T g / sqrt(eps).  An infinity or NaN stays in its own head."""
    import decode_attention_rq_gb300 as rq
    cfg = config(rq)
    ws = torch.empty(rq.rq_norm_rope_workspace_bytes(128), dtype=torch.uint8, device="cuda")
    start = torch.zeros(2, dtype=torch.int32, device="cuda")
    none = torch.empty((2, 4, 0, 128), dtype=BF, device="cuda")
    dw = torch.full((128,), 7.0, device="cuda")
    rq.rq_norm_rope(cfg, none, None, None, None, 1e-6, start)
    rq.rq_norm_rope_backward(cfg, none, None, none, None, None, None, 1e-6, start, None, None, None, dw, None, ws, ws.numel())
    assert bool((dw == 0).all())
    x = torch.zeros((2, 4, 3, 128), device="cuda")
    g = torch.randn_like(x)
    y, dx = torch.full_like(x, 9), torch.empty_like(x)
    rq.rq_norm_rope(cfg, x, None, None, None, 0.25, start, None, y)
    assert bool((y == 0).all())
    rq.rq_norm_rope_backward(cfg, x, None, g, None, None, None, 0.25, start, None, dx, None, dw, None, ws, ws.numel())
    ref, size = spin(rq, cfg, f64(g), positions([0, 0], 3), back=True)
    close(dx, 2 * ref, 2 * size * 2.0 ** -18, F)
    assert bool((dw == 0).all())
    for bad in (float("inf"), float("nan")):
        for r in (128, 58):
            c = config(rq, rotary_dim=r)
            z = torch.randn((2, 4, 3, 128), device="cuda")
            keep = torch.empty_like(z)
            rq.rq_norm_rope(c, z, None, None, None, 1e-6, start, None, keep)
            z[1, 2, 1, 100] = bad
            rq.rq_norm_rope(c, z, None, None, None, 1e-6, start, None, y)
            hit = torch.zeros((2, 4, 3), dtype=torch.bool, device="cuda")
            hit[1, 2, 1] = True
            assert torch.equal(y[~hit], keep[~hit]) and bool(torch.isnan(y[1, 2, 1]).any())


def test_gradient_of_a_broadcast_tensor():
    """A gradient whose strides are zero (the sum's), and inputs of a broadcast row."""
    rq, cfg, x, w, _, _, pos = inputs(CASES[1], 8)
    start = torch.tensor(CASES[1][11], dtype=torch.int32).cuda()
    q = x[:1, :, :4].transpose(1, 2).cuda().expand(2, 4, 300, 128)
    g = torch.randn(128, device="cuda").to(BF).expand(2, 4, 300, 128)
    out, dw = torch.empty((2, 4, 300, 128), dtype=BF, device="cuda"), torch.empty(128, device="cuda")
    ws = torch.empty(rq.rq_norm_rope_workspace_bytes(128), dtype=torch.uint8, device="cuda")
    rq.rq_norm_rope_backward(cfg, q, None, g, None, w[0].cuda(), None, 1e-6, start, None, out, None, dw, None, ws, ws.numel())
    dx, dwr, bar, wbar = backward(rq, cfg, f64(q), f64(w[0]), 1e-6, pos, f64(g))
    close(out, dx, bar * 2.0 ** -18, BF)
    close(dw, dwr, wbar * (2.0 ** -18 + 2400 * 2.0 ** -24), F)
    with pytest.raises(rq.RqError):      # its own place for the result has two results in one
        rq.rq_norm_rope(cfg, q, None, None, None, 1e-6, start)


def test_other_stream():
    rq, cfg, x, w, _, _, pos = inputs(CASES[0])
    start = torch.tensor(CASES[0][11], dtype=torch.int32).cuda()
    q, wq = x[:, :, :16].transpose(1, 2).cuda(), w[0].cuda()
    out = torch.zeros_like(q.contiguous())
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    rq.rq_norm_rope(cfg, q, None, wq, None, 1e-6, start, None, out, stream=s)
    s.synchronize()
    ref, size = forward(rq, cfg, f64(q), f64(w[0]), 1e-6, pos)
    close(out, ref, size * 2.0 ** -18, BF)


@pytest.mark.parametrize("inter", [0, 1])
@pytest.mark.parametrize("dtype", [BF, HF, F])
def test_widths_and_rotated_parts(dtype, inter):
    """Every way in which a head can be split into rotated, other and no channels of a group of lanes."""
    for d in (16, 24, 32, 40, 48, 56, 64, 72, 80, 88, 96, 104, 112, 120, 128, 136, 160, 192, 200, 256, 264, 320, 384, 504, 512):
        for r in sorted({min(d, 256) - (min(d, 256) - x) % 2 for x in (2, 8, 16, 24, 32, 48, 64, 96, 128, 192, 256, d, d - 2)
                         if x <= d}):
            case = (dtype, F, d, r, inter, 0, 0, 1, 2, 1, 5, [d + r], False)
            rq, cfg, x, w, g, _, pos = inputs(case, d + r)
            start, ws = torch.tensor([d + r], dtype=torch.int32).cuda(), torch.empty(
                rq.rq_norm_rope_workspace_bytes(d), dtype=torch.uint8, device="cuda")
            q, k, qg, kg = (heads(z.cuda(), a, b) for z in (x, g) for a, b in ((0, 2), (2, 3)))
            qo, ko = torch.full_like(q.contiguous(), 99), torch.full_like(k.contiguous(), 99)
            wq, wk, dw = w[0].cuda(), w[1].cuda(), torch.full((2, d), 7.0, device="cuda")
            rq.rq_norm_rope(cfg, q, k, wq, wk, 1e-5, start, None, qo, ko)
            for got, z, v in ((qo, q, w[0]), (ko, k, w[1])):
                ref, size = forward(rq, cfg, f64(z), f64(v), 1e-5, pos)
                close(got, ref, size * 2.0 ** -18, dtype, f"{d} {r}")
            rq.rq_norm_rope_backward(cfg, q, k, qg, kg, wq, wk, 1e-5, start, None, qo, ko, dw[0], dw[1], ws, ws.numel())
            for got, gw, z, v, y, nh in ((qo, dw[0], q, w[0], qg, 2), (ko, dw[1], k, w[1], kg, 1)):
                dx, dwr, bar, wbar = backward(rq, cfg, f64(z), f64(v), 1e-5, pos, f64(y))
                close(got, dx, bar * 2.0 ** -18, dtype, f"dx {d} {r}")
                close(gw, dwr, wbar * (2.0 ** -18 + 5 * nh * 2.0 ** -24), F, f"dw {d} {r}")


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("d,r", [(128, 64), (128, 58), (256, 128), (512, 256), (511, 254)])
@pytest.mark.parametrize("top,eps", [(2.0 ** 60, 1e-6), (2.0 ** -50, 0.0)])
def test_ends_of_the_range(dtype, d, r, top, eps):
    """Magnitudes up to 2^60, every channel there in one head; with eps = 0 down to vectors whose largest is 2^-50."""
    case = (dtype, F, d, r, 0, 0, 0, 1, 3, 1, 5, [9], False)
    rq, cfg, x, w, g, _, pos = inputs(case, d)
    x = (x.float().sign() * top * (0.5 + 0.5 * torch.rand(x.shape, generator=torch.Generator().manual_seed(d)))).to(dtype)
    x[:, :, 0] = top
    x[:, :, 1, 1:] = 0                               # one channel alone
    x[:, :, 1, 0] = top
    start, dev, dg, wd = torch.tensor([9], dtype=torch.int32).cuda(), x.cuda(), g.cuda(), [v.cuda() for v in w]
    q, k, qg, kg = heads(dev, 0, 3), heads(dev, 3, None), heads(dg, 0, 3), heads(dg, 3, None)
    out = torch.full_like(dev, 99)
    rq.rq_norm_rope(cfg, q, k, *wd, eps, start, None, heads(out, 0, 3), heads(out, 3, None))
    for got, z, v in ((heads(out, 0, 3), q, w[0]), (heads(out, 3, None), k, w[1])):
        ref, size = forward(rq, cfg, f64(z), f64(v), eps, pos)
        close(got, ref, size * 2.0 ** -18, dtype)
    dw, ws = torch.full((2, d), 7.0, device="cuda"), torch.empty(rq.rq_norm_rope_workspace_bytes(d), dtype=torch.uint8,
                                                                 device="cuda")
    rq.rq_norm_rope_backward(cfg, q, k, qg, kg, *wd, eps, start, None, heads(out, 0, 3), heads(out, 3, None), dw[0], dw[1],
                             ws, ws.numel())
    for got, gw, nh, z, v, y in ((heads(out, 0, 3), dw[0], 3, q, w[0], qg), (heads(out, 3, None), dw[1], 1, k, w[1], kg)):
        dx, dwr, bar, wbar = backward(rq, cfg, f64(z), f64(v), eps, pos, f64(y))
        close(got, dx, bar * 2.0 ** -18, dtype, "dx")
        close(gw, dwr, wbar * (2.0 ** -18 + 5 * nh * 2.0 ** -24), F, "dw")


LONG = [
    # as CASES: several items a CTA, across tokens, their number no multiple of the grid's
    (BF, F, 128, 128, 0, 0, 0, 2, 5, 2, 4099, [0, 50000], False),
    (HF, HF, 96, 64, 1, 0, 0, 2, 3, 2, 3001, [7, 1], True),
    (F, F, 512, 256, 0, 0, 0, 2, 3, 1, 701, [9, 5], False),          # two slots a lane
    (BF, F, 128, 58, 0, 0, 0, 2, 5, 2, 2501, [5, 900], False),       # the kernel for any alignment
    (F, BF, 511, 254, 0, 0, 0, 2, 3, 1, 601, [3, 4], False),
]


@pytest.mark.parametrize("case", LONG, ids=[f"{i}" for i in range(len(LONG))])
def test_prompts(case):
    """Forward into another tensor and in place, backward over the inputs: a CTA walks along heads and from token to token."""
    rq, cfg, x, w, g, offs, pos = inputs(case, 11)
    dtype, d, B, Hq, H, n = case[0], case[2], case[7], case[8], case[9], case[10]
    start, offs = torch.tensor(case[11], dtype=torch.int32).cuda(), None if offs is None else offs.cuda()
    dev, dg, wd = x.cuda(), g.cuda(), [v.cuda() for v in w]
    q, k, qg, kg = heads(dev, 0, Hq), heads(dev, Hq, None), heads(dg, 0, Hq), heads(dg, Hq, None)
    refs = [forward(rq, cfg, f64(z), f64(v), 1e-6, pos) for z, v in ((q, w[0]), (k, w[1]))]
    back = [backward(rq, cfg, f64(z), f64(v), 1e-6, pos, f64(y)) for z, v, y in ((q, w[0], qg), (k, w[1], kg))]
    out = torch.full_like(dev, 99)
    rq.rq_norm_rope(cfg, q, k, *wd, 1e-6, start, offs, heads(out, 0, Hq), heads(out, Hq, None))
    same = dev.clone()
    rq.rq_norm_rope(cfg, heads(same, 0, Hq), heads(same, Hq, None), *wd, 1e-6, start, offs)
    assert torch.equal(out, same)
    for got, (ref, size) in zip((heads(out, 0, Hq), heads(out, Hq, None)), refs):
        close(got, ref, size * 2.0 ** -18, dtype)
    dw, ws = torch.full((2, d), 7.0, device="cuda"), torch.empty(rq.rq_norm_rope_workspace_bytes(d), dtype=torch.uint8,
                                                                 device="cuda")
    rq.rq_norm_rope_backward(cfg, q, k, qg, kg, *wd, 1e-6, start, offs, None, None, dw[0], dw[1], ws, ws.numel())
    for got, gw, nh, (dx, dwr, bar, wbar) in ((q, dw[0], Hq, back[0]), (k, dw[1], H, back[1])):
        close(got, dx, bar * 2.0 ** -18, dtype, "dx")
        close(gw, dwr, wbar * (2.0 ** -18 + B * n * nh * 2.0 ** -24), F, "dw")
