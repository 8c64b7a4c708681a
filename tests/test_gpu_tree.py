"""GPU: attention of drafted tokens (rq_tree_attention) against float64.

Bar: |gpu - float64| <= 2e-3 + 2^-8 |float64| + 2 * 2^-11 sum p |v|: the library's
bar for decode attention on O(1) data, half a BF16 step for the rounded result, and
the half steps of 11-bit operands in the value sum.  That sum is of products p v, with
p and v (the anchor's part c a of it) each rounded to 11 significant bits, half a step
or 2^-11 of the value: a product is off by at most 2 * 2^-11 of p |v| to first order.
Where channels are outliers (values of 8 to 30), few keys share the weight and the values
cancel, that exceeds 2e-3.  The residual's part R^T r, at most about 1, separates c a from
v by 2^-10, inside the 2e-3; queries are BF16 and so exact in 11 bits, only R q rounds:
a score moves by some 2^-11 |R q| |r| scale, 2e-4 at most.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from rq_harness import Case, GpuCache, kv_for, rotation32
from test_gpu_paged import PagedCache, _table

pytestmark = pytest.mark.gpu

ATOL, RTOL, VTOL = 2e-3, 2.0 ** -8, 2 * 2.0 ** -11
FILL = 7.0          # what output rows hold before the call


def tree_masks(seed, B, T, kind="tree"):
    """bool [B, T, T]: node t sees token j."""
    rng = np.random.default_rng(seed)
    see = np.zeros((B, T, T), dtype=bool)
    for b in range(B):
        for t in range(T):
            if kind == "any":
                see[b, t] = rng.random(T) < 0.5
                continue
            p = int(rng.integers(-1, t)) if t else -1
            if p >= 0:
                see[b, t] = see[b, p]
            see[b, t, t] = True
    return see


def mask_words(see):
    B, T, _ = see.shape
    words = -(-T // 64)
    bits = np.zeros((B, T, words * 64), dtype=np.uint64)
    bits[..., :T] = see
    w = (bits.reshape(B, T, words, 64) << np.arange(64, dtype=np.uint64)).sum(-1, dtype=np.uint64)
    return torch.from_numpy(w.view(np.int64).copy())


def bf16(rng, *shape):
    t = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16)
    return t, t.double().numpy()


class Ref:
    """Float64 results and, per element, sum p |v|."""

    def __init__(self, out, size):
        self.out, self.size = out, size

    def __getitem__(self, at):
        return Ref(self.out[at], self.size[at])


def reference(obuf, geom, R, case, layer, group, loop, q, kn, vn, see, counts, lens, scale):
    B, Hq, T, d = q.shape
    qpk = Hq // case.H
    out, size = np.full(q.shape, FILL), np.zeros(q.shape)
    for b in range(B):
        n, m = int(lens[b]), int(counts[b])
        for h in range(case.H):
            K, V = oracle.reconstruct(obuf, geom, R, layer, group, b, h, loop, n, case.chained)
            for hq in range(h * qpk, (h + 1) * qpk):
                for t in range(m):
                    vis = np.nonzero(see[b, t, :m])[0]
                    keys = np.concatenate([K, kn[b, h, vis]])
                    vals = np.concatenate([V, vn[b, h, vis]])
                    if len(keys) == 0:
                        out[b, hq, t] = 0.0
                        continue
                    s = keys @ q[b, hq, t] * scale
                    with np.errstate(invalid="ignore"):
                        p = np.exp(s - s.max())
                        out[b, hq, t] = (p / p.sum()) @ vals
                        size[b, hq, t] = (p / p.sum()) @ np.abs(vals)
    return Ref(out, size)


def call(gpu, layer, group, loop, q, kn, vn, mask, counts, lens, scale, out=None, ws=None):
    rq = gpu.rq
    B, Hq, T, d = q.shape
    if ws is None:
        size = rq.rq_tree_workspace_bytes(gpu.cfg, B, T)
        assert size > 0
        ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    if out is None:
        out = torch.full((B, Hq, T, d), FILL, dtype=torch.bfloat16, device="cuda")
    dev = [None if x is None else x.cuda().contiguous() for x in (q, kn, vn, mask)]
    cnt = None if counts is None else torch.tensor([int(c) for c in counts], dtype=torch.int32, device="cuda")
    sl = torch.tensor([int(n) for n in lens], dtype=torch.int32, device="cuda")
    rq.rq_tree_attention(gpu.handle, layer, group, loop, B, T, dev[0], dev[1], dev[2], dev[3], cnt, sl, scale, out,
                         ws, ws.numel())
    torch.cuda.synchronize()
    assert ws[:16].view(torch.int32).tolist() == [0, 0, 0, 0]
    return out


def filled(case, seed, ntok, paged=False, layer=0, group=0):
    R32, R = rotation32(case.d, kind=case.rotation)
    if paged:
        table, pages = _table(case, seed=seed)
        gpu = PagedCache(case, R32, table, pages)
    else:
        gpu = GpuCache(case, R32)
    geom = oracle.Geometry(case.L, case.P, case.G, case.H, case.d, case.g, case.B, case.Nmax)
    obuf = np.zeros(geom.total_bytes, dtype=np.uint8)
    kvb, kv = kv_for(case, seed, ntok, anchor_is_base=case.P == 4)
    gpu.append(layer, group, kvb, [0] * case.B)
    oracle.append(obuf, geom, R, layer, group, kv, np.zeros(case.B, dtype=np.int64), chained=case.chained,
                  rotation=case.rotation)
    return gpu, obuf, geom, R


def check(out, ref, what):
    got = out.double().cpu().numpy()
    err = np.abs(got - ref.out) - RTOL * np.abs(ref.out) - VTOL * ref.size
    worst = float(err.max())
    assert worst <= ATOL, f"{what}: {worst:.3e} beyond half a BF16 step"
    return worst


CASES = [
    # d, g, H, Hq, P, T, lens, counts, paged, chained, rotation, kind
    (128, 32, 2, 2, 4, 4, [200], None, False, False, "dense", "tree"),
    (128, 32, 2, 2, 4, 1, [256, 0, 65], None, False, False, "dense", "tree"),
    (128, 16, 3, 3, 4, 17, [300, 1, 128], [17, 1, 5], False, False, "dense", "tree"),
    (96, 32, 5, 5, 4, 25, [190, 64], [25, 9], True, False, "dense", "any"),
    (96, 16, 2, 4, 4, 33, [63, 129], None, False, False, "dense", "tree"),
    (128, 32, 2, 8, 4, 13, [250, 130], [13, 0], True, False, "dense", "tree"),
    (128, 32, 1, 4, 4, 64, [127, 255], None, False, False, "hadamard", "tree"),
    (128, 32, 1, 1, 4, 65, [100], None, False, False, "dense", "any"),
    (128, 16, 1, 2, 4, 130, [70, 5], [130, 77], True, False, "hadamard", "tree"),
    (128, 32, 1, 1, 4, 256, [300], None, False, False, "dense", "tree"),
    (128, 32, 2, 2, 4, 9, [200, 30], None, False, True, "dense", "tree"),
    (96, 32, 1, 2, 8, 6, [150], None, True, True, "dense", "any"),
    (128, 32, 1, 3, 2, 21, [90, 64], None, False, False, "dense", "tree"),
    (96, 32, 1, 1, 1, 12, [77], None, False, False, "dense", "tree"),
]


@pytest.mark.parametrize("d,g,H,Hq,P,T,lens,counts,paged,chained,rotation,kind", CASES)
def test_tree_matches_float64(d, g, H, Hq, P, T, lens, counts, paged, chained, rotation, kind):
    B = len(lens)
    case = Case(L=1, P=P, G=1, H=H, d=d, g=g, B=B, Nmax=max(max(lens), 1) + 30, chained=chained, rotation=rotation,
                Hq=Hq)
    gpu, obuf, geom, R = filled(case, 40 + T, max(max(lens), 1), paged)
    rng = np.random.default_rng(T)
    see = tree_masks(T, B, T, kind)
    cnt = counts or [T] * B
    scale = 1 / math.sqrt(d)
    for loop in range(P):
        qb, q = bf16(rng, B, Hq, T, d)
        kb, kn = bf16(rng, B, H, T, d)
        vb, vn = bf16(rng, B, H, T, d)
        out = call(gpu, 0, 0, loop, qb, kb, vb, mask_words(see), counts, lens, scale)
        ref = reference(obuf, geom, R, case, 0, 0, loop, q, kn, vn, see, cnt, lens, scale)
        worst = check(out, ref, f"loop {loop}")
        for b in range(B):       # rows behind the node count are left as they were
            assert (out[b, :, cnt[b]:] == FILL).all()
        print(f"loop {loop}: {worst:.2e}")
    gpu.close()


def test_single_token_agrees_with_the_decode_call_and_null_mask_is_a_sequence():
    case = Case(L=1, P=4, G=1, H=4, d=128, g=32, B=3, Nmax=512)
    gpu, obuf, geom, R = filled(case, 5, 500)
    rng = np.random.default_rng(0)
    lens, scale = [500, 77, 0], 1 / math.sqrt(128)
    for loop in (0, 3):
        qb, _ = bf16(rng, 3, 4, 1, 128)
        kb, _ = bf16(rng, 3, 4, 1, 128)
        vb, _ = bf16(rng, 3, 4, 1, 128)
        one = gpu.decode(0, 0, loop, qb[:, :, 0], kb[:, :, 0], vb[:, :, 0], lens, scale)
        out = call(gpu, 0, 0, loop, qb, kb, vb, None, None, lens, scale)
        ref = reference(obuf, geom, R, case, 0, 0, loop, qb.double().numpy(), kb.double().numpy(),
                        vb.double().numpy(), np.ones((3, 1, 1), dtype=bool), [1] * 3, lens, scale)
        check(out, ref, f"loop {loop}")
        check(out, Ref(one.double().cpu().numpy()[:, :, None], ref.size), f"loop {loop}, decode call")
    T = 70
    qb, q = bf16(rng, 3, 4, T, 128)
    kb, kn = bf16(rng, 3, 4, T, 128)
    vb, vn = bf16(rng, 3, 4, T, 128)
    see = np.tril(np.ones((3, T, T), dtype=bool))
    out = call(gpu, 0, 0, 1, qb, kb, vb, None, [T, 66, 3], lens, scale)
    ref = reference(obuf, geom, R, case, 0, 0, 1, q, kn, vn, see, [T, 66, 3], lens, scale)
    check(out, ref, "sequence")
    gpu.close()


def test_rows_without_a_key_are_zero_and_hidden_values_may_be_anything():
    """A node with an empty mask on an empty row gives zero; infinities and NaN in
    hidden nodes and behind the node count enter no other result."""
    case = Case(L=1, P=4, G=1, H=2, d=128, g=32, B=2, Nmax=256, Hq=4)
    gpu, obuf, geom, R = filled(case, 6, 200)
    rng = np.random.default_rng(1)
    T, lens, counts, scale = 12, [0, 150], [10, 9], 1 / math.sqrt(128)
    see = tree_masks(3, 2, T)
    see[:, :, 4] = False
    see[:, 4, 4] = True                   # node 4 is seen by itself alone
    see[0, 7] = False                     # row 0 has no cache: nothing at all
    qb, q = bf16(rng, 2, 4, T, 128)
    kb, kn = bf16(rng, 2, 2, T, 128)
    vb, vn = bf16(rng, 2, 2, T, 128)
    ref = reference(obuf, geom, R, case, 0, 0, 2, q, kn, vn, see, counts, lens, scale)
    kb[:, :, 4], vb[:, :, 4] = float("nan"), float("inf")
    kb[:, :, 10:], vb[:, :, 10:], qb[:, :, 10:] = float("inf"), float("nan"), float("nan")
    kb[1, :, 9], vb[1, :, 9] = float("nan"), float("nan")
    out = call(gpu, 0, 0, 2, qb, kb, vb, mask_words(see), counts, lens, scale)
    assert (out[0, :, 7] == 0).all()
    assert not torch.isfinite(out[:, :, 4]).any()
    keep = [t for t in range(T) if t != 4]
    check(out[:, :, keep], ref[:, :, keep], "hidden infinities")
    gpu.close()


@pytest.mark.parametrize("gain", [8.0, 64.0, 1e-3])
def test_peaky_and_flat_softmax(gain):
    """Queries far from O(1): nearly all weight on one key, or none preferred; one
    query is a cached key, so the running maximum moves late in the row."""
    case = Case(L=1, P=4, G=1, H=1, d=128, g=32, B=1, Nmax=1024)
    gpu, obuf, geom, R = filled(case, 9, 1000)
    rng = np.random.default_rng(2)
    T, scale = 8, 1 / math.sqrt(128)
    K, _ = oracle.reconstruct(obuf, geom, R, 0, 0, 0, 0, 1, 1000)
    q = rng.standard_normal((1, 1, T, 128)) * gain
    q[0, 0, 3] = K[990] * min(gain, 1.0)
    qb = torch.from_numpy(q.astype(np.float32)).to(torch.bfloat16)
    kb, kn = bf16(rng, 1, 1, T, 128)
    vb, vn = bf16(rng, 1, 1, T, 128)
    see = tree_masks(8, 1, T)
    out = call(gpu, 0, 0, 1, qb, kb, vb, mask_words(see), None, [1000], scale)
    ref = reference(obuf, geom, R, case, 0, 0, 1, qb.double().numpy(), kn, vn, see, [T], [1000], scale)
    got = out.double().cpu().numpy()
    # 11-bit operands move a score by about 2^-11 sqrt(sum (q_i k_i)^2) scale, six deviations taken
    # over 1000 keys; a weight moves by as much, the result by that times the spread of V (about 9)
    move = 6 * 2.0 ** -11 * scale * math.sqrt(2) * np.sqrt((qb.double().numpy()[0, 0][:, None] ** 2 * K[None] ** 2).sum(-1)).max()
    tol = max(ATOL, 9 * move)
    off = np.abs(got - ref.out)
    assert (off <= tol + RTOL * np.abs(ref.out) + VTOL * ref.size).all(), off.max()
    gpu.close()


def test_layers_groups_and_larger_batch():
    case = Case(L=2, P=4, G=2, H=2, d=128, g=32, B=5, Nmax=320)
    lens, T, scale = [300, 0, 64, 129, 257], 10, 1 / math.sqrt(128)
    gpu, obuf, geom, R = filled(case, 12, 300, layer=1, group=1)
    rng = np.random.default_rng(4)
    qb, q = bf16(rng, 5, 2, T, 128)
    kb, kn = bf16(rng, 5, 2, T, 128)
    vb, vn = bf16(rng, 5, 2, T, 128)
    see = tree_masks(2, 5, T)
    out = call(gpu, 1, 1, 0, qb, kb, vb, mask_words(see), None, lens, scale)
    check(out, reference(obuf, geom, R, case, 1, 1, 0, q, kn, vn, see, [T] * 5, lens, scale), "layer 1, group 1")
    gpu.close()


def test_captured_and_replayed_on_another_stream():
    """The call in a captured graph, replayed with new inputs, and on a stream of its own."""
    case = Case(L=1, P=4, G=1, H=4, d=128, g=32, B=2, Nmax=512)
    gpu, obuf, geom, R = filled(case, 15, 400)
    rq, T, scale, lens = gpu.rq, 16, 1 / math.sqrt(128), [400, 210]
    rng = np.random.default_rng(6)
    see = tree_masks(5, 2, T)
    mask, sl = mask_words(see).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    q, k, v = (bf16(rng, 2, 4, T, 128)[0].cuda() for _ in range(3))
    out = torch.zeros((2, 4, T, 128), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(rq.rq_tree_workspace_bytes(gpu.cfg, 2, T), dtype=torch.uint8, device="cuda")

    def go():
        rq.rq_tree_attention(gpu.handle, 0, 0, 1, 2, T, q, k, v, mask, None, sl, scale, out, ws, ws.numel())

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go()
    torch.cuda.synchronize()
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for rep in range(3):
        out.zero_()
        if rep:
            q.copy_(bf16(rng, 2, 4, T, 128)[0])
        graph.replay()
        torch.cuda.synchronize()
        if rep == 0:
            assert torch.equal(out, first)
        ref = reference(obuf, geom, R, case, 0, 0, 1, q.double().cpu().numpy(), k.double().cpu().numpy(),
                        v.double().cpu().numpy(), see, [T, T], lens, scale)
        check(out, ref, f"replay {rep}")
    assert ws[:16].view(torch.int32).tolist() == [0, 0, 0, 0]
    gpu.close()


def test_bad_page_is_flagged_not_followed():
    case = Case(L=1, P=4, G=1, H=2, d=128, g=32, B=1, Nmax=256)
    R32, R = rotation32(128)
    table, pages = _table(case, seed=1)
    gpu = PagedCache(case, R32, table, pages)
    kvb, _ = kv_for(case, 3, 200)
    gpu.append(0, 0, kvb, [0])
    gpu.table[0, 1] = pages + 9
    gpu.table[0, 2] = -1
    rng = np.random.default_rng(0)
    T = 5
    q, k, v = (bf16(rng, 1, 2, T, 128)[0].cuda() for _ in range(3))
    out = torch.zeros((1, 2, T, 128), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(gpu.rq.rq_tree_workspace_bytes(gpu.cfg, 1, T), dtype=torch.uint8, device="cuda")
    sl = torch.tensor([200], dtype=torch.int32, device="cuda")
    gpu.rq.rq_tree_attention(gpu.handle, 0, 0, 0, 1, T, q, k, v, None, None, sl, 0.09, out, ws, ws.numel())
    torch.cuda.synchronize()
    assert ws[:16].view(torch.int32).tolist() == [0, 0, 1, 0]
    assert torch.isfinite(out.float()).all()
    gpu.close()
