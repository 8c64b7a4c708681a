"""GPU: tree attention, page operations and rotary positions at their limits -- many partial states,
storage behind 4 GB, calls that overlap, calls in a row without a wait, refusals."""
import math

import numpy as np
import pytest
import torch

import oracle
from rq_harness import Case, GpuCache, kv_for, rotation32
from test_gpu_paged import PagedCache
from test_gpu_tree import bf16, call, check, filled, mask_words, reference, tree_masks

pytestmark = pytest.mark.gpu


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("d,loop,T,Hq", [(128, 0, 5, 1), (128, 3, 40, 1), (96, 1, 3, 2)])
def test_one_head_spread_over_many_sms(d, loop, T, Hq):
    """A long row with a single KV head: 67 partial states, more than the merge holds weights of at a time."""
    n = 8500
    case = Case(L=1, P=4, G=1, H=1, d=d, g=32, B=1, Nmax=n + 10, Hq=Hq)
    gpu, obuf, geom, R = filled(case, 71, n)
    rng = np.random.default_rng(3)
    qb, q = bf16(rng, 1, Hq, T, d)
    kb, kn = bf16(rng, 1, 1, T, d)
    vb, vn = bf16(rng, 1, 1, T, d)
    see, scale = tree_masks(9, 1, T), 1 / math.sqrt(d)
    out = call(gpu, 0, 0, loop, qb, kb, vb, mask_words(see), None, [n], scale)
    check(out, reference(obuf, geom, R, case, 0, 0, loop, q, kn, vn, see, [T], [n], scale), f"loop {loop}")
    gpu.close()


@pytest.mark.parametrize("d,Hq,H,T,chained", [(128, 16, 1, 1, False), (96, 24, 2, 1, False), (128, 40, 1, 7, False),
                                              (128, 20, 2, 1, True)])
def test_many_query_heads_of_a_key_head(d, Hq, H, T, chained):
    case = Case(L=1, P=4, G=1, H=H, d=d, g=32, B=3, Nmax=600, Hq=Hq, chained=chained)
    gpu, obuf, geom, R = filled(case, 72, 590)
    rng = np.random.default_rng(4)
    lens, scale, see = [590, 0, 64], 1 / math.sqrt(d), tree_masks(10, 3, T)
    for loop in (1, 3):
        qb, q = bf16(rng, 3, Hq, T, d)
        kb, kn = bf16(rng, 3, H, T, d)
        vb, vn = bf16(rng, 3, H, T, d)
        out = call(gpu, 0, 0, loop, qb, kb, vb, mask_words(see), None, lens, scale)
        check(out, reference(obuf, geom, R, case, 0, 0, loop, q, kn, vn, see, [T] * 3, lens, scale), f"loop {loop}")
    gpu.close()


@pytest.mark.parametrize("d,rotation,loops", [(128, "dense", (0, 3)), (128, "hadamard", (1,)), (96, "dense", (2, 3))])
def test_enough_queries_for_blocks_of_16_in_the_merge(d, rotation, loops):
    """160 (row, KV head) pairs of 17 queries: 320 merge blocks of 16, more than two an SM."""
    B, H, T, n = 10, 16, 17, 70
    case = Case(L=1, P=4, G=1, H=H, d=d, g=32, B=B, Nmax=n, rotation=rotation)
    gpu, obuf, geom, R = filled(case, 77, n)
    rng = np.random.default_rng(14)
    lens, counts = [n - 7 * b for b in range(B)], [T - (b % 4) for b in range(B)]
    see, scale = tree_masks(15, B, T), 1 / math.sqrt(d)
    for loop in loops:
        qb, q = bf16(rng, B, H, T, d)
        kb, kn = bf16(rng, B, H, T, d)
        vb, vn = bf16(rng, B, H, T, d)
        out = call(gpu, 0, 0, loop, qb, kb, vb, mask_words(see), counts, lens, scale)
        check(out, reference(obuf, geom, R, case, 0, 0, loop, q, kn, vn, see, counts, lens, scale), f"loop {loop}")
    gpu.close()


@pytest.mark.parametrize("alphas", [(0.2, -0.05, 0.004), (-1.5, 12.0, 1e-6)])
def test_coefficients_far_from_one(alphas):
    """Loops that are small, negative or large multiples of their anchor."""
    n, T, H = 150, 6, 2
    case = Case(L=1, P=4, G=1, H=H, d=128, g=32, B=1, Nmax=200)
    R32, R = rotation32(128)
    gpu = GpuCache(case, R32)
    rng = np.random.default_rng(21)
    base = rng.standard_normal((1, 2, 1, H, n, 128))
    loops = [a * base + 0.02 * rng.standard_normal(base.shape) for a in alphas] + [base]
    kvb = torch.from_numpy(np.concatenate(loops).astype(np.float32)).to(torch.bfloat16)
    geom = oracle.Geometry(1, 4, 1, H, 128, 32, 1, 200)
    obuf = np.zeros(geom.total_bytes, dtype=np.uint8)
    gpu.append(0, 0, kvb, [0])
    oracle.append(obuf, geom, R, 0, 0, kvb.double().numpy(), np.zeros(1, dtype=np.int64))
    see, scale = tree_masks(22, 1, T), 1 / math.sqrt(128)
    for loop in range(3):
        qb, q = bf16(rng, 1, H, T, 128)
        kb, kn = bf16(rng, 1, H, T, 128)
        vb, vn = bf16(rng, 1, H, T, 128)
        out = call(gpu, 0, 0, loop, qb, kb, vb, mask_words(see), None, [n], scale)
        check(out, reference(obuf, geom, R, case, 0, 0, loop, q, kn, vn, see, [T], [n], scale), f"loop {loop}")
    gpu.close()


def test_more_rows_than_a_warp():
    """70 rows, some of them empty: the work's split over rows is summed 32 at a time."""
    B, T = 70, 3
    case = Case(L=1, P=2, G=1, H=1, d=128, g=32, B=B, Nmax=200)
    gpu, obuf, geom, R = filled(case, 73, 140)
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 141, B)]
    lens[0] = lens[31] = lens[32] = lens[69] = 0
    counts = [int(x) for x in rng.integers(0, T + 1, B)]
    qb, q = bf16(rng, B, 1, T, 128)
    kb, kn = bf16(rng, B, 1, T, 128)
    vb, vn = bf16(rng, B, 1, T, 128)
    see, scale = tree_masks(11, B, T), 1 / math.sqrt(128)
    out = call(gpu, 0, 0, 0, qb, kb, vb, mask_words(see), counts, lens, scale)
    check(out, reference(obuf, geom, R, case, 0, 0, 0, q, kn, vn, see, counts, lens, scale), "70 rows")
    gpu.close()


def test_pages_and_tree_behind_4_gigabytes():
    """Pages at both ends of a pool of more than 2^32 bytes: a copy moves every layer's block, and a
    tree call reads the last layer's far pages as it reads the same bytes in near ones."""
    L, H, n, T = 24, 16, 130, 6
    case = Case(L=L, P=4, G=1, H=H, d=128, g=32, B=1, Nmax=192)
    R32, R = rotation32(128)
    pages = 480
    gpu = PagedCache(case, R32, np.array([[1, 0, 2]]), pages)
    assert gpu.nbytes > 2 ** 32
    kvb, _ = kv_for(case, 74, n)
    for layer in (0, L - 1):
        gpu.append(layer, 0, kvb, [0])
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    rq = gpu.rq
    rq.rq_pages_copy(gpu.handle, 3, ints(0, 1, 2), ints(pages - 1, pages - 2, pages - 3), status)
    pool = gpu.buf.view(L, pages, -1)
    assert torch.equal(pool[:, pages - 3:].flip(1), pool[:, :3])
    assert (pool[L - 1, pages - 3:] != 0).any(-1).all() and (pool[0, 3:pages - 3] == 0).all()
    rng = np.random.default_rng(6)
    qb, kb, vb = (bf16(rng, 1, H, T, 128)[0] for _ in range(3))
    res = []
    for table in ([1, 0, 2], [pages - 2, pages - 1, pages - 3]):
        gpu.table.copy_(torch.tensor([table], dtype=torch.int32))
        for layer in (0, L - 1):
            res.append(call(gpu, layer, 0, 2, qb, kb, vb, None, None, [n], 0.09))
    assert all(torch.equal(res[0], r) for r in res[1:])
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")     # compaction brings them back
    refs[pages - 3:] = 1
    used, ws = ints(0), torch.zeros(rq.rq_pages_workspace_bytes(gpu.cfg, pages), dtype=torch.uint8, device="cuda")
    pool[:, :3] = 0
    rq.rq_pages_compact(gpu.handle, refs, used, status, ws, ws.numel())
    assert used.item() == 3 and gpu.table[0].tolist() == [1, 2, 0] and status.tolist() == [0, 0, 0, 0]
    assert torch.equal(call(gpu, L - 1, 0, 2, qb, kb, vb, None, None, [n], 0.09), res[0])
    gpu.close()


def test_rope_of_more_than_2_to_31_elements():
    """Rotated in place; rows far apart get what the same positions get in a small tensor."""
    import decode_attention_rq_gb300 as rq
    n = (1 << 24) + 40
    cfg = rq.rq_rope_config(head_dim=128, rotary_dim=128, theta=10000.0)
    x = torch.empty((1, 1, n, 128), dtype=torch.bfloat16, device="cuda")
    row = torch.randn(64, 128, device="cuda").to(torch.bfloat16)
    for t in (0, n // 2, n - 64):
        x[0, 0, t:t + 64] = row
    x.view(torch.int16)[0, 0, 64:70] = 0
    rq.rq_rope(cfg, x, None, None)
    for t in (0, n // 2, n - 64):
        y = row[None, None].clone()
        rq.rq_rope(cfg, y, None, ints(t))
        assert torch.equal(x[:, :, t:t + 64], y)
    assert (x[0, 0, 64:70] == 0).all()


def test_calls_on_two_streams_at_once():
    """Two tree calls that may overlap, a workspace each, give what they give alone."""
    case = Case(L=1, P=4, G=1, H=16, d=128, g=32, B=2, Nmax=2048)
    gpu = GpuCache(case, rotation32(128)[0])
    gpu.append(0, 0, kv_for(case, 75, 2000)[0], [0, 0])
    rq, T, sl = gpu.rq, 16, ints(2000, 1500)
    rng = np.random.default_rng(7)
    mask = mask_words(tree_masks(12, 2, T)).cuda()
    ins = [[bf16(rng, 2, 16, T, 128)[0].cuda() for _ in range(3)] for _ in range(2)]
    size = rq.rq_tree_workspace_bytes(gpu.cfg, 2, T)
    ws = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    out = [torch.zeros((2, 16, T, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    def go(i, loop):
        rq.rq_tree_attention(gpu.handle, 0, 0, loop, 2, T, *ins[i], mask, None, sl, 0.09, out[i], ws[i], size)

    alone = []
    for i in range(2):
        go(i, 2 * i + 1)
        torch.cuda.synchronize()
        alone.append(out[i].clone())
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for i in range(2):
            out[i].zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    go(i, 2 * i + 1)
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(out[i], alone[i]) and ws[i][:16].view(torch.int32).tolist() == [0] * 4
    gpu.close()


def test_a_run_of_calls_without_waits():
    """Tree attention, rotation in place, appends and decode calls queued in one stream over the same
    buffers give, bit for bit, what they give with a wait behind each."""
    T, H, B = 8, 4, 2
    case = Case(L=1, P=4, G=1, H=H, d=128, g=32, B=B, Nmax=512)
    R32, _ = rotation32(128)
    rng = np.random.default_rng(8)
    steps = 12
    fresh = [bf16(rng, 4, 2, B, H, T, 128)[0].cuda() for _ in range(steps)]
    queries = [bf16(rng, B, H, T, 128)[0].cuda() for _ in range(steps)]
    kvb, _ = kv_for(case, 76, 300)
    results = []
    for wait in (True, False):
        gpu = GpuCache(case, R32)
        rq = gpu.rq
        gpu.append(0, 0, kvb, [0] * B)
        cfg = rq.rq_rope_config(head_dim=128, rotary_dim=128, theta=10000.0)
        sl, mask = ints(300, 300), mask_words(tree_masks(13, B, T)).cuda()
        ws = torch.zeros(rq.rq_tree_workspace_bytes(gpu.cfg, B, T), dtype=torch.uint8, device="cuda")
        q, kv = torch.empty_like(queries[0]), torch.empty_like(fresh[0])
        out = torch.zeros_like(q)
        one, got = torch.zeros((B, H, 128), device="cuda"), []
        torch.cuda.synchronize()

        def pause():
            if wait:
                torch.cuda.synchronize()

        for i in range(steps):
            q.copy_(queries[i]); pause()
            kv.copy_(fresh[i]); pause()
            for loop in range(4):
                rq.rq_rope(cfg, q if loop == 0 else None, kv[loop, 0], sl); pause()
                rq.rq_tree_attention(gpu.handle, 0, 0, loop, B, T, q, kv[loop, 0], kv[loop, 1], mask, None, sl, 0.09, out,
                                     ws, ws.numel()); pause()
                got.append(out.clone()); pause()
                rq.rq_decode_attention(gpu.handle, 0, 0, loop, B, q[:, :, 0].contiguous(), kv[loop, 0, :, :, 0].contiguous(),
                                       kv[loop, 1, :, :, 0].contiguous(), sl, 0.09, one, gpu.ws, gpu.ws_bytes); pause()
                got.append(one.clone()); pause()
            rq.rq_append(gpu.handle, 0, 0, B, kv, sl, T, gpu.status); pause()
            sl.add_(T); pause()
        torch.cuda.synchronize()
        assert ws[:16].view(torch.int32).tolist() == [0] * 4
        results.append([x.cpu() for x in got])
        gpu.close()
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_tree_refusals():
    case = Case(L=2, P=4, G=2, H=2, d=128, g=32, B=2, Nmax=256)
    R32, _ = rotation32(128)
    gpu = GpuCache(case, R32)
    rq, T = gpu.rq, 4
    q, k, v, out = (torch.zeros((2, 2, T, 128), dtype=torch.bfloat16, device="cuda") for _ in range(4))
    mask = torch.zeros((2, T, 1), dtype=torch.int64, device="cuda")
    sl = ints(0, 0)
    size = rq.rq_tree_workspace_bytes(gpu.cfg, 2, T)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    good = dict(layer=0, group=0, loop=0, batch=2, n_nodes=T, q=q, k_new=k, v_new=v, mask=mask, node_counts=None,
                seq_lens=sl, softmax_scale=0.1, out=out, workspace=ws, workspace_bytes=size)
    rq.rq_tree_attention(gpu.handle, **good)

    def fails(status, **kw):
        with pytest.raises(rq.RqError) as e:
            rq.rq_tree_attention(gpu.handle, **{**good, **kw})
        assert e.value.status == status, (kw, e.value)

    INVALID, ALIGN, CAPACITY, UNSUPPORTED, WORKSPACE = 1, 2, 3, 6, 4
    for name, bad in (("layer", 2), ("layer", -1), ("group", 2), ("loop", 4), ("loop", -1), ("batch", 0), ("n_nodes", 0)):
        fails(INVALID, **{name: bad})
    for name in ("q", "k_new", "v_new", "seq_lens", "out", "workspace"):
        fails(INVALID, **{name: None})
    fails(INVALID, q=q.cpu())
    fails(INVALID, out=out.float())
    fails(INVALID, q=q.transpose(1, 2))
    fails(INVALID, out=out[:1])
    fails(INVALID, v_new=v[:1])
    fails(INVALID, q=q[0, 0, 0])
    fails(INVALID, mask=mask[:1])
    fails(INVALID, seq_lens=sl[:1])
    fails(INVALID, node_counts=sl.long())
    fails(INVALID, workspace=ws[:-16])
    fails(WORKSPACE, workspace_bytes=size - 1)
    fails(INVALID, n_nodes=128, mask=None)      # longer than the tensors
    fails(UNSUPPORTED, n_nodes=257, mask=None, q=q.data_ptr(), k_new=k.data_ptr(), v_new=v.data_ptr())
    fails(CAPACITY, batch=3, mask=None, seq_lens=sl.data_ptr())
    for name, x in (("q", q), ("k_new", k), ("v_new", v), ("mask", mask), ("seq_lens", sl), ("out", out)):
        fails(ALIGN, **{name: x.data_ptr() + 4})
    torch.cuda.synchronize()
    assert (out == 0).all() and ws[:16].view(torch.int32).tolist() == [0] * 4
    gpu.close()


def test_more_steps_than_32_bits_hold_are_refused():
    """Many long rows of a paged cache can make more steps than the kernels' int32 counts hold."""
    case = Case(L=1, P=1, G=1, H=64, d=128, g=32, B=8, Nmax=1 << 24, Hq=64 * 16)
    R32, _ = rotation32(128)
    gpu = PagedCache(case, R32, np.full((8, 1 << 18), -1), 1)
    rq, T = gpu.rq, 256
    q, out = (torch.zeros((8, 1024, T, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k, v = (torch.zeros((8, 64, T, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = torch.zeros(rq.rq_tree_workspace_bytes(gpu.cfg, 8, T), dtype=torch.uint8, device="cuda")
    with pytest.raises(rq.RqError) as e:      # 8 * 64 * 64 blocks of queries, 2^17 steps each
        rq.rq_tree_attention(gpu.handle, 0, 0, 0, 8, T, q, k, v, None, None, ints(*[0] * 8), 0.1, out, ws, ws.numel())
    assert e.value.status == 6
    T = 1                                     # 8 * 64 blocks
    rq.rq_tree_attention(gpu.handle, 0, 0, 0, 8, T, q, k, v, None, None, ints(*[0] * 8), 0.1, out, ws, ws.numel())
    torch.cuda.synchronize()
    assert ws[:16].view(torch.int32).tolist() == [0] * 4
    gpu.close()
