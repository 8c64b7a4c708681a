"""GPU: speculative steps over a branching paged cache, the operators together.

A prompt is appended to row 0 and forked to two more rows, which share its pages.
Each step rotates the drafted nodes' queries and keys at their positions, attends
with every loop, accepts a path of a different length per row, reserves pages (the
first write to a shared page copies it), appends, and gives back what was reserved
too far.  In between a row is forked over another and the pool is packed.  Held against
the float64 oracle throughout: attention within the bar of test_gpu_tree, and the
bytes of every whole tile of every row equal to those of a contiguous cache that got the
same tokens."""
import math

import numpy as np
import pytest
import torch

import oracle
from rq_harness import Case, rotation32
from test_gpu_rope import angles, config
from test_gpu_tree import FILL, check, mask_words, reference, tree_masks

pytestmark = pytest.mark.gpu


def rotated(rq, cfg, x, pos):
    """BF16 tensor rotated in float64 and rounded, for comparison; x [B, H, n, d], pos [B, n]."""
    ang, mag = angles(rq, cfg, pos)
    z = x.double().numpy()
    h = cfg.rotary_dim // 2
    a, b = z[..., :h], z[..., h:2 * h]
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    return np.concatenate([a * c - b * s, b * c + a * s], -1)


def test_speculative_steps_over_forked_rows():
    import decode_attention_rq_gb300 as rq
    case = Case(L=1, P=4, G=1, H=2, d=128, g=32, B=3, Nmax=320, Hq=4)
    B, P, H, Hq, d, T = case.B, case.P, case.H, case.Hq, case.d, 7
    R32, R = rotation32(d)
    cfg = rq.rq_config(1, P, 1, H, d, 32, B, case.Nmax, rq.RQ_MODE_SHARED, Hq)
    pages, tiles = 16, 5
    pool = torch.zeros(rq.rq_cache_paged_bytes(cfg, pages), dtype=torch.uint8, device="cuda")
    table = torch.full((B, tiles), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    used = torch.zeros(4, dtype=torch.int32, device="cuda")
    rotation = torch.from_numpy(R32).cuda()          # kept alive as long as the cache
    handle = rq.rq_cache_create_paged(cfg, pages, pool, pool.numel(), table, tiles, rotation)
    pws = torch.zeros(rq.rq_pages_workspace_bytes(cfg, pages), dtype=torch.uint8, device="cuda")
    tws = torch.zeros(rq.rq_tree_workspace_bytes(cfg, B, T), dtype=torch.uint8, device="cuda")
    rope = config(rq, head_dim=d, rotary_dim=d)
    geom = oracle.Geometry(1, P, 1, H, d, 32, B, case.Nmax)
    obuf = np.zeros(geom.total_bytes, dtype=np.uint8)
    rng = np.random.default_rng(11)
    scale = 1 / math.sqrt(d)

    def ints(x):
        return torch.tensor([int(v) for v in x], dtype=torch.int32, device="cuda")

    def draw(*shape):
        x = rng.standard_normal(shape).astype(np.float32)
        return torch.from_numpy(x).to(torch.bfloat16)

    def same_tiles(lens):
        torch.cuda.synchronize()
        t = table.cpu().numpy()
        got = pool.cpu().numpy().reshape(pages, -1)
        for b in range(B):     # this row's tiles where the table has them, all others on a page of their own
            alone = np.where((np.arange(B)[:, None] == b) & (t >= 0), t, pages)
            one = oracle.paged_pool(obuf, geom, alone, pages + 1).reshape(pages + 1, -1)
            for tile in range(lens[b] // 64):
                assert t[b, tile] >= 0
                assert np.array_equal(got[t[b, tile]], one[t[b, tile]]), (b, tile)

    # the prompt, its keys rotated at positions 0 ..
    n0 = 100
    kv = draw(P, 2, 1, H, n0, d).cuda()
    for p in range(P):
        rq.rq_rope(rope, None, kv[p, 0], None)
    rq.rq_pages_reserve(handle, 1, ints([0]), n0, refs, status, pws, pws.numel())
    rq.rq_append(handle, 0, 0, 1, kv, ints([0]), n0, status)
    for b in range(B):
        oracle.append(obuf, geom, R, 0, 0, kv.double().cpu().numpy().repeat(B, axis=2), np.zeros(B, dtype=np.int64), rows=[b])
    rq.rq_pages_fork(handle, 2, ints([0, 0]), ints([1, 2]), refs, status)
    lens = [n0] * B
    assert refs.tolist()[:2] == [3, 3]
    same_tiles(lens)

    for step in range(4):
        seq = ints(lens)
        see = tree_masks(20 + step, B, T)
        depth = see.sum(-1) - 1
        offs = torch.from_numpy(depth.astype(np.int32)).cuda()
        pos = np.asarray(lens)[:, None] + depth
        q_raw, kv_raw = draw(P, B, Hq, T, d), draw(P, 2, B, H, T, d)
        q, kv = q_raw.cuda(), kv_raw.cuda()
        for loop in range(P):
            rq.rq_rope(rope, q[loop], kv[loop, 0], seq, offs)
            # one rounding of an exact value: half a BF16 step, and float32 arithmetic (test_gpu_rope)
            exact = rotated(rq, rope, kv_raw[loop, 0], pos)
            size = np.abs(exact) * 2.0 ** -8 + 2.0 ** -21 * 12
            assert (np.abs(kv[loop, 0].double().cpu().numpy() - exact) <= size).all()
            out = torch.full((B, Hq, T, d), FILL, dtype=torch.bfloat16, device="cuda")
            rq.rq_tree_attention(handle, 0, 0, loop, B, T, q[loop], kv[loop, 0], kv[loop, 1],
                                 mask_words(see).cuda(), None, seq, scale, out, tws, tws.numel())
            ref = reference(obuf, geom, R, case, 0, 0, loop, q[loop].double().cpu().numpy(),
                            kv[loop, 0].double().cpu().numpy(), kv[loop, 1].double().cpu().numpy(), see, [T] * B,
                            lens, scale)
            check(out, ref, f"step {step}, loop {loop}")
        # a path of every row's tree: the ancestors of a node, of different lengths
        paths = [np.nonzero(see[b, (3 * step + 2 * b) % T])[0] for b in range(B)]
        n = max(len(p) for p in paths)
        take = np.stack([np.concatenate([p, np.full(n - len(p), p[-1])]) for p in paths])      # padded: overwritten later
        index = torch.from_numpy(take).cuda()
        chosen = torch.stack([kv[:, :, b][:, :, :, index[b]] for b in range(B)], 2).contiguous()
        rq.rq_pages_reserve(handle, B, seq, n, refs, status, pws, pws.numel())
        rq.rq_append(handle, 0, 0, B, chosen, seq, n, status)
        oracle.append(obuf, geom, R, 0, 0, chosen.double().cpu().numpy(), np.asarray(lens))
        lens = [ln + len(p) for ln, p in zip(lens, paths)]
        rq.rq_pages_free(handle, B, ints(range(B)), ints(lens), refs, status)
        same_tiles(lens)
        if step == 1:      # row 2 gives up its branch and takes row 1's
            rq.rq_pages_fork(handle, 1, ints([1]), ints([2]), refs, status)
            lens[2] = lens[1]
            size = geom.region_offset(0, 0, 1, 0) - geom.region_offset(0, 0, 0, 0)
            obuf[2 * size: 3 * size] = obuf[size: 2 * size]
        if step == 2:
            rq.rq_pages_compact(handle, refs, used, status, pws, pws.numel())
            same_tiles(lens)
            assert int(used[0]) == int((refs > 0).sum()) and bool((refs[: int(used[0])] > 0).all())
    assert status.tolist() == [0, 0, 0, 0] and tws[:16].view(torch.int32).tolist() == [0, 0, 0, 0]
    rq.rq_pages_free(handle, B, ints(range(B)), None, refs, status)
    assert int(refs.sum()) == 0
    rq.rq_cache_destroy(handle)
