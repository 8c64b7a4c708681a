"""The binding refuses tensors that are too short for the cache they are used with, before the library is called.

The library and the device are stood in for (a call that gets through is recorded, nothing is launched), so that
short tensors meet no kernel; CPU tensors count as the device's."""
import pytest
import torch

INVALID = 1
H, HQ, D, B, PAGES = 4, 8, 128, 3, 10


class Stub:
    """Accepts every call and hands out handles."""

    def __init__(self):
        self.calls, self.handles = [], 0

    def rq_status_string(self, status):
        return b"refused"

    def __getattr__(self, name):
        def call(*args):
            if name.startswith("rq_cache_create"):
                self.handles += 1
                args[-1]._obj.value = 4096 * self.handles
            self.calls.append(name)
            return 0
        return call


@pytest.fixture
def rq(monkeypatch):
    import __graft_entry__
    __graft_entry__.build()
    import decode_attention_rq_gb300 as rq
    monkeypatch.setattr(rq, "lib", Stub())
    monkeypatch.setattr(rq, "_device", lambda: (rq._setup(), -1)[1])
    yield rq


def config(rq, **kw):
    base = dict(num_layers=1, loops_per_group=4, num_groups=1, num_heads=H, head_dim=D, group_size=32, max_batch=B,
                max_seq_len=256, mode=0, num_query_heads=HQ)
    base.update(kw)
    return rq.rq_config(**base)


def ints(n):
    return torch.zeros(n, dtype=torch.int32)


def halves(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def refused(rq, fn, *args, **kw):
    before = list(rq.lib.calls)
    with pytest.raises(rq.RqError) as e:
        fn(*args, stream=0, **kw)
    assert e.value.status == INVALID
    assert rq.lib.calls == before            # nothing reached the library


def tree(rq, handle, T=5, **kw):
    a = dict(q=halves(B, HQ, T, D), k_new=halves(B, H, T, D), v_new=halves(B, H, T, D), mask=None, node_counts=None,
             seq_lens=ints(B), softmax_scale=0.1, out=halves(B, HQ, T, D),
             workspace=torch.zeros(64, dtype=torch.uint8), workspace_bytes=64)
    a.update(kw)
    return (handle, 0, 0, 0, B, T), a


@pytest.mark.parametrize("paged", [False, True])
def test_tree_tensors_with_too_few_heads(rq, paged):
    h = (rq.rq_cache_create_paged(config(rq), PAGES, 16, 1, 16, 4, 16) if paged else
         rq.rq_cache_create(config(rq), 16, 1, 16))
    T = 5
    pos, kw = tree(rq, h)
    rq.rq_tree_attention(*pos, **kw, stream=0)
    assert rq.lib.calls[-1] == "rq_tree_attention"
    for name, heads in (("q", HQ), ("out", HQ), ("k_new", H), ("v_new", H)):
        for short in (halves(B, 1, T, D), halves(B, heads - 1, T, D), halves(B, heads, T, 96), halves(B, heads, T - 1, D),
                      halves(B - 1, heads, T, D), halves(B * heads * T * D - 1)):
            pos, kw = tree(rq, h, **{name: short})
            refused(rq, rq.rq_tree_attention, *pos, **kw)
    # every tensor too short by the same factor, the KV heads' count for the query heads
    pos, kw = tree(rq, h, q=halves(B, 1, T, D), k_new=halves(B, 1, T, D), v_new=halves(B, 1, T, D), out=halves(B, 1, T, D))
    refused(rq, rq.rq_tree_attention, *pos, **kw)
    pos, kw = tree(rq, h, q=halves(B, H, T, D), out=halves(B, H, T, D))
    refused(rq, rq.rq_tree_attention, *pos, **kw)
    # addresses are the caller's word, and do not take the check from the others
    pos, kw = tree(rq, h, q=4096, k_new=4096, v_new=halves(B, 1, T, D))
    refused(rq, rq.rq_tree_attention, *pos, **kw)
    pos, kw = tree(rq, h, q=4096, k_new=4096, out=halves(B, 1, T, D))
    refused(rq, rq.rq_tree_attention, *pos, **kw)
    # longer ones are no harm, each by itself
    pos, kw = tree(rq, h, q=halves(B + 1, HQ, T, D), k_new=halves(B, H + 1, T, D))
    rq.rq_tree_attention(*pos, **kw, stream=0)


def test_multi_head_cache_and_width_96(rq):
    h = rq.rq_cache_create(config(rq, head_dim=96, num_query_heads=0), 16, 1, 16)
    T = 5
    full = dict(q=halves(B, H, T, 96), k_new=halves(B, H, T, 96), v_new=halves(B, H, T, 96), out=halves(B, H, T, 96))
    pos, kw = tree(rq, h, **full)
    rq.rq_tree_attention(*pos, **kw, stream=0)
    for name in full:
        pos, kw = tree(rq, h, **{**full, name: halves(B, H - 1, T, 96)})
        refused(rq, rq.rq_tree_attention, *pos, **kw)


def page_calls(rq, h, refs):
    w = torch.zeros(64, dtype=torch.uint8)
    return [(rq.rq_pages_fork, (h, 2, ints(2), ints(2), refs)), (rq.rq_pages_free, (h, 2, ints(2), None, refs)),
            (rq.rq_pages_reserve, (h, B, ints(B), 1, refs, None, w, 64)),
            (rq.rq_pages_compact, (h, refs, ints(1), None, w, 64))]


def test_counts_of_every_page(rq):
    h = rq.rq_cache_create_paged(config(rq), PAGES, 16, 1, 16, 4, 16)
    for fn, args in page_calls(rq, h, ints(PAGES)) + page_calls(rq, h, 4096):
        fn(*args, stream=0)
    for n in (0, 1, PAGES - 1):
        for fn, args in page_calls(rq, h, ints(n)):
            refused(rq, fn, *args)


def test_a_handle_given_out_again_has_its_new_shape(rq):
    small, large = config(rq, num_heads=1, num_query_heads=0), config(rq)
    h = rq.rq_cache_create(small, 16, 1, 16)
    rq.rq_cache_destroy(h)
    rq.lib.handles -= 1
    assert rq.rq_cache_create(large, 16, 1, 16) == h
    T = 5
    pos, kw = tree(rq, h, q=halves(B, 1, T, D), k_new=halves(B, 1, T, D), v_new=halves(B, 1, T, D), out=halves(B, 1, T, D))
    refused(rq, rq.rq_tree_attention, *pos, **kw)
    rq.rq_cache_destroy(h)
    # the configuration is taken as it was at creation
    h = rq.rq_cache_create_paged(large, PAGES, 16, 1, 16, 4, 16)
    large.num_heads = large.num_query_heads = 1
    pos, kw = tree(rq, h, k_new=halves(B, 1, T, D))
    refused(rq, rq.rq_tree_attention, *pos, **kw)


@pytest.mark.gpu
def test_short_tensors_on_the_device():
    from rq_harness import Case, rotation32
    from test_gpu_paged import PagedCache, _table
    case = Case(L=1, P=4, G=1, H=H, d=D, g=32, B=B, Nmax=128, Hq=HQ)
    table, pages = _table(case)
    gpu = PagedCache(case, rotation32(D)[0], table, pages)
    rq, T = gpu.rq, 5
    ws = torch.zeros(rq.rq_tree_workspace_bytes(gpu.cfg, B, T), dtype=torch.uint8, device="cuda")
    full = dict(q=halves(B, HQ, T, D).cuda(), k_new=halves(B, H, T, D).cuda(), v_new=halves(B, H, T, D).cuda(), mask=None,
                node_counts=None, seq_lens=ints(B).cuda(), softmax_scale=0.1, out=halves(B, HQ, T, D).cuda(), workspace=ws,
                workspace_bytes=ws.numel())
    rq.rq_tree_attention(gpu.handle, 0, 0, 0, B, T, **full)
    for name in ("q", "k_new", "v_new", "out"):
        with pytest.raises(rq.RqError) as e:
            rq.rq_tree_attention(gpu.handle, 0, 0, 0, B, T, **{**full, name: full[name][:, 1:].contiguous()})
        assert e.value.status == INVALID
    w = torch.zeros(rq.rq_pages_workspace_bytes(gpu.cfg, pages), dtype=torch.uint8, device="cuda")
    refs = ints(pages).cuda()
    rq.rq_pages_reserve(gpu.handle, B, ints(B).cuda(), 1, refs, None, w, w.numel())
    with pytest.raises(rq.RqError) as e:
        rq.rq_pages_reserve(gpu.handle, B, ints(B).cuda(), 1, refs[:-1], None, w, w.numel())
    assert e.value.status == INVALID
    torch.cuda.synchronize()
    gpu.close()
