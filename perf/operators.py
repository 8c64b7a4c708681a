"""What the speculative-decoding and branching operators are measured on.

Three operators beside the single-token decode attention: attention of a tree
of drafted tokens over the compressed cache, the page operations of the paged
cache, and rotary positions.  `run` computes each either in plain torch
operations (own = False) or through the library's entry points (own = True).
"""
import math

import torch

own = False

# ---------------------------------------------------------------------------
# cases


def listed():
    return [
        # tree attention: the smallest call, one layer of the toy shape with a chain-like draft of four
        dict(name="tree_toy", op="tree", H=2, Hq=2, d=128, g=32, B=1, N=256, T=4, loop=1, paged=False, ragged=False),
        # one residual-loop call of an Ouro-shaped step at 8k, batch 4, sixteen drafted tokens
        dict(name="tree_ouro8k_b4", op="tree", H=16, Hq=16, d=128, g=32, B=4, N=8192, T=16, loop=1, paged=False,
             ragged=False),
        # 16k context over a paged cache, a wide tree of odd size
        dict(name="tree_ouro16k_b2_paged", op="tree", H=16, Hq=16, d=128, g=32, B=2, N=16384, T=61, loop=2,
             paged=True, ragged=False),
        # Huginn-shaped heads of width 96, rows of different lengths and draft sizes, the anchor loop
        dict(name="tree_huginn_anchor", op="tree", H=55, Hq=55, d=96, g=32, B=2, N=4096, T=25, loop=3, paged=False,
             ragged=True),
        # grouped-query heads (four per KV head), groups of 16 channels, batch 8
        dict(name="tree_gqa_b8", op="tree", H=16, Hq=64, d=128, g=16, B=8, N=8192, T=13, loop=0, paged=False,
             ragged=True),
        # pages: 32 beams (8 prompts x 4) about to write their next token into shared last pages
        dict(name="pages_reserve_beams", op="reserve", L=24, G=1, H=16, d=128, g=32, P=4, rows=32, share=4, tiles=4,
             pages=128),
        # pages: a beam permutation of 64 rows at 16k; table and counts only, latency
        dict(name="pages_fork_64", op="fork", L=1, G=1, H=1, d=128, g=32, P=4, rows=64, tiles=256, pages=20000),
        # pages: single pages of a Huginn-shaped cache moved by an explicit list
        dict(name="pages_copy_huginn", op="copy", L=4, G=8, H=55, d=96, g=32, P=4, rows=4, tiles=8, pages=40, n=5),
        # pages: a fragmented pool packed to the front (50 of 120 pages in use move)
        dict(name="pages_compact", op="compact", L=24, G=1, H=16, d=128, g=32, P=4, rows=8, tiles=16, pages=256,
             used=120, n=50),
        # rotary: q and k of one token per row, batch 4: latency
        dict(name="rope_token", op="rope", B=4, n=1, Hq=16, H=16, d=128, r=128, inter=False, inverse=False,
             scaling="none", dtype="bf16", far=8192, tree=False),
        # rotary: a prompt of 8k, batch 4, frequencies scaled by parts for a longer context
        dict(name="rope_prompt_8k", op="rope", B=4, n=8192, Hq=16, H=16, d=128, r=128, inter=False, inverse=False,
             scaling="parts", dtype="bf16", far=0, tree=False),
        # rotary: the gradient in 32 bits, neighbouring pairs, part of a width-96 head, an odd length
        dict(name="rope_backward_odd", op="rope", B=2, n=1021, Hq=55, H=55, d=96, r=64, inter=True, inverse=True,
             scaling="linear", dtype="fp32", far=100000, tree=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "rope", "rope", "copy", "fork", "reserve", "free", "compact"])
    if op == "tree":
        d = rng.choice([128, 128, 96])
        qpk = rng.choice([1, 1, 2, 4])
        H = rng.choice([2, 5, 16, 16, 20])
        B = rng.choice([1, 2, 3, 4, 8])
        T = _log(rng, 1, 64)
        N = _log(rng, 30, 16384)
        while B * H * N > 16 * 6 * 8192 or B * H * N * T * qpk > 16 * 6 * 8192 * 46:
            N = max(30, N // 2)
            T = max(1, (2 * T) // 3)
        return dict(op=op, H=H, Hq=H * qpk, d=d, g=rng.choice([16, 32]), B=B, N=N, T=T, loop=rng.randrange(4),
                    paged=rng.random() < 0.5, ragged=rng.random() < 0.6)
    if op == "rope":
        d = rng.choice([64, 96, 128, 128])
        n = _log(rng, 1, 8192)
        B = rng.choice([1, 2, 3, 4])
        H = rng.choice([1, 4, 16])
        return dict(op=op, B=B, n=n, Hq=H * rng.choice([1, 2]) if n < 2048 else H, H=H, d=d,
                    r=rng.choice([d, d, d // 2, d - 6]), inter=rng.random() < 0.5, inverse=rng.random() < 0.4,
                    scaling=rng.choice(["none", "linear", "base", "parts"]),
                    dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]) if n < 2048 else "bf16",
                    far=rng.choice([0, 8192, 1000000]), tree=n <= 64 and rng.random() < 0.5)
    if op == "copy":
        pages = rng.randrange(6, 40)
        return dict(op=op, L=rng.choice([1, 2, 4]), G=rng.choice([1, 8]), H=rng.choice([1, 3, 16, 55]), d=96, g=32,
                    P=4, rows=2, tiles=4, pages=pages, n=rng.randrange(1, pages // 2 + 1))
    if op == "reserve":
        share = rng.choice([1, 2, 4, 5])
        rows = share * rng.randrange(1, 7)
        tiles = rng.randrange(1, 6)
        return dict(op=op, L=rng.choice([1, 4, 24]), G=1, H=rng.choice([2, 16]), d=128, g=rng.choice([16, 32]), P=4,
                    rows=rows, share=share, tiles=tiles, pages=rows * (tiles + 1) + rng.randrange(0, 30))
    if op == "compact":
        pages = rng.randrange(20, 200)
        used = rng.randrange(4, pages // 2)
        return dict(op=op, L=rng.choice([1, 2, 8]), G=1, H=rng.choice([1, 16]), d=128, g=32, P=rng.choice([2, 4]),
                    rows=4, tiles=-(-used // 4) + 1, pages=pages, used=used, n=rng.randrange(0, used // 2 + 1))
    rows = rng.randrange(2, 65)
    tiles = _log(rng, 2, 256)
    return dict(op=op, L=1, G=1, H=1, d=128, g=32, P=4, rows=rows, tiles=tiles, pages=rows * tiles + 100)


# ---------------------------------------------------------------------------
# the cache's bytes (the layout that the library states in its header)

_P = 4          # loops per group of the tree cases


def _tile_bytes(d, g):
    ng = d // g
    return 64 * d // 2 + 64 * ng * 2, 64 * d // 4 + 64 * ng * 2 + 128   # anchor tile, residual tile


def _head_block(d, g, P):
    a, r = _tile_bytes(d, g)
    return 2 * a + 2 * (P - 1) * r


def _e4m3(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _coded(x, g, bits):
    """x [..., tokens, d] float32 -> codes uint8, metadata bytes [..., tokens, ng, 2]."""
    q = x.unflatten(-1, (-1, g))
    lo, hi = q.amin(-1, keepdim=True), q.amax(-1, keepdim=True)
    o8, s8 = _e4m3(lo), _e4m3((hi - lo) / (2 ** bits - 1))
    s = s8.float()
    k = torch.where(s > 0, (q - o8.float()) / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(q))
    codes = k.round().clamp(0, 2 ** bits - 1).to(torch.uint8).flatten(-2)
    meta = torch.stack([s8.view(torch.uint8), o8.view(torch.uint8)], -1).squeeze(-2)
    return codes, meta


def _pack_tiles(codes, meta, c, bits, kv):
    """codes [R, nt, 64, d], meta [R, nt, 64, ng, 2], c [R, nt, 64] bf16 or None -> bytes [R, nt, tile]."""
    R, nt, _, d = codes.shape
    if kv == 0:                                    # token-major: neighbouring channels share a byte
        per = 8 // bits
        b = codes.view(R, nt, 64, d // per, per)
        out = sum(b[..., m] << (bits * m) for m in range(per))
    else:                                          # channel-major words of 8 or 16 tokens
        t = codes.transpose(2, 3)
        if bits == 4:
            b = t.reshape(R, nt, d, 8, 2, 4)       # word, nibble, byte
            out = b[..., 0, :] | (b[..., 1, :] << 4)
        else:
            b = t.reshape(R, nt, d, 4, 4, 4)       # word, field m, byte
            out = sum(b[..., m, :] << (2 * m) for m in range(4))
    parts = [out.reshape(R, nt, -1), meta.reshape(R, nt, -1)]
    if c is not None:
        parts.append(c.contiguous().view(torch.uint8).reshape(R, nt, -1))
    return torch.cat(parts, -1)


def _unpack(tiles, d, g, bits, kv, dtype):
    """bytes [R, nt, tile] -> dequantised values [R, nt * 64, d] and, for residual tiles, c [R, nt * 64]."""
    R, nt, _ = tiles.shape
    ng, nb = d // g, 64 * d * bits // 8
    raw = tiles[..., :nb]
    if kv == 0:
        per = 8 // bits
        b = raw.reshape(R, nt, 64, d // per)
        codes = torch.stack([(b >> (bits * m)) & (2 ** bits - 1) for m in range(per)], -1).reshape(R, nt, 64, d)
    elif bits == 4:
        b = raw.reshape(R, nt, d, 8, 4)
        codes = torch.stack([b & 15, b >> 4], -2).reshape(R, nt, d, 64).transpose(2, 3)
    else:
        b = raw.reshape(R, nt, d, 4, 4)
        codes = torch.stack([(b >> (2 * m)) & 3 for m in range(4)], -2).reshape(R, nt, d, 64).transpose(2, 3)
    meta = tiles[..., nb:nb + 128 * ng].contiguous().view(torch.float8_e4m3fn).reshape(R, nt, 64, ng, 2).to(dtype)
    x = codes.to(dtype).unflatten(-1, (ng, g)) * meta[..., :1] + meta[..., 1:]
    x = x.flatten(-2).reshape(R, nt * 64, d)
    c = None
    if bits == 2:
        c = tiles[..., nb + 128 * ng:].contiguous().view(torch.bfloat16).reshape(R, nt * 64).to(dtype)
    return x, c


# ---------------------------------------------------------------------------
# tree attention

_ALPHA = (0.7, 0.85, 0.95)


def _lens(case):
    B, N = case["B"], case["N"]
    if not case["ragged"]:
        return [N] * B
    return [max(0, N - (N * b) // (2 * B) - 7 * b) for b in range(B)]


def _counts(case):
    B, T = case["B"], case["T"]
    return [max(1, T - (b % 3) * (T // 5)) for b in range(B)] if case["ragged"] else [T] * B


def _tree_inputs(case, seed, dev):
    gen = torch.Generator(device=dev).manual_seed(seed)
    H, Hq, d, g, B, N, T, loop = (case[k] for k in ("H", "Hq", "d", "g", "B", "N", "T", "loop"))

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    nt = -(-(N + T) // 64)
    a_tile, r_tile = _tile_bytes(d, g)
    plane_a, plane_r = nt * a_tile, nt * r_tile
    region = 2 * plane_a + 2 * (_P - 1) * plane_r
    buf = torch.zeros((B * H, region), dtype=torch.uint8, device=dev)
    for kv in range(2):                            # anchor and this loop's residual; outlier channels as in the recipe
        x = normal(B * H, nt, 64, d)
        for ch in (3, 77):
            x[..., ch] *= 8
        codes, meta = _coded(x, g, 4)
        buf[:, kv * plane_a:(kv + 1) * plane_a] = _pack_tiles(codes, meta, None, 4, kv).reshape(B * H, -1)
        del x, codes, meta
        if loop < _P - 1:
            codes, meta = _coded(0.3 * normal(B * H, nt, 64, d), g, 2)
            c = (_ALPHA[loop] + 0.02 * normal(B * H, nt, 64)).to(torch.bfloat16)
            at = 2 * plane_a + (2 * loop + kv) * plane_r
            buf[:, at:at + plane_r] = _pack_tiles(codes, meta, c, 2, kv).reshape(B * H, -1)
            del codes, meta
    a = torch.randn((d, d), generator=torch.Generator().manual_seed(seed), dtype=torch.float64)
    R, tri = torch.linalg.qr(a)
    R = (R * torch.sign(torch.diagonal(tri))).float().to(dev)
    q = normal(B, Hq, T, d).to(torch.bfloat16)
    k_new, v_new = normal(B, H, T, d).to(torch.bfloat16), normal(B, H, T, d).to(torch.bfloat16)
    # a tree per row: node t hangs under a random earlier node, or under the cached text
    parent = (torch.rand((B, T), generator=gen, device=dev) * (torch.arange(T, device=dev) + 1)).long() - 1
    see = torch.zeros((B, T, T), dtype=torch.bool, device=dev)
    rows = torch.arange(B, device=dev)
    for t in range(T):
        if t:
            p = parent[:, t]
            see[:, t] = see[rows, p.clamp(min=0)] & (p >= 0)[:, None]
        see[:, t, t] = True
    words = -(-T // 64)
    bits = torch.zeros((B, T, words * 64), dtype=torch.int64, device=dev)
    bits[..., :T] = see.long()
    shift = torch.arange(64, device=dev)
    mask = (bits.view(B, T, words, 64) << shift).sum(-1)
    s = dict(case=case, R=R, q=q, k_new=k_new, v_new=v_new, mask=mask.contiguous(), scale=1 / math.sqrt(d),
             lens=_lens(case), counts=_counts(case))
    s["seq"] = torch.tensor(s["lens"], dtype=torch.int32, device=dev)
    s["count"] = torch.tensor(s["counts"], dtype=torch.int32, device=dev)
    if case["paged"]:                              # the same tiles spread over a pool by a shuffled table
        pages = B * nt + 3
        table = torch.randperm(pages, generator=gen, device=dev)[:B * nt].view(B, nt)
        pool = torch.zeros((pages, H, _head_block(d, g, _P)), dtype=torch.uint8, device=dev)
        off, src = 0, 0
        for plane in range(2 * _P):
            tb = a_tile if plane < 2 else r_tile
            t = buf[:, src:src + nt * tb].view(B, H, nt, tb).permute(0, 2, 1, 3).reshape(B * nt, H, tb)
            pool[:, :, off:off + tb].index_copy_(0, table.flatten(), t)
            off, src = off + tb, src + nt * tb
        s.update(buf=pool, pages=pages, table=table.to(torch.int32).contiguous())
    else:
        s.update(buf=buf)
    s["nt"] = nt
    return s


def _row_planes(s, b, nt, dtype):
    """K and V of row b's first nt tiles, rebuilt: [H, nt * 64, d] each."""
    case = s["case"]
    d, g, H, loop = case["d"], case["g"], case["H"], case["loop"]
    a_tile, r_tile = _tile_bytes(d, g)
    R = s["R"].to(dtype)
    out = []
    for kv in range(2):
        if case["paged"]:
            blocks = s["buf"][s["table"][b, :nt].long()].transpose(0, 1)           # [H, nt, head block]
            at = 2 * a_tile + (2 * loop + kv) * r_tile
            anchor, res = blocks[..., kv * a_tile:(kv + 1) * a_tile], blocks[..., at:at + r_tile]
        else:
            rows = s["buf"][b * H:(b + 1) * H]
            pa, pr = s["nt"] * a_tile, s["nt"] * r_tile
            at = 2 * pa + (2 * loop + kv) * pr
            anchor = rows[:, kv * pa:kv * pa + nt * a_tile].reshape(H, nt, a_tile)
            res = rows[:, at:at + nt * r_tile]         # nothing there for the anchor loop
        x, _ = _unpack(anchor, d, g, 4, kv, dtype)
        if loop < _P - 1:
            r, c = _unpack(res.reshape(H, nt, r_tile), d, g, 2, kv, dtype)
            x = c[..., None] * x + r @ R
        out.append(x)
    return out


def _tree_plain(s):
    case = s["case"]
    H, Hq, T = case["H"], case["Hq"], case["T"]
    qpk = Hq // H
    for b in range(case["B"]):
        n, m = s["lens"][b], s["counts"][b]
        K, V = _row_planes(s, b, -(-n // 64), torch.float32)
        K = torch.cat([K[:, :n], s["k_new"][b, :, :m].float()], 1)
        V = torch.cat([V[:, :n], s["v_new"][b, :, :m].float()], 1)
        q = s["q"][b, :, :m].float().reshape(H, qpk * m, -1)
        S = (q @ K.transpose(1, 2)) * s["scale"]
        bit = (s["mask"][b, :m, :, None] >> torch.arange(64, device=S.device)) & 1
        hide = bit.reshape(m, -1)[:, :m] == 0
        S.view(H, qpk, m, n + m)[..., n:].masked_fill_(hide, -math.inf)
        E = torch.exp(S - S.amax(-1, keepdim=True))
        O = (E @ V) / E.sum(-1, keepdim=True)
        s["out"][b, :, :m] = O.reshape(Hq, m, -1).to(torch.bfloat16)
    return s["out"]


def _byte_view(s, b, kv, loop):
    """Tiles of one plane of row b as bytes [H, nt, tile]; loop None: the anchor."""
    case = s["case"]
    H, nt = case["H"], s["nt"]
    sizes = [n for n in _tile_bytes(case["d"], case["g"])[:1] for _ in range(2)]
    sizes += [_tile_bytes(case["d"], case["g"])[1]] * (2 * (_P - 1))
    i = kv if loop is None else 2 + 2 * loop + kv
    if case["paged"]:
        pool = s["buf"][s["table"][b].long()]
        return pool[..., sum(sizes[:i]):sum(sizes[:i + 1])].permute(1, 0, 2)
    return s["buf"][b * H:(b + 1) * H, nt * sum(sizes[:i]):nt * sum(sizes[:i + 1])].unflatten(1, (nt, sizes[i]))


def _values(tiles, d, g, bits, kv, n):
    """Tokens 0..n-1 of a plane from the byte and bit where the layout keeps each code, in 64 bits: [H, n, d]."""
    dev = tiles.device
    t, ch = torch.arange(n, device=dev)[:, None], torch.arange(d, device=dev)[None]
    slot = t % 64
    if kv == 0:
        at, bit = slot * (d * bits // 8) + ch * bits // 8, (ch * bits) % 8
    else:
        run = 32 // bits                           # tokens in a word
        at, bit = ch * (8 * bits) + 4 * (slot // run) + slot % 4, bits * ((slot % run) // 4)
    code = (tiles[:, t // 64, at].long() >> bit) & (2 ** bits - 1)
    at = 8 * d * bits + (slot * (d // g) + ch // g) * 2
    f8 = tiles.contiguous().view(torch.float8_e4m3fn)
    return code * f8[:, t // 64, at].double() + f8[:, t // 64, at + 1].double()


def _tree_exact(case, seed):
    s = _tree_inputs(case, seed, "cuda")
    H, Hq, T, B, d, g, loop = (case[k] for k in ("H", "Hq", "T", "B", "d", "g", "loop"))
    if 4 * Hq * T * sum(s["lens"]) * d > 2e12:
        return None
    out = torch.zeros((B, Hq, T, d), dtype=torch.float64, device="cuda")
    for b in range(B):
        n, m = s["lens"][b], s["counts"][b]
        cached = []
        for kv in range(2):
            x = _values(_byte_view(s, b, kv, None), d, g, 4, kv, n)
            if loop < _P - 1:
                tiles = _byte_view(s, b, kv, loop)
                c = tiles[..., -128:].contiguous().view(torch.bfloat16).flatten(1)[:, :n].double()
                x = torch.einsum("hn,hnd->hnd", c, x)
                x += torch.einsum("ij,hni->hnj", s["R"].double(), _values(tiles, d, g, 2, kv, n))
            cached.append(x)
        words = s["mask"][b, :m].cpu().tolist()
        see = torch.tensor([[(w[j // 64] >> (j % 64)) & 1 for j in range(m)] for w in words], dtype=torch.bool,
                           device="cuda")
        ok = torch.cat([torch.ones((m, n), dtype=torch.bool, device="cuda"), see], 1)
        for h in range(Hq):
            kv = h // (Hq // H)
            keys = torch.cat([cached[0][kv], s["k_new"][b, kv, :m].double()])
            values = torch.cat([cached[1][kv], s["v_new"][b, kv, :m].double()])
            logits = torch.einsum("td,nd->tn", s["q"][b, h, :m].double(), keys) * s["scale"]
            w = torch.softmax(logits.masked_fill(~ok, -math.inf), -1)
            out[b, h, :m] = torch.einsum("tn,nd->td", w, values)
    return out


# ---------------------------------------------------------------------------
# pages


def _pages_inputs(case, seed, dev):
    gen = torch.Generator(device=dev).manual_seed(seed)
    op, rows, tiles, pages = case["op"], case["rows"], case["tiles"], case["pages"]
    planes = case["L"] * case["G"]
    page = case["H"] * _head_block(case["d"], case["g"], case["P"])
    pool = torch.randint(0, 256, (planes, pages, page), dtype=torch.uint8, generator=gen, device=dev)
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    table = torch.full((rows, tiles + 2), -1, dtype=torch.int32, device=dev)
    s = dict(case=case, pool=pool)

    def ints(x):
        return torch.as_tensor(x, dtype=torch.int32, device=dev).contiguous()

    if op == "copy":                               # sources and targets apart, in no order
        s.update(src=order[:case["n"]].contiguous(), dst=order[case["n"]:2 * case["n"]].contiguous())
        table[:, :tiles] = 0
    elif op == "reserve":                          # every prompt's rows share all their pages; the last is half full
        share = case["share"]
        own_pages = order[:rows // share * tiles].view(rows // share, tiles)
        table[:, :tiles] = own_pages.repeat_interleave(share, 0)
        lens = [(tiles - 1) * 64 + 1 + (17 * (b // share)) % 63 for b in range(rows)]
        s.update(seq=ints(lens), lens=lens)
    elif op == "compact":                          # n pages in use lie at or above `used`, as many holes below it
        used, n = case["used"], case["n"]
        low = torch.randperm(used, generator=gen, device=dev)[n:]
        high = used + torch.randperm(pages - used, generator=gen, device=dev)[:n]
        live = torch.cat([low, high])
        live = live[torch.randperm(used, generator=gen, device=dev)].to(torch.int32)
        flat = torch.full((rows * tiles,), -1, dtype=torch.int32, device=dev)
        flat[:used] = live
        table[:, :tiles] = flat.view(rows, tiles)
    else:                                          # fork, free: every row full of its own pages
        table[:, :tiles] = order[:rows * tiles].view(rows, tiles)
        if op == "fork":                           # beams: each target row takes a random parent, all at once
            parents = torch.randint(0, rows, (rows,), generator=gen, device=dev)
            s.update(src=ints(parents), dst=ints(torch.randperm(rows, generator=gen, device=dev)))
        else:                                      # every second row is cut back to a shorter length
            which = torch.randperm(rows, generator=gen, device=dev)[:max(1, rows // 2)]
            keep = (torch.rand((which.numel(),), generator=gen, device=dev) * (tiles * 64)).int()
            s.update(rows=ints(which), keep=ints(keep))
    flat = table[table >= 0].long()
    refs = torch.zeros((pages,), dtype=torch.int32, device=dev)
    refs.index_add_(0, flat, torch.ones_like(flat, dtype=torch.int32))
    s.update(table0=table, refs0=refs, table=table.clone(), refs=refs.clone(),
             status=torch.zeros((4,), dtype=torch.int32, device=dev),
             used=torch.zeros((4,), dtype=torch.int32, device=dev))
    return s


def _pages_plain(s):
    case, op, pool, table, refs = s["case"], s["case"]["op"], s["pool"], s["table"], s["refs"]
    if op == "copy":
        pool[:, s["dst"].long()] = pool[:, s["src"].long()]
        return pool
    table.copy_(s["table0"])
    refs.copy_(s["refs0"])
    one = torch.ones((), dtype=torch.int32, device=pool.device)
    if op == "reserve":
        # the token at lens[b] lands in the last tile (shared by `share` rows): all holders but the last get a
        # copy on the lowest free pages, in row order
        b = torch.arange(case["rows"], device=pool.device)
        t = s["seq"].long() // 64
        old = table[b, t].long()
        last = torch.full((case["pages"],), -1, dtype=torch.long, device=pool.device)
        last.scatter_reduce_(0, old, b, "amax")
        move = (refs[old] > 1) & (last[old] != b)
        b, t, old = b[move], t[move], old[move]
        new = (refs == 0).nonzero().flatten()[:b.numel()]
        pool[:, new] = pool[:, old]
        table[b, t] = new.int()
        refs.index_add_(0, old, -one.expand(b.numel()))
        refs[new] = 1
        return pool, table, refs
    if op == "fork":
        src, dst = s["src"].long(), s["dst"].long()
        fresh, gone = table[src], table[dst]
        for rows, sign in ((fresh, one), (gone, -one)):
            flat = rows[rows >= 0].long()
            refs.index_add_(0, flat, sign.expand(flat.numel()))
        table[dst] = fresh
        return table, refs
    if op == "free":
        rows = s["rows"].long()
        first = (s["keep"].long() + 63) // 64
        drop = torch.arange(table.shape[1], device=pool.device) >= first[:, None]
        old = table[rows]
        flat = old[drop & (old >= 0)].long()
        refs.index_add_(0, flat, -one.expand(flat.numel()))
        table[rows] = torch.where(drop & (old >= 0), -one, old)
        return table, refs
    live = refs > 0
    used = live.sum()
    index = torch.arange(case["pages"], device=pool.device)
    src = index[live & (index >= used)]
    dst = index[~live & (index < used)]
    pool[:, dst] = pool[:, src]
    to = index.clone()
    to[src] = dst
    table.copy_(torch.where(table >= 0, to[table.long().clamp(min=0)].int(), table))
    refs[dst] = refs[src]
    refs[src] = 0
    s["used"][0] = used
    return pool, table, refs, s["used"][:1]


# ---------------------------------------------------------------------------
# rotary positions

_DT = dict(bf16=torch.bfloat16, fp16=torch.float16, fp32=torch.float32)
_THETA, _FACTOR, _LENGTH, _LOW, _HIGH, _MAG = 10000.0, 4.0, 8192, 1.0, 32.0, 1.138629436111989


def _rope_inputs(case, seed, dev):
    gen = torch.Generator(device=dev).manual_seed(seed)
    B, n, Hq, H, d = (case[k] for k in ("B", "n", "Hq", "H", "d"))
    dt = _DT[case["dtype"]]
    # one projection's output, [row, token, head, channel]: q and k are strided views of it
    x = torch.randn((B, n, Hq + H, d), generator=gen, device=dev).to(dt)
    q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:].transpose(1, 2)
    start = (torch.rand((B,), generator=gen, device=dev) * (case["far"] + 1)).int()
    depth = None
    if case["tree"]:
        depth = (torch.rand((B, n), generator=gen, device=dev) * 8).int()
    return dict(case=case, q=q, k=k, start=start, depth=depth,
                q_out=torch.empty((B, Hq, n, d), dtype=dt, device=dev),
                k_out=torch.empty((B, H, n, d), dtype=dt, device=dev))


def _freqs(case, dtype, dev):
    r = case["r"]
    i = torch.arange(r // 2, dtype=dtype, device=dev)
    theta = _THETA * (_FACTOR ** (r / (r - 2)) if case["scaling"] == "base" else 1.0)
    f = theta ** (-2.0 * i / r)
    if case["scaling"] == "linear":
        f = f / _FACTOR
    if case["scaling"] == "parts":                 # fast frequencies stay, slow ones are divided, a ramp between
        keep = ((_LENGTH * f / (2 * math.pi) - _LOW) / (_HIGH - _LOW)).clamp(0, 1)
        f = f * (keep + (1 - keep) / _FACTOR)
    return f


def _magnitude(case):
    return _MAG if case["scaling"] == "parts" else 1.0


def _rope_plain(s):
    case = s["case"]
    r, n = case["r"], case["n"]
    dev = s["q"].device
    pos = s["start"][:, None] + (s["depth"] if s["depth"] is not None else torch.arange(n, device=dev))
    angle = pos.double()[..., None] * _freqs(case, torch.float64, dev)       # far positions: 64 bits
    if case["inverse"]:
        angle = -angle
    cos = (torch.cos(angle) * _magnitude(case)).float()[:, None]
    sin = (torch.sin(angle) * _magnitude(case)).float()[:, None]
    for x, y in ((s["q"], s["q_out"]), (s["k"], s["k_out"])):
        z = x.float()
        if case["inter"]:
            a, b = z[..., 0:r:2], z[..., 1:r:2]
        else:
            a, b = z[..., :r // 2], z[..., r // 2:r]
        u, w = a * cos - b * sin, b * cos + a * sin
        turned = torch.stack([u, w], -1).flatten(-2) if case["inter"] else torch.cat([u, w], -1)
        y.copy_(torch.cat([turned, z[..., r:]], -1))
    return s["q_out"], s["k_out"]


def _rope_exact(case, seed):
    s = _rope_inputs(case, seed, "cuda")
    r, h = case["r"], case["r"] // 2
    base = _THETA * (_FACTOR ** (r / (r - 2)) if case["scaling"] == "base" else 1.0)
    f = [math.exp(-2.0 * i / r * math.log(base)) for i in range(h)]
    if case["scaling"] == "linear":
        f = [x / _FACTOR for x in f]
    if case["scaling"] == "parts":
        keep = [min(1.0, max(0.0, (_LENGTH * x / math.tau - _LOW) / (_HIGH - _LOW))) for x in f]
        f = [x * y + x * (1.0 - y) / _FACTOR for x, y in zip(f, keep)]
    f = torch.tensor(f, dtype=torch.float64, device="cuda")
    step = s["depth"] if s["depth"] is not None else torch.arange(case["n"], device="cuda")
    turn = torch.polar(torch.full((), _magnitude(case), dtype=torch.float64, device="cuda"),
                       (s["start"][:, None] + step).double()[..., None] * f)  # complex numbers on a circle
    if case["inverse"]:
        turn = turn.conj()
    out = []
    for x in (s["q"], s["k"]):
        z = x.double().clone()
        first, second = (slice(0, r, 2), slice(1, r, 2)) if case["inter"] else (slice(0, h), slice(h, r))
        w = torch.complex(z[..., first].contiguous(), z[..., second].contiguous()) * turn[:, None]
        z[..., first], z[..., second] = w.real, w.imag
        out.append(z)
    return tuple(out)


# ---------------------------------------------------------------------------
# the library's calls


class _Handle:
    """A cache handle that is given back with the state."""

    def __init__(self, rq, value):
        self.rq, self.value = rq, value

    def __del__(self):
        try:
            self.rq.rq_cache_destroy(self.value)
        except Exception:
            pass


def _own_state(s):
    import decode_attention_rq_gb300 as rq
    case, op = s["case"], s["case"]["op"]
    s["rq"] = rq
    if op == "tree":
        s["R"] = s["R"].contiguous()               # the library takes R row by row
        cfg = rq.rq_config(1, _P, 1, case["H"], case["d"], case["g"], case["B"], s["nt"] * 64, rq.RQ_MODE_SHARED,
                           case["Hq"])
        if case["paged"]:
            h = rq.rq_cache_create_paged(cfg, s["pages"], s["buf"], s["buf"].numel(), s["table"], s["nt"], s["R"])
        else:
            h = rq.rq_cache_create(cfg, s["buf"], s["buf"].numel(), s["R"])
        size = rq.rq_tree_workspace_bytes(cfg, case["B"], case["T"])
    elif op == "rope":
        kind = dict(none=rq.RQ_ROPE_PLAIN, linear=rq.RQ_ROPE_LINEAR, base=rq.RQ_ROPE_BASE, parts=rq.RQ_ROPE_PARTS)
        s["rope"] = rq.rq_rope_config(head_dim=case["d"], rotary_dim=case["r"], interleaved=int(case["inter"]),
                                      inverse=int(case["inverse"]), scaling=kind[case["scaling"]],
                                      original_len=_LENGTH, theta=_THETA, factor=_FACTOR, low_turns=_LOW,
                                      high_turns=_HIGH, magnitude=_magnitude(case))
        return s
    else:
        cfg = rq.rq_config(case["L"], case["P"], case["G"], case["H"], case["d"], case["g"], case["rows"],
                           case["tiles"] * 64, rq.RQ_MODE_HADAMARD if case["d"] == 128 else rq.RQ_MODE_SHARED, 0)
        R = None if case["d"] == 128 else torch.eye(case["d"], device=s["pool"].device)
        s["R"] = R
        if op == "copy":                           # lists start on a 16-byte boundary
            s.update(src=s["src"].clone(), dst=s["dst"].clone())
        h = rq.rq_cache_create_paged(cfg, case["pages"], s["pool"], s["pool"].numel(), s["table"],
                                     s["table"].shape[1], R)
        size = rq.rq_pages_workspace_bytes(cfg, case["pages"])
    s["handle"] = _Handle(rq, h)
    s["ws"] = torch.zeros((max(size, 16),), dtype=torch.uint8, device="cuda")
    return s


def _tree_own(s):
    c = s["case"]
    s["rq"].rq_tree_attention(s["handle"].value, 0, 0, c["loop"], c["B"], c["T"], s["q"], s["k_new"], s["v_new"],
                              s["mask"], s["count"], s["seq"], s["scale"], s["out"], s["ws"], s["ws"].numel())
    return s["out"]


def _pages_own(s):
    rq, c, op, h = s["rq"], s["case"], s["case"]["op"], s["handle"].value
    if op == "copy":
        rq.rq_pages_copy(h, c["n"], s["src"], s["dst"], s["status"])
        return s["pool"]
    s["table"].copy_(s["table0"])
    s["refs"].copy_(s["refs0"])
    if op == "reserve":
        rq.rq_pages_reserve(h, c["rows"], s["seq"], 1, s["refs"], s["status"], s["ws"], s["ws"].numel())
        return s["pool"], s["table"], s["refs"]
    if op == "fork":
        rq.rq_pages_fork(h, c["rows"], s["src"], s["dst"], s["refs"], s["status"])
        return s["table"], s["refs"]
    if op == "free":
        rq.rq_pages_free(h, s["rows"].numel(), s["rows"], s["keep"], s["refs"], s["status"])
        return s["table"], s["refs"]
    rq.rq_pages_compact(h, s["refs"], s["used"], s["status"], s["ws"], s["ws"].numel())
    return s["pool"], s["table"], s["refs"], s["used"][:1]


def _rope_own(s):
    s["rq"].rq_rope(s["rope"], s["q"], s["k"], s["start"], s["depth"], s["q_out"], s["k_out"])
    return s["q_out"], s["k_out"]


# ---------------------------------------------------------------------------
# what the tools call


def prepare(case, seed):
    if case["op"] == "tree":
        s = _tree_inputs(case, seed, "cuda")
        s["out"] = torch.zeros((case["B"], case["Hq"], case["T"], case["d"]), dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "rope":
        s = _rope_inputs(case, seed, "cuda")
    else:
        s = _pages_inputs(case, seed, "cuda")
    return _own_state(s) if own else s


def run(state):
    op = state["case"]["op"]
    if op == "tree":
        return _tree_own(state) if own else _tree_plain(state)
    if op == "rope":
        return _rope_own(state) if own else _rope_plain(state)
    return _pages_own(state) if own else _pages_plain(state)


def exact(case, seed):
    if case["op"] == "tree":
        return _tree_exact(case, seed)
    if case["op"] == "rope":
        return _rope_exact(case, seed)
    return None


def work(case):
    op = case["op"]
    if op == "tree":
        d, g, H, Hq = case["d"], case["g"], case["H"], case["Hq"]
        a_tile, r_tile = _tile_bytes(d, g)
        per_token = 2 * (a_tile + (r_tile if case["loop"] < _P - 1 else 0)) / 64
        cached = sum(_lens(case))
        nodes = sum(_counts(case))
        keys = sum(m * (n + m) for n, m in zip(_lens(case), _counts(case)))
        return {"bytes": cached * H * per_token + nodes * d * 2 * (2 * Hq + 2 * H), "flops": 4 * Hq * keys * d}
    if op == "rope":
        size = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
        total = case["B"] * case["n"] * (case["Hq"] + case["H"]) * case["d"]
        return {"bytes": 2 * size * total, "flops": 6 * total * case["r"] // (2 * case["d"])}
    table, refs = case["rows"] * (case["tiles"] + 2) * 4, case["pages"] * 4
    page = case["L"] * case["G"] * case["H"] * _head_block(case["d"], case["g"], case["P"])
    if op == "copy":
        return {"bytes": 2 * case["n"] * page, "flops": 0}
    if op == "reserve":
        moved = case["rows"] - case["rows"] // case["share"]
        return {"bytes": 2 * moved * page + 2 * table + 2 * refs, "flops": 0}
    if op == "compact":
        return {"bytes": 2 * case["n"] * page + 2 * table + 2 * refs, "flops": 0}
    return {"bytes": 3 * table + 2 * refs, "flops": 0}
