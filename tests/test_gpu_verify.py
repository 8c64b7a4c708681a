"""GPU: verification of drafted tokens (rq_verify) against a walk in float64 on the host.

Results are whole numbers and have to be equal.  The kernel's products and differences are float32 and its sums true to
about 2^-40; the host repeats the float32 steps (NumPy rounds each operation) and sums in float64, so that a decision could differ
only where a border lies within about 2^-40 of the random number (inputs have 24 bits), or where z's rounding to
float32 falls the other way, as rarely."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, HF, F = torch.bfloat16, torch.float16, torch.float32


def walk(rule, target, draft, tokens, parents, n, accept, sample):
    """One row, NumPy float32 arrays -> path, next."""
    V = target.shape[1]
    prob = lambda x: np.clip(np.nan_to_num(x, nan=0.0, posinf=np.inf, neginf=-np.inf), 0, 1).astype(np.float32)
    if n == 0:
        return [], -1
    path = [0]
    if rule:
        best = lambda t: int(np.argmax(np.where(np.isnan(target[t]), -np.inf, target[t])))
        for t in range(1, n):
            if parents[t] == path[-1] and parents[t] < t and tokens[t] == best(path[-1]):
                path.append(t)
        return path, best(path[-1])
    r, z = prob(target[0]), np.float32(1)
    for t in range(1, n):
        x = tokens[t]
        if parents[t] != path[-1] or parents[t] >= t or not 0 <= x < V:
            continue
        q = prob(draft[parents[t]]) if draft is not None else None
        qx = q[x] if draft is not None else np.float32(1)
        if np.float32(accept[t]) * (z * qx) < r[x]:
            path.append(t)
            r, z = prob(target[t]), np.float32(1)
            continue
        if draft is not None:
            r = np.maximum(r - z * q, np.float32(0))
        else:
            r = r.copy()
            r[x] = 0
        z = np.float32(r.astype(np.float64).sum())
    if not r.max() > 0:
        r = prob(target[path[-1]])
    c = np.cumsum(r.astype(np.float64))
    if not c[-1] > 0:
        return path, -1
    w = min(max(float(np.nan_to_num(sample)), 0.0), 1 - 2.0 ** -24)
    return path, int(np.nonzero(c > w * c[-1])[0][0])


def make(seed, B, T, V, dtype, tree=True, draft=True, guess=0.5, sharp=2.0):
    rng = np.random.default_rng(seed)
    z = sharp * rng.standard_normal((B, T, V)).astype(np.float32)
    p = np.exp(z - z.max(-1, keepdims=True))
    y = z + 0.7 * rng.standard_normal((B, T, V)).astype(np.float32)
    q = np.exp(y - y.max(-1, keepdims=True))
    p, q = (torch.from_numpy(v / v.sum(-1, keepdims=True)).to(dtype) for v in (p, q))
    parents = np.zeros((B, T), dtype=np.int32)
    tokens = np.zeros((B, T), dtype=np.int32)
    qn = q.double().numpy()
    for b in range(B):
        for t in range(1, T):
            parents[b, t] = max(0, t - 1 - int(rng.random() ** 2 * 4)) if tree else t - 1
            c = np.cumsum(qn[b, parents[b, t]])
            tokens[b, t] = (int(p[b, parents[b, t]].float().argmax()) if rng.random() < guess
                            else min(V - 1, np.searchsorted(c, rng.random() * c[-1], side="right")))
    accept = rng.random((B, T)).astype(np.float32)
    sample = rng.random(B).astype(np.float32)
    return p, q if draft else None, tokens, parents, accept, sample


def run(rq, rule, p, q, tokens, parents, counts, accept, sample, stream=None):
    dev = lambda x: None if x is None else (x if isinstance(x, torch.Tensor) else torch.from_numpy(x)).cuda()
    B, T = tokens.shape
    path = torch.full((B, T), 77, dtype=torch.int32, device="cuda")
    n = torch.full((B,), 77, dtype=torch.int32, device="cuda")
    nxt = torch.full((B,), 77, dtype=torch.int32, device="cuda")
    args = [p if p.is_cuda else p.cuda(), q if q is None or q.is_cuda else q.cuda()] + [
        dev(x) for x in (tokens, parents, counts, accept, sample)]
    torch.cuda.synchronize()
    rq.rq_verify(rule, *args, path, n, nxt, stream=stream)
    torch.cuda.synchronize()
    return path.cpu().numpy(), n.cpu().numpy(), nxt.cpu().numpy()


def check(got, rule, p, q, tokens, parents, counts, accept, sample):
    path, n, nxt = got
    P = p.float().cpu().numpy()
    Q = None if q is None else q.float().cpu().numpy()
    T = tokens.shape[1]
    par = parents if parents is not None else np.broadcast_to(np.arange(-1, T - 1), tokens.shape)
    for b in range(len(tokens)):
        m = T if counts is None else min(max(int(counts[b]), 0), T)
        ref, tok = walk(rule, P[b], None if Q is None else Q[b], tokens[b], par[b], m, accept[b], sample[b])
        assert n[b] == len(ref) and path[b].tolist() == ref + [-1] * (T - len(ref)), (b, path[b], ref)
        assert nxt[b] == tok, (b, nxt[b], tok)


@pytest.mark.parametrize("dtype", [F, BF, HF])
@pytest.mark.parametrize("B,T,V", [(1, 1, 1), (2, 3, 2), (3, 5, 31), (2, 9, 1000), (3, 16, 4096), (2, 7, 4097), (2, 33, 8200),
                                   (2, 6, 20000), (1, 12, 50257), (1, 4, 131072), (1, 3, 262144), (40, 256, 67)])
@pytest.mark.parametrize("tree,draft", [(True, True), (False, True), (True, False)])
def test_sample(dtype, B, T, V, tree, draft):
    import decode_attention_rq_gb300 as rq
    case = make(B + T + V, B, T, V, dtype, tree, draft)
    p, q, tokens, parents, accept, sample = case
    parents = parents if tree else None
    check(run(rq, 0, p, q, tokens, parents, None, accept, sample), 0, p, q, tokens, parents, None, accept, sample)


@pytest.mark.parametrize("dtype", [F, BF])
@pytest.mark.parametrize("V", [1, 5, 4096, 50257, 131071])
def test_greedy(dtype, V):
    """Ties in BF16, logits of both signs, NaN and infinities."""
    import decode_attention_rq_gb300 as rq
    rng = np.random.default_rng(V)
    z = torch.from_numpy(4 * rng.standard_normal((4, 9, V)).astype(np.float32)).to(dtype)
    z[1, 0] = -z[1, 0].abs()
    z[2, :, V // 2] = float("nan")
    z[2, 1, V // 3] = float("inf")
    z[3, 0] = -float("inf")
    z[3, 2] = float("nan")
    _, _, tokens, parents, accept, sample = make(V, 4, 9, V, dtype)
    zf = torch.where(torch.isnan(z.float()), -torch.inf, z.float())
    for b in range(4):
        for t in range(1, 9):
            if rng.random() < 0.7:
                tokens[b, t] = int(np.argmax(zf[b, parents[b, t]].numpy()))
    check(run(rq, 1, z, None, tokens, parents, None, None, None), 1, z, None, tokens, parents, None, accept, sample)


def test_ragged_rows_and_bad_nodes():
    """Counts of 0, 1, more than T and below 0; parents that do not come first, tokens outside the vocabulary."""
    import decode_attention_rq_gb300 as rq
    p, q, tokens, parents, accept, sample = make(3, 8, 10, 300, F)
    counts = np.array([0, 1, 10, 99, -3, 5, 7, 2], dtype=np.int32)
    parents[2, 4], parents[2, 5], parents[3, 1], parents[5, 2] = 4, 7, -5, 1 << 30
    tokens[2, 1], tokens[3, 2], tokens[6, 1] = -1, 300, 1 << 30
    check(run(rq, 0, p, q, tokens, parents, counts, accept, sample), 0, p, q, tokens, parents, counts, accept, sample)
    check(run(rq, 1, p, None, tokens, parents, counts, None, None), 1, p, None, tokens, parents, counts, accept, sample)


def test_probabilities_out_of_range():
    """NaN, infinities, negative values, rows of zeros; random numbers at and beyond the ends of [0, 1)."""
    import decode_attention_rq_gb300 as rq
    p, q, tokens, parents, accept, sample = make(4, 12, 6, 5000, F)
    p[0, :, 7], p[1, :, 8], p[2], p[3, :, 4] = float("nan"), float("inf"), 0.0, -3.0
    q[4, :, 5], q[5], q[6, :, 6] = float("nan"), 0.0, float("inf")
    q[7] = p[7]                                      # nothing is left after a rejection
    accept[7] = 1.0
    sample[8:12] = [0.0, 1.0, np.nan, 1 - 2.0 ** -24]
    accept[9], accept[10] = -1.0, np.nan
    check(run(rq, 0, p, q, tokens, parents, None, accept, sample), 0, p, q, tokens, parents, None, accept, sample)
    check(run(rq, 0, p, None, tokens, parents, None, accept, sample), 0, p, None, tokens, parents, None, accept, sample)


def test_the_same_token_twice():
    """Siblings of one token, with and without a draft distribution."""
    import decode_attention_rq_gb300 as rq
    p, q, tokens, parents, accept, sample = make(5, 16, 8, 64, F, sharp=0.5)
    parents[:] = 0
    tokens[:] = tokens[:, 1:2]
    accept[:] = 0.999
    for d in (q, None):
        check(run(rq, 0, p, d, tokens, parents, None, accept, sample), 0, p, d, tokens, parents, None, accept, sample)


@pytest.mark.parametrize("dtype", [F, BF])
def test_strides(dtype):
    """Views: a vocabulary inside a padded one, rows and nodes swapped, a draft of T - 1 nodes, one shared by the rows."""
    import decode_attention_rq_gb300 as rq
    p, q, tokens, parents, accept, sample = make(6, 3, 5, 9000, dtype)
    wide = torch.full((5, 3, 9011), 0.25, dtype=dtype, device="cuda")
    wide[:, :, 3:9003] = p.transpose(0, 1).cuda()
    target = wide.transpose(0, 1)[:, :, 3:9003]
    draft = q[:, :4].contiguous().cuda()
    check(run(rq, 0, target, draft, tokens, parents, None, accept, sample), 0, p, q, tokens, parents, None, accept, sample)
    one = q[:1].cuda().expand(3, 5, 9000)
    check(run(rq, 0, target, one, tokens, parents, None, accept, sample), 0, p, q[:1].expand(3, 5, 9000), tokens, parents,
          None, accept, sample)


def test_frequencies_follow_the_target():
    """Many rows of one small problem: the first token that comes out is distributed as p.  4 sigma of a binomial."""
    import decode_attention_rq_gb300 as rq
    rng = np.random.default_rng(9)
    B, T, V = 40000, 4, 6
    p = np.array([0.4, 0.3, 0.15, 0.1, 0.05, 0.0], dtype=np.float32)
    q = np.array([0.1, 0.2, 0.3, 0.1, 0.2, 0.1], dtype=np.float32)
    parents = np.zeros((B, T), dtype=np.int32)               # three siblings drawn from q
    tokens = rng.choice(V, size=(B, T), p=q / q.astype(np.float64).sum()).astype(np.int32)
    P = torch.from_numpy(p).expand(B, T, V).cuda()
    Q = torch.from_numpy(q).expand(B, T, V).cuda()
    accept, sample = rng.random((B, T)).astype(np.float32), rng.random(B).astype(np.float32)
    path, n, nxt = run(rq, 0, P, Q, tokens, parents, None, accept, sample)
    first = np.where(n > 1, tokens[np.arange(B), path[:, 1]], nxt)
    got = np.bincount(first, minlength=V) / B
    assert (np.abs(got - p) <= 4 * np.sqrt(p * (1 - p) / B) + 1e-12).all(), got


def test_storage_behind_4gb_and_another_stream():
    import decode_attention_rq_gb300 as rq
    B, T, V = 3, 70, 20011
    p, q, tokens, parents, accept, sample = make(10, B, 4, V, BF)
    big = torch.zeros((B, 2, 36000, V), dtype=BF, device="cuda")     # 4.3e9 elements: rows lie 1.4e9 elements apart
    big[:, 1, :4] = p.cuda()
    check(run(rq, 0, big[:, 1, :4], q, tokens, parents, None, accept, sample, torch.cuda.Stream()), 0, p, q, tokens,
          parents, None, accept, sample)


@pytest.mark.parametrize("dtype", [F, BF])
@pytest.mark.parametrize("B,T,V", [(44, 5, 50257), (1, 256, 131072), (70, 256, 1003)])
def test_greedy_of_many_values(dtype, B, T, V):
    """More than 32 MB of target rows: one node after another."""
    import decode_attention_rq_gb300 as rq
    g = torch.Generator(device="cuda").manual_seed(V)
    z = torch.randn(B, T, V, generator=g, device="cuda").to(dtype)
    best = torch.nan_to_num(z.float()).argmax(-1).cpu().numpy()
    rng = np.random.default_rng(V)
    parents = np.array([[max(0, t - 1 - int(rng.random() ** 2 * 4)) for t in range(T)] for _ in range(B)], dtype=np.int32)
    tokens = rng.integers(0, V, (B, T)).astype(np.int32)
    for b in range(B):
        for t in range(1, T):
            if rng.random() < 0.6:
                tokens[b, t] = best[b, parents[b, t]]
    counts = rng.integers(0, T + 1, B).astype(np.int32) if B > 1 else None
    path, n, nxt = run(rq, 1, z, None, tokens, parents, counts, None, None)
    for b in range(B):
        m = T if counts is None else counts[b]
        ref = [0] if m else []
        for t in range(1, m):
            if parents[b, t] == ref[-1] and tokens[b, t] == best[b, ref[-1]]:
                ref.append(t)
        assert n[b] == len(ref) and path[b].tolist() == ref + [-1] * (T - len(ref)), b
        assert nxt[b] == (best[b, ref[-1]] if ref else -1), b


@pytest.mark.parametrize("V", [17, 40, 5000, 70001])
@pytest.mark.parametrize("step", [1, 37, 4000])
def test_siblings_that_take_nearly_all(V, step):
    """No draft distribution: each sibling refused takes half of what is left, twelve times; some tokens come twice."""
    import decode_attention_rq_gb300 as rq
    B, T = 24, 16
    rng = np.random.default_rng(V + step)
    p = torch.from_numpy(2.0 ** -16 * rng.random((B, T, V))).float() / V
    where = (np.arange(T) * step + 3) % V
    for i, x in enumerate(where):
        p[:, 0, x] = 2.0 ** -(i + 1)
    if V == 17:
        p[B // 2:, 0, 12:] = 0
    tokens = np.broadcast_to(where.astype(np.int32), (B, T)).copy()
    tokens[:, 1:] = tokens[:, :-1]                       # node t: the t-th heaviest
    tokens[::3, 5] = tokens[::3, 4]
    parents = np.zeros((B, T), dtype=np.int32)
    counts = np.arange(B, dtype=np.int32) % (T + 1)
    accept = (1 - 2.0 ** -10 * rng.random((B, T))).astype(np.float32)
    sample = rng.random(B).astype(np.float32)
    check(run(rq, 0, p, None, tokens, parents, counts, accept, sample), 0, p, None, tokens, parents, counts, accept, sample)


def test_graphs_and_calls_at_once():
    """Both rules captured into a graph each, replayed on two streams at once with inputs that change in between, beside
    eager calls; greedy by nodes at once and by nodes in turn (more than 32 MB of target rows)."""
    import decode_attention_rq_gb300 as rq
    dev = lambda x: torch.from_numpy(x).cuda()
    sets = []
    for rule, B, T, V in ((0, 5, 9, 9000), (1, 5, 9, 9001), (1, 30, 6, 50257)):
        cases = [make(60 + i, B, T, V, F, guess=0.8) for i in range(2)]
        p, q, tokens, parents, accept, sample = cases[0]
        ins = [p.cuda(), q.cuda() if rule == 0 else None] + [dev(x) for x in (tokens, parents)]
        ins += [None] + ([dev(accept), dev(sample)] if rule == 0 else [None, None])
        out = [torch.full(s, 77, dtype=torch.int32, device="cuda") for s in ((B, T), (B,), (B,))]
        sets.append((rule, cases, ins, out))

    def go(s, out=None):
        rq.rq_verify(s[0], *s[2], *(out or s[3]))

    def fill(s, i):
        p, q, tokens, parents, accept, sample = s[1][i]
        for x, y in zip(s[2], (p, q, dev(tokens), dev(parents), None, dev(accept), dev(sample))):
            if x is not None:
                x.copy_(y)

    for s in sets:
        go(s)
    torch.cuda.synchronize()
    graphs, streams = [], [torch.cuda.Stream() for _ in sets]
    for s in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            go(s)
            go(s)
    for i in (1, 0):
        for s in sets:
            fill(s, i)
            for x in s[3]:
                x.fill_(77)
        torch.cuda.synchronize()
        eager = [[torch.empty_like(x) for x in s[3]] for s in sets]
        for _ in range(3):
            for g, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
            for s, e in zip(sets, eager):
                go(s, e)
        torch.cuda.synchronize()
        for s, e in zip(sets, eager):
            p, q, tokens, parents, accept, sample = s[1][i]
            for got in (s[3], e):
                check([x.cpu().numpy() for x in got], s[0], p, q if s[0] == 0 else None, tokens, parents, None, accept, sample)


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("V", [40, 5000, 70001])
def test_refusals_side_by_side(V, kept):
    """No draft distribution: siblings next to each other, their probabilities spread over 2^30, all refused, with nothing
    or a little left beside them and half of all elsewhere.  The samples count as 0: the next token is the first of anything."""
    import decode_attention_rq_gb300 as rq
    B, T, at = 96, 9, V // 3
    rng = np.random.default_rng(V)
    p = np.zeros((B, T, V), dtype=np.float32)
    p[:, 0, V - 1] = 0.5
    p[:, 0, at:at + T - 1] = rng.random((B, T - 1)) * 2.0 ** -(4 + 30 * rng.random((B, T - 1)))
    if kept:
        p[:, 0, at + T] = 2.0 ** -(40 + 20 * rng.random(B))
    tokens = np.full((B, T), at, dtype=np.int32)
    for b in range(B):
        tokens[b, 1:] += rng.permutation(T - 1).astype(np.int32)
    parents, accept = np.zeros((B, T), dtype=np.int32), np.ones((B, T), dtype=np.float32)
    sample = np.array([0.0, -1.0, np.nan, -0.0], dtype=np.float32)[np.arange(B) % 4]
    p = torch.from_numpy(p)
    check(run(rq, 0, p, None, tokens, parents, None, accept, sample), 0, p, None, tokens, parents, None, accept, sample)
