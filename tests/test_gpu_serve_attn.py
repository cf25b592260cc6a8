"""gqa_attn_fwd_varlen and gqa_attn_fwd_tree against a 64-bit implementation, element by
element, with tolerances derived from the kernels' roundings (see serve_ref)."""
import numpy as np
import pytest

from tests import serve_ref as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import gqa_exact_attention_b200 as G  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.load_serve()
    yield
    assert G.gqa_serve_device_status(reset=True) == 0, "an in-kernel wait timed out"


def randn(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).bfloat16()


def f64(t):
    return t.double().cpu().numpy()


def cu(lens, start=0):
    return torch.tensor(np.concatenate([[start], start + np.cumsum(lens)]), dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- packed prompts

def varlen_ref(q, k, v, cq, ck, causal, scale):
    """Over [total, H, d] host arrays in 64 bits: out, lse, tolerances, and the rows of a sequence."""
    Tq, Hq, d = q.shape
    out, tol = np.zeros((Tq, Hq, d)), np.zeros((Tq, Hq, d))
    lse, ltol = np.full((Hq, Tq), -np.inf), np.zeros((Hq, Tq))
    inside = np.zeros(Tq, dtype=bool)
    for a, b, c, e in zip(cq[:-1], cq[1:], ck[:-1], ck[1:]):
        see = R.causal(b - a, e - c) if causal else np.ones((b - a, e - c), dtype=bool)
        out[a:b], lse[:, a:b], tol[a:b], ltol[:, a:b] = R.attn(q[a:b], k[c:e], v[c:e], see, scale)
        inside[a:b] = True
    return out, lse, tol, ltol, inside


def run_varlen(rng, lq, lk, Hq, Hk, d, causal, bf16=False, start=0, after=0, scale=None):
    tq, tk = start + sum(lq) + after, start + sum(lk) + after
    q, k, v = randn(rng, tq, Hq, d), randn(rng, tk, Hk, d), randn(rng, tk, Hk, d)
    cq, ck = cu(lq, start), cu(lk, start)
    dt = torch.bfloat16 if bf16 else torch.float32
    out = torch.full((tq, Hq, d), 7.0, dtype=dt, device="cuda")
    lse = torch.full((Hq, tq), 7.0, device="cuda")
    G.gqa_attn_fwd_varlen(q.cuda(), k.cuda(), v.cuda(), cq, ck, out=out, lse=lse, causal=causal, scale=scale)
    torch.cuda.synchronize()
    s = d ** -0.5 if scale is None else scale
    o, l, tol, ltol, inside = varlen_ref(f64(q), f64(k), f64(v), cq.cpu().numpy(), ck.cpu().numpy(), causal, s)
    R.check(out[torch.from_numpy(inside).cuda()], lse[:, torch.from_numpy(inside).cuda()], o[inside],
            l[:, inside], tol[inside], ltol[:, inside], bf16)
    outside = torch.from_numpy(~inside).cuda()
    assert (out[outside] == 7.0).all() and (lse[:, outside] == 7.0).all()


VARLEN = [
    # query lengths, key lengths (None: the same), Hq, Hk, d
    ([1], None, 8, 2, 64),
    ([5], None, 1, 1, 128),
    ([0, 1, 2, 0, 63, 64, 65], None, 8, 2, 128),
    ([127, 128, 129, 33], None, 8, 2, 64),
    ([256, 0, 257, 255], None, 4, 4, 128),       # g = 1
    ([300, 41, 42, 43], None, 6, 2, 64),         # g = 3: 42 positions a tile
    ([90, 700], None, 8, 1, 128),                # g = 8
    ([50, 3, 130], None, 130, 1, 64),            # g = 130: a group above one tile's rows
    ([20, 30], None, 48, 1, 64),                 # g = 48
    ([1, 1, 1, 7], [900, 1, 127, 2000], 8, 2, 128),      # single queries behind contexts
    ([100, 1, 64], [333, 129, 64], 8, 2, 64),
    ([300, 10, 70], [100, 0, 1], 4, 2, 64),      # fewer keys than queries: rows without a key
]


@pytest.mark.parametrize("case", range(len(VARLEN)))
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
def test_varlen(case, causal, bf16):
    lq, lk, Hq, Hk, d = VARLEN[case]
    rng = np.random.default_rng(100 + case)
    run_varlen(rng, lq, lk or lq, Hq, Hk, d, causal, bf16)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bf16", [False, True])
def test_varlen_rows_outside_the_sequences_stay(d, bf16):
    run_varlen(np.random.default_rng(7), [70, 0, 200, 3], [70, 5, 210, 3], 8, 2, d, True, bf16, start=5, after=150)


@pytest.mark.parametrize("scale", [-0.3, 0.0, 2.5])
def test_varlen_scales(scale):
    run_varlen(np.random.default_rng(8), [150, 40], [150, 300], 4, 2, 64, True, scale=scale)


@pytest.mark.parametrize("B", [700, 1500])
def test_varlen_many_sequences(B):
    rng = np.random.default_rng(9)
    lens = [int(x) for x in rng.integers(0, 40, B)]
    run_varlen(rng, lens, lens, 4, 2, 64, True)


@pytest.mark.parametrize("Hq,Hk,d", [(32, 32, 128), (64, 8, 64), (24, 8, 128), (32, 8, 64)])
@pytest.mark.parametrize("causal", [False, True])
def test_varlen_many_tiles(Hq, Hk, d, causal):
    """Enough tiles for several rounds of two-tile units on every SM, of ragged sequences."""
    rng = np.random.default_rng(15)
    lens = [800, 0, 1100, 5, 700, 257, 512, 1, 640, 900]
    run_varlen(rng, lens, lens, Hq, Hk, d, causal, bf16=True, start=3, after=70)
    run_varlen(rng, lens, [x + 100 * (i % 3) for i, x in enumerate(lens)], Hq, Hk, d, causal)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_varlen_neighbours_do_not_leak(d, causal):
    """Infinities and NaN in every other sequence leave the ones between them as they are."""
    rng = np.random.default_rng(10)
    lens = [50, 77, 130, 200, 1, 129]
    q, k, v = (randn(rng, sum(lens), H, d).cuda() for H in (8, 2, 2))
    c = cu(lens)
    a, la = G.gqa_attn_fwd_varlen(q, k, v, c, causal=causal)
    at = np.concatenate([[0], np.cumsum(lens)])
    q2, k2, v2 = q.clone(), k.clone(), v.clone()
    for b in (1, 3, 5):
        for t, x in ((q2, float("nan")), (k2, float("inf")), (v2, float("nan"))):
            t[at[b]:at[b + 1]] = x
    o, lo = G.gqa_attn_fwd_varlen(q2, k2, v2, c, causal=causal)
    torch.cuda.synchronize()
    for b in (0, 2, 4):
        assert torch.equal(o[at[b]:at[b + 1]], a[at[b]:at[b + 1]])
        assert torch.equal(lo[:, at[b]:at[b + 1]], la[:, at[b]:at[b + 1]])


@pytest.mark.parametrize("d", [64, 128])
def test_varlen_columns_of_one_projection(d):
    rng = np.random.default_rng(11)
    lens, Hq, Hk = [100, 37, 256], 8, 2
    qkv = randn(rng, sum(lens), Hq + 2 * Hk, d).cuda()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    a = G.gqa_attn_fwd_varlen(q, k, v, cu(lens), causal=True)
    b = G.gqa_attn_fwd_varlen(q.contiguous(), k.contiguous(), v.contiguous(), cu(lens), cu(lens), causal=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_varlen_without_rows_or_keys():
    rng = np.random.default_rng(12)
    q = randn(rng, 9, 4, 64).cuda()
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    out, lse = G.gqa_attn_fwd_varlen(q, none, none, cu([4, 5]), cu([0, 0]))
    assert (out == 0).all() and torch.isneginf(lse).all()
    out, lse = G.gqa_attn_fwd_varlen(q[:0], none, none, cu([0, 0]))
    assert out.shape == (0, 4, 64) and lse.shape == (4, 0)


def test_varlen_bounds_are_clamped():
    """Bounds below 0 or past the rows are read as 0 and the number of rows."""
    rng = np.random.default_rng(13)
    q, k, v = (randn(rng, 100, H, 64).cuda() for H in (4, 2, 2))
    wild = torch.tensor([-5, 40, 10 ** 6], dtype=torch.int32, device="cuda")
    tame = torch.tensor([0, 40, 100], dtype=torch.int32, device="cuda")
    a, b = G.gqa_attn_fwd_varlen(q, k, v, wild, causal=True), G.gqa_attn_fwd_varlen(q, k, v, tame, causal=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_varlen_equals_the_dense_forward_on_equal_lengths():
    """Each side rounds its own weights to bf16, relatively by at most 2^-8 (their sum keeps them
    unrounded), so each output is within 2^-8 sum_j w_j |v_j| <= 2^-8 max |v| of the definition
    (and fp32 steps, 2 % of that), and the two are within twice that of each other."""
    rng = np.random.default_rng(14)
    B, S, Hq, Hk, d = 3, 300, 8, 2, 128
    q, k, v = randn(rng, B, S, Hq, d).cuda(), randn(rng, B, S, Hk, d).cuda(), randn(rng, B, S, Hk, d).cuda()
    o, l = G.gqa_attn_fwd(q, k, v, causal=True)
    a, la = G.gqa_attn_fwd_varlen(q.flatten(0, 1), k.flatten(0, 1), v.flatten(0, 1), cu([S] * B), causal=True)
    assert (a.view(B, S, Hq, d) - o).abs().max() <= 2 * 1.02 * 2.0 ** -8 * v.float().abs().max()
    assert (la.view(Hq, B, S).transpose(0, 1) - l).abs().max() <= 1e-3


# ---------------------------------------------------------------- trees over a cache

def bits(see):
    T = see.shape[-1]
    W = (T + 31) // 32
    full = np.zeros(see.shape[:-1] + (W * 32,), dtype=np.uint64)
    full[..., :T] = see
    w = (full.reshape(see.shape[:-1] + (W, 32)) << np.arange(32, dtype=np.uint64)).sum(-1)
    return torch.from_numpy(w.astype(np.uint32).view(np.int32)).cuda()


def tree(rng, T):
    see = np.zeros((T, T), dtype=bool)
    for i in range(T):
        p = int(rng.integers(max(-1, i - 5), i)) if i else -1
        if p >= 0:
            see[i] = see[p]
        see[i, i] = True
    return see


def run_tree(rng, lens, T, Hq, Hk, d, page, n=None, see=None, shared=False, bf16=False, cap=None,
             poison=True):
    B = len(lens)
    cap = cap or max(max(lens), 1) + 5
    nodes = [min(T, L) if n is None else min(max(n[b], 0), T, L) for b, L in enumerate(lens)]
    if see is None:
        see = np.stack([tree(rng, T) for _ in range(1 if shared else B)])
    q = randn(rng, B, T, Hq, d)
    kv = [randn(rng, B, cap, Hk, d) for _ in range(2)]
    dirty = [x.clone() for x in kv]
    if poison:  # what lies past a sequence's keys does not matter
        for x, bad in zip(dirty, (float("inf"), float("nan"))):
            for b, L in enumerate(lens):
                x[b, L:] = bad
    args = dict(tree_lens=None if n is None else torch.tensor(n, dtype=torch.int32, device="cuda"),
                out_dtype=torch.bfloat16 if bf16 else torch.float32)
    if page:
        M = -(-cap // page)
        perm = rng.permutation(B * M + 3)
        table = np.empty((B, M), dtype=np.int32)
        pools = [torch.full((B * M + 3, page, Hk, d), float("nan")).bfloat16() for _ in range(2)]
        for b in range(B):
            used = -(-lens[b] // page)
            table[b] = perm[b * M:b * M + M]
            for pool, x in zip(pools, dirty):
                for j in range(M):
                    rows = x[b, j * page:(j + 1) * page]
                    pool[table[b, j], :len(rows)] = rows
            table[b, used:] = rng.choice([-1, 10 ** 9, B * M + 3], M - used)  # never used
        args["block_table"] = torch.from_numpy(table).cuda()
        k, v = (x.cuda() for x in pools)
    else:
        k, v = (x.cuda() for x in dirty)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = G.gqa_attn_fwd_tree(q.cuda(), k, v, bits(see[0] if shared else see), sl, **args)
    torch.cuda.synchronize()
    for b, L in enumerate(lens):
        m = nodes[b]
        ok = np.zeros((T, L), dtype=bool)
        ok[:m] = True
        ok[:m, L - m:] = see[0 if shared else b][:m, :m]
        o, l, tol, ltol = R.attn(f64(q[b]), f64(kv[0][b, :L]), f64(kv[1][b, :L]), ok, d ** -0.5)
        R.check(out[b], lse[b], o, l, tol, ltol, bf16, f"sequence {b}")
    return q, k, v, sl, args, out, lse


TREE = [
    # lengths, T, Hq, Hk, d
    ([1], 1, 1, 1, 64),
    ([300, 1, 129, 5], 8, 8, 2, 64),
    ([300, 31, 200, 128, 0], 31, 8, 2, 128),
    ([500, 64, 127], 33, 8, 2, 64),          # T across two words, tiles of 132 rows
    ([257, 600], 65, 4, 4, 128),             # g = 1
    ([400, 90], 61, 6, 2, 128),              # g = 3
    ([1000, 150, 97], 96, 8, 1, 64),         # many tiles
    ([200, 40], 20, 130, 1, 64),             # a group above one tile's rows
    ([3000, 100], 4, 32, 8, 128),
]


@pytest.mark.parametrize("case", range(len(TREE)))
@pytest.mark.parametrize("page", [0, 16, 64, 256])
@pytest.mark.parametrize("bf16", [False, True])
def test_tree(case, page, bf16):
    lens, T, Hq, Hk, d = TREE[case]
    run_tree(np.random.default_rng(200 + case), lens, T, Hq, Hk, d, page, bf16=bf16)


@pytest.mark.parametrize("page", [0, 32])
def test_tree_lens(page):
    run_tree(np.random.default_rng(30), [300, 300, 300, 300, 2], 12, 8, 2, 128, page, n=[12, 0, 5, -3, 12])
    run_tree(np.random.default_rng(31), [140, 135, 129], 40, 8, 2, 64, page, n=[33, 32, 100])


@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("T", [7, 40])
def test_tree_any_mask(T, page):
    """Bits of any kind: rows that see nothing of the tree, everything, later nodes."""
    rng = np.random.default_rng(32)
    see = rng.random((3, T, T)) < 0.5
    see[0, 0], see[0, 1], see[1, T - 1] = False, True, False
    run_tree(rng, [T, 333, 128 + T // 2], T, 8, 2, 64, page, see=see)


def test_tree_rows_that_see_no_key():
    rng = np.random.default_rng(33)
    see = np.zeros((2, 5, 5), dtype=bool)
    see[1, 2, 3] = True
    run_tree(rng, [5, 5], 5, 4, 2, 64, 16, see=see)  # no context: only one row has a key


@pytest.mark.parametrize("page", [0, 64])
def test_tree_shared_mask(page):
    run_tree(np.random.default_rng(34), [100, 260, 31], 24, 8, 2, 128, page, shared=True)


@pytest.mark.parametrize("offset", [-1, 0, 1, 31, 32, 33, 100])
def test_tree_across_a_block_border(offset):
    """The tree's first key at every kind of place in a 128-key block."""
    T = 50
    run_tree(np.random.default_rng(35), [256 + offset + T], T, 4, 1, 64, 0)


def test_tree_of_a_chain_is_causal_attention():
    rng = np.random.default_rng(36)
    T = 9
    q, k, v, sl, args, out, lse = run_tree(rng, [77, 200, 9], T, 8, 2, 128, 0, see=np.tril(np.ones((3, T, T), dtype=bool)),
                                           poison=False)
    o, l = G.gqa_attn_fwd_kvcache(q.cuda(), k, v, sl, causal=True)
    # two roundings of the weights, as in the comparison with the dense forward
    assert (o - out).abs().max() <= 2 * 1.02 * 2.0 ** -8 * v.float().abs().max() and (l - lse).abs().max() <= 1e-3


def test_tree_entry_outside_the_pool_reads_zeros():
    rng = np.random.default_rng(37)
    B, T, Hq, Hk, d, page, L = 1, 3, 4, 2, 64, 16, 100
    q, k, v = randn(rng, B, T, Hq, d), randn(rng, 8, page, Hk, d), randn(rng, 8, page, Hk, d)
    table = np.array([[3, 8, 5, -1, 0, 1, 2]], dtype=np.int32)
    see = np.tril(np.ones((1, T, T), dtype=bool))
    out, lse = G.gqa_attn_fwd_tree(q.cuda(), k.cuda(), v.cuda(), bits(see), torch.tensor([L], dtype=torch.int32, device="cuda"),
                                   block_table=torch.from_numpy(table).cuda())
    rows = lambda x: np.concatenate([f64(x[p]) if 0 <= p < 8 else np.zeros((page, Hk, d)) for p in table[0]])[:L]  # noqa: E731
    ok = np.ones((T, L), dtype=bool)
    ok[:, L - T:] = see[0]
    R.check(out[0], lse[0], *R.attn(f64(q[0]), rows(k), rows(v), ok, d ** -0.5))


# ---------------------------------------------------------------- streams, graphs, repeats

def _both(rng, scale=1):
    lens = [scale * x for x in (300, 17, 128, 999)]
    q, k, v = (randn(rng, sum(lens), H, 128).cuda() for H in (32, 8, 8))
    c = cu(lens)
    tq = randn(rng, 3, 10, 8, 128).cuda()
    kc, vc = randn(rng, 3, 700, 2, 128).cuda(), randn(rng, 3, 700, 2, 128).cuda()
    mask = bits(np.stack([tree(rng, 10) for _ in range(3)]))
    sl = torch.tensor([700, 10, 400], dtype=torch.int32, device="cuda")

    def call():
        return (*G.gqa_attn_fwd_varlen(q, k, v, c, causal=True), *G.gqa_attn_fwd_tree(tq, kc, vc, mask, sl))
    return call, (q, tq)


@pytest.mark.parametrize("scale", [1, 4])
def test_repeats_and_other_streams_give_the_same_bits(scale):
    call, _ = _both(np.random.default_rng(40), scale)
    want = call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = call()
    again = call()  # at the same time as the other stream's
    torch.cuda.synchronize()
    for a, b, c in zip(want, got, again):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("scale", [1, 4])
def test_captured_graphs(scale):
    """Two graphs, replayed in turn and at once with new inputs, give what the calls give."""
    pairs = []
    for seed in (41, 42):
        call, inputs = _both(np.random.default_rng(seed), scale)
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = call()
        pairs.append((call, inputs, graph, got))
    for _, inputs, _, _ in pairs:
        for x in inputs:
            x.mul_(-0.5)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for (_, _, graph, _), s in zip(pairs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for call, _, _, got in pairs:
        for a, b in zip(got, call()):
            assert torch.equal(a, b)


# ---------------------------------------------------------------- nothing else is written

class Canary:
    """A tensor inside a buffer of a pattern that no result has."""

    def __init__(self, shape, dtype, pad=4096):
        self.n, self.pad = int(np.prod(shape)), pad
        self.buf = torch.full((self.n + 2 * pad,), -123.0, dtype=dtype, device="cuda")
        self.t = self.buf[pad:pad + self.n].view(shape)

    def untouched(self):
        return bool((self.buf[:self.pad] == -123.0).all() and (self.buf[self.pad + self.n:] == -123.0).all())

    def written(self):
        return not bool((self.t == -123.0).any())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lens,Hq,Hk,d", [([33, 1, 0, 127], 6, 2, 64), ([700, 900, 1, 640, 513], 32, 8, 128),
                                          ([300, 5000], 8, 2, 64), ([900, 700, 650], 64, 8, 64)])
def test_varlen_writes_its_outputs_and_nothing_else(lens, Hq, Hk, d, dtype):
    rng = np.random.default_rng(50)
    q, k, v = (randn(rng, sum(lens), H, d).cuda() for H in (Hq, Hk, Hk))
    out, lse = Canary((sum(lens), Hq, d), dtype), Canary((Hq, sum(lens)), torch.float32)
    G.gqa_attn_fwd_varlen(q, k, v, cu(lens), out=out.t, lse=lse.t, causal=True)
    torch.cuda.synchronize()
    assert out.untouched() and lse.untouched() and out.written() and lse.written()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,Hq,Hk,d", [(1, 8, 2, 64), (31, 8, 2, 128), (45, 8, 2, 128), (100, 6, 2, 64)])
def test_tree_writes_its_outputs_and_nothing_else(T, Hq, Hk, d, dtype):
    rng = np.random.default_rng(51)
    B, cap = 3, 1500
    q, k, v = randn(rng, B, T, Hq, d).cuda(), randn(rng, B, cap, Hk, d).cuda(), randn(rng, B, cap, Hk, d).cuda()
    sl = torch.tensor([1500, 7, 0], dtype=torch.int32, device="cuda")
    out, lse = Canary((B, T, Hq, d), dtype), Canary((B, Hq, T), torch.float32)
    G.gqa_attn_fwd_tree(q, k, v, bits(tree(rng, T)), sl, out=out.t, lse=lse.t)
    torch.cuda.synchronize()
    assert out.untouched() and lse.untouched() and out.written() and lse.written()


@pytest.mark.parametrize("cap", [600, 20000])
def test_one_sequence_shared_by_all_ctas(cap):
    """A unit in many parts: one kv head, one long sequence."""
    run_tree(np.random.default_rng(52), [cap], 5, 4, 1, 128, 64)
    run_varlen(np.random.default_rng(53), [3], [cap], 4, 1, 64, True, bf16=True)


def test_a_given_stream():
    rng = np.random.default_rng(55)
    lens = [64, 300]
    a, b, c = (randn(rng, sum(lens), H, 64).cuda() for H in (4, 2, 2))
    x = G.gqa_attn_fwd_varlen(a, b, c, cu(lens), causal=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y = G.gqa_attn_fwd_varlen(a, b, c, cu(lens), causal=True, stream=s)
    s.synchronize()
    assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    with pytest.raises(ValueError):
        G.gqa_attn_fwd_varlen(a, b, c, cu(lens), stream=7)


def test_random_shapes_of_the_whole_range():
    """Shapes drawn over the range, against the 64-bit implementation on a sample of heads."""
    rng = np.random.default_rng(56)
    for _ in range(12):
        Hk, g, d = int(rng.choice([1, 2, 4])), int(rng.choice([1, 2, 3, 5, 8])), int(rng.choice([64, 128]))
        B = int(rng.integers(1, 7))
        lq = [int(x) for x in rng.integers(0, int(rng.choice([5, 80, 600])), B)]
        lk = [a + int(x) for a, x in zip(lq, rng.integers(0, int(rng.choice([1, 900])), B))]
        run_varlen(rng, lq, lk, Hk * g, Hk, d, bool(rng.integers(2)), bool(rng.integers(2)),
                   start=int(rng.integers(0, 3)), after=int(rng.integers(0, 200)))
        T = int(rng.choice([1, 3, 17, 64, 90]))
        lens = [int(x) for x in rng.integers(0, 1500, B)]
        run_tree(rng, lens, T, Hk * g, Hk, d, int(rng.choice([0, 16, 32, 128, 512])),
                 n=[int(x) for x in rng.integers(0, T + 2, B)] if rng.integers(2) else None, bf16=bool(rng.integers(2)))


def test_more_sequences_than_a_cta_sums_up():
    """Above 1024 sequences a kernel in front sums up the schedule: units that are split and units
    that are not, prompts and trees."""
    rng = np.random.default_rng(57)
    lens = [0] * 2000
    for b in rng.integers(0, 2000, 60):
        lens[b] = int(rng.integers(1, 9))
    run_varlen(rng, lens, lens, 4, 2, 64, True)
    short = [int(x) for x in rng.integers(0, 40, 1100)]
    run_tree(rng, short, 2, 2, 1, 64, 0)
    run_tree(rng, short[:1090] + [700] * 10, 2, 2, 1, 64, 16)
    run_tree(rng, short, 70, 2, 1, 64, 16)  # two tiles


def test_outputs_of_a_given_stream_come_from_its_memory():
    """Memory freed on the current stream may still be in use there, so that a call on another
    stream must not be given it for its outputs."""
    rng = np.random.default_rng(57)
    T, Hq = 5000, 8
    a, b, c = (randn(rng, T, H, 64).cuda() for H in (Hq, 2, 2))
    bounds = cu([T])
    refs, lens = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    table, to = torch.full((2, 2), -1, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    x = G.gqa_attn_fwd_varlen(a, b, c, bounds)
    st = G.gqa_cache_resize(table, lens, refs, 16, to)
    torch.cuda.synchronize()
    expect = [x[0].clone(), x[1].clone(), st.clone()]
    s = torch.cuda.Stream()
    was = [t.data_ptr() for t in (*x, st)]
    del x, st  # the current stream has these to give
    y = G.gqa_attn_fwd_varlen(a, b, c, bounds, stream=s)
    st = G.gqa_cache_resize(table, lens, refs, 16, to, stream=s)
    s.synchronize()
    got = [*y, st]
    assert all(torch.equal(p, q) for p, q in zip(expect, got))
    assert not set(was) & {t.data_ptr() for t in got}
    assert torch.cuda.current_stream() != s
