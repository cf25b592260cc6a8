"""gqa_cache_resize, gqa_cache_fork and gqa_cache_compact: state and pools equal, value for value,
what a program of one request after the other gives, over long random runs and at the borders;
and a run of all serving calls together."""
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


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Both:
    """The calls on the device beside the model on the host."""

    def __init__(self, S, M, P, ps, layers=2, Hk=2, d=64, seed=0, dtype=torch.bfloat16):
        g = torch.Generator().manual_seed(seed)
        # int16 or int8 patterns: every value is exact on both sides
        self.bits = torch.int8 if dtype.itemsize == 1 else torch.int16
        shape = (layers, P, ps, Hk, d)
        raw = [torch.randint(-100, 100, shape, dtype=self.bits, generator=g) for _ in range(2)]
        self.k, self.v = (x.cuda().view(dtype) for x in raw)
        self.model = R.Pages(S, M, P, ps, [x.numpy().reshape(layers, P, ps, Hk * d).copy() for x in raw])
        self.table, self.lens, self.refs = ints(self.model.table), ints(self.model.lens), ints(self.model.refs)
        self.state = (self.table, self.lens, self.refs)

    def same(self, status, want):
        torch.cuda.synchronize()
        m = self.model
        assert status.cpu().tolist() == list(want)
        assert np.array_equal(self.lens.cpu().numpy(), m.lens)
        assert np.array_equal(self.refs.cpu().numpy(), m.refs)
        assert np.array_equal(self.table.cpu().numpy(), m.table)
        for t, x in zip((self.k, self.v), m.pools):
            assert np.array_equal(t.view(self.bits).cpu().numpy().reshape(x.shape), x)

    def resize(self, slots, new):
        st = G.gqa_cache_resize(*self.state, self.model.ps, ints(new), None if slots is None else ints(slots))
        want = self.model.resize(list(range(len(new))) if slots is None else list(slots), list(new))
        self.same(st, want)
        return want

    def fork(self, parents, children):
        st = G.gqa_cache_fork(self.k, self.v, *self.state, ints(parents), ints(children))
        want = self.model.fork(list(parents), list(children))
        self.same(st, want)
        return want

    def compact(self, keep, m, n=None):
        st = G.gqa_cache_compact(self.k, self.v, *self.state, ints(keep), ints(m), None if n is None else ints(n))
        want = self.model.compact(keep, m, n)
        self.same(st, want)
        return want


@pytest.mark.parametrize("seed", range(6))
def test_random_runs(seed):
    rng = np.random.default_rng(seed)
    S, ps = int(rng.integers(3, 40)), int(rng.choice([16, 32]))
    M = int(rng.integers(2, 12))
    c = Both(S, M, int(rng.integers(S, 4 * S)), ps, layers=int(rng.integers(1, 4)), Hk=int(rng.choice([1, 2, 5])),
             d=int(rng.choice([64, 128])), seed=seed, dtype=[torch.bfloat16, torch.float8_e4m3fn][seed & 1])
    seen = set()
    for _ in range(40):
        op = rng.integers(3)
        n = int(rng.integers(1, S + 1))
        if op == 0:
            slots = rng.integers(-1, S + 1, n)  # some twice, some out of range
            near = c.model.lens[np.clip(slots, 0, S - 1)] + rng.integers(-20, 40, n)
            new = np.where(rng.random(n) < 0.3, rng.integers(-1, M * ps + 2, n), near)
            seen |= set(c.resize(slots.tolist(), np.where(rng.random(n) < 0.2, 0, new).tolist()))
        elif op == 1:
            seen |= set(c.fork(rng.integers(-1, S, n).tolist(), rng.integers(0, S + 1, n).tolist()))
        else:
            T = int(rng.integers(1, 40))
            keep = np.sort(np.argsort(rng.random((S, T)), 1), 1)
            m = rng.integers(0, T + 1, S)
            tree_lens = rng.integers(-1, T + 3, S) if rng.random() < 0.5 else None
            for s in range(S):  # mostly proper lists
                nodes = min(T if tree_lens is None else max(int(tree_lens[s]), 0), T, int(c.model.lens[s]))
                m[s] = rng.integers(0, nodes + 1)
                keep[s, :m[s]] = np.sort(rng.permutation(nodes)[:m[s]])
                if rng.random() < 0.1 and m[s] > 1:
                    keep[s, 1] = keep[s, 0]
            seen |= set(c.compact(keep.tolist(), m.tolist(), None if tree_lens is None else tree_lens.tolist()))
    assert {R.DONE, R.INVALID} <= seen


def test_resize_takes_the_lowest_pages_first_and_reuses_those_given_up():
    c = Both(4, 8, 10, 16)
    assert c.resize([2, 0], [40, 17]) == [0, 0]
    assert c.table[2, :3].tolist() == [0, 1, 2] and c.table[0, :2].tolist() == [3, 4]
    assert c.resize([2, 1], [0, 16 * 8]) == [0, 0]  # slot 1 gets slot 2's pages in the same call
    assert c.resize([3], [1]) == [R.NO_PAGES] and c.resize([0], [0]) == [0] and c.resize([3], [1]) == [0]


def test_resize_too_few_pages():
    c = Both(6, 8, 9, 16)
    # the second does not fit, so neither do later ones that need pages; the third needs none
    assert c.resize([0, 1, 2, 3], [64, 16 * 6, 0, 16]) == [0, R.NO_PAGES, 0, R.NO_PAGES]
    assert c.resize([1, 0, 3], [10 ** 6, 16, 16]) == [R.INVALID, 0, 0]


def test_resize_shared_pages():
    c = Both(4, 8, 20, 16)
    c.resize([0], [50])
    assert c.fork([0], [1]) == [0]
    assert c.resize([1], [20]) == [R.SHARED]  # row 20's page is the parent's too
    assert c.resize([1], [32]) == [0]         # whole shared pages may stay
    assert c.resize([0, 1], [0, 33]) == [0, 0]
    assert c.resize([1], [20]) == [0]         # the parent is gone


def test_fork_replaces_children_and_refuses_tangles():
    c = Both(8, 8, 40, 16)
    c.resize([0, 1, 2], [70, 16, 5])
    assert c.fork([0, 0, 1, 2], [3, 4, 5, 6]) == [0] * 4
    assert c.fork([1, 1, 0], [3, 4, 5]) == [0] * 3           # last step's children replaced
    assert c.fork([0, 3, 9, 2, 2, 1], [3, 7, 6, 8, 5, 5]) == [R.INVALID, 0, R.INVALID, R.INVALID, 0, R.INVALID]
    assert c.fork([2, 2], [2, 4]) == [0, 0]                  # a slot as its own child stays
    assert c.fork([7, 0], [2, 2]) == [0, R.INVALID]


def test_fork_without_pages_leaves_the_child_empty():
    c = Both(5, 4, 7, 16)
    c.resize([0], [16 * 3 + 1])
    assert c.fork([0, 0, 0, 0], [1, 2, 3, 4]) == [0, 0, 0, R.NO_PAGES]
    assert c.lens[4].item() == 0 and (c.table[4] == -1).all()


@pytest.mark.parametrize("ps", [16, 64])
def test_compact_borders(ps):
    c = Both(6, 6, 40, ps, layers=3)
    c.resize(None, [ps, ps - 1, 2 * ps, 3, ps + 7, 0])
    T = 9
    keep = [[0, 1, 2] + [0] * 6, [8] + [0] * 8, list(range(9)), [2] + [0] * 8, [0] * 9, [0] * 9]
    c.resize(None, [ps + 9, ps + 8, 2 * ps + 9, 3 + 4, ps + 7, 0])
    assert c.compact(keep, [3, 1, 9, 1, 0, 0], [9, 9, 9, 4, 0, 3]) == [0] * 6
    assert c.lens.tolist() == [ps + 3, ps, 2 * ps + 9, 4, ps + 7, 0]
    assert c.compact([[1, 1]] + [[0, 1]] * 5, [2, 3, -1, 0, 2, 1], None) == [2, 2, 2, 0, 0, 2]


def test_compact_refuses_shared_pages():
    c = Both(3, 6, 20, 16)
    c.resize([0], [32])
    c.fork([0], [1])
    assert c.compact([[3], [0], [0]], [0, 0, 0], [4, 0, 0]) == [R.SHARED, 0, 0]
    c.resize([1], [0])
    # (nodes are counted up to T: the list has a place for each of the four)
    assert c.compact([[0, 3, 0, 0], [0] * 4, [0] * 4], [2, 0, 0], [4, 0, 0]) == [0, 0, 0]


def test_larger_than_one_round_of_requests():
    """More requests than threads of a block, more pages than a pass over them."""
    rng = np.random.default_rng(3)
    S = 3000
    c = Both(S, 4, 9000, 16, layers=1, Hk=1)
    c.resize(None, rng.integers(0, 60, S).tolist())
    c.resize(rng.permutation(S)[:2500].tolist(), rng.integers(0, 64, 2500).tolist())
    c.fork([0] * 1200, (1 + rng.permutation(S - 1)[:1200]).tolist())
    with pytest.raises(G.GqaError):
        G.gqa_cache_resize(*c.state, 16, ints([0] * 4097), ints([0] * 4097))


def test_long_sequences():
    """Tables of more entries than a warp's turn."""
    c = Both(3, 700, 2500, 16, layers=1, Hk=1)
    c.resize([0, 2], [11000, 300])
    c.fork([0, 0], [1, 2])
    c.resize([0, 1], [0, 5333 // 16 * 16])
    c.resize([1], [9000])


def test_one_layer_pools_and_no_requests():
    c = Both(3, 4, 8, 16, layers=1)
    c.k, c.v = c.k[0], c.v[0]
    c.resize([0], [20])
    c.fork([0], [2])
    c.fork([], [])
    c.resize([], [])
    c.compact([[1]] * 3, [0, 0, 1], [1, 0, 1])


def test_captured_and_on_another_stream():
    c = Both(6, 8, 30, 16)
    c.resize([0, 1], [50, 20])
    start = [x.clone() for x in c.state]
    to, back, slots = ints([30, 64, 5]), ints([50, 20, 0]), ints([0, 1, 5])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        G.gqa_cache_resize(*c.state, 16, to, slots)
        G.gqa_cache_fork(c.k, c.v, *c.state, ints([0]), ints([3]))
        G.gqa_cache_resize(*c.state, 16, ints([0]), ints([3]))
        G.gqa_cache_resize(*c.state, 16, back, slots)
    torch.cuda.synchronize()
    par, kid, none = ints([0]), ints([3]), ints([0])
    with torch.cuda.graph(graph):
        st = [G.gqa_cache_resize(*c.state, 16, to, slots),
              G.gqa_cache_fork(c.k, c.v, *c.state, par, kid),
              G.gqa_cache_resize(*c.state, 16, none, kid),
              G.gqa_cache_resize(*c.state, 16, back, slots)]
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all((x == 0).all() for x in st)
    assert torch.equal(c.lens, start[1]) and c.refs.sum() == start[2].sum()


def test_a_serving_step_of_all_calls():
    """Prompts, their pages, samples of one, drafts, a verification, the accepted tokens, the next
    token: the paged forward over the pages equals attention over the tokens themselves."""
    rng = np.random.default_rng(5)
    Hq, Hk, d, ps, S, M, P = 8, 2, 64, 16, 6, 12, 60
    rn = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).bfloat16().cuda()  # noqa: E731
    kp, vp = (torch.full((1, P, ps, Hk, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.full((S, M), -1, dtype=torch.int32, device="cuda")
    lens, refs = ints([0] * S), ints([0] * P)
    state = (table, lens, refs)
    prompt = [37, 80, 16]
    cq = ints(np.concatenate([[0], np.cumsum(prompt)]))
    q, k, v = rn(sum(prompt), Hq, d), rn(sum(prompt), Hk, d), rn(sum(prompt), Hk, d)
    out, _ = G.gqa_attn_fwd_varlen(q, k, v, cq, causal=True)
    tokens = {s: [k[a:b], v[a:b]] for s, a, b in zip(range(3), cq[:-1].tolist(), cq[1:].tolist())}

    def write(s, at, kk, vv):  # a program's own write of new rows
        pos = torch.arange(at, at + len(kk), device="cuda")
        page = table[s].long()[pos // ps]
        kp[0, page, pos % ps], vp[0, page, pos % ps] = kk, vv

    assert (G.gqa_cache_resize(*state, ps, ints(prompt), ints([0, 1, 2])) == 0).all()
    for s in range(3):
        write(s, 0, *tokens[s])
    assert (G.gqa_cache_fork(kp, vp, *state, ints([0, 0, 1]), ints([3, 4, 5])) == 0).all()
    tokens.update({3: tokens[0], 4: tokens[0], 5: tokens[1]})

    T = 6
    grown = [len(tokens[s][0]) + T for s in range(S)]
    assert (G.gqa_cache_resize(*state, ps, ints(grown)) == 0).all()
    kd, vd = rn(S, T, Hk, d), rn(S, T, Hk, d)
    for s in range(S):
        write(s, grown[s] - T, kd[s], vd[s])
    paths = [[0, 2, 5], [0], [1, 3], [], [0, 1, 2, 3, 4, 5], [4]]
    see = np.tril(np.ones((S, T, T), dtype=bool))
    words = torch.from_numpy((see << np.arange(T)).sum(-1).astype(np.int32)[..., None]).cuda()
    qd = rn(S, T, Hq, d)
    o, l = G.gqa_attn_fwd_tree(qd, kp[0], vp[0], words, lens, block_table=table)
    f = lambda x: x.double().cpu().numpy()  # noqa: E731
    for s in range(S):
        kk, vv = torch.cat([tokens[s][0], kd[s]]), torch.cat([tokens[s][1], vd[s]])
        R.check(o[s], l[s], *R.attn(f(qd[s]), f(kk), f(vv), R.causal(T, len(kk)), d ** -0.5))
        tokens[s] = [torch.cat([tokens[s][i], x[s][paths[s]]]) for i, x in enumerate((kd, vd))]
    keep = ints([p + [0] * (T - len(p)) for p in paths])
    assert (G.gqa_cache_compact(kp, vp, *state, keep, ints([len(p) for p in paths])) == 0).all()
    assert lens.tolist() == [len(tokens[s][0]) for s in range(S)]

    for pool in (kp, vp):  # rows that no sequence has hold NaN; the paged forward wants them finite
        pool.nan_to_num_()
    q1 = rn(S, 1, Hq, d)
    o, l = G.gqa_attn_fwd_paged(q1, kp[0], vp[0], table, lens)
    for s in range(S):
        see = np.ones((1, len(tokens[s][0])), dtype=bool)
        R.check(o[s], l[s], *R.attn(f(q1[s]), f(tokens[s][0]), f(tokens[s][1]), see, d ** -0.5))
    assert (G.gqa_cache_resize(*state, ps, ints([0] * S)) == 0).all()
    assert (refs == 0).all() and (table == -1).all()
