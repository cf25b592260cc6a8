"""NaN and infinities in Q and K of the serving attention calls: a row that sees a score which is
NaN or +inf gives NaN, a score of -inf weighs nothing, and no other row changes, whether a unit
is split over the CTAs or not."""
import numpy as np
import pytest

from tests import serve_ref as R
from tests.test_gpu_serve_attn import bits, cu, f64, randn, tree

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


def check(out, lse, q, k, v, see, scale, what):
    """One sequence: out [S, Hq, d] and lse [Hq, S] of the device; q, k, v in 64 bits, see [S, L]."""
    g = q.shape[1] // k.shape[1]
    clean = lambda x: np.nan_to_num(x, nan=0.0, posinf=0.0, neginf=0.0)  # noqa: E731
    n_bad = 0
    for h in range(q.shape[1]):
        kk, vv = k[:, h // g], v[:, h // g]
        with np.errstate(invalid="ignore"):
            x = scale * (q[:, h] @ kk.T)
        bad = (see & ~(x < np.inf)).any(1)
        keep = see & (x > -np.inf)  # (no such key's row has an infinity, nor such a query's)
        o, l, tol, ltol = R.attn(clean(q[:, h:h + 1]), clean(kk[:, None]), vv[:, None], keep, scale)
        assert torch.isnan(out[bad, h]).all() and torch.isnan(lse[h, bad]).all(), f"{what}, head {h}: a NaN is lost"
        good = ~bad
        R.check(out[good, h], lse[h, good], o[good, 0], l[0, good], tol[good, 0], ltol[0, good], what=f"{what}, head {h}")
        n_bad += int(bad.sum())
    return n_bad


KINDS = ["nan key", "nan query", "inf key", "inf blocks", "inf everywhere"]


def spoil(rng, kind, q, k):
    """Values that are not finite in one sequence's q [S, Hq, d] and k [L, Hk, d]."""
    S, L = len(q), len(k)
    if S == 0 or L == 0:
        return
    for h in range(k.shape[1]):
        j = int(rng.integers(max(0, L - S), L)) if rng.integers(2) else int(rng.integers(L))
        if kind == "nan key":
            k[j, h, int(rng.integers(k.shape[2]))] = float("nan")
        elif kind == "inf key":  # +inf or -inf, by the sign of each query's first element
            k[j, h, 0] = float("inf")
        elif kind == "inf blocks":  # the first blocks of the row: nothing is summed up there
            k[:max(min(L - 1, 300), 1), h, 0] = float("inf")
        elif kind == "inf everywhere":
            k[:, h, 0] = float("-inf")
    if kind == "nan query":
        for _ in range(3):
            q[int(rng.integers(S)), int(rng.integers(q.shape[1])), int(rng.integers(q.shape[2]))] = float("nan")


VARLEN = {  # query lengths, keys before them, Hq, Hk
    "whole units": ([60, 1, 130, 200], [0, 0, 0, 0], 8, 2),
    "split units": ([30, 1, 0, 300], [900, 3000, 5, 1200], 8, 2),
    "list": ([700, 200, 640, 512], [0, 300, 17, 128], 16, 4),
}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("case", VARLEN)
def test_varlen(case, kind, d):
    lq, more, Hq, Hk = VARLEN[case]
    lk = [a + b for a, b in zip(lq, more)]
    rng = np.random.default_rng(70)
    q, k, v = randn(rng, sum(lq), Hq, d), randn(rng, sum(lk), Hk, d), randn(rng, sum(lk), Hk, d)
    cq, ck = cu(lq), cu(lk)
    at = list(zip(cq[:-1].tolist(), cq[1:].tolist(), ck[:-1].tolist(), ck[1:].tolist()))
    for i, (a, b, c, e) in enumerate(at):
        if i != 1:  # (one sequence stays as it is)
            spoil(rng, kind, q[a:b], k[c:e])
    out, lse = G.gqa_attn_fwd_varlen(q.cuda(), k.cuda(), v.cuda(), cq, ck, causal=True)
    torch.cuda.synchronize()
    out, lse = out.cpu(), lse.cpu()
    n_bad = [check(out[a:b], lse[:, a:b], f64(q[a:b]), f64(k[c:e]), f64(v[c:e]), R.causal(b - a, e - c), d ** -0.5,
                   f"sequence {i}") for i, (a, b, c, e) in enumerate(at)]
    assert n_bad[1] == 0 and sum(n_bad) > 0


TREE = {  # lengths, T, Hq, Hk
    "whole units": ([400, 90, 128], 9, 8, 2),
    "split units": ([3000, 700, 1100], 9, 8, 2),
    "two tiles": ([1500, 100, 300], 80, 8, 2),
}


@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("case", TREE)
def test_tree(case, kind, d, page):
    lens, T, Hq, Hk = TREE[case]
    rng = np.random.default_rng(71)
    B, cap = len(lens), -(-max(lens) // 64) * 64
    if case == "whole units":
        cap = 448
    q, k, v = randn(rng, B, T, Hq, d), randn(rng, B, cap, Hk, d), randn(rng, B, cap, Hk, d)
    for b in (0, 2):
        spoil(rng, kind, q[b], k[b, :lens[b]])
    see = np.stack([tree(rng, T) for _ in range(B)])
    args = {}
    kd, vd = k.cuda(), v.cuda()
    if page:
        M = cap // page
        args["block_table"] = torch.arange(B * M, dtype=torch.int32, device="cuda").view(B, M)
        kd, vd = kd.view(B * M, page, Hk, d), vd.view(B * M, page, Hk, d)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = G.gqa_attn_fwd_tree(q.cuda(), kd, vd, bits(see), sl, **args)
    torch.cuda.synchronize()
    out, lse = out.cpu(), lse.cpu()
    n_bad = []
    for b, L in enumerate(lens):
        ok = np.ones((T, L), dtype=bool)
        ok[:, L - T:] = see[b]
        n_bad.append(check(out[b], lse[b], f64(q[b]), f64(k[b, :L]), f64(v[b, :L]), ok, d ** -0.5, f"sequence {b}"))
    assert n_bad[1] == 0 and sum(n_bad) > 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_at_every_place_of_a_block(d, bad):
    """128 kv heads, each with one bad key, at every place of an unmasked block."""
    rng = np.random.default_rng(72)
    H = L = 128
    q, k, v = randn(rng, 5, H, d).abs() + 0.5, randn(rng, L, H, d), randn(rng, L, H, d)
    k[torch.arange(L), torch.arange(H), 0] = bad
    out, lse = G.gqa_attn_fwd_varlen(q.cuda(), k.cuda(), v.cuda(), cu([5]), cu([L]))
    assert torch.isnan(out).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("d", [64, 128])
def test_negative_scale(d):
    """With scale < 0 the reference maximum is the scores' minimum."""
    rng = np.random.default_rng(73)
    lq, lk = [200, 40], [1300, 700]
    q, k, v = randn(rng, sum(lq), 4, d), randn(rng, sum(lk), 2, d), randn(rng, sum(lk), 2, d)
    for a, b, c, e in ((0, 200, 0, 1300), (200, 240, 1300, 2000)):
        for kind in ("nan query", "inf blocks"):
            spoil(rng, kind, q[a:b], k[c:e])
    out, lse = G.gqa_attn_fwd_varlen(q.cuda(), k.cuda(), v.cuda(), cu(lq), cu(lk), causal=True, scale=-0.1)
    torch.cuda.synchronize()
    out, lse = out.cpu(), lse.cpu()
    for a, b, c, e in ((0, 200, 0, 1300), (200, 240, 1300, 2000)):
        assert check(out[a:b], lse[:, a:b], f64(q[a:b]), f64(k[c:e]), f64(v[c:e]), R.causal(b - a, e - c), -0.1, "scale") > 0


@pytest.mark.parametrize("T", [9, 80])
def test_rows_past_the_tree_stay_zero(T):
    """Rows i >= n_b get 0 and -inf whatever their queries and the keys hold."""
    rng = np.random.default_rng(74)
    q, k, v = randn(rng, 2, T, 8, 64), randn(rng, 2, 900, 2, 64), randn(rng, 2, 900, 2, 64)
    n = [T // 2, 0]
    q[0, n[0]:], k[1, 5] = float("nan"), float("nan")
    see = np.ones((2, T, T), dtype=bool)
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out, lse = G.gqa_attn_fwd_tree(q.cuda(), k.cuda(), v.cuda(), bits(see), ints(900, 700), tree_lens=ints(*n))
    for b in range(2):
        assert (out[b, n[b]:] == 0).all() and torch.isneginf(lse[b, :, n[b]:]).all()
    assert torch.isfinite(out).all() and torch.isfinite(lse[0, :, :n[0]]).all()
