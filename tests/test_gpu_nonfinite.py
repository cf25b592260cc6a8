"""NaN and infinities in Q and K of the forward's entry points: a row that sees a score which is
NaN or +inf gives NaN, a score of -inf weighs nothing, and no other row changes, in every
schedule (splits, packed heads, one or two tiles).  Other rows keep the parity tolerances."""
import numpy as np
import pytest

from tests import parity as P

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import gqa_exact_attention_b200 as G  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.load()
    yield
    assert G.gqa_attn_device_status(reset=True) == 0, "an in-kernel wait timed out"


def randn(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).bfloat16()


def spoil(rng, kind, q, k):
    """One sequence's q [S, Hq, d] and k [L, Hk, d]."""
    S, L = len(q), len(k)
    for h in range(k.shape[1]):
        j = int(rng.integers(max(0, L - S), L)) if rng.integers(2) else int(rng.integers(L))
        if kind == "nan key":
            k[j, h, int(rng.integers(k.shape[2]))] = float("nan")
        elif kind == "inf key":  # +inf or -inf, by the sign of each query's first element
            k[j, h, 0] = float("inf")
        elif kind == "inf blocks":
            k[:max(min(L - 1, 300), 1), h, 0] = float("inf")
        elif kind == "inf everywhere":
            k[:, h, 0] = float("-inf")
    if kind == "nan query":
        for _ in range(3):
            q[int(rng.integers(S)), int(rng.integers(q.shape[1])), int(rng.integers(q.shape[2]))] = float("nan")


def check(out, lse, q, k, v, causal, scale):
    """One sequence: out [S, Hq, d] and lse [Hq, S] of the device, host tensors q, k, v."""
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    q, k, v = (x.double().numpy() for x in (q, k, v))
    S, L, g = len(q), len(k), q.shape[1] // k.shape[1]
    see = np.arange(L)[None] <= np.arange(S)[:, None] + (L - S) if causal else np.ones((S, L), dtype=bool)
    n_bad = 0
    for h in range(q.shape[1]):
        with np.errstate(invalid="ignore"):
            x = scale * (q[:, h] @ k[:, h // g].T)
        bad = (see & ~(x < np.inf)).any(1)
        assert np.isnan(out[bad, h]).all() and np.isnan(lse[h, bad]).all(), f"head {h}: a NaN is lost"
        x = np.where(see & ~bad[:, None], x, -np.inf)
        m = np.where(x.max(1) > -np.inf, x.max(1), 0.0)
        p = np.exp(x - m[:, None])
        l = p.sum(1)
        o = (p / np.where(l > 0, l, 1)[:, None]) @ v[:, h // g]
        with np.errstate(divide="ignore"):
            P.check(out[~bad, h], lse[h, ~bad], o[~bad], (m + np.log(l))[~bad], f"head {h}")
        n_bad += int(bad.sum())
    return n_bad


KINDS = ["nan key", "nan query", "inf key", "inf blocks", "inf everywhere"]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Sq,Sk,Hq,Hk,pack,splits", [
    (1, 900, 8, 2, 1, 1), (1, 900, 8, 2, 1, 4), (3, 1500, 4, 4, 0, 3), (300, 700, 8, 2, 1, 1), (300, 700, 4, 2, 0, 1),
    (200, 1100, 6, 2, 1, 3)])
def test_forward(Sq, Sk, Hq, Hk, pack, splits, kind, d):
    rng = np.random.default_rng(80)
    q, k, v = randn(rng, 2, Sq, Hq, d), randn(rng, 2, Sk, Hk, d), randn(rng, 2, Sk, Hk, d)
    spoil(rng, kind, q[0], k[0])
    for causal in (False, True):
        out, lse = G.gqa_attn_fwd(q.cuda(), k.cuda(), v.cuda(), causal=causal, pack_gqa=pack, num_splits=splits)
        n = [check(out[b], lse[b], q[b], k[b], v[b], causal, P.default_scale(d)) for b in range(2)]
        assert n[1] == 0 and (n[0] > 0 or causal or kind in ("inf everywhere", "inf key", "inf blocks"))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("splits", [1, 4])
def test_kvcache_and_paged(kind, splits):
    rng = np.random.default_rng(81)
    B, Sq, Hq, Hk, d, page, cap = 3, 2, 8, 2, 128, 64, 1024
    lens = [1000, 130, 600]
    q, k, v = randn(rng, B, Sq, Hq, d), randn(rng, B, cap, Hk, d), randn(rng, B, cap, Hk, d)
    for b in (0, 2):
        spoil(rng, kind, q[b], k[b, :lens[b]])
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    table = torch.arange(B * cap // page, dtype=torch.int32, device="cuda").view(B, -1)
    pages = [x.cuda().view(-1, page, Hk, d) for x in (k, v)]
    for out, lse in (G.gqa_attn_fwd_kvcache(q.cuda(), k.cuda(), v.cuda(), sl, causal=True, num_splits=splits),
                     G.gqa_attn_fwd_paged(q.cuda(), *pages, table, sl, causal=True, num_splits=splits)):
        n = [check(out[b], lse[b], q[b], k[b, :L], v[b, :L], True, P.default_scale(d)) for b, L in enumerate(lens)]
        assert n[1] == 0


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("Sq", [1, 200])
def test_fp8_nan(Sq, splits):
    """e4m3 has NaN and no infinities."""
    rng = np.random.default_rng(82)
    q, k, v = (randn(rng, 1, S, H, 128).to(torch.float8_e4m3fn) for S, H in ((Sq, 4), (700, 2), (700, 2)))
    k.view(torch.uint8)[0, 350, 1, 7] = 0x7f
    out, lse = G.gqa_attn_fwd_fp8(q.cuda(), k.cuda(), v.cuda(), 1.0, 1.0, 1.0, num_splits=splits)
    assert torch.isnan(out[0, :, 2:]).all() and torch.isnan(lse[0, 2:]).all()
    assert torch.isfinite(out[0, :, :2]).all() and torch.isfinite(lse[0, :2]).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_at_every_place_of_a_block(d, bad):
    """128 kv heads, each with one bad key, at every place of an unmasked block."""
    rng = np.random.default_rng(83)
    H = L = 128
    q, k, v = randn(rng, 1, 5, H, d).abs() + 0.5, randn(rng, 1, L, H, d), randn(rng, 1, L, H, d)
    k[0, torch.arange(L), torch.arange(H), 0] = bad
    out, lse = G.gqa_attn_fwd(q.cuda(), k.cuda(), v.cuda())
    assert torch.isnan(out).all() and torch.isnan(lse).all()
