"""Bounds of packed prompts that decrease: sequences that start before the end of an earlier one
cover rows with unspecified values, every other sequence gets its own result, and nothing else
is written."""
import numpy as np
import pytest

from tests.test_gpu_serve_attn import Canary, randn

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


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("Hq,Hk,d,T,again", [(32, 8, 128, 8192, 8), (16, 4, 64, 8192, 40), (8, 2, 64, 500, 3)])
@pytest.mark.parametrize("causal", [False, True])
def test_a_sequence_behind_overlapping_ones_is_written(Hq, Hk, d, T, again, causal):
    """[0, T/2) many times over (more tile groups than the rows have), then [T/2, T)."""
    rng = np.random.default_rng(90)
    q, k, v = (randn(rng, T, H, d).cuda() for H in (Hq, Hk, Hk))
    bounds = ints([0, T // 2] * again + [T // 2, T, 7, 9])  # (and a last one inside the first rows)
    out, lse = Canary((T, Hq, d), torch.float32), Canary((Hq, T), torch.float32)
    G.gqa_attn_fwd_varlen(q, k, v, bounds, out=out.t, lse=lse.t, causal=causal)
    torch.cuda.synchronize()
    assert out.untouched() and lse.untouched()
    a = T // 2
    o, l = G.gqa_attn_fwd_varlen(q, k, v, ints([a, T]), causal=causal)
    # (the schedule goes by the number of sequences: two roundings of the weights, as in the
    # comparison with the dense forward)
    assert (out.t[a:] - o[a:]).abs().max() <= 2 * 1.02 * 2.0 ** -8 * v.float().abs().max()
    assert (lse.t[:, a:] - l[:, a:]).abs().max() <= 1e-3


def test_the_list_takes_each_ordered_sequence_once():
    """Bounds that go back now and then, and more sequences than the warps look at in one turn."""
    rng = np.random.default_rng(91)
    n, L = 90, 150
    T = n * L
    q, k, v = (randn(rng, T, H, 128).cuda() for H in (32, 8, 8))
    bounds, good = [0], []
    for i in range(n):
        good.append((i * L, (i + 1) * L))
        bounds.append((i + 1) * L)
        if i % 7 == 3 and i < 40:
            bounds += [L // 2, (i + 1) * L]  # back to the first sequence's middle: overlaps the ones before
    out, lse = torch.full((T, 32, 128), 7.0, device="cuda"), torch.full((32, T), 7.0, device="cuda")
    G.gqa_attn_fwd_varlen(q, k, v, ints(bounds), out=out, lse=lse, causal=True)
    o, l = G.gqa_attn_fwd_varlen(q, k, v, ints([0] + [b for _, b in good]), causal=True)
    torch.cuda.synchronize()
    # rows behind the last sequence that goes back belong to ordered sequences alone
    for a, b in good[39:]:
        assert torch.equal(out[a:b], o[a:b]) and torch.equal(lse[:, a:b], l[:, a:b])
