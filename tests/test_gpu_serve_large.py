"""The serving operators where offsets pass 32 bits: a pool and packed rows of more than 2^31
elements.  What lies far out must equal the same data lying near."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import gqa_exact_attention_b200 as G  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.load_serve()
    yield
    torch.cuda.empty_cache()
    assert G.gqa_serve_device_status(reset=True) == 0, "an in-kernel wait timed out"


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def test_pages_past_2_to_31_elements():
    ps, Hk, d, near, layers = 64, 8, 128, 40, 2
    far = 2 ** 31 // (ps * Hk * d) + 3  # the pool's pages before the ones in use, in each layer
    P = far + near
    gen = torch.Generator(device="cuda").manual_seed(1)
    small = [torch.randn((layers, near, ps, Hk, d), generator=gen, device="cuda").bfloat16() for _ in range(2)]
    large = [torch.zeros((layers, P, ps, Hk, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for a, b in zip(large, small):
        a[:, far:] = b
    S, M, T = 3, 10, 7
    lens = [500, 64, 300]
    rng = np.random.default_rng(2)
    perm = rng.permutation(near)
    table = np.full((S, M), -1)
    at = 0
    for s, L in enumerate(lens):
        n = -(-L // ps)
        table[s, :n] = perm[at:at + n]
        at += n

    def state(first):
        t = np.where(table >= 0, table + first, -1)
        refs = np.zeros(first + near, dtype=np.int64)
        refs[t[t >= 0]] = 1
        refs[:first] = 1  # the pages before are somebody else's
        return ints(t), ints(lens), ints(refs)

    q = torch.randn((S, T, 32, d), generator=gen, device="cuda").bfloat16()
    mask = ints(rng.integers(0, 2 ** T, (S, T, 1)))
    n, keep, m = ints([T, 3, 0]), ints([[0, 3, 5, 6, 0, 0, 0], [2] + [0] * 6, [0] * 7]), ints([4, 1, 0])
    got = []
    for pools, first in ((small, 0), (large, far)):
        st = state(first)
        out = []
        for layer in range(layers):
            out += G.gqa_attn_fwd_tree(q, pools[0][layer], pools[1][layer], mask, st[1], block_table=st[0], tree_lens=n)
        assert (G.gqa_cache_compact(*pools, *st, keep, m, tree_lens=n) == 0).all()
        assert (G.gqa_cache_resize(*st, ps, ints([0]), ints([1])) == 0).all()
        assert (G.gqa_cache_fork(*pools, *st, ints([0]), ints([1])) == 0).all()
        got.append([*out, st[1], torch.where(st[0] >= 0, st[0] - first, st[0]), st[2][first:],
                    *(x[:, first:] for x in pools)])
    torch.cuda.synchronize()
    for a, b in zip(*got):
        assert torch.equal(a, b)
    for x in large:  # nothing was written before them
        assert not x[:, :far].any()


def test_packed_rows_past_2_to_31_elements():
    Hq, Hk, d, L = 128, 8, 128, 128
    B = 2 ** 31 // (Hq * d * L) + 2
    gen = torch.Generator(device="cuda").manual_seed(3)
    k = torch.randn((B * L, Hk, d), generator=gen, device="cuda").bfloat16()
    v = torch.randn((B * L, Hk, d), generator=gen, device="cuda").bfloat16()
    q = torch.zeros((B * L, Hq, d), dtype=torch.bfloat16, device="cuda")
    q[-3 * L:] = torch.randn((3 * L, Hq, d), generator=gen, device="cuda").bfloat16()
    cu = ints(np.arange(B + 1) * L)
    out, lse = G.gqa_attn_fwd_varlen(q, k, v, cu, causal=True, out_dtype=torch.bfloat16)
    o, l = G.gqa_attn_fwd_varlen(q[-3 * L:], k[-3 * L:], v[-3 * L:], ints(np.arange(4) * L), causal=True,
                                 out_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    # two schedules: each rounds its own weights (2^-8, with 2 % for fp32 steps) and its output
    near = 2 * 1.02 * 2.0 ** -8 * v[-3 * L:].float().abs().max() + 2 * 2.0 ** -8 * o.float().abs().max()
    assert (out[-3 * L:].float() - o.float()).abs().max() <= near
    assert (lse[:, -3 * L:] - l).abs().max() <= 1e-3
    # queries of zeros weigh their keys alike: row i of a sequence is the mean of v[0..i]
    for b in (0, B // 2):
        want = v[b * L:(b + 1) * L].double().cumsum(0) / torch.arange(1, L + 1, device="cuda").view(-1, 1, 1)
        got = out[b * L:(b + 1) * L].view(L, Hk, Hq // Hk, d).double()
        assert (got - want[:, :, None]).abs().max() <= 2.02 * 2.0 ** -8 * v.float().abs().max()
