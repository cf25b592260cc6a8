"""The most requests that one call takes (4096), whose sets fill the shared memory of the plan's
blocks, against the model of one request after the other."""
import numpy as np
import pytest

from tests import serve_ref as R
from tests.test_gpu_cache_pages import Both

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import gqa_exact_attention_b200 as G  # noqa: E402

MOST = G.GQA_CACHE_MAX_REQUESTS


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.load_serve()


@pytest.mark.parametrize("P", [13000, 5000, 3000])
def test_forks(P):
    """With pages for all (the parents have at most 3 pages each and a child takes one: 600 + 4096
    < 5000), and with pages for some."""
    rng = np.random.default_rng(95)
    S = MOST + 300
    c = Both(S, 3, P, 16, layers=1, Hk=1)
    c.resize(None, rng.integers(0, 40, 200).tolist())  # 200 parents
    kids = 200 + rng.permutation(S - 200)
    st = c.fork(rng.integers(0, 200, MOST).tolist(), kids[:MOST].tolist())
    assert (R.NO_PAGES in st) == (P == 3000) and R.DONE in st
    # again, with children named twice, out of range and among the parents
    c.fork(rng.integers(-1, 260, MOST).tolist(), rng.integers(150, S + 1, MOST).tolist())


@pytest.mark.parametrize("P", [13000, 5000])
def test_resizes(P):
    rng = np.random.default_rng(96)
    S = MOST + 300
    c = Both(S, 3, P, 16, layers=1, Hk=1)
    c.resize(rng.permutation(S)[:MOST].tolist(), rng.integers(0, 49, MOST).tolist())
    c.resize(None, rng.integers(0, 49, MOST).tolist())
    c.resize(rng.integers(-1, S + 1, MOST).tolist(), rng.integers(-1, 50, MOST).tolist())
