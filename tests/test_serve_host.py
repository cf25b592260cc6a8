"""The serving operators on the host: the library exports what the header declares, invalid
arguments are refused before anything is launched, and the binding's checks."""
import os
import re
import subprocess

import pytest

import gqa_exact_attention_b200 as G

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gqa_serve.h")


def declared():
    return sorted(set(re.findall(r"GQA_API\s+gqa_status\s+(gqa_\w+)\s*\(", open(HEADER).read())))


def test_library_exports_what_the_header_declares():
    G.load_serve()
    assert declared() == ["gqa_attn_fwd_tree", "gqa_attn_fwd_varlen", "gqa_cache_compact", "gqa_cache_fork",
                          "gqa_cache_resize", "gqa_serve_device_status"]
    out = subprocess.run(["nm", "-D", "--defined-only", G.serve_lib_path], capture_output=True, text=True,
                         check=True).stdout
    exported = {ln.split()[-1] for ln in out.splitlines() if " T " in ln}
    assert {s for s in exported if s.startswith("gqa")} == set(declared())


def test_header_compiles_as_c():
    src = f'#include "{HEADER}"\nint main(void) {{ return (int)GQA_CACHE_DONE; }}\n'
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-x", "c", "-", "-o", os.devnull], input=src,
                       text=True, capture_output=True)
    assert r.returncode == 0, r.stderr


NULL = None
# what valid arguments give here: no device, or one that is no B200 (the pointers are never read)
NO_GPU = (6, 8)


def varlen(q=16, qs=0, k=16, ks=0, v=16, vs=0, cq=16, ck=16, out=16, dt=0, lse=16, B=2, tq=8, tk=8, Hq=4, Hk=2,
           d=64, scale=0.125, causal=1):
    return G.load_serve().gqa_attn_fwd_varlen(q, qs, k, ks, v, vs, cq, ck, out, dt, lse, B, tq, tk, Hq, Hk, d,
                                              scale, causal, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=NULL), 1), (dict(k=NULL), 1), (dict(v=NULL), 1), (dict(cq=NULL), 1), (dict(ck=NULL), 1),
    (dict(out=NULL), 1), (dict(lse=NULL), 1),
    (dict(B=0), 2), (dict(tq=-1), 2), (dict(tk=-1), 2), (dict(Hq=0), 2), (dict(Hk=0), 2), (dict(dt=2), 2),
    (dict(scale=float("nan")), 2),
    (dict(qs=255), 2), (dict(qs=260), 2), (dict(ks=120), 2), (dict(vs=64), 2), (dict(qs=-256), 2), (dict(ks=1 << 40), 2),
    (dict(tq=1 << 30), 2), (dict(B=1 << 30), 2), (dict(tk=1 << 30), 2),
    (dict(Hq=6, Hk=4), 3), (dict(d=96), 4), (dict(q=24), 5), (dict(out=8), 5), (dict(cq=18), 5), (dict(ck=17), 5),
])
def test_varlen_refusals(kw, code):
    assert varlen(**kw) == code


def tree(q=16, k=16, v=16, table=16, M=4, P=8, page=16, lens=16, mask=16, shared=0, tl=NULL, out=16, dt=0, lse=16,
         B=2, T=4, Sk=0, Hq=4, Hk=2, d=64, scale=0.125):
    return G.load_serve().gqa_attn_fwd_tree(q, k, v, table, M, P, page, lens, mask, shared, tl, out, dt, lse, B, T,
                                            Sk, Hq, Hk, d, scale, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=NULL), 1), (dict(k=NULL), 1), (dict(v=NULL), 1), (dict(lens=NULL), 1), (dict(mask=NULL), 1),
    (dict(out=NULL), 1), (dict(lse=NULL), 1),
    (dict(B=0), 2), (dict(T=0), 2), (dict(M=0), 2), (dict(P=0), 2), (dict(page=8), 2), (dict(page=48), 2),
    (dict(dt=-1), 2), (dict(scale=float("inf")), 2), (dict(table=NULL, Sk=0), 2),
    (dict(M=1 << 27), 2), (dict(P=1 << 27), 2), (dict(B=1 << 20, T=1 << 10), 2), (dict(table=NULL, Sk=1 << 30), 2),
    (dict(Hq=5), 3), (dict(d=80), 4),
    (dict(q=8), 5), (dict(table=18), 5), (dict(lens=17), 5), (dict(mask=18), 5), (dict(tl=18), 5),
])
def test_tree_refusals(kw, code):
    assert tree(**kw) == code


def resize(table=16, lens=16, refs=16, S=4, M=4, P=8, page=16, slots=16, new=16, n=2, status=16):
    return G.load_serve().gqa_cache_resize(table, lens, refs, S, M, P, page, slots, new, n, status, None)


def fork(k=16, v=32, layers=2, row=256, table=16, lens=16, refs=16, S=4, M=4, P=8, page=16, par=16, kid=16, n=2,
         status=16):
    return G.load_serve().gqa_cache_fork(k, v, layers, row, table, lens, refs, S, M, P, page, par, kid, n, status,
                                         None)


def compact(k=16, v=32, layers=2, row=256, table=16, lens=16, refs=16, S=4, M=4, P=8, page=16, keep=16, m=16,
            tl=NULL, T=4, status=16):
    return G.load_serve().gqa_cache_compact(k, v, layers, row, table, lens, refs, S, M, P, page, keep, m, tl, T,
                                            status, None)


STATE = [(dict(table=NULL), 1), (dict(lens=NULL), 1), (dict(refs=NULL), 1), (dict(status=NULL), 1),
         (dict(S=0), 2), (dict(M=0), 2), (dict(P=0), 2), (dict(page=8), 2), (dict(page=24), 2), (dict(page=-16), 2),
         (dict(M=1 << 27), 2), (dict(P=1 << 27), 2), (dict(table=18), 5), (dict(lens=17), 5), (dict(refs=18), 5),
         (dict(status=18), 5)]
POOLS = [(dict(k=NULL), 1), (dict(v=NULL), 1), (dict(layers=0), 2), (dict(row=0), 2), (dict(row=24), 2),
         (dict(row=1 << 25), 2), (dict(k=24), 5), (dict(v=40), 5)]


@pytest.mark.parametrize("kw,code", STATE + [(dict(new=NULL), 1), (dict(n=-1), 2), (dict(n=4097), 2),
                                             (dict(slots=18), 5), (dict(new=17), 5)])
def test_resize_refusals(kw, code):
    assert resize(**kw) == code


@pytest.mark.parametrize("kw,code", STATE + POOLS + [(dict(par=NULL), 1), (dict(kid=NULL), 1), (dict(n=4097), 2),
                                                     (dict(par=18), 5), (dict(kid=17), 5)])
def test_fork_refusals(kw, code):
    assert fork(**kw) == code


@pytest.mark.parametrize("kw,code", STATE + POOLS + [(dict(keep=NULL), 1), (dict(m=NULL), 1), (dict(T=0), 2),
                                                     (dict(keep=18), 5), (dict(m=17), 5), (dict(tl=18), 5)])
def test_compact_refusals(kw, code):
    assert compact(**kw) == code


def test_no_gpu_is_an_error_not_a_fallback():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for call in (varlen, tree, resize, fork, compact):
        assert call() in NO_GPU
    assert tree(table=NULL, Sk=64, tl=16, shared=1) in NO_GPU
    assert varlen(qs=512, ks=512, vs=512) in NO_GPU


def _i(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _h(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_the_binding_refuses_host_tensors_and_wrong_types():
    with pytest.raises(ValueError):
        G.gqa_attn_fwd_varlen(_h(8, 4, 64), _h(8, 2, 64), _h(8, 2, 64), _i(3))
    with pytest.raises(ValueError):
        G.gqa_attn_fwd_varlen(_h(8, 256), _h(8, 2, 64), _h(8, 2, 64), _i(3))
    with pytest.raises(ValueError):
        G.gqa_attn_fwd_tree(_h(2, 4, 4, 64), _h(2, 16, 2, 64), _h(2, 16, 2, 64), _i(2, 4, 1), _i(2))
    with pytest.raises(ValueError):
        G.gqa_cache_resize(_i(4, 4), _i(4), _i(8), 16, _i(4))
    with pytest.raises(ValueError):
        G.gqa_cache_fork(_h(8, 16, 2, 64), _h(8, 16, 2, 64), _i(4, 4), _i(4), _i(8), _i(1), _i(1))
    with pytest.raises(ValueError):
        G.gqa_cache_compact(_h(8, 16, 2, 64), _h(8, 16, 2, 64), _i(4, 4), _i(4), _i(8), _i(4, 2), _i(4))


def test_ranges_cut_the_steps_without_a_gap():
    """The arithmetic of the ranges schedule: CTA c takes steps [floor(all c / n), floor(all (c + 1)
    / n)), and the CTA of step x is ((x + 1) n - 1) // all; no range is empty when n <= all."""
    import random
    r = random.Random(1)
    for _ in range(300):
        n = r.randint(1, 300)
        steps = r.choice([n, n + 1, r.randint(n, 10 * n), r.randint(n, 10 ** 9)])
        start = [steps * c // n for c in range(n + 1)]
        assert start[0] == 0 and start[n] == steps and all(a < b for a, b in zip(start, start[1:]))
        for x in [0, steps - 1] + [r.randrange(steps) for _ in range(30)] + [s for s in start[:-1][:40]]:
            c = ((x + 1) * n - 1) // steps
            assert start[c] <= x < start[c + 1]
