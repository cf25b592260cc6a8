"""Failure paths of the serving operators: a bounded wait that runs out, and scratch that cannot
be had; and the first call of a process made in a stream capture.  The wait runs out on purpose at a barrier that nothing completes (the GPU stays healthy);
each case runs in a process of its own."""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

_CHILD = r"""
import json, os, sys, time
sys.path.insert(0, os.getcwd())
import torch
import gqa_exact_attention_b200 as G

G.load_serve()
kind = sys.argv[1]
gen = torch.Generator(device="cuda").manual_seed(1)
rn = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()
if kind.startswith("varlen"):
    lens = [700, 40, 260] if kind == "varlen ranges" else [700, 900, 640, 512, 1100, 800]
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).int()
    q, k, v = rn(sum(lens), 32, 128), rn(sum(lens), 8, 128), rn(sum(lens), 8, 128)
    run = lambda: G.gqa_attn_fwd_varlen(q, k, v, cu, causal=True)
else:
    T = 8 if kind == "tree" else 80
    q, k, v = rn(3, T, 8, 64), rn(3, 900, 2, 64), rn(3, 900, 2, 64)
    mask = torch.randint(-2 ** 31, 2 ** 31 - 1, (3, T, (T + 31) // 32), generator=gen, device="cuda").int()
    lens = torch.tensor([900, 100, 500], device="cuda").int()
    run = lambda: G.gqa_attn_fwd_tree(q, k, v, mask, lens)
want = run()
torch.cuda.synchronize()
res = {"before": G.gqa_serve_device_status(reset=True)}
os.environ["GQA_WAIT_TIMEOUT_MS"] = "20"
os.environ["GQA_FAULT_INJECT_STALL"] = "1"
t0 = time.time()
run()
torch.cuda.synchronize()
res["seconds"] = time.time() - t0
res["stalled"] = G.gqa_serve_device_status(reset=True)
del os.environ["GQA_FAULT_INJECT_STALL"], os.environ["GQA_WAIT_TIMEOUT_MS"]
got = run()
torch.cuda.synchronize()
res["after"] = G.gqa_serve_device_status(reset=True)
res["same"] = all(torch.equal(a, b) for a, b in zip(want, got))
os.environ["GQA_FAULT_INJECT_ALLOC"] = "1"
out, lse = (torch.full_like(x, float("nan")) for x in want)
try:
    (G.gqa_attn_fwd_varlen(q, k, v, cu, causal=True, out=out, lse=lse) if kind.startswith("varlen")
     else G.gqa_attn_fwd_tree(q, k, v, mask, lens, out=out, lse=lse))
    res["alloc"] = 0
except G.GqaError as e:
    res["alloc"] = e.status
torch.cuda.synchronize()
res["untouched"] = bool(torch.isnan(out).all() and torch.isnan(lse).all())
print("RESULT " + json.dumps(res), flush=True)
"""


@pytest.mark.parametrize("kind", ["varlen ranges", "varlen list", "tree", "tree of two tiles"])
def test_waits_run_out_and_scratch_is_missing(kind):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    env = {k: v for k, v in os.environ.items() if not k.startswith("GQA_")}
    r = subprocess.run([sys.executable, "-c", _CHILD, kind], cwd=ROOT, env=env, capture_output=True, text=True, timeout=120)
    lines = [ln for ln in r.stdout.splitlines() if ln.startswith("RESULT ")]
    assert lines, r.stdout + r.stderr
    res = json.loads(lines[0][7:])
    assert res["before"] == 0 and res["after"] == 0 and res["same"]
    assert res["stalled"] == 9 and res["seconds"] < 30
    assert res["alloc"] == 7 and res["untouched"]


_FIRST = r"""
import os, sys
sys.path.insert(0, os.getcwd())
import torch
import gqa_exact_attention_b200 as G

rn = lambda *s: torch.randn(s, device="cuda").bfloat16()
ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
kind = sys.argv[1]
if kind == "varlen":
    q, k, v, cu = rn(3000, 32, 128), rn(3000, 8, 128), rn(3000, 8, 128), ints(0, 1000, 3000)
    f = lambda: G.gqa_attn_fwd_varlen(q, k, v, cu, causal=True)
elif kind == "tree":
    q, k, v, mask, lens = rn(2, 8, 32, 128), rn(2, 4000, 8, 128), rn(2, 4000, 8, 128), ints(*[1] * 8).view(8, 1), ints(4000, 3000)
    f = lambda: G.gqa_attn_fwd_tree(q, k, v, mask, lens)
else:
    table, lens, refs = ints(*[-1] * 32).view(4, 8), ints(0, 0, 0, 0), ints(*[0] * 40)
    kp, vp, new, a, b = rn(2, 40, 16, 2, 64), rn(2, 40, 16, 2, 64), ints(20, 30, 0, 0), ints(0, 1), ints(2, 3)
    f = lambda: (G.gqa_cache_resize(table, lens, refs, 16, new), G.gqa_cache_fork(kp, vp, table, lens, refs, a, b))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    x = f()
graph.replay()
torch.cuda.synchronize()
y = f()
torch.cuda.synchronize()
assert all(torch.equal(s, t) for s, t in zip(x, y))
print("SAME", flush=True)
"""


@pytest.mark.parametrize("kind", ["varlen", "tree", "cache"])
def test_the_first_call_of_a_process_in_a_capture(kind):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    r = subprocess.run([sys.executable, "-c", _FIRST, kind], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert "SAME" in r.stdout, r.stdout + r.stderr
