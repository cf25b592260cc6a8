"""The coefficients of the serving softmax's polynomial 2^x as its header states them, and a
float32 restatement of its steps.  Error of a value: the polynomial's own (BOUND's first term,
which the tests hold against the least possible), and the roundings of its evaluation: the last
fma by half a step of a value in [0.7, 1.42], the three before it scaled by |f| <= 1/2 each:
below 2^-23 together."""
import os
import re

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
FOLDER = os.path.join(os.path.dirname(HERE), "gqa_exact_attention_b200", "csrc_serve")
HEADER = os.path.join(FOLDER, "exp2_poly4.cuh")
BOUND = 2.84e-6 + 2.0 ** -23


def constants():
    src = open(HEADER).read()
    return [np.float32(float(re.search(rf"\bc{i} = ([-0-9.e]+)f", src).group(1))) for i in (1, 2, 3, 4)]


def _fma(a, b, c):  # a * b is exact in 64 bits; one addition there, then rounding to 32
    return (a.astype(np.float64) * np.asarray(b, dtype=np.float64) + np.float64(c)).astype(np.float32)


def poly4(x):
    c1, c2, c3, c4 = constants()
    x = np.maximum(np.asarray(x, dtype=np.float32), np.float32(-126.0))
    t = x + np.float32(12582912.0)
    f = x - (t - np.float32(12582912.0))
    q = _fma(f, c4, c3)
    for c in (c2, c1, np.float32(1.0)):
        q = _fma(q, f, c)
    bits = q.view(np.int32).astype(np.int64) + (t.view(np.int32).astype(np.int64) << 23)
    return (bits & 0xFFFFFFFF).astype(np.uint32).view(np.float32)


def points():
    return np.concatenate([np.linspace(-125.0, 8.0, 1_000_001), np.linspace(-1, 1, 100_001), np.arange(-126, 9),
                           [-127.5, -1000.0, -np.inf]]).astype(np.float32)


def check(x, y):
    ok = x >= -125.0
    rel = np.abs(y[ok].astype(np.float64) / np.exp2(x[ok].astype(np.float64)) - 1.0)
    assert rel.max() <= BOUND, rel.max()
    whole = ok & (x == np.rint(x))
    assert np.array_equal(y[whole], np.exp2(x[whole].astype(np.float64)).astype(np.float32))
    assert (y[x <= -126.0] == np.float32(2.0 ** -126)).all()
