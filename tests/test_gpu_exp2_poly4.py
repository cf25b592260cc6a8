"""The device code of the serving softmax's polynomial 2^x, compiled from its header into a small
probe, against exact 2^x and the host restatement of its steps."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from tests import exp2_poly4_ref as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def test_device_polynomial(tmp_path):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    out = str(tmp_path / "libprobe.so")
    subprocess.run(["nvcc", "-O3", "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-Xcompiler",
                    "-fPIC", "-I", R.FOLDER, "-I", os.path.join(os.path.dirname(R.FOLDER), "csrc"), "-o", out,
                    os.path.join(R.HERE, "exp2_poly4_probe.cu")], check=True)
    lib = ctypes.CDLL(out)
    lib.exp2_poly4_eval.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int]
    x = R.points()
    xd = torch.from_numpy(x).cuda()
    yd = torch.empty_like(xd)
    assert lib.exp2_poly4_eval(xd.data_ptr(), yd.data_ptr(), xd.numel()) == 0
    y = yd.cpu().numpy()
    R.check(x, y)
    # the same steps: equal up to one step (the host emulates fma in 64 bits)
    assert np.abs(y.view(np.int32).astype(np.int64) - R.poly4(x).view(np.int32).astype(np.int64)).max() <= 1
