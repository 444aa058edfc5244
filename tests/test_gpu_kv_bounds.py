"""The debug build's device-side bounds checks in the paged cache's kernels: the addresses of cached rows and their
exponents, the outputs' places and those of the scratch between stretches.  Built into the test-hook library and run in a
child process, as in test_gpu_debug_bounds.py."""
import json
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from long_context_decode_bit_b200 import build, fathom

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_cache_checks_pass_and_report(tmp_path):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import _kv_bounds_child as child
    lib = build.build(test_hooks=True)
    npz = str(tmp_path / "kv_bounds.npz")
    env = dict(os.environ, FATHOM_LIB=lib)
    env.pop(child.SHRINK, None)
    env.pop("FATHOM_TEST_WITHHOLD_TILE", None)
    r = subprocess.run([sys.executable, os.path.join(HERE, "_kv_bounds_child.py"), npz], env=env, capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-4000:]
    seen = json.loads(r.stdout.strip().splitlines()[-1])
    assert seen["lib"] == lib and len(seen["status"]) == len(child.CASES)
    assert all(st == fathom.OK for st in seen["status"].values()), seen["status"]
    # The checked build gives the product library's results.
    fathom.load()
    saved = np.load(npz)
    for fmt, layout, i in child.CASES:
        for name, x in child.outputs(fmt, layout, child.SHAPES[i]).items():
            assert np.array_equal(saved[f"{fmt}/{layout}/{i}/{name}"], x, equal_nan=True), (fmt, layout, i, name)
    # A failed check reaches the host, clears, and the next calls are right again.
    for key, got in seen["shrunk"].items():
        assert got == [fathom.ERR_BOUNDS, fathom.ERR_BOUNDS, fathom.OK, True, fathom.OK], (key, got)
