"""A bounded wait of the chunk attention that runs out is reported, not hung on.

The roles of ``kv_chunk_kernel`` wait for one another on mbarriers with a poll limit that a correct launch never
reaches, so the test uses the build of the library made for it (``build(test_hooks=True)``: a poll limit of 65536 and a
switch that withholds one arrival), in a child process.  Nothing faults: every role gives up, products and copies on
their way are waited for, tensor memory is freed (the next launch, which needs all of it, runs), and the status reaches
the host."""
import json
import os
import subprocess
import sys

import pytest
import torch

from long_context_decode_bit_b200 import build, fathom

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_withheld_tile_reports_timeout_and_context_recovers():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import _kv_timeout_child as child
    lib = build.build(test_hooks=True)
    env = dict(os.environ, FATHOM_LIB=lib)
    env.pop(child.WITHHOLD, None)
    r = subprocess.run([sys.executable, os.path.join(HERE, "_kv_timeout_child.py")], env=env, capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-4000:]
    seen = [json.loads(line) for line in r.stdout.strip().splitlines()]
    assert [(s["fmt"], s["D"], s["tile"]) for s in seen] == [(f, d, t) for f, d in child.CASES for t in child.TILES]
    for s in seen:
        assert s["lib"] == lib
        assert s["before"] == fathom.OK
        assert s["withheld"] == fathom.ERR_TIMEOUT, s
        assert s["others_equal"], s       # other CTAs' rows are as they should be
        assert s["clear"] == fathom.ERR_TIMEOUT and s["after"] == fathom.OK, s
        assert s["again_equal"] and s["end"] == fathom.OK, s
