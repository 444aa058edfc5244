"""Child process of test_gpu_kv_timeout.py, run on the test-hook build of the library (``FATHOM_LIB`` names it).  Prints
one JSON line for each case with what it saw.

A chunk's attention runs normally, then with one arrival withheld for one tile of one CTA
(``FATHOM_TEST_WITHHOLD_TILE``): that tile never fills, so the warp that issues the products, the softmax warps and the
load warps run out of polls one after another, leave their loops, wait for their products and copies and end.  Then it
runs normally again."""
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
sys.path.insert(0, os.path.join(ROOT, "tests"))

import torch  # noqa: E402

from _kv import fill, make_batch, make_cache  # noqa: E402
from long_context_decode_bit_b200 import fathom  # noqa: E402

WITHHOLD = "FATHOM_TEST_WITHHOLD_TILE"
CASES = [(fmt, D) for fmt in ("bf16", "int8", "e4m3") for D in (64, 128, 160, 256)]
TILES = (0, 1, 2, 5)    # K0, V0, K1, V2
H = 32                  # groups: enough CTAs that each takes all tokens of its rows


def main():
    lib = fathom.load()._name
    for fmt, D in CASES:
        lens = [(100, 900), (50, 300)]
        assert fathom.paged_attention_workspace_bytes(H, 4, D, 150, 2, 100, 900) == 0
        pages, table, cu, length = make_batch(lens, 64)
        cache = make_cache(fathom, fmt, pages, H, D, 64)
        fill(fathom, cache, lens, table)
        q = torch.randn((150, 4 * H, D), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").bfloat16()

        def call():
            out = torch.full_like(q, 7.0)
            fathom.paged_attention(cache, q, table, cu, length, 100, 900, out=out)
            torch.cuda.synchronize()
            return out
        want = call()
        for tile in TILES:
            got = {"lib": lib, "fmt": fmt, "D": D, "tile": tile, "before": fathom.device_status()}
            os.environ[WITHHOLD] = str(tile)
            try:
                out = call()
            finally:
                del os.environ[WITHHOLD]
            got["withheld"] = fathom.device_status()
            got["others_equal"] = torch.equal(out[:, 4:], want[:, 4:]) and torch.equal(out[100:], want[100:])
            got["clear"] = fathom.device_status(clear=True)
            got["after"] = fathom.device_status()
            got["again_equal"] = torch.equal(call(), want)
            got["end"] = fathom.device_status()
            print(json.dumps(got), flush=True)


if __name__ == "__main__":
    main()
