"""Child process of test_gpu_kv_bounds.py, run on the test-hook build of the library (``FATHOM_LIB`` names it), whose
device-side bounds checks are on.  Writes, reads and attends over caches in all formats and layouts (every check must
pass), saves the outputs for the parent to compare with the product library's, then makes the checks fail on purpose
(``FATHOM_TEST_SHRINK_CAP=1``: they allow half of the cache; skipped accesses are never out of bounds) and reports what
the host sees.  Prints one JSON line."""
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
sys.path.insert(0, os.path.join(ROOT, "tests"))

import numpy as np  # noqa: E402
import torch  # noqa: E402

from _kv import make_batch, make_cache  # noqa: E402
from long_context_decode_bit_b200 import fathom  # noqa: E402

SHRINK = "FATHOM_TEST_SHRINK_CAP"
#        H, G, D, page, [(new, length)]: single tokens, a few rows, chunks; the last pages partly filled
SHAPES = [(2, 4, 128, 64, [(1, 1), (1, 3000)]), (3, 1, 32, 16, [(1, 333), (1, 17)]), (1, 5, 96, 16, [(3, 129), (2, 31)]),
          (2, 4, 128, 32, [(100, 1000), (7, 7)]), (1, 8, 64, 256, [(40, 700), (0, 9)]), (1, 3, 256, 64, [(50, 500), (1, 65)]),
          (2, 2, 160, 128, [(4, 77), (33, 200)])]
CASES = [(fmt, layout, i) for fmt in ("bf16", "int8", "e4m3") for layout in ("head", "token", "layer")
         for i in range(len(SHAPES))]


def outputs(fmt, layout, shape):
    """What the four operators give for a case."""
    H, G, D, page, lens = shape
    pages, table, cu, length = make_batch(lens, page, spare=1)
    table[0, 0] = pages        # one page that is not there
    cache = make_cache(fathom, fmt, pages, H, D, page, layout)
    g = torch.Generator(device="cuda").manual_seed(D)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    total = sum(t for _, t in lens)
    everything = torch.tensor(np.cumsum([0] + [t for _, t in lens]), dtype=torch.int32, device="cuda")
    fathom.kv_write(cache, rand(total, H, D), rand(total, H, D), table, everything, length)
    out = {"k": None, "v": None}
    out["k"], out["v"] = fathom.kv_read(cache, table, everything, length, total, dtype=torch.float32)
    rows, new, most = int(cu[-1]), max(n for n, _ in lens), max(t for _, t in lens)
    q = rand(rows, H * G, D)
    for name, dt in (("bf16", torch.bfloat16), ("fp32", torch.float32)):
        out[name] = fathom.paged_attention(cache, q.to(dt), table, cu, length, new, most).float()
    n = lens[0][1]
    idx = torch.randint(0, n, (H, 300), generator=g, device="cuda").to(torch.int32)
    cnt = torch.full((H,), 290, dtype=torch.int32, device="cuda")
    out["union"] = fathom.paged_union_attention(cache, rand(H, G, D), table[0], n, idx, cnt)
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in out.items()}


def main(out_path):
    seen = {"lib": fathom.load()._name, "status": {}, "shrunk": {}}
    saved = {}
    for fmt, layout, i in CASES:
        for name, x in outputs(fmt, layout, SHAPES[i]).items():
            saved[f"{fmt}/{layout}/{i}/{name}"] = x
        seen["status"][f"{fmt}/{layout}/{i}"] = fathom.device_status()
    np.savez(out_path, **saved)
    for fmt in ("bf16", "int8", "e4m3"):
        for i in range(len(SHAPES)):
            os.environ[SHRINK] = "1"
            try:
                outputs(fmt, "head", SHAPES[i])
            finally:
                del os.environ[SHRINK]
            got = [fathom.device_status(), fathom.device_status(clear=True), fathom.device_status()]
            again = outputs(fmt, "head", SHAPES[i])
            same = all(np.array_equal(x, saved[f"{fmt}/head/{i}/{name}"], equal_nan=True) for name, x in again.items())
            seen["shrunk"][f"{fmt}/{i}"] = got + [same, fathom.device_status()]
    print(json.dumps(seen))


if __name__ == "__main__":
    main(sys.argv[1])
