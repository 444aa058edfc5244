"""The 64-bit oracle of the paged KV cache against things it was not written from: torch's own 8-bit
conversion, brute force over the exponents, and a softmax over the concatenated rows."""
import math

import numpy as np
import pytest
import torch

from oracle import kv as okv


def test_e4m3_patterns_are_torchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(np.isnan(t), np.isnan(okv.e4m3_table()))
    ok = ~np.isnan(t)
    assert np.array_equal(t[ok], okv.e4m3_table()[ok])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("scale", [1.0, 3e-5, 1e4, 1e-33])
def test_encode_is_the_least_exponent_that_fits(fmt, scale):
    rng = np.random.default_rng(3)
    x = (rng.standard_normal(64) * scale).astype(np.float32)
    codes, byte = okv.encode(x, fmt)
    for i in range(2):
        blk, e = x[32 * i:32 * i + 32].astype(np.float64), int(byte[i]) - 127
        m = np.abs(blk).max()

        def fits(t):
            return round(math.ldexp(m, -t)) <= 127 if fmt == "int8" else math.ldexp(m, -t) <= 464
        assert fits(e) or e == 7
        assert e == okv.LOWEST or not fits(e - 1)
        y = np.ldexp(blk, -e)
        got = codes[32 * i:32 * i + 32]
        if fmt == "int8":
            assert np.array_equal(got, np.rint(y).astype(np.int8))
        else:
            t = torch.tensor(np.clip(y, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
            assert np.array_equal(got, t)


def test_encode_edges():
    x = np.zeros(32, np.float32)
    for fmt in ("int8", "e4m3"):
        codes, byte = okv.encode(x, fmt)
        assert byte[0] == 27 and not codes.any()
    # 127.5 rounds to 128 (even), which is no code: the exponent goes up; just below it stays
    for top, e in ((127.5, 1), (np.nextafter(np.float32(127.5), np.float32(0)), 0), (127.0, 0), (64.0, 0), (63.7, -1)):
        x[5] = -top
        assert okv.encode(x, "int8")[1][0] == e + 127, top
    for top, e in ((464.0, 0), (np.nextafter(np.float32(464), np.float32(500)), 1), (448.0, 0), (256.0, 0)):
        x[5] = top
        assert okv.encode(x, "e4m3")[1][0] == e + 127, top
    x[5] = 1e9   # above the largest kept magnitude
    codes, byte = okv.encode(x, "e4m3")
    assert okv.decode(codes, byte, "e4m3")[5] == 57344.0
    for bad in (np.inf, -np.inf, np.nan):
        x[5] = bad
        codes, byte = okv.encode(x, "int8")
        assert byte[0] == 255 and not codes.any() and np.isnan(okv.decode(codes, byte, "int8")).all()


def test_bf16_bits_are_torchs():
    x = np.random.default_rng(1).standard_normal(1000).astype(np.float32) * np.float32(1e-3)
    assert np.array_equal(okv.bf16_bits(x), torch.tensor(x).bfloat16().view(torch.int16).numpy().view(np.uint16))


@pytest.mark.parametrize("fmt", ["bf16", "int8", "e4m3"])
def test_write_read_attend_against_concatenated_rows(fmt):
    rng = np.random.default_rng(5)
    H, G, D, page = 2, 3, 32, 16
    lens = [(3, 20), (1, 1), (4, 33)]
    table = np.array([[4, 0, -1], [2, -1, -1], [1, 3, 5]], np.int32)
    total = sum(t for _, t in lens)
    cu_all = np.cumsum([0] + [t for _, t in lens])
    length = np.array([t for _, t in lens])
    dt = {"bf16": np.uint16, "int8": np.int8, "e4m3": np.uint8}[fmt]
    zero = [np.zeros((6, H, page, D), dt), np.zeros((6, H, page, D), dt)]
    zero += [None, None] if fmt == "bf16" else [np.zeros((6, H, page, 1), np.uint8) for _ in range(2)]
    k, v = (rng.standard_normal((total, H, D)).astype(np.float32) for _ in range(2))
    cache = okv.write(zero, fmt, k, v, table, cu_all, length)
    rk, rv = okv.read(cache, fmt, table, cu_all, length, total)
    step = {"bf16": 2.0 ** -8, "int8": 2.0 ** -6, "e4m3": 2.0 ** -4}[fmt]   # of the block's largest, or of the value
    for x, r in ((k, rk), (v, rv)):
        ref = np.abs(x).max(-1, keepdims=True) if fmt == "int8" else np.maximum(np.abs(x), 1e-3)
        assert (np.abs(r.transpose(1, 0, 2) - x) <= step * ref).all()
    cu = np.cumsum([0] + [n for n, _ in lens])
    q = rng.standard_normal((cu[-1], H * G, D))
    out, mag, _ = okv.attend(cache, fmt, q, table, cu, length, 0.2)
    for b, (n, t) in enumerate(lens):
        for i in range(n):
            for hq in range(H * G):
                h = hq // G
                see = t - n + i + 1
                K, V = rk[h, cu_all[b]:cu_all[b] + see], rv[h, cu_all[b]:cu_all[b] + see]
                w = torch.softmax(torch.tensor(K @ q[cu[b] + i, hq] * 0.2), 0).numpy()
                assert np.allclose(out[cu[b] + i, hq], w @ V, rtol=1e-12, atol=1e-13)
    idx = np.array([[0, 5, 19, -1], [2, 3, 25, 7]], np.int32)   # 25 lies beyond sequence 0
    u, _, _ = okv.union_attend(cache, fmt, q[:2].reshape(2, H * G, D)[:, :G], table[0], 20, idx, np.array([3, 4]), 0.2)
    for h, keep in ((0, [0, 5, 19]), (1, [2, 3, 7])):
        w = torch.softmax(torch.tensor(rk[h, keep] @ q[h, 0] * 0.2), 0).numpy()
        assert np.allclose(u[h, 0], w @ rv[h, keep], rtol=1e-12, atol=1e-13)


def test_rows_that_see_nothing_are_zero():
    cache = [np.ones((1, 1, 16, 32), np.int8)] * 2 + [np.full((1, 1, 16, 1), 127, np.uint8)] * 2
    q = np.ones((5, 1, 32))
    # five new rows of a sequence of two tokens: the first three lie before it
    out, _, _ = okv.attend(cache, "int8", q, np.array([[0]]), [0, 5], [2], 1.0)
    assert (out[:3] == 0).all() and (out[3:] == 1).all()
    out, _, _ = okv.attend(cache, "int8", q, np.array([[7]]), [0, 5], [5], 1.0)   # a page id that names nothing
    assert (out == 0).all()
