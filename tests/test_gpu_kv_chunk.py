"""Attention of prompt chunks over the paged cache against the 64-bit oracle, at the places where its tiles (256 query
rows, 128 tokens), its ring of tiles and its stretches of tokens begin and end."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import kv as okv
from _kv import TYPES, check_attention, fill, host, make_batch, make_cache

pytestmark = pytest.mark.gpu
DEV = "cuda"


def queries(shape, seed, dtype=torch.bfloat16, loud=2.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (loud * torch.randn(shape, generator=g, device=DEV)).to(dtype)


def both(fathom, cache, fmt, q, table, cu, length, new, most, causal=True, scale=None):
    out = fathom.paged_attention(cache, q, table, cu, length, new, most, causal=causal, scale=scale)
    ref = okv.attend(host(cache), fmt, q.float().cpu().numpy(), table.cpu().numpy(), cu.cpu().numpy(), length.cpu().numpy(),
                     cache.D ** -0.5 if scale is None else scale, causal)
    check_attention(out, ref, most, cache.D, q.dtype)
    return out


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("fmt", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("H,G,D,page,lens", [
    (1, 1, 128, 64, [(128, 128)]),                    # one row tile, one tile of tokens
    (1, 1, 128, 64, [(129, 129), (127, 127)]),
    (1, 8, 64, 16, [(32, 128), (33, 129), (31, 1)]),  # one row over a row tile
    (1, 2, 128, 16, [(128, 256), (128, 255), (128, 257)]),
    (2, 4, 128, 128, [(65, 2000)]),                   # the ring goes round
    (1, 3, 64, 32, [(200, 3001)]),
    (1, 5, 128, 256, [(260, 1500), (1, 900), (0, 10)]),
    (3, 7, 64, 64, [(19, 700), (100, 101)]),
    (1, 1, 256, 64, [(128, 128), (129, 129), (64, 64)]),   # beyond 128 channels: one row tile, 64 tokens
    (1, 4, 256, 16, [(33, 65), (32, 63), (16, 3000)]),
    (2, 2, 160, 32, [(70, 1000), (0, 5)]),
    (1, 8, 224, 256, [(40, 777)]),
    (1, 3, 192, 128, [(50, 320), (300, 301)]),
])
def test_edges_of_tiles(fathom_gpu, fmt, causal, H, G, D, page, lens):
    lens = [(min(n, t), t) for n, t in lens]
    pages, table, cu, length = make_batch(lens, page, seed=D + G)
    cache = make_cache(fathom_gpu, fmt, pages, H, D, page, ("head", "token", "layer")[(G + H) % 3])
    fill(fathom_gpu, cache, lens, table, seed=G)
    q = queries((int(cu[-1]), H * G, D), 4)
    both(fathom_gpu, cache, fmt, q, table, cu, length, max(n for n, _ in lens), max(t for _, t in lens), causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("layout", ["head", "token", "layer"])
@pytest.mark.parametrize("fmt", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("H,G,D,page,lens", [(2, 4, 96, 64, [(60, 500), (20, 129)]), (3, 5, 32, 16, [(130, 999)]),
                                             (1, 1, 96, 16, [(300, 300), (1, 5000)]), (1, 3, 32, 256, [(33, 3000), (40, 40)])])
def test_widths_between(fathom_gpu, fmt, causal, layout, H, G, D, page, lens):
    """32 and 96 channels, taken as 64 and 128 with zeros behind: what lies behind a row in the cache is not used."""
    pages, table, cu, length = make_batch(lens, page, seed=D)
    cache = make_cache(fathom_gpu, fmt, pages, H, D, page, layout)
    if fmt != "bf16":
        cache.k_scale.fill_(255), cache.v_scale.fill_(255)
    else:
        cache.k.fill_(float("nan")), cache.v.fill_(float("nan"))
    fill(fathom_gpu, cache, lens, table, seed=G)
    q = queries((int(cu[-1]), H * G, D), 4)
    both(fathom_gpu, cache, fmt, q, table, cu, length, max(n for n, _ in lens), max(t for _, t in lens), causal)


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_maximum_that_keeps_growing(fathom_gpu, fmt, D):
    """Keys that point at the queries more and more along the sequence, by steps smaller and larger than the 2^8 below
    which the running maximum stays; then the other way round."""
    lens = [(150, 1300)]
    pages, table, cu, length = make_batch(lens, 64)
    base = torch.randn(D, generator=torch.Generator().manual_seed(1)).to(DEV)
    for grow in (0.002, 0.02, 0.2, -0.02):
        cache = make_cache(fathom_gpu, fmt, pages, 1, D, 64)
        t = torch.arange(1300, device=DEV, dtype=torch.float32)
        k = (base[None] * (grow * (t if grow > 0 else t - 1300))[:, None] + 0.1 * queries((1300, D), 5, torch.float32))[:, None]
        v = queries((1300, 1, D), 6, torch.float32)
        one = torch.tensor([0, 1300], dtype=torch.int32, device=DEV)
        fathom_gpu.kv_write(cache, k.contiguous(), v, table, one, length)
        q = (base[None, None] + 0.1 * queries((150, 2, D), 7, torch.float32)).to(torch.bfloat16)
        both(fathom_gpu, cache, fmt, q, table, cu, length, 150, 1300)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("new", [1, 100])
def test_pages_missing_in_the_middle(fathom_gpu, new, dtype):
    """Entries of the table that name no page: their tokens are left out, by whole tiles and within tiles."""
    for page in (16, 64, 256):
        lens = [(new, 1500), (new, 700)]
        pages, table, cu, length = make_batch(lens, page)
        cache = make_cache(fathom_gpu, "int8", pages, 2, 128, page)
        fill(fathom_gpu, cache, lens, table)
        table[0, 1] = -1
        table[0, 3:3 + 256 // page] = pages
        table[1, 0] = 1 << 30
        table[1, 2] = -7
        both(fathom_gpu, cache, "int8", queries((2 * new, 8, 128), 4, TYPES[dtype]), table, cu, length, new, 1500)


@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("fmt", ["bf16", "int8", "e4m3"])
def test_nan_keys_are_not_hidden(fathom_gpu, fmt, new):
    """A NaN among the keys a row sees makes the row NaN, also where no other key is left; other sequences stay."""
    lens = [(new, new), (new, new + 30)]
    pages, table, cu, length = make_batch(lens, 64)
    cache = make_cache(fathom_gpu, fmt, pages, 1, 128, 64)
    k, v = torch.ones(2 * new + 30, 1, 128, device=DEV), torch.ones(2 * new + 30, 1, 128, device=DEV)
    k[:new] = float("nan")
    everything = torch.tensor([0, new, 2 * new + 30], dtype=torch.int32, device=DEV)
    fathom_gpu.kv_write(cache, k, v, table, everything, length)
    for dt in TYPES.values():
        out = fathom_gpu.paged_attention(cache, queries((2 * new, 4, 128), 4, dt), table, cu, length, new, new + 30)
        assert out[:new].isnan().all() and not out[new:].isnan().any()


def test_many_stretches(fathom_gpu):
    """A session long enough for the tokens to be cut into stretches, against the same call cut otherwise (bounded by a
    larger max_len) within the bound of both, and run twice with equal results."""
    n = 20000
    for new, G in ((1, 4), (12, 2), (40, 4), (300, 2)):
        lens = [(new, n)]
        pages, table, cu, length = make_batch(lens, 64)
        cache = make_cache(fathom_gpu, "int8", pages, 1, 128, 64)
        fill(fathom_gpu, cache, lens, table)
        q = queries((new, G, 128), 4)
        few = torch.arange(0, new, 1 + new // 8)
        ref = okv.attend(host(cache), "int8", q.float().cpu().numpy(), table.cpu().numpy(), cu.cpu().numpy(),
                         length.cpu().numpy(), 128 ** -0.5)
        ref = tuple(np.asarray(x)[few.numpy()] for x in ref)
        out = fathom_gpu.paged_attention(cache, q, table, cu, length, new, n)
        assert torch.equal(out, fathom_gpu.paged_attention(cache, q, table, cu, length, new, n))
        check_attention(out[few], ref, n, 128, torch.bfloat16)
        check_attention(fathom_gpu.paged_attention(cache, q, table, cu, length, new, 100 * n)[few], ref, n, 128, torch.bfloat16)
    assert fathom_gpu.device_status() == fathom_gpu.OK


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("span", [10, 40])
@pytest.mark.parametrize("D,new", [(128, 1), (96, 1), (64, 5), (128, 100), (256, 3)])
def test_blocks_of_very_different_sizes(fathom_gpu, fmt, dtype, span, D, new):
    """Powers of two 2^-span .. 2^span among the blocks of K, V and q, small blocks of K where q is large: operands hold
    them all exactly."""
    n = 300
    lens = [(new, n)]
    pages, table, cu, length = make_batch(lens, 64)
    cache = make_cache(fathom_gpu, fmt, pages, 1, D, 64)
    g = torch.Generator(device=DEV).manual_seed(span + D)
    size = lambda *shape: torch.exp2(torch.randint(-span, span + 1, shape, generator=g, device=DEV).float())  # noqa: E731
    chan = size(1, 1, D // 32, 1)
    k = (queries((n, 1, D // 32, 32), 1, torch.float32) * chan).flatten(2)
    v = (queries((n, 1, D // 32, 32), 2, torch.float32) * size(n, 1, D // 32, 1)).flatten(2)
    cu_all = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    fathom_gpu.kv_write(cache, k.contiguous(), v.contiguous(), table, cu_all, length)
    q = (queries((new, 4, D // 32, 32), 3, torch.float32) / chan).flatten(2).to(TYPES[dtype])
    both(fathom_gpu, cache, fmt, q, table, cu, length, new, n)


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
@pytest.mark.parametrize("D", [32, 64, 128, 160, 256])
def test_again_and_again(fathom_gpu, fmt, D):
    """Many calls one behind another, over maxima that grow often (products and softmax meet in every order): the same
    result each time, and no wait that ran out."""
    lens = [(256, 8000), (100, 4000)]
    pages, table, cu, length = make_batch(lens, 64)
    cache = make_cache(fathom_gpu, fmt, pages, 4, D, 64)
    k = torch.randn(12000, 4, D, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    k *= torch.cat([torch.linspace(0.1, 12, 8000), torch.linspace(0.1, 12, 4000)]).to(DEV)[:, None, None]
    v = torch.randn(12000, 4, D, generator=torch.Generator(device=DEV).manual_seed(2), device=DEV)
    fathom_gpu.kv_write(cache, k, v, table, torch.tensor([0, 8000, 12000], dtype=torch.int32, device=DEV), length)
    q = queries((356, 16, D), 4)
    want = fathom_gpu.paged_attention(cache, q, table, cu, length, 256, 8000)
    got = [fathom_gpu.paged_attention(cache, q, table, cu, length, 256, 8000) for _ in range(40)]
    assert fathom_gpu.device_status() == fathom_gpu.OK
    assert all(torch.equal(g, want) for g in got)
    few = torch.tensor([0, 100, 255, 256, 300, 355])
    ref = okv.attend(host(cache), fmt, q.float().cpu().numpy(), table.cpu().numpy(), cu.cpu().numpy(), length.cpu().numpy(),
                     D ** -0.5)
    check_attention(want[few], tuple(x[few.numpy()] for x in ref), 8000, D, torch.bfloat16)


@pytest.mark.parametrize("new", [1, 100])
def test_first_call_under_capture(new):
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, os.path.join(here, "_capture_child.py"), str(new)], cwd=os.path.dirname(here),
                       env=dict(os.environ, PYTHONPATH=os.path.dirname(here)), capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("new", [2, 100])
def test_row_bounds_that_make_no_sense(fathom_gpu, new):
    """Offsets below zero, beyond the rows, or decreasing: no row outside the call's is read or written, and sequences
    whose own bounds are sound get their results."""
    lens = [(new, 300)] * 4
    pages, table, cu, length = make_batch(lens, 64)
    cache = make_cache(fathom_gpu, "int8", pages, 2, 128, 64)
    fill(fathom_gpu, cache, lens, table)
    for dt in TYPES.values():
        q = queries((4 * new + 64, 8, 128), 4, dt)
        mid = q[32:-32]
        good = fathom_gpu.paged_attention(cache, mid, table, cu, length, new, 300)
        for bad in ([-5, new, 2 * new, 3 * new, 4 * new], [0, new, 2 * new, 1 << 30, 4 * new], [0, new, 2 * new, new, 0],
                    [1 << 30, new, 2 * new, 3 * new, 7 * new], [-(1 << 31), new, 2 * new, -7, (1 << 31) - 1]):
            c = torch.tensor(bad, dtype=torch.int32, device=DEV)
            out = torch.full((4 * new + 64, 8, 128), 7.0, dtype=dt, device=DEV)
            fathom_gpu.paged_attention(cache, mid, table, c, length, new, 300, out=out[32:-32])
            assert torch.equal(out[32 + new:32 + 2 * new], good[new:2 * new])
            assert (out[:32] == 7.0).all() and (out[-32:] == 7.0).all()
            kv = [torch.full((2, 4 * new + 64, 128), 7.0, device=DEV) for _ in range(2)]
            fathom_gpu.kv_read(cache, table, c, length, 4 * new, out=[t[:, 32:-32] for t in kv])
            assert all((t[:, :32] == 7.0).all() and (t[:, -32:] == 7.0).all() for t in kv)


def test_one_place_for_two_outputs(fathom_gpu):
    pages, table, cu, length = make_batch([(5, 30)], 16)
    cache = make_cache(fathom_gpu, "int8", pages, 1, 64, 16)
    out = torch.zeros(1, 5, 64, device=DEV)
    with pytest.raises(fathom_gpu.FathomError):
        fathom_gpu.kv_read(cache, table, cu, length, 5, out=(out, out))


@pytest.mark.parametrize("fmt,D", [("bf16", 128), ("int8", 64), ("int8", 256)])
def test_two_chunks_at_once(fathom_gpu, fmt, D):
    """Two calls on two streams, many times over, each with scratch of its own: the results of one call alone."""
    lens = [(300, 5000), (150, 2500)]
    pages, table, cu, length = make_batch(lens, 32)
    cache = make_cache(fathom_gpu, fmt, pages, 2, D, 32)
    fill(fathom_gpu, cache, lens, table)
    qs = [queries((450, 8, D), 4 + i) for i in range(2)]
    want = [fathom_gpu.paged_attention(cache, q, table, cu, length, 300, 5000) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(fathom_gpu.paged_attention(cache, qs[i], table, cu, length, 300, 5000))
            got[i].append(fathom_gpu.paged_attention(cache, qs[i], table, cu, length, 300, 5000, stream=s))   # named instead
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[i]) for i in range(2) for x in got[i])
    assert fathom_gpu.device_status() == fathom_gpu.OK
