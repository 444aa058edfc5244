"""The paged KV cache on the GPU against the 64-bit oracle: what is written and read back bit for bit, attention
within the bounds of its roundings, over formats, widths, layouts, page sizes, ragged batches and empty rows."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import kv as okv
from _kv import FORMATS, TYPES, check_attention, fill, host, make_batch, make_cache

pytestmark = pytest.mark.gpu
DEV = "cuda"


def rand(shape, seed, dtype=torch.float32, spread=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(shape, generator=g, device=DEV)
    if spread:   # blocks of very different sizes
        x = x * torch.exp2(torch.randint(-20, 20, shape[:-1] + (1,), generator=g, device=DEV).float())
    return x.to(dtype)


def assert_same_cache(cache, want):
    for got, ref in zip(host(cache), want):
        assert (got is None) == (ref is None)
        assert got is None or np.array_equal(got, ref)


@pytest.mark.parametrize("layout", ["head", "token", "layer"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("fmt", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("H,D,page,lens", [(3, 96, 16, [(5, 40), (1, 1), (17, 17)]), (2, 128, 64, [(1, 200)]),
                                           (1, 32, 32, [(70, 100), (3, 33)]), (2, 256, 128, [(9, 130)])])
def test_write_and_read_exact(fathom_gpu, fmt, dtype, layout, H, D, page, lens):
    pages, table, cu, length = make_batch(lens, page)
    cache = make_cache(fathom_gpu, fmt, pages, H, D, page, layout)
    before = host(cache)
    total = int(cu[-1])
    k, v = rand((total, H, D), 1, TYPES[dtype]), rand((total, H, D), 2, TYPES[dtype])
    k[0, 0, :32] = 0.0
    fathom_gpu.kv_write(cache, k, v, table, cu, length)
    tn, cn, ln = table.cpu().numpy(), cu.cpu().numpy(), length.cpu().numpy()
    want = okv.write(before, fmt, k.float().cpu().numpy(), v.float().cpu().numpy(), tn, cn, ln)
    assert_same_cache(cache, want)
    ref = okv.read(want, fmt, tn, cn, ln, total)
    for out in ("fp32", "bf16"):
        got = fathom_gpu.kv_read(cache, table, cu, length, total, dtype=TYPES[out])
        for g, r in zip(got, ref):
            assert g.dtype == TYPES[out] and np.array_equal(g.float().cpu().numpy().astype(np.float64), r)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_write_borders(fathom_gpu, fmt):
    """Largest magnitudes next to where the exponent changes, ties, zeros, subnormal and huge rows, infinities, NaN."""
    tops = [127.5, np.nextafter(np.float32(127.5), np.float32(0)), 127.0, 63.75, 464.0,
            np.nextafter(np.float32(464), np.float32(1e9)), 448.0, 232.0, 1e-38, 1e-45, 3e38, 3.4028234e38, 57344.0, 65504.0,
            2.0 ** -94, 2.0 ** -95, np.inf, -np.inf, np.nan, 0.0]
    rng = np.random.default_rng(7)
    x = rng.uniform(-1, 1, (len(tops), 1, 32)).astype(np.float32)
    with np.errstate(all="ignore"):
        for i, t in enumerate(tops):
            x[i] *= np.float32(t) if np.isfinite(t) else np.float32(1)
            x[i, 0, i % 32] = t
    half = np.arange(32, dtype=np.float32) + np.float32(0.5)   # ties of the rounding
    half[0] = 127.0
    x = np.concatenate([x, half[None, None], -half[None, None]])
    x = np.where(np.isnan(x) & ~np.isnan(np.append(tops, [0, 0])[:, None, None]), 0, x).astype(np.float32)
    n = len(x)
    pages, table, cu, length = make_batch([(n, n)], 16)
    cache = make_cache(fathom_gpu, fmt, pages, 1, 32, 16)
    before = host(cache)
    t = torch.tensor(x, device=DEV)
    fathom_gpu.kv_write(cache, t, -t, table, cu, length)
    args = table.cpu().numpy(), cu.cpu().numpy(), length.cpu().numpy()
    want = okv.write(before, fmt, x, -x, *args)
    assert_same_cache(cache, want)
    got = fathom_gpu.kv_read(cache, table, cu, length, n, dtype=torch.float32)
    for g, r in zip(got, okv.read(want, fmt, *args, n)):
        assert np.array_equal(g.cpu().numpy().astype(np.float64), r, equal_nan=True)


def test_rows_of_other_strides_and_alignment(fathom_gpu):
    """Inputs cut out of a wider tensor, off by one element; outputs [rows][H][D] and odd; only one of K and V."""
    lens = [(21, 50), (2, 9)]
    pages, table, cu, length = make_batch(lens, 16)
    total = int(cu[-1])
    wide = rand((total, 2, 3, 131), 3, spread=False)
    for dtype in (torch.float32, torch.bfloat16):
        w = wide.to(dtype)
        for cut in (slice(0, 128), slice(1, 129)):
            k, v = w[:, 0, :, cut], w[:, 1, :, cut]
            cache = make_cache(fathom_gpu, "int8", pages, 3, 128, 16)
            before = host(cache)
            fathom_gpu.kv_write(cache, k, v, table, cu, length)
            want = okv.write(before, "int8", k.float().cpu().numpy(), v.float().cpu().numpy(), table.cpu().numpy(),
                             cu.cpu().numpy(), length.cpu().numpy())
            assert_same_cache(cache, want)
            ref = fathom_gpu.kv_read(cache, table, cu, length, total, dtype=dtype)
            flat = [torch.empty((total, 3, 128), dtype=dtype, device=DEV).transpose(0, 1) for _ in range(2)]
            odd = [torch.empty((3, total, 131), dtype=dtype, device=DEV)[:, :, 1:129] for _ in range(2)]
            for out in (flat, odd):
                fathom_gpu.kv_read(cache, table, cu, length, total, out=out)
                assert all(torch.equal(a, b) for a, b in zip(out, ref))
            one = torch.empty_like(ref[1])
            got = fathom_gpu.kv_read(cache, table, cu, length, total, out=(None, one))
            assert got[0] is None and torch.equal(one, ref[1])


def test_rows_of_no_sequence_and_pages_that_name_nothing(fathom_gpu):
    """Rows behind the last sequence, positions before 0 and beyond the table, ids out of range: nothing is written
    for them, they read as zeros (rows of no sequence are left alone)."""
    page, H, D = 16, 2, 64
    table = torch.tensor([[3, -1, 9, 1], [0, 2, 99999, -5]], dtype=torch.int32, device=DEV)   # 5 pages
    cu = torch.tensor([0, 70, 110], dtype=torch.int32, device=DEV)
    length = torch.tensor([64, 38], dtype=torch.int32, device=DEV)   # sequence 0: rows from position -6 on; 1: from -2
    total = 117
    cache = make_cache(fathom_gpu, "int8", 5, H, D, page)
    cache.k.fill_(7), cache.k_scale.fill_(120)
    before = host(cache)
    k, v = rand((total, H, D), 5), rand((total, H, D), 6)
    fathom_gpu.kv_write(cache, k, v, table, cu, length)
    args = table.cpu().numpy(), cu.cpu().numpy(), length.cpu().numpy()
    want = okv.write(before, "int8", k.cpu().numpy(), v.cpu().numpy(), *args)
    assert_same_cache(cache, want)
    out = [torch.full((H, total, D), 5.0, device=DEV) for _ in range(2)]
    fathom_gpu.kv_read(cache, table, cu, length, total, out=out)
    for g, r in zip(out, okv.read(want, "int8", *args, total)):
        r[:, 110:] = 5.0
        assert np.array_equal(g.cpu().numpy().astype(np.float64), r)
    for causal in (True, False):
        for dt in (torch.float32, torch.bfloat16):
            q = rand((total, H * 3, D), 8, dt, spread=False)
            o = torch.full_like(q, 5.0)
            fathom_gpu.paged_attention(cache, q, table, cu, length, 70, 64, causal=causal, out=o)
            ref = okv.attend(want, "int8", q.float().cpu().numpy(), *args, D ** -0.5, causal)
            check_attention(o, ref, 64, D, dt)
            assert (o[110:] == 5.0).all()
            assert not causal or (o[:6] == 0).all()


SHAPES = [
    # H, G, D, page, lens
    (2, 4, 128, 64, [(1, 1)]),
    (2, 4, 128, 64, [(1, 300), (1, 64), (1, 65), (1, 1000)]),
    (3, 1, 64, 16, [(1, 17), (1, 1), (1, 333)]),
    (1, 8, 128, 32, [(1, 2777)]),
    (2, 5, 96, 16, [(1, 129), (3, 31)]),
    (1, 3, 32, 128, [(2, 500), (1, 3)]),
    (2, 2, 256, 64, [(4, 77), (1, 200)]),
    (1, 7, 160, 16, [(5, 90)]),
    (1, 4, 128, 64, [(4, 700), (2, 129)]),
    (2, 4, 128, 64, [(33, 33), (64, 500), (1, 127), (0, 40)]),
    (1, 5, 128, 16, [(130, 777), (7, 40), (100, 100)]),
    (1, 1, 64, 256, [(300, 300), (129, 1500)]),
    (2, 3, 64, 32, [(57, 200), (90, 91)]),
    (1, 8, 128, 128, [(65, 1025)]),
    (1, 6, 192, 64, [(20, 150)]),
    (1, 4, 224, 16, [(40, 99)]),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("fmt", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("H,G,D,page,lens", SHAPES)
def test_attention(fathom_gpu, fmt, dtype, H, G, D, page, lens):
    pages, table, cu, length = make_batch(lens, page, seed=H + G)
    cache = make_cache(fathom_gpu, fmt, pages, H, D, page, ("head", "token", "layer")[(G + D // 32) % 3])
    fill(fathom_gpu, cache, lens, table, seed=D)
    total = int(cu[-1])
    q = rand((total, H * G, D), 4, TYPES[dtype], spread=False) * 2
    new, most = max(n for n, _ in lens), max(t for _, t in lens)
    args = host(cache), fmt, q.float().cpu().numpy(), table.cpu().numpy(), cu.cpu().numpy(), length.cpu().numpy()
    for causal in (True, False):
        out = fathom_gpu.paged_attention(cache, q, table, cu, length, new, most, causal=causal)
        check_attention(out, okv.attend(*args, D ** -0.5, causal), most, D, TYPES[dtype])
    assert torch.equal(out, fathom_gpu.paged_attention(cache, q, table, cu, length, new, most, causal=False))


@pytest.mark.parametrize("new", [1, 6, 150])
@pytest.mark.parametrize("fmt", ["bf16", "int8", "e4m3"])
def test_what_lies_beyond_the_length_is_not_used(fathom_gpu, fmt, new):
    """Infinities and NaN behind the last token of the last page, and in pages of nobody."""
    lens = [(new, 200), (min(new, 77), 77)]
    pages, table, cu, length = make_batch(lens, 64)
    cache = make_cache(fathom_gpu, fmt, pages, 2, 128, 64)
    if fmt == "bf16":
        cache.k.fill_(float("nan")), cache.v.fill_(float("inf"))
    else:
        raw = (lambda t: t.view(torch.uint8)) if fmt == "e4m3" else (lambda t: t)
        raw(cache.k).fill_(0x7f), raw(cache.v).fill_(0x7f), cache.k_scale.fill_(255), cache.v_scale.fill_(254)
    fill(fathom_gpu, cache, lens, table)
    q = rand((int(cu[-1]), 8, 128), 4, torch.bfloat16, spread=False)
    out = fathom_gpu.paged_attention(cache, q, table, cu, length, new, 200)
    ref = okv.attend(host(cache), fmt, q.float().cpu().numpy(), table.cpu().numpy(), cu.cpu().numpy(),
                     length.cpu().numpy(), 128 ** -0.5)
    check_attention(out, ref, 200, 128, torch.bfloat16)


@pytest.mark.parametrize("new,G", [(1, 4), (40, 4), (200, 1)])
def test_bounds_smaller_than_the_batch(fathom_gpu, new, G):
    """max_new and max_len below the batch's own: the first max_new rows over the first max_len tokens."""
    lens = [(new + 3, 900), (2, 100)]
    pages, table, cu, length = make_batch(lens, 64)
    cache = make_cache(fathom_gpu, "int8", pages, 1, 128, 64)
    fill(fathom_gpu, cache, lens, table)
    for dt in (torch.bfloat16, torch.float32):
        q = rand((int(cu[-1]), G, 128), 4, dt, spread=False)
        out = torch.full_like(q, 5.0)
        fathom_gpu.paged_attention(cache, q, table, cu, length, new, 500, out=out)
        ref = okv.attend(host(cache), "int8", q.float().cpu().numpy(), table.cpu().numpy(), cu.cpu().numpy(),
                         length.cpu().numpy(), 128 ** -0.5, max_new=new, max_len=500)
        check_attention(out, ref, 500, 128, dt)
        assert (out[torch.tensor(np.isnan(ref[0]), device=DEV)] == 5.0).all()


def test_scores_far_apart(fathom_gpu):
    """Scores of thousands, of one key far above the rest, all equal, and of a negative scale."""
    lens = [(3, 260), (140, 260)]
    pages, table, cu, length = make_batch(lens, 64)
    for fmt in FORMATS:
        cache = make_cache(fathom_gpu, fmt, pages, 1, 128, 64)
        fill(fathom_gpu, cache, lens, table, scale=30.0)
        for dt in (torch.bfloat16, torch.float32):
            q = rand((143, 2, 128), 4, dt, spread=False)
            q[1] = 0
            for scale in (1.0, -0.3, 0.0, 1e-30):
                out = fathom_gpu.paged_attention(cache, q, table, cu, length, 140, 260, scale=scale)
                ref = okv.attend(host(cache), fmt, q.float().cpu().numpy(), table.cpu().numpy(), cu.cpu().numpy(),
                                 length.cpu().numpy(), scale)
                check_attention(out, ref, 260, 128, dt)


def test_query_strides(fathom_gpu):
    """Queries cut out of a fused projection, 16-byte aligned and not."""
    lens = [(5, 80), (90, 91)]
    pages, table, cu, length = make_batch(lens, 16)
    cache = make_cache(fathom_gpu, "e4m3", pages, 2, 64, 16)
    fill(fathom_gpu, cache, lens, table)
    for dt in (torch.bfloat16, torch.float32):
        wide = rand((95, 11, 73), 4, dt, spread=False)
        for cut in (slice(0, 64), slice(3, 67)):
            q = wide[:, 2:8, cut]
            a = fathom_gpu.paged_attention(cache, q, table, cu, length, 90, 91)
            b = fathom_gpu.paged_attention(cache, q.contiguous(), table, cu, length, 90, 91)
            assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("H,G,D,page,n,M", [(2, 4, 128, 64, 700, 300), (3, 8, 64, 16, 90, 100), (1, 1, 32, 32, 40, 1),
                                            (2, 5, 96, 16, 333, 1000), (2, 2, 256, 128, 600, 257), (1, 3, 160, 64, 500, 2049)])
def test_union_attention(fathom_gpu, fmt, H, G, D, page, n, M):
    lens = [(1, n)]
    pages, table, _, _ = make_batch(lens, page)
    cache = make_cache(fathom_gpu, fmt, pages, H, D, page, "token")
    fill(fathom_gpu, cache, lens, table)
    g = torch.Generator().manual_seed(9)
    idx = torch.randint(-3, n + 5, (H, M), generator=g, dtype=torch.int32)   # unsorted, repeated, out of range
    count = torch.tensor([M, M // 2, -6][:H], dtype=torch.int32)
    q = rand((H, G, D), 4, spread=False)
    out = fathom_gpu.paged_union_attention(cache, q, table, n, idx.to(DEV), count.to(DEV))
    ref = okv.union_attend(host(cache), fmt, q.cpu().numpy(), table.cpu().numpy()[0], n, idx.numpy(), count.numpy(), D ** -0.5)
    check_attention(out, ref, M, D, torch.float32)
    zero = fathom_gpu.paged_union_attention(cache, q, table, n, idx.to(DEV), torch.zeros_like(count).to(DEV))
    assert (zero == 0).all()


def test_scan_to_attention_over_the_cache(fathom_gpu):
    """As used: write a prompt in chunks, attend each chunk, read the keys back for the index, plan, scan, top-k, and
    attend over the winners; then a token, with the index's tail packed again from the cache."""
    H, G, D, page, n, k = 2, 4, 128, 64, 1500, 64
    cache = fathom_gpu.KVCache.empty(40, H, D, page, dtype=torch.int8)
    table = torch.randperm(40, generator=torch.Generator().manual_seed(1))[None, :24].to(torch.int32).to(DEV)
    keys, vals = rand((n + 1, H, D), 1, torch.bfloat16, False), rand((n + 1, H, D), 2, torch.bfloat16, False)
    tok_q = rand((1, H * G, D), 3, torch.bfloat16, False)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    for lo, hi in ((0, 700), (700, 1499), (1499, 1500)):
        fathom_gpu.kv_write(cache, keys[lo:hi], vals[lo:hi], table, i32(0, hi - lo), i32(hi))
        q = rand((hi - lo, H * G, D), 10 + lo, torch.bfloat16, False)
        out = fathom_gpu.paged_attention(cache, q, table, i32(0, hi - lo), i32(hi), hi - lo, hi)
        few = torch.arange(0, hi - lo, 97)
        ref = okv.attend(host(cache), "int8", q.float().cpu().numpy(), table.cpu().numpy(), [0, hi - lo], [hi], D ** -0.5)
        check_attention(out[few], tuple(x[few.numpy()] for x in ref), hi, D, torch.bfloat16)
    kr, vr = fathom_gpu.kv_read(cache, table, i32(0, n), i32(n), n)
    planes, scales = fathom_gpu.pack(kr, nb_stride_words=32)
    _, s2, _ = fathom_gpu.calibrate(kr)
    # one token more: written, and the index's last block packed again from what the cache holds
    fathom_gpu.kv_write(cache, keys[n:], vals[n:], table, i32(0, 1), i32(n + 1))
    b0 = n // 64
    tail = n + 1 - 64 * b0
    kt, _ = fathom_gpu.kv_read(cache, table, i32(0, tail), i32(n + 1), tail)
    fathom_gpu.pack_range(kt, planes, scales, b0)
    kall, vall = fathom_gpu.kv_read(cache, table, i32(0, n + 1), i32(n + 1), n + 1)
    whole = fathom_gpu.pack(kall, nb_stride_words=32)
    assert torch.equal(planes, whole[0]) and torch.equal(scales, whole[1])
    qf = tok_q.view(H, G, D).float()
    step = fathom_gpu.Step(planes, scales, n + 1, s2, G, k)
    _, uni, cnt = step.run(qf)
    got = fathom_gpu.paged_union_attention(cache, qf, table, n + 1, uni, cnt)
    ref = okv.union_attend(host(cache), "int8", qf.cpu().numpy(), table.cpu().numpy()[0], n + 1, uni.cpu().numpy(),
                           cnt.cpu().numpy(), D ** -0.5)
    check_attention(got, ref, uni.shape[1], D, torch.float32)
    # the same rows through the dense cache: the two attend alike within their rounding
    dense = fathom_gpu.union_attention(kall, vall, qf, uni, cnt)
    check_attention(dense, ref, uni.shape[1], D, torch.float32)


@pytest.mark.parametrize("new", [1, 100])
def test_captured_replayed_and_on_another_stream(fathom_gpu, new):
    lens = [(new, 3000), (1, 400)]
    pages, table, cu, length = make_batch(lens, 64)
    cache = make_cache(fathom_gpu, "int8", pages, 2, 128, 64)
    fill(fathom_gpu, cache, lens, table)
    q = rand((int(cu[-1]), 8, 128), 4, torch.bfloat16, spread=False)
    k, v = rand((int(cu[-1]), 2, 128), 5, torch.bfloat16), rand((int(cu[-1]), 2, 128), 6, torch.bfloat16)
    out = torch.empty_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        fathom_gpu.kv_write(cache, k, v, table, cu, length)
        fathom_gpu.paged_attention(cache, q, table, cu, length, new, 3000, out=out)
        with torch.cuda.graph(graph, stream=s):
            fathom_gpu.kv_write(cache, k, v, table, cu, length)
            fathom_gpu.paged_attention(cache, q, table, cu, length, new, 3000, out=out)
    for seed, at in ((20, 2500), (21, 2999)):
        k.copy_(rand(k.shape, seed, torch.bfloat16))
        q.copy_(rand(q.shape, seed + 5, torch.bfloat16, False))
        length[0] = at   # another length on each replay
        graph.replay()
        torch.cuda.synchronize()
        want = fathom_gpu.paged_attention(cache, q, table, cu, length, new, 3000)
        assert torch.equal(out, want)
        ref = okv.attend(host(cache), "int8", q.float().cpu().numpy(), table.cpu().numpy(), cu.cpu().numpy(),
                         length.cpu().numpy(), 128 ** -0.5)
        check_attention(out, ref, 3000, 128, torch.bfloat16)


def test_two_calls_at_once(fathom_gpu):
    """The same batch on two streams, each call with its own workspace, many times over: the results of one call."""
    lens = [(1, 9000), (1, 5000)]
    pages, table, cu, length = make_batch(lens, 64)
    cache = make_cache(fathom_gpu, "int8", pages, 2, 128, 64)
    fill(fathom_gpu, cache, lens, table)
    qs = [rand((2, 8, 128), 4 + i, torch.bfloat16, False) for i in range(2)]
    want = [fathom_gpu.paged_attention(cache, q, table, cu, length, 1, 9000) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(fathom_gpu.paged_attention(cache, qs[i], table, cu, length, 1, 9000))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[i]) for i in range(2) for x in got[i])


def test_offsets_past_32_bits(fathom_gpu):
    """A cache whose last pages lie beyond 2^31 elements (the pool is touched only where a token is written)."""
    H, D, page = 8, 128, 256
    pages = 9000                                     # 9000 x 8 x 256 x 128 = 2.36e9 elements
    k, v = (torch.empty((pages, H, page, D), dtype=torch.int8, device=DEV) for _ in range(2))
    s = [torch.empty((pages, H, page, D // 32), dtype=torch.uint8, device=DEV) for _ in range(2)]
    cache = fathom_gpu.KVCache(k, v, *s)
    lens = [(3, 300), (150, 400)]
    table = torch.tensor([[8999, 8997], [8998, 8996]], dtype=torch.int32, device=DEV)
    cu, length = torch.tensor([0, 3, 153], dtype=torch.int32, device=DEV), torch.tensor([300, 400], dtype=torch.int32, device=DEV)
    fill(fathom_gpu, cache, lens, table)
    small = fathom_gpu.KVCache(k[8996:].clone(), v[8996:].clone(), s[0][8996:].clone(), s[1][8996:].clone())
    q = rand((153, H, D), 4, torch.bfloat16, spread=False)
    a = fathom_gpu.paged_attention(cache, q, table, cu, length, 150, 400)
    b = fathom_gpu.paged_attention(small, q, table - 8996, cu, length, 150, 400)
    assert torch.equal(a, b)
    ref = okv.attend(host(small), "int8", q.float().cpu().numpy(), (table - 8996).cpu().numpy(), cu.cpu().numpy(),
                     length.cpu().numpy(), D ** -0.5)
    check_attention(b, ref, 400, D, torch.bfloat16)
    kr = fathom_gpu.kv_read(cache, table, cu, length, 153)
    assert all(torch.equal(x, y) for x, y in zip(kr, fathom_gpu.kv_read(small, table - 8996, cu, length, 153)))


def test_refusals_on_the_device(fathom_gpu):
    lens = [(2, 100)]
    pages, table, cu, length = make_batch(lens, 64)
    cache = make_cache(fathom_gpu, "int8", pages, 2, 128, 64)
    q = rand((2, 8, 128), 4, torch.bfloat16, False)
    with pytest.raises(ValueError):
        fathom_gpu.paged_attention(cache, q.cpu(), table, cu, length, 2, 100)
    with pytest.raises(ValueError):
        fathom_gpu.paged_attention(cache, q, table, cu, length, 2, 100, out=torch.empty_like(q.float()))
    big = fathom_gpu.KVCache.empty(64, 2, 128, 64)
    need = fathom_gpu.paged_attention_workspace_bytes(2, 4, 128, 2, 1, 2, 4096)
    if need:
        with pytest.raises(fathom_gpu.FathomError, match="too small"):
            fathom_gpu.paged_attention(big, q, table, cu, length, 2, 4096, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    host_q = torch.zeros(2, 8, 128)   # pageable host memory: refused by the library itself
    st = fathom_gpu.lib().fathom_paged_attention(
        cache._ref, fathom_gpu._kv_rows(cache, table, cu, length, 2), ctypes.c_void_p(host_q.data_ptr()), 0, 8 * 128, 128, 4, 2,
        100, 1, 0.1, q.data_ptr(), torch.empty(1 << 24, dtype=torch.uint8, device=DEV).data_ptr(), 1 << 24, None)
    assert st == fathom_gpu.ERR_INVALID_ARG
