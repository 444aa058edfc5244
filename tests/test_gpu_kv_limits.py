"""The paged KV cache and its attention at the ends of the number formats, against the 64-bit oracle."""
import numpy as np
import pytest
import torch

from oracle import kv as okv
from _kv import check_attention, host, make_batch, make_cache

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("new", [1, 10, 100])
@pytest.mark.parametrize("fmt", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("D", [64, 96, 128, 256])
def test_largest_fp32_queries(fathom_gpu, fmt, D, new):
    """fp32 queries of 3.4e38, which round to an infinity in bf16, against keys small enough for finite scores."""
    lens = [(new, 300)]
    pages, table, cu, length = make_batch(lens, 64)
    cache = make_cache(fathom_gpu, fmt, pages, 1, D, 64)
    g = torch.Generator(device=DEV).manual_seed(D)
    rand = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    k = rand(300, 1, D)
    k[..., :32] *= 2.0 ** -95
    fathom_gpu.kv_write(cache, k, rand(300, 1, D), table, torch.tensor([0, 300], dtype=torch.int32, device=DEV), length)
    q = rand(new, 4, D)
    q[..., :32] = torch.where(q[..., :32] > 0, 3.4e38, -3.4e38)
    q[:, 1, :32] = torch.finfo(torch.float32).max
    scale = 2.0 ** -34
    out = fathom_gpu.paged_attention(cache, q, table, cu, length, new, 300, scale=scale)
    ref = okv.attend(host(cache), fmt, q.cpu().numpy(), table.cpu().numpy(), cu.cpu().numpy(), length.cpu().numpy(), scale)
    check_attention(out, ref, 300, D, torch.float32)
    idx = torch.arange(300, dtype=torch.int32, device=DEV)[None]
    got = fathom_gpu.paged_union_attention(cache, q[-1:].contiguous(), table, 300, idx, torch.tensor([300], dtype=torch.int32, device=DEV),
                                           scale=scale)
    check_attention(got, tuple(x[-1:] for x in ref), 300, D, torch.float32)


def bf16_of(x):
    """Nearest bf16 value of fp32 values in 64 bits, ties to even (beyond the largest: infinity), NaN as NaN."""
    with np.errstate(all="ignore"):
        a = np.abs(x.astype(np.float64))
        step = np.exp2(np.maximum(np.floor(np.log2(np.where((a > 0) & np.isfinite(a), a, 1.0))), -126) - 7)
        y = np.where(np.isfinite(a), np.rint(a / step) * step, a)
    return np.copysign(np.where(y >= 2.0 ** 128, np.inf, y), x)


@pytest.mark.parametrize("shift", [0, 1])   # rows on 16 bytes, and not
def test_bf16_pages_keep_infinities_and_nan(fathom_gpu, shift):
    """What a bf16 cache holds of infinities, NaN, values around the largest and the least, and ties; the channels beside
    them are as they were."""
    f = np.float32
    ends = np.array([np.inf, -np.inf, np.nan, 3.3895314e38, 3.39615e38, np.nextafter(f(3.3961775e38), f(0)), 3.3961775e38, 3.4028235e38,
                     -3.4028235e38, 1e-45, -1e-45, 9.2e-41, 4.6e-41, 1.1754944e-38, 1.1754942e-38, 0.0, -0.0, 1.00390625,
                     1.01171875, -1.00390625], f)
    x = np.random.default_rng(3).standard_normal((len(ends) + 3, 2, 64)).astype(f)
    for i, e in enumerate(ends):
        x[i, 0, (7 * i) % 64] = e
        x[i, 1, (11 * i + 5) % 64] = e
    n = len(x)
    pages, table, cu, length = make_batch([(n, n)], 16)
    args = table.cpu().numpy(), cu.cpu().numpy(), length.cpu().numpy()
    for dtype in (torch.float32, torch.bfloat16):
        cache = make_cache(fathom_gpu, "bf16", pages, 2, 64, 16)
        wide = torch.zeros(n, 2, 64 + 8, device=DEV, dtype=dtype)
        rows = wide[..., shift:shift + 64]
        rows.copy_(torch.tensor(x))
        fathom_gpu.kv_write(cache, rows, rows, table, cu, length)
        want = bf16_of(x).transpose(1, 0, 2)
        for got in okv.read(host(cache), "bf16", *args, n):
            assert np.array_equal(got, want, equal_nan=True)
        for out in (torch.float32, torch.bfloat16):
            for got in fathom_gpu.kv_read(cache, table, cu, length, n, dtype=out):
                assert np.array_equal(got.float().cpu().numpy().astype(np.float64), want, equal_nan=True)


@pytest.mark.parametrize("new", [1, 60])
def test_infinities_in_bf16_pages(fathom_gpu, new):
    """A value that is infinite makes its channel of the rows that see it infinite (or NaN, of fp32 queries), and NaN where
    there is one of the other sign; a key that is infinite makes them NaN (its score and the largest one are).  Rows of other sequences stay."""
    lens = [(new, new + 20), (new, new + 20), (new, 90)]
    pages, table, cu, length = make_batch(lens, 16)
    g = torch.Generator(device=DEV).manual_seed(1)
    n = sum(t for _, t in lens)
    k, v = (torch.randn((n, 1, 64), generator=g, device=DEV) for _ in range(2))
    v[3, 0, 5], v[4, 0, 6], v[5, 0, 6] = np.inf, np.inf, -np.inf        # sequence 0
    k[new + 20 + 2] = np.inf                                             # sequence 1
    cache = make_cache(fathom_gpu, "bf16", pages, 1, 64, 16)
    everything = torch.tensor([0, new + 20, 2 * new + 40, n], dtype=torch.int32, device=DEV)
    fathom_gpu.kv_write(cache, k, v, table, everything, length)
    for dt in (torch.float32, torch.bfloat16):
        q = torch.randn((3 * new, 4, 64), generator=g, device=DEV).abs().to(dt)   # that key's score is infinite
        out = fathom_gpu.paged_attention(cache, q, table, cu, length, new, 90).float()
        first = out[:new]
        # Of fp32 queries a weight is three parts, and where it has no more than 16 bits the last is 0: 0 * inf is NaN.
        assert ((first[..., 5] == np.inf) | (first[..., 5].isnan() & (dt == torch.float32))).all()
        assert first[..., 6].isnan().all()
        rest = torch.ones(64, dtype=torch.bool, device=DEV)
        rest[5:7] = False
        assert first[..., rest].isfinite().all()
        assert out[new:2 * new].isnan().all() and out[2 * new:].isfinite().all()


@pytest.mark.parametrize("new", [1, 60])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_scores_up_to_where_they_overflow(fathom_gpu, dtype, new):
    """The largest scale: the one key with a score of 2.2e38 is the row's answer, one of 2.4e38 makes it NaN, one of -2.4e38
    takes no part."""
    D, n = 64, 80
    lens = [(new, n)]
    pages, table, cu, length = make_batch(lens, 16)
    g = torch.Generator(device=DEV).manual_seed(1)
    everything = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    q = torch.zeros((new, 2, D), device=DEV, dtype=dtype)
    q[..., 0] = 1.0
    for top in (2.203125, 2.40625, -2.40625):      # bf16 values
        k, v = torch.zeros((n, 1, D), device=DEV), torch.randn((n, 1, D), generator=g, device=DEV).bfloat16().float()
        k[7, 0, 0] = top
        cache = make_cache(fathom_gpu, "bf16", pages, 1, D, 16)
        fathom_gpu.kv_write(cache, k, v, table, everything, length)
        out = fathom_gpu.paged_attention(cache, q, table, cu, length, new, n, causal=False, scale=1e38).double()
        if top > 2.3:
            assert out.isnan().all()
        elif top > 0:
            assert torch.equal(out, v[7].double().expand_as(out))
        else:
            rest = torch.cat([v[:7], v[8:]]).double().mean(0)
            assert ((out - rest).abs() <= rest.abs() * 2.0 ** -8 + 2.0 ** -8).all()   # weights of 1, 79 of them; output in bf16


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("new", [1, 10, 100])
@pytest.mark.parametrize("fmt,D", [("bf16", 64), ("int8", 128), ("e4m3", 96), ("bf16", 256), ("int8", 160)])
def test_scores_whose_steps_are_large(fathom_gpu, fmt, D, new, dtype):
    """Scores so large that fp32 holds them in steps of 2 and more: the largest one's value is the answer, two that are equal
    share it, and causal rows over scores that grow from token to token have their own token's value."""
    n = 400
    lens = [(new, n)]
    pages, table, cu, length = make_batch(lens, 64)
    g = torch.Generator(device=DEV).manual_seed(D)
    everything = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    base = torch.where(torch.rand(D, generator=g, device=DEV) < 0.5, -1.0, 1.0)      # q . k = D times the keys' factor
    v = torch.randint(-7, 8, (n, 1, D), generator=g, device=DEV).float()             # values that every format holds
    q = (base * torch.tensor([1.0, 0.5, 2.0], device=DEV)[:, None]).expand(new, 3, D).contiguous().to(dtype)
    two = torch.full((n,), 0.5, device=DEV)
    two[7] = two[251] = 1.75
    at = torch.arange(n, device=DEV)
    grow = 2.0 ** (at // 8 - 35).float() * (1 + at % 8 / 8)   # 4 bits each, up to 30720 (E4M3 ends at 57344)
    scales = (2.0 ** 20, 2.0 ** 23, 2.0 ** 26, 1.37e9, 2.0 ** 40, -2.0 ** 30)
    for factor, causal, want, more in ((two, False, (v[7] + v[251]) / 2, (1.37e20, 2.0 ** 100, -2.0 ** 110)),
                                       (grow, True, v[n - new:], ())):
        cache = make_cache(fathom_gpu, fmt, pages, 1, D, 64)
        fathom_gpu.kv_write(cache, (factor[:, None, None] * base).contiguous(), v, table, everything, length)
        for scale in scales + more:
            out = fathom_gpu.paged_attention(cache, q if scale > 0 else -q, table, cu, length, new, n, causal=causal, scale=scale)
            assert torch.equal(out.float(), want.expand(new, 3, D)), (scale, causal)


@pytest.mark.parametrize("new", [1, 64])
def test_long_sums_of_fp32_queries(fathom_gpu, new):
    """A million tokens whose values are all the same: that value, within the roundings to nearest of a stretch's sums.  The
    weights and the values go into sums of their own, each with a rounding of at most 2^-24 for every 16-token tile of a
    warp (a quarter of a stretch), then for every stretch and warp that is joined; 64 for a tile's own sum, the weights'
    exponentials and the division."""
    H, G, D, page, n = 8, 4, 128, 256, 1 << 20
    g = torch.Generator(device=DEV).manual_seed(1)
    k = torch.randint(-60, 61, (n // page, H, page, D), generator=g, dtype=torch.int8, device=DEV)
    exps = [torch.full((n // page, H, page, D // 32), 127 - e, dtype=torch.uint8, device=DEV) for e in (5, 6)]
    cache = fathom_gpu.KVCache(k, torch.full_like(k, 93), *exps)
    table = torch.arange(n // page, dtype=torch.int32, device=DEV)[None]
    q = torch.randn((new, H * G, D), generator=g, device=DEV)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    out = fathom_gpu.paged_attention(cache, q, table, i32(0, new), i32(n), new, n, causal=False)
    scratch = fathom_gpu.paged_attention_workspace_bytes(H, G, D, new, 1, new, n, torch.float32)
    stretches = scratch // (new * H * G * (4 * D + 8))
    tiles = -(-n // stretches // 64)
    bound = (2 * tiles + 2 * (-(-stretches // 16) + 16) + 64) * 2.0 ** -24
    assert ((out.double() / (93 / 64) - 1).abs() <= bound).all()
