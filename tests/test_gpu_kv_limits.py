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
