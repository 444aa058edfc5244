"""Shared by the tests of the paged KV cache: caches in several layouts, ragged batches, tolerances."""
import numpy as np
import torch

from oracle import kv as okv

FORMATS = {"bf16": torch.bfloat16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def host(cache):
    """A KVCache as the oracle's numpy cache."""
    def bits(t):
        if t is None:
            return None
        if t.dtype == torch.bfloat16:
            return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
        if t.dtype == torch.float8_e4m3fn:
            return t.view(torch.uint8).contiguous().cpu().numpy()
        return t.contiguous().cpu().numpy()
    return [bits(cache.k), bits(cache.v), bits(cache.k_scale), bits(cache.v_scale)]


def make_cache(fathom, fmt, pages, H, D, page_tokens, layout="head", device="cuda"):
    """A zeroed cache: pages of [H][tokens][D] ("head"), of [tokens][H][D] ("token"), or
    the second of three layers of one tensor ("layer")."""
    dt = FORMATS[fmt]
    raw = torch.uint8 if fmt == "e4m3" else dt

    def one(width, dtype, view):
        if layout == "head":
            return torch.zeros(pages, H, page_tokens, width, dtype=dtype, device=device).view(view)
        if layout == "token":
            return torch.zeros(pages, page_tokens, H, width, dtype=dtype, device=device).view(view).transpose(1, 2)
        return torch.zeros(pages, 3, H, page_tokens, width, dtype=dtype, device=device).view(view)[:, 1]
    data = [one(D, raw, dt) for _ in range(2)]
    scales = [None, None] if fmt == "bf16" else [one(D // okv.BLOCK, torch.uint8, torch.uint8) for _ in range(2)]
    return fathom.KVCache(*data, *scales)


def make_batch(lens, page_tokens, spare=2, seed=0, device="cuda"):
    """Page table, cu and length of sequences [(new, total)], pages in random order; unused entries are -1."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-max(total, 0) // page_tokens) for _, total in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    cu = torch.tensor(np.cumsum([0] + [n for n, _ in lens]), dtype=torch.int32)
    length = torch.tensor([t for _, t in lens], dtype=torch.int32)
    return pages, table.to(device), cu.to(device), length.to(device)


def fill(fathom, cache, lens, table, seed=0, dtype=torch.float32, scale=1.0):
    """Write every token of every sequence, random rows."""
    dev = cache.k.device
    g = torch.Generator(device=dev).manual_seed(seed)
    cu = torch.tensor(np.cumsum([0] + [max(t, 0) for _, t in lens]), dtype=torch.int32, device=dev)
    length = torch.tensor([max(t, 0) for _, t in lens], dtype=torch.int32, device=dev)
    total = int(cu[-1])
    k, v = (scale * torch.randn(total, cache.H, cache.D, generator=g, device=dev) for _ in range(2))
    if total:
        fathom.kv_write(cache, k.to(dtype), v.to(dtype), table, cu, length)
    return k, v


def tolerance(ref, mag, l1, keys, D, dtype):
    """Bound of |out - ref|.  A score is a sum of D products, at most three bf16 parts of each, in matrix steps of 16:
    at most 3 D/16 + 4 roundings of 2^-23 of its partial sums, so it is off by ds = (3 D/16 + 4) 2^-23 l1 and a weight
    by 2 ds relatively (numerator and denominator; exp adds 2 ulp to each).  The value sum adds keys/16 + 64 such
    roundings (steps of 16 keys, partial results joined) of sums no larger than mag = sum |p v|.  bf16 queries: the
    weights enter the value product in bf16 at worst (half a step: 2^-8), and the output is rounded to bf16."""
    ds = (3 * D / 16 + 4) * 2.0 ** -23 * l1[..., None]
    tol = mag * (2 * ds + 2.0 ** -20 + (keys / 16 + 64) * 2.0 ** -23) + 1e-30
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (mag + np.abs(ref))
    return tol


def check_attention(out, want, keys, D, dtype):
    ref, mag, l1 = want
    got = out.float().cpu().numpy().astype(np.float64)
    live = ~np.isnan(ref)
    err, tol = np.abs(got - ref), tolerance(ref, mag, l1, keys, D, dtype)
    bad = live & ~(err <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{int(bad.sum())} of {int(live.sum())} values out of tolerance; first at {i}: "
                             f"got {got[i]!r}, want {ref[i]!r}, error {err[i]:.3g} > {tol[i]:.3g}")
