"""A call that is given a stream: what it allocates belongs to that stream.  The allocator hands a block out again at
once to the stream it belongs to, since the order of that stream's work protects it; a block of another stream may still
be in use by work queued there."""
import contextlib
import inspect

import pytest
import torch

from long_context_decode_bit_b200 import fathom


class _Library:
    """Every entry point of the library, doing nothing; sizes are 4096."""

    def __getattr__(self, name):
        return lambda *args: 4096 if name.endswith("_bytes") else 4 if name == "fathom_nb_stride" else 0


def _calls():
    """Each function that takes a stream, with arguments that make it allocate whatever it can."""
    f32, i32 = (lambda *s: torch.zeros(s)), (lambda *s: torch.zeros(s, dtype=torch.int32))
    H, G, D, n, k, M = 2, 4, 64, 100, 8, 32
    keys, q = f32(H, n, D), f32(H, G, D)
    planes, scales = torch.zeros(H, D, 4, 4, dtype=torch.int64), torch.zeros(H, D, 4, dtype=torch.int16)
    active, count = torch.zeros(H, D, dtype=torch.int16), i32(H)
    codes, exps = torch.zeros(3, H, 64, D, dtype=torch.int8), torch.zeros(3, H, 64, 2, dtype=torch.uint8)
    cache = fathom.KVCache(codes, codes.clone(), exps, exps.clone())
    table, cu, length = i32(1, 2), torch.tensor([0, 5], dtype=torch.int32), torch.tensor([100], dtype=torch.int32)
    rows = f32(5, H, D)
    return {
        "pack": (keys,), "pack_rotated": (keys, f32(H, D, D)), "pack_range": (keys[:, :64], planes, scales, 0),
        "plan": (f32(H, D), q, 48), "plan_fixed": (q, 16), "layer_budgets": (f32(H, D), q, 1, 100),
        "scan": (planes, scales, n, active, count, q, fathom.SCAN_CANDIDATE, k),
        "nibbles_from_planes": (planes, n), "nibbles_tm_from_planes": (planes, n),
        "topk": (H, G, n, k, f32(H, G, n)), "dequant_rows": (planes, scales, n, i32(H, M)),
        "scan_topk_noalloc": (planes, scales, n, active, count, q, k), "calibrate": (keys, n, True, True),
        "union_attention": (keys, keys, q, i32(H, M), count),
        "kv_write": (cache, rows, rows.clone(), table, cu, length), "kv_read": (cache, table, cu, length, 5),
        "paged_attention": (cache, f32(5, H * G, D), table, cu, length, 5, 100),
        "paged_union_attention": (cache, q, table, n, i32(H, M), count),
        "device_status": (),
    }


def test_every_function_with_a_stream_is_listed():
    takes = {name for name, f in vars(fathom).items() if inspect.isfunction(f) and not name.startswith("_")
             and "stream" in inspect.signature(f).parameters}
    assert takes == set(_calls())


@pytest.mark.parametrize("name", sorted(_calls()))
def test_allocations_belong_to_the_stream(monkeypatch, name):
    class Stream:
        cuda_stream = 0x5000
    stream, current, made, kept = Stream(), ["the caller's"], [], []

    @contextlib.contextmanager
    def on(s):
        current.append(s)
        yield
        current.pop()
    args = _calls()[name]
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current[-1])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: kept.append((t.data_ptr(), s)))
    for where, what in ((torch, "empty"), (torch, "zeros"), (torch, "empty_like"), (torch, "empty_strided"),
                        (torch.Tensor, "new_empty")):
        def spy(*a, _make=getattr(where, what), **kw):
            t = _make(*a, **kw)
            made.append((t, current[-1]))
            return t
        monkeypatch.setattr(where, what, spy)
    monkeypatch.setattr(fathom, "lib", _Library)
    monkeypatch.setattr(fathom, "_kv_here", lambda *a: None)
    monkeypatch.setattr(fathom, "_paged_workspace", lambda *a: 4096)
    monkeypatch.setattr(fathom, "_union_workspace", lambda *a: 4096)
    out = getattr(fathom, name)(*args, stream=stream)
    assert all(where is stream for _, where in made)
    # what is handed to the caller stays until the caller's own stream is done with it
    got = {t.data_ptr() for t in (out if isinstance(out, tuple) else (out,)) if isinstance(t, torch.Tensor)}
    for t, _ in made:
        assert t.data_ptr() not in got or (t.data_ptr(), "the caller's") in kept
    assert current == ["the caller's"]


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["pack", "union_attention", "kv_read", "paged_attention", "paged_union_attention"])
def test_blocks_in_use_on_the_callers_stream_are_left_alone(fathom_gpu, name):
    """Work queued on the caller's stream still writes to tensors freed there when a call is made on another stream:
    the call's results and its scratch are elsewhere."""
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    H, G, D, n, M = 2, 4, 128, 9000, 1024
    keys, vals, q = rand(H, n, D).bfloat16(), rand(H, n, D).bfloat16(), rand(H, G, D)
    cache = fathom_gpu.KVCache.empty(150, H, D, 64, device=dev)
    table = torch.randperm(150, generator=torch.Generator().manual_seed(2))[None, :141].to(torch.int32).to(dev)
    fathom_gpu.kv_write(cache, keys.transpose(0, 1), vals.transpose(0, 1), table, i32(0, n), i32(n))
    uni = torch.randint(0, n, (H, M), generator=g, device=dev).sort(1).values.to(torch.int32)
    cnt = i32(M, 700)
    call = {"pack": lambda **kw: fathom_gpu.pack(keys, **kw),
            "union_attention": lambda **kw: fathom_gpu.union_attention(keys, vals, q, uni, cnt, **kw),
            "kv_read": lambda **kw: fathom_gpu.kv_read(cache, table, i32_0n, i32_n, n, **kw),
            "paged_attention": lambda **kw: fathom_gpu.paged_attention(cache, token, table, i32_01, i32_n, 1, n, **kw),
            "paged_union_attention": lambda **kw: fathom_gpu.paged_union_attention(cache, q, table, n, uni, cnt, **kw)}[name]
    i32_0n, i32_01, i32_n, token = i32(0, n), i32(0, 1), i32(n), q.view(1, H * G, D).bfloat16()
    tuple_of = lambda x: x if isinstance(x, tuple) else (x,)  # noqa: E731
    want = [t.clone() for t in tuple_of(call())]
    sizes = [t.numel() * t.element_size() for t in want] + \
        [fathom_gpu.paged_attention_workspace_bytes(H, G, D, 1, 1, 1, n), 1 << 16, 1 << 20]
    big, side = rand(4096, 4096), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(30):          # some tens of milliseconds
        big @ big
    for size in 4 * sizes:       # and behind them, writes to blocks that are free again as soon as they are queued
        torch.empty(max(size, 1), dtype=torch.uint8, device=dev).fill_(0x7f)
    got = tuple_of(call(stream=side))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_current_stream_by_torchs_public_api(monkeypatch):
    """The current stream is found without the short way that torch offers itself, too."""
    import importlib.util
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    spec = importlib.util.spec_from_file_location("fathom_again", fathom.__file__, submodule_search_locations=None)
    again = importlib.util.module_from_spec(spec)
    again.__package__ = fathom.__package__
    spec.loader.exec_module(again)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: type("S", (), {"cuda_stream": 0x7000 + dev}))
    assert again._stream(None) == 0x7003
