"""The paged KV cache's entry points refuse what they cannot do before anything reaches a GPU (none is needed here)."""
import ctypes

import pytest
import torch

from long_context_decode_bit_b200 import build, fathom


@pytest.fixture(scope="module")
def lib():
    build.build()
    return fathom.load()


FAKE = 4096   # an aligned address that is never dereferenced


def cache(**kw):
    f = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, pages=8, page_stride=8 * 64 * 128, head_stride=64 * 128,
             token_stride=128, scale_page_stride=8 * 64 * 4, scale_head_stride=64 * 4, scale_token_stride=4, H=8, D=128,
             page_tokens=64, format=fathom.KV_INT8)
    f.update(kw)
    return ctypes.byref(fathom._KvCacheStruct(**f))


def rows(**kw):
    f = dict(table=FAKE, cu=FAKE, length=FAKE, table_stride=4, rows=10, table_pages=4, B=2)
    f.update(kw)
    return ctypes.byref(fathom._KvRowsStruct(**f))


BAD_CACHES = [(dict(format=3), fathom.ERR_INVALID_ARG), (dict(format=-1), fathom.ERR_INVALID_ARG),
              (dict(H=-1), fathom.ERR_INVALID_ARG), (dict(pages=-1), fathom.ERR_INVALID_ARG),
              (dict(pages=1 << 31), fathom.ERR_INVALID_ARG), (dict(D=48), fathom.ERR_UNSUPPORTED),
              (dict(D=288), fathom.ERR_UNSUPPORTED), (dict(H=65536), fathom.ERR_UNSUPPORTED),
              (dict(page_tokens=8), fathom.ERR_UNSUPPORTED), (dict(page_tokens=48), fathom.ERR_UNSUPPORTED),
              (dict(page_tokens=512), fathom.ERR_UNSUPPORTED), (dict(token_stride=127), fathom.ERR_INVALID_ARG),
              (dict(page_stride=-16), fathom.ERR_INVALID_ARG), (dict(scale_token_stride=3), fathom.ERR_INVALID_ARG),
              (dict(k=FAKE + 8), fathom.ERR_UNSUPPORTED), (dict(token_stride=136), fathom.ERR_UNSUPPORTED),
              (dict(scale_token_stride=5), fathom.ERR_UNSUPPORTED), (dict(v_scale=FAKE + 2), fathom.ERR_UNSUPPORTED),
              (dict(k=None), fathom.ERR_INVALID_ARG)]
BAD_ROWS = [(dict(B=-1), fathom.ERR_INVALID_ARG), (dict(B=65536), fathom.ERR_INVALID_ARG),
            (dict(rows=-1), fathom.ERR_INVALID_ARG), (dict(rows=1 << 31), fathom.ERR_INVALID_ARG),
            (dict(table_pages=-1), fathom.ERR_INVALID_ARG)]


def calls(lib, c, w):
    big = 1 << 40
    yield lib.fathom_kv_write(c, w, FAKE, FAKE, 1, 1024, 128, None)
    yield lib.fathom_kv_read(c, w, FAKE, FAKE, 1, 10 * 128, 128, None)
    yield lib.fathom_paged_attention(c, w, FAKE, 1, 4096, 128, 4, 5, 256, 1, 0.1, FAKE, FAKE, big, None)


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches(lib, kw, status):
    if kw.get("D") == 48:
        kw = dict(kw, token_stride=128)
    assert set(calls(lib, cache(**kw), rows())) == {status}
    assert lib.fathom_paged_union_attention(cache(**kw), FAKE, 4, 200, FAKE, 4, FAKE, FAKE, 512, 0.1, FAKE, FAKE, 1 << 40,
                                            None) == status


@pytest.mark.parametrize("kw,status", BAD_ROWS)
def test_bad_rows(lib, kw, status):
    assert set(calls(lib, cache(), rows(**kw))) == {status}


def test_no_structs(lib):
    assert set(calls(lib, None, rows())) == {fathom.ERR_INVALID_ARG}
    assert set(calls(lib, cache(), None)) == {fathom.ERR_INVALID_ARG}


def test_nothing_to_do(lib):
    for c, w in ((cache(H=0), rows()), (cache(), rows(B=0)), (cache(), rows(rows=0))):
        assert set(calls(lib, c, w)) == {fathom.OK}


def test_bad_arguments(lib):
    c, w = cache(), rows()
    assert lib.fathom_kv_write(c, w, FAKE, FAKE, 2, 1024, 128, None) == fathom.ERR_INVALID_ARG      # no such type
    assert lib.fathom_kv_write(c, w, FAKE, FAKE, 1, -1, 128, None) == fathom.ERR_INVALID_ARG
    assert lib.fathom_kv_write(c, w, FAKE + 1, FAKE, 1, 1024, 128, None) == fathom.ERR_UNSUPPORTED
    assert lib.fathom_kv_read(c, w, FAKE, FAKE, 1, 9 * 128, 128, None) == fathom.ERR_INVALID_ARG    # rows overlap
    assert lib.fathom_kv_read(c, w, FAKE, FAKE, 1, 128, 7 * 128, None) == fathom.ERR_INVALID_ARG
    assert lib.fathom_kv_read(c, w, None, None, 1, 10 * 128, 128, None) == fathom.ERR_INVALID_ARG   # nothing wanted

    def attend(q_dtype=1, G=4, max_new=5, max_len=256, scale=0.1, q=FAKE, out=FAKE, ws=FAKE, ws_bytes=1 << 40):
        return lib.fathom_paged_attention(c, w, q, q_dtype, 4096, 128, G, max_new, max_len, 1, scale, out, ws, ws_bytes, None)
    assert attend(q_dtype=2) == fathom.ERR_INVALID_ARG
    assert attend(G=0) == fathom.ERR_UNSUPPORTED and attend(G=9) == fathom.ERR_UNSUPPORTED
    assert attend(max_new=-1) == fathom.ERR_INVALID_ARG and attend(max_len=-1) == fathom.ERR_INVALID_ARG
    assert attend(max_new=0) == fathom.OK
    assert attend(scale=float("nan")) == fathom.ERR_INVALID_ARG
    assert attend(scale=float("inf")) == fathom.ERR_INVALID_ARG
    assert attend(q=FAKE + 1) == fathom.ERR_UNSUPPORTED and attend(q_dtype=0, out=FAKE + 2) == fathom.ERR_UNSUPPORTED

    def union(G=4, n=200, M=512, scale=0.1, table_pages=4, q=FAKE):
        return lib.fathom_paged_union_attention(c, FAKE, table_pages, n, q, G, FAKE, FAKE, M, scale, FAKE, FAKE, 1 << 40, None)
    assert union(G=9) == fathom.ERR_UNSUPPORTED
    for kw in (dict(n=-1), dict(n=1 << 31), dict(M=0), dict(M=65537), dict(scale=float("nan")), dict(table_pages=-1)):
        assert union(**kw) == fathom.ERR_INVALID_ARG
    assert union(q=FAKE + 2) == fathom.ERR_UNSUPPORTED


def test_workspace_sizes(lib):
    ws = lib.fathom_paged_attention_workspace_bytes
    assert ws(8, 9, 128, 10, 1, 10, 100, 1) == 0 and ws(8, 4, 100, 10, 1, 10, 100, 1) == 0
    assert ws(8, 4, 128, 0, 1, 10, 100, 1) == 0 and ws(8, 4, 128, 10, 1, 10, 100, 7) == 0
    # a bound on a sequence's rows above the rows there are asks for no more
    assert ws(8, 4, 128, 10, 1, 1000, 131072, 1) == ws(8, 4, 128, 10, 1, 10, 131072, 1)
    assert lib.fathom_paged_union_attention_workspace_bytes(1, 4, 128, 0) == 0
    assert lib.fathom_paged_union_attention_workspace_bytes(1, 9, 128, 64) == 0


def test_small_workspace(lib):
    need = lib.fathom_paged_attention_workspace_bytes(8, 4, 128, 2, 2, 1, 131072, 1)
    if need:
        assert lib.fathom_paged_attention(cache(), rows(rows=2), FAKE, 1, 4096, 128, 4, 1, 131072, 1, 0.1, FAKE, FAKE,
                                          need - 1, None) == fathom.ERR_WORKSPACE
    need = lib.fathom_paged_union_attention_workspace_bytes(8, 4, 128, 2048)
    if need:
        assert lib.fathom_paged_union_attention(cache(), FAKE, 4, 200, FAKE, 4, FAKE, FAKE, 2048, 0.1, FAKE, FAKE,
                                                need - 1, None) == fathom.ERR_WORKSPACE


def test_binding_checks():
    k = torch.zeros(4, 2, 16, 64, dtype=torch.int8)
    s = torch.zeros(4, 2, 16, 2, dtype=torch.uint8)
    with pytest.raises(TypeError):
        fathom.KVCache(k.float(), k.float())
    with pytest.raises(ValueError):
        fathom.KVCache(k, k.clone())                                  # no scales
    with pytest.raises(ValueError):
        fathom.KVCache(k, k.clone(), s, s[:, :, :, :1])
    with pytest.raises(ValueError):
        fathom.KVCache(k, k[:, :1], s, s)
    with pytest.raises(ValueError):
        fathom.KVCache(k.bfloat16(), k.bfloat16(), s, s)              # scales without codes
    with pytest.raises(ValueError):
        fathom.KVCache(k.transpose(2, 3), k.transpose(2, 3), s, s)
    c = fathom.KVCache(k, k.clone(), s, s.clone())
    assert c._struct.scale_token_stride == 2 and c._struct.head_stride == 16 * 64
    table, cu, length = torch.zeros(1, 4, dtype=torch.int32), torch.tensor([0, 3], dtype=torch.int32), torch.tensor([3], dtype=torch.int32)
    x = torch.zeros(3, 2, 64)
    with pytest.raises(ValueError, match="current CUDA device"):
        fathom.kv_write(c, x, x.clone(), table, cu, length)           # a cache in host memory
    with pytest.raises(TypeError):
        fathom.kv_write(c, x.half(), x.half(), table, cu, length)
    with pytest.raises(TypeError):
        fathom.kv_write(c, x, x.clone(), table.long(), cu, length)
    with pytest.raises(ValueError):
        fathom.kv_write(c, x[:, :1], x[:, :1], table, cu, length)
    with pytest.raises(ValueError):
        fathom.kv_write(c, x, x.clone(), table, cu[:1], length)
    with pytest.raises(ValueError):
        fathom.paged_attention(c, torch.zeros(3, 3, 64), table, cu, length, 3, 3)   # 3 heads over 2 groups
    with pytest.raises(ValueError):
        fathom.kv_read(c, table, cu, length, 3, out=(None, None))
    with pytest.raises(ValueError):
        fathom.paged_union_attention(c, torch.zeros(2, 2, 64).bfloat16(), table, 3, cu[None], length)


def test_largest_sizes(lib):
    """Sizes beyond what a token or a row of queries may be counted to."""
    def attend(rows_=10, max_new=5, max_len=256, G=4, scale=0.1):
        return lib.fathom_paged_attention(cache(), rows(rows=rows_), FAKE, 1, 4096, 128, G, max_new, max_len, 1, scale, FAKE + 2,
                                          FAKE + 1, 1 << 62, None)
    assert attend(max_len=(1 << 30) + 1) == fathom.ERR_UNSUPPORTED
    assert attend(rows_=(1 << 28) + 1, max_new=1 << 30, G=8) == fathom.ERR_UNSUPPORTED
    assert attend(scale=1.1e38) == fathom.ERR_INVALID_ARG and attend(scale=-1.1e38) == fathom.ERR_INVALID_ARG
    ws = lib.fathom_paged_attention_workspace_bytes
    for max_len in (1, 1 << 30):   # a bound that covers any replay of a graph asks for no unbounded scratch
        for new in (1, 2, 40, 5000):
            assert ws(8, 4, 128, new, 1, new, max_len, 1) <= 160 * 592 * 8 * 4 * 136


def test_workspace_that_is_not_what_it_says():
    wide = torch.zeros(1, dtype=torch.uint8).expand(1 << 20)   # one byte that calls itself a mebibyte
    with pytest.raises(ValueError, match="contiguous"):
        fathom._workspace(wide, 1 << 20, wide, None)


def test_workspace_of_sizes_that_are_refused(lib):
    """The query knows the bounds of the call: nothing to give for more tokens, query rows, rows or sequences than it takes."""
    ws = lib.fathom_paged_attention_workspace_bytes
    for max_len in ((1 << 30) + 1, 1 << 31, (1 << 32) - 1, 1 << 32, 1 << 33, 1 << 62):
        for dtype in (0, 1):
            for rows_, B, new in ((2, 2, 1), (300, 300, 1), (300, 1, 300), (90000, 300, 300), (5000, 1, 5000)):
                assert ws(8, 4, 128, rows_, B, new, max_len, dtype) == 0
    assert ws(8, 8, 128, (1 << 28) + 1, 1, 1 << 28, 1 << 20, 1) == 0          # rows of queries that no int counts
    assert ws(1, 1, 128, 1 << 31, 1, 1, 1 << 20, 1) == 0 and ws(1, 1, 128, 1 << 62, 1, 1, 1 << 20, 1) == 0
    assert ws(1, 1, 128, 10, 1 << 16, 1, 1 << 20, 1) == 0
    assert ws(1, 1, 128, 1, 1, 1, 1 << 30, 1) > 0


def test_largest_write(lib):
    """A write is refused for its size where its CTAs pass what a launch takes, and only there (of two faults the size's is
    reported first; these pointers are the other)."""
    wide = dict(H=65535, D=256, token_stride=256, head_stride=64 * 256, page_stride=65535 * 64 * 256, scale_token_stride=8,
                scale_head_stride=64 * 8, scale_page_stride=65535 * 64 * 8)

    def write(n):   # n * 65535 * 16 threads, 256 to a CTA
        return lib.fathom_kv_write(cache(**wide), rows(rows=n), FAKE, FAKE, 1, 65535 * 256, 256, None)
    most = ((1 << 31) - 1) * 16 // 65535
    assert write(300000) == write(most) == fathom.ERR_INVALID_ARG
    assert write(most + 1) == fathom.ERR_UNSUPPORTED


def test_a_cache_keeps_its_tensors():
    """The addresses that calls use are those of the tensors it was made over: another tensor in an attribute's place would
    leave them pointing at freed memory."""
    k, s = torch.zeros(4, 2, 16, 64, dtype=torch.int8), torch.zeros(4, 2, 16, 2, dtype=torch.uint8)
    c = fathom.KVCache(k, k.clone(), s, s.clone())
    for name in ("k", "v", "k_scale", "v_scale", "H", "D", "page_tokens", "format"):
        old = getattr(c, name)
        with pytest.raises(AttributeError, match="another KVCache"):
            setattr(c, name, old.clone() if isinstance(old, torch.Tensor) else old)
        assert getattr(c, name) is old
        with pytest.raises(AttributeError):
            delattr(c, name)
    c.label = "a user's own"
    assert c._struct.k == c.k.data_ptr() and c._struct.v_scale == c.v_scale.data_ptr()


def test_cache_of_no_groups():
    k, s = torch.zeros(4, 0, 16, 64, dtype=torch.int8), torch.zeros(4, 0, 16, 2, dtype=torch.uint8)
    c = fathom.KVCache(k, k.clone(), s, s.clone())
    table, cu, length = torch.zeros(1, 4, dtype=torch.int32), torch.tensor([0, 3], dtype=torch.int32), torch.tensor([3], dtype=torch.int32)
    for heads in (0, 4):
        with pytest.raises(ValueError, match=r"q must be \[rows\]"):
            fathom.paged_attention(c, torch.zeros(3, heads, 64), table, cu, length, 3, 3)
