"""Cases of the paged key/value cache: writing it (in 16 or 8 bits), reading it back, attention of a chunk of new
tokens over it, and attention over the rows that a scan's top-k chose.

A cache is pages of ``page`` tokens, [pages][H][page][D]; a sequence is a row of the page table.  In the 8-bit
formats every 32 channels of a row share one power of two, 2^(b - 127), b the byte kept beside the codes:
``int8`` keeps round(x 2^-e), ``e4m3`` the 8-bit float of x 2^-e.  A call names, for each sequence, its length
and how many of its last tokens the call's rows are.

``run`` computes plain forms with elementary torch operations, or, where ``own`` is true, calls the framework.
"""
import random

import torch

own = False

BLOCK = 32
LOWEST = -100   # smallest exponent of a block's power of two


# ---------------------------------------------------------------- the cases

def _case(name, op, fmt, dtype, H, G, D, page, B=1, new=(1, 1), kv=(1, 1), mix=0, k=0, causal=True):
    return {"name": name, "op": op, "fmt": fmt, "dtype": dtype, "H": H, "G": G, "D": D, "page": page, "B": B,
            "new_lo": new[0], "new_hi": new[1], "kv_lo": kv[0], "kv_hi": kv[1], "mix": mix, "k": k, "causal": causal}


def listed():
    return [
        # One new token of one session, one layer of 8 heads: the write of every decode step, and the read of it.
        _case("write-token", "write", "int8", "bf16", 8, 4, 128, 64, kv=(32768, 32768)),
        # A prefill of 32k tokens of one layer, written once.
        _case("write-prefill", "write", "int8", "bf16", 8, 4, 128, 64, new=(32768, 32768), kv=(32768, 32768)),
        # Chunks of several sessions at other widths: fp32 rows, 8-bit floats, small pages, odd lengths.
        _case("write-ragged", "write", "e4m3", "fp32", 3, 1, 96, 16, B=17, new=(1, 611), kv=(700, 5000), mix=3),
        # The tail block of a session read back, for the index to be packed again.
        _case("read-tail", "read", "int8", "fp32", 8, 4, 128, 64, new=(37, 37), kv=(131072, 131072)),
        # A whole 128k session's layer read back in the index's input layout.
        _case("read-session", "read", "int8", "bf16", 8, 4, 128, 64, new=(131072, 131072), kv=(131072, 131072)),
        # One token of one 128k session: the dense decode step of a layer.
        _case("decode-128k", "attend", "int8", "bf16", 8, 4, 128, 64, kv=(131072, 131072)),
        # One token each of many sessions of uneven lengths, 16-bit cache.
        _case("decode-batch", "attend", "bf16", "bf16", 8, 8, 64, 32, B=24, kv=(1, 32768), mix=5),
        # A chunk of a long prompt over what is there already: the largest.
        _case("chunk-128k", "attend", "bf16", "bf16", 8, 4, 128, 64, new=(2048, 2048), kv=(131072, 131072)),
        # Chunks of several sessions, odd lengths and a group of five, 8-bit cache.
        _case("chunk-ragged", "attend", "int8", "bf16", 4, 5, 128, 16, B=5, new=(1, 700), kv=(700, 9001), mix=7),
        # A short prompt at fp32 precision.
        _case("chunk-fp32", "attend", "e4m3", "fp32", 2, 4, 96, 64, B=2, new=(129, 333), kv=(333, 2049), mix=9),
        # The winners of one layer's scan at 128k, fetched from the 8-bit cache.
        _case("union-layer", "union", "int8", "fp32", 8, 4, 128, 64, kv=(131072, 131072), k=512),
        # The winners of all 288 layer-heads at 32k.
        _case("union-step", "union", "int8", "fp32", 288, 4, 128, 64, kv=(32768, 32768), k=512, mix=1),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(("write", "read", "attend", "attend", "attend", "union"))
    fmt = rng.choice(("bf16", "int8", "e4m3"))
    D = rng.choice((32, 64, 64, 96, 128, 128, 128, 160, 256))
    page = rng.choice((16, 32, 64, 128))
    H = rng.randint(1, 12)
    mix = rng.randrange(1 << 20)
    if op == "union":
        H = _log(rng, 1, 128)
        kv = _log(rng, 1100, 60000) if H < 32 else _log(rng, 1100, 20000)
        return _nameless(_case("", op, fmt, "fp32", H, rng.randint(1, 8), D, page, kv=(kv, kv), mix=mix, k=_log(rng, 1, 1024)))
    if op in ("write", "read"):
        B = _log(rng, 1, 40)
        hi = _log(rng, 1, 40000 // B)
        kv = _log(rng, hi, 2 * hi + 3000)
        return _nameless(_case("", op, fmt, rng.choice(("bf16", "fp32")), H, 1, D, page, B=B, new=(_log(rng, 1, hi), hi),
                               kv=(hi, kv), mix=mix))
    G = rng.randint(1, 8)
    if rng.random() < 0.4:   # single tokens
        B = _log(rng, 1, 48)
        kv = _log(rng, 1, 400000 // (B * (D // 32)))
        return _nameless(_case("", op, fmt, rng.choice(("bf16", "bf16", "fp32")), H, G, D, page, B=B,
                               kv=(_log(rng, 1, kv), kv), mix=mix))
    B = _log(rng, 1, 8)
    dtype = rng.choice(("bf16", "bf16", "bf16", "fp32"))
    hi = _log(rng, 2, 2048 // B if dtype == "bf16" else 300)
    kv = _log(rng, hi, 600000 // (B * max(H, 4) * (D // 32)) + hi)
    return _nameless(_case("", op, fmt, dtype, H, G, D, page, B=B, new=(_log(rng, 1, hi), hi), kv=(hi, kv), mix=mix,
                           causal=rng.random() < 0.85))


def _nameless(case):
    return {k: v for k, v in case.items() if k != "name"}


def _lengths(case):
    """[(rows of the call, length)] of each sequence."""
    rng = random.Random(case["mix"])
    spread = [(_log(rng, case["new_lo"], case["new_hi"]), _log(rng, case["kv_lo"], case["kv_hi"])) for _ in range(case["B"])]
    spread[0] = (case["new_hi"], case["kv_hi"])   # the bounds are reached
    return [(min(n, kv), kv) for n, kv in spread]


# ---------------------------------------------------------------- the inputs

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _power(e):
    """2^e as fp32, for whole e in -126 .. 127."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _encode(x, fmt):
    """Codes and exponent bytes of rows x [..., D] (fp32 values)."""
    if fmt == "bf16":
        return x.to(torch.bfloat16), None
    blocks = x.unflatten(-1, (-1, BLOCK))
    top = blocks.abs().amax(-1)
    mant, ex = torch.frexp(top)                       # top = mant 2^ex, mant in [1/2, 1)
    if fmt == "int8":
        e = (ex - 7 + (mant >= 255 / 256)).clamp(LOWEST, 121)
    else:
        e = (ex - 9 + (mant > 29 / 32)).clamp(LOWEST, 7)
    e = torch.where(top > 0, e, torch.full_like(e, LOWEST))
    y = blocks * _power(-e)[..., None]
    if fmt == "int8":
        codes = y.round().clamp(-127, 127).to(torch.int8)
    else:
        codes = y.clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes.flatten(-2), (e + 127).to(torch.uint8)


def _decode(codes, scale):
    """fp32 values of codes [..., D]."""
    if scale is None:
        return codes.float()
    return (codes.float().unflatten(-1, (-1, BLOCK)) * _power(scale.to(torch.int32) - 127)[..., None]).flatten(-2)


def _rows(shape, g, dev):
    """Key rows as under a QK norm: unit mean square."""
    z = torch.randn(shape, generator=g, device=dev)
    return z * z.square().mean(-1, keepdim=True).rsqrt()


def _pages(count, case, g, dev):
    """A filled cache."""
    H, D, page, fmt = case["H"], case["D"], case["page"], case["fmt"]
    step = max(1, (1 << 27) // (H * page * D))
    parts = []
    for at in range(0, count, step):
        shape = (min(step, count - at), H, page, D)
        parts.append(_encode(_rows(shape, g, dev), fmt) + _encode(torch.randn(shape, generator=g, device=dev), fmt))
    k, ks, v, vs = [None if p[0] is None else torch.cat(p) for p in zip(*parts)]
    return k, v, ks, vs


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1_000_003 + case["mix"])
    H, G, D, page, B = case["H"], case["G"], case["D"], case["page"], case["B"]
    lens = _lengths(case)
    need = [-(-kv // page) for _, kv in lens]
    count = sum(need) + 3
    order = torch.randperm(count, generator=g, device=dev).to(torch.int32)
    starts = [sum(need[:b]) for b in range(B)]
    wide = max(need)
    at = torch.arange(wide, device=dev)[None, :].expand(B, wide)
    first = torch.tensor(starts, device=dev)[:, None]
    held = at < torch.tensor(need, device=dev)[:, None]
    table = torch.where(held, order[(first + at).clamp(max=count - 1)], torch.full((1,), -1, dtype=torch.int32, device=dev))
    cu = torch.tensor([sum(n for n, _ in lens[:b]) for b in range(B + 1)], dtype=torch.int32, device=dev)
    length = torch.tensor([kv for _, kv in lens], dtype=torch.int32, device=dev)
    rows = sum(n for n, _ in lens)
    dtype = _TYPES[case["dtype"]]
    state = {"case": case, "table": table.contiguous(), "cu": cu, "length": length, "rows": rows,
             "max_new": max(n for n, _ in lens), "max_len": max(kv for _, kv in lens)}
    if case["op"] == "write":
        shape = (count, H, page, D)
        held_as = {"bf16": torch.bfloat16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}[case["fmt"]]
        k, v = (torch.zeros(shape, dtype=torch.uint8 if case["fmt"] == "e4m3" else held_as, device=dev) for _ in range(2))
        if case["fmt"] == "e4m3":
            k, v = k.view(held_as), v.view(held_as)
        ks, vs = (None, None) if case["fmt"] == "bf16" else \
            (torch.zeros(shape[:3] + (D // BLOCK,), dtype=torch.uint8, device=dev) for _ in range(2))
        state["new_k"] = _rows((rows, H, D), g, dev).to(dtype)
        state["new_v"] = torch.randn(rows, H, D, generator=g, device=dev).to(dtype)
    else:
        k, v, ks, vs = _pages(count, case, g, dev)
    state["pages"] = (k, v, ks, vs)
    if case["op"] in ("attend", "union"):
        q = torch.randn((rows, H * G, D) if case["op"] == "attend" else (H, G, D), generator=g, device=dev)
        loud = torch.randperm(D, generator=g, device=dev)[:max(1, D // 12)]
        q[..., loud] *= 5.0
        state["q"] = q.to(torch.bfloat16).to(dtype)   # bf16 values, as a model's queries
    if case["op"] == "union":
        n, M = case["kv_hi"], G * min(case["k"], case["kv_hi"])
        keep = min(M, n)
        pick = torch.rand(H, n, generator=g, device=dev).argsort(1)[:, :keep].sort(1).values.to(torch.int32)
        cnt = torch.randint((keep + G - 1) // G, keep + 1, (H,), generator=g, device=dev).to(torch.int32)
        pad = torch.full((H, M - keep), -1, dtype=torch.int32, device=dev)
        idx = torch.cat([pick, pad], 1)
        state["union"] = torch.where(torch.arange(M, device=dev)[None, :] < cnt[:, None], idx, torch.full_like(idx, -1)).contiguous()
        state["count"] = cnt
        state["n"] = n
    if own:
        from long_context_decode_bit_b200 import fathom
        state["cache"] = fathom.KVCache(k, v, ks, vs)
    return state


# ---------------------------------------------------------------- one pass

def _places(s):
    """Page, offset and validity of the call's rows, and their sequence."""
    cu, page = s["cu"].long(), s["case"]["page"]
    r = torch.arange(s["rows"], device=cu.device)
    b = torch.searchsorted(cu[1:], r, right=True)
    pos = s["length"].long()[b] - cu[b + 1] + r
    return s["table"][b, pos // page].long(), pos % page, b, pos


def _plain_write(s):
    fmt, page = s["case"]["fmt"], s["case"]["page"]
    where, off, _, _ = _places(s)
    k, v, ks, vs = s["pages"]
    raw = (lambda t: t.view(torch.uint8)) if fmt == "e4m3" else (lambda t: t)
    kc, kb = _encode(s["new_k"].float(), fmt)
    vc, vb = _encode(s["new_v"].float(), fmt)
    raw(k)[where, :, off] = raw(kc)
    raw(v)[where, :, off] = raw(vc)
    if fmt != "bf16":
        ks[where, :, off] = kb
        vs[where, :, off] = vb
    return _plain_read(s) + ([] if fmt == "bf16" else [ks, vs])


def _plain_read(s):
    where, off, _, _ = _places(s)
    k, v, ks, vs = s["pages"]
    fp8 = s["case"]["fmt"] == "e4m3"
    take = lambda t: t.view(torch.uint8)[where, :, off].view(t.dtype) if fp8 and t.dtype != torch.uint8 else t[where, :, off]  # noqa: E731
    dtype = _TYPES[s["case"]["dtype"]]
    return [_decode(take(c), None if b is None else take(b)).transpose(0, 1).to(dtype).contiguous() for c, b in ((k, ks), (v, vs))]


def _sequence_rows(s, at):
    """K and V, fp32, of the tokens at positions ``at`` [..., L] of table rows [..., pages] -> [..., L, H, D]."""
    k, v, ks, vs = s["pages"]
    page = s["case"]["page"]
    fp8 = s["case"]["fmt"] == "e4m3"
    where = torch.gather(s["table"].long(), 1, at // page).clamp(min=0)
    off = at % page
    take = lambda t: t.view(torch.uint8)[where, :, off].view(t.dtype) if fp8 and t.dtype != torch.uint8 else t[where, :, off]  # noqa: E731
    return [_decode(take(c), None if b is None else take(b)) for c, b in ((k, ks), (v, vs))]


def _plain_attend(s):
    c = s["case"]
    H, G, D, B, T, L = c["H"], c["G"], c["D"], c["B"], s["max_new"], s["max_len"]
    dev = s["cu"].device
    cu, length = s["cu"].long(), s["length"].long()
    new = cu[1:] - cu[:-1]
    t = torch.arange(T, device=dev)
    valid = t[None, :] < new[:, None]
    row = (cu[:-1, None] + t[None, :]).clamp(max=s["rows"] - 1)
    q = s["q"][row].float().view(B, T, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * T, D)
    last = torch.where(valid, (length - new)[:, None] + t[None, :] if c["causal"] else (length - 1)[:, None].expand(B, T),
                       torch.full((1,), -1, device=dev))
    at = torch.arange(L, device=dev)[None, :].expand(B, L).contiguous()
    K, V = _sequence_rows(s, torch.minimum(at, (length - 1)[:, None]))
    score = q @ K.permute(0, 2, 3, 1)                              # [B][H][G T][L]
    score *= D ** -0.5
    hide = (at[:, None, :] > last[:, :, None])[:, None, None]      # [B][1][1][T][L]
    score.view(B, H, G, T, L).masked_fill_(hide, float("-inf"))
    score -= score.amax(-1, keepdim=True).clamp(min=-1e30)
    score.exp_()
    total = score.sum(-1, keepdim=True)
    out = (score @ V.transpose(1, 2)) / total.clamp(min=1e-30)
    out = out.view(B, H, G, T, D).permute(0, 3, 1, 2, 4).reshape(B, T, H * G, D)
    return out[valid].to(s["q"].dtype)


def _plain_union(s):
    c = s["case"]
    idx, live = s["union"].long(), torch.arange(s["union"].shape[1], device=s["count"].device)[None, :] < s["count"][:, None]
    idx = idx.clamp(min=0)
    page = c["page"]
    where, off = s["table"].long()[0][idx // page], idx % page
    head = torch.arange(c["H"], device=idx.device)[:, None].expand_as(idx)
    k, v, ks, vs = s["pages"]
    fp8 = c["fmt"] == "e4m3"
    take = lambda t: t.view(torch.uint8)[where, head, off].view(t.dtype) if fp8 and t.dtype != torch.uint8 else t[where, head, off]  # noqa: E731
    K, V = (_decode(take(x), None if b is None else take(b)) for x, b in ((k, ks), (v, vs)))
    score = (s["q"].float() @ K.transpose(1, 2)) * c["D"] ** -0.5
    score = score.masked_fill(~live[:, None, :], float("-inf"))
    score = (score - score.amax(-1, keepdim=True)).exp()
    return (score @ V) / score.sum(-1, keepdim=True)


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        from long_context_decode_bit_b200 import fathom
        cache, table, cu, length = s["cache"], s["table"], s["cu"], s["length"]
        if op == "write":
            fathom.kv_write(cache, s["new_k"], s["new_v"], table, cu, length)
        if op in ("write", "read"):
            got = list(fathom.kv_read(cache, table, cu, length, s["rows"], dtype=_TYPES[s["case"]["dtype"]]))
            return got + ([] if op == "read" or cache.k_scale is None else [cache.k_scale, cache.v_scale])
        if op == "attend":
            return fathom.paged_attention(cache, s["q"], table, cu, length, s["max_new"], s["max_len"],
                                          causal=s["case"]["causal"])
        return fathom.paged_union_attention(cache, s["q"], table, s["n"], s["union"], s["count"])
    return {"write": _plain_write, "read": _plain_read, "attend": _plain_attend, "union": _plain_union}[op](s)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    H, G, D = case["H"], case["G"], case["D"]
    lens = _lengths(case)
    held = 2 * D if case["fmt"] == "bf16" else D + D // BLOCK      # bytes of a cached row
    wide = 2 if case["dtype"] == "bf16" else 4
    rows = sum(n for n, _ in lens)
    if case["op"] == "write":   # in, written, and read back
        return {"bytes": 2 * rows * H * (2 * D * wide + 2 * held), "flops": 0}
    if case["op"] == "read":
        return {"bytes": 2 * rows * H * (D * wide + held), "flops": 0}
    if case["op"] == "attend":
        keys = sum(n * kv - (n * (n - 1) // 2 if case["causal"] else 0) for n, kv in lens)
        return {"bytes": 2 * H * held * sum(kv for _, kv in lens) + 2 * rows * H * G * D * wide, "flops": 4 * D * H * G * keys}
    keep = min(G * min(case["k"], case["kv_hi"]), case["kv_hi"])
    mean = ((keep + G - 1) // G + keep) / 2
    return {"bytes": H * mean * (2 * held + 4) + 2 * H * G * D * wide, "flops": 4 * D * H * G * mean}


# ---------------------------------------------------------------- the definition, in 64 bits

def _value64(codes, scale):
    if scale is None:
        return codes.double()
    e = scale.double().sub(127).repeat_interleave(BLOCK, -1)
    return codes.to(torch.float32).double() * torch.exp2(e)


def _one_sequence(s, b, kv):
    """K and V [H][kv][D] of sequence b in 64 bits."""
    page = s["case"]["page"]
    ids = s["table"][b, : -(-kv // page)].long()
    out = []
    for codes, scale in ((s["pages"][0], s["pages"][2]), (s["pages"][1], s["pages"][3])):
        sel = codes.view(torch.uint8)[ids].view(codes.dtype) if codes.dtype == torch.float8_e4m3fn else codes[ids]
        x = _value64(sel, None if scale is None else scale[ids])
        out.append(x.transpose(0, 1).flatten(1, 2)[:, :kv])
    return out


def _quantised64(x, fmt):
    """The values and exponent bytes that rows x stand for once kept, in 64 bits."""
    if fmt == "bf16":
        return x.to(torch.bfloat16).double(), None
    x = x.double().reshape(*x.shape[:-1], -1, BLOCK)
    top = x.abs().max(-1, keepdim=True).values
    whole = torch.floor(torch.log2(top.clamp(min=2.0 ** -149)))
    whole = whole + (torch.exp2(whole + 1) <= top).double() - (torch.exp2(whole) > top).double()   # log2 may round over a border
    if fmt == "int8":     # the least e with round(top 2^-e) <= 127
        e = whole - 6
        e = e + (top / torch.exp2(e) >= 127.5).double()
        e = e.clamp(LOWEST, 121)
    else:                 # the least e with top 2^-e within half a step of 448
        e = whole - 8
        e = e + (top / torch.exp2(e) > 464).double()
        e = e.clamp(LOWEST, 7)
    e = torch.where(top > 0, e, torch.full_like(e, LOWEST))
    y = x / torch.exp2(e)
    if fmt == "int8":
        y = torch.round(y).clamp(-127, 127)
    else:                 # three bits after the leading one, steps of 2^-9 below 2^-6
        y = y.clamp(-448, 448)
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))).clamp(min=-6) - 3)
        y = torch.round(y / step) * step
    return (y * torch.exp2(e)).flatten(-2), (e[..., 0] + 127).to(torch.uint8)


def exact(case, seed):
    s = prepare(case, seed)
    lens, H, G, D = _lengths(case), case["H"], case["G"], case["D"]
    page = case["page"]
    if case["op"] == "write":
        vals, bytes_ = [], []
        for new, scale in ((s["new_k"], s["pages"][2]), (s["new_v"], s["pages"][3])):
            x, b = _quantised64(new, case["fmt"])
            vals.append(x.transpose(0, 1).contiguous())
            if b is not None:
                scale = scale.clone()
                row = 0
                for i, (n, kv) in enumerate(lens):
                    pos = torch.arange(kv - n, kv, device=scale.device)
                    scale[s["table"][i].long()[pos // page], :, pos % page] = b[row:row + n]
                    row += n
                bytes_.append(scale)
        return vals + bytes_
    if case["op"] == "read":
        both = []
        for i, (n, kv) in enumerate(lens):
            both.append([x[:, kv - n:] for x in _one_sequence(s, i, kv)])
        return [torch.cat(x, 1) for x in zip(*both)]
    if case["op"] == "union":
        out = torch.zeros(H, G, D, dtype=torch.float64, device=s["q"].device)
        ids, n = s["table"][0].long(), case["kv_hi"]
        counts = s["count"].tolist()
        for h in range(H):
            at = s["union"][h, :counts[h]].long()
            kv = []
            for codes, scale in ((s["pages"][0], s["pages"][2]), (s["pages"][1], s["pages"][3])):
                raw = codes.view(torch.uint8) if codes.dtype == torch.float8_e4m3fn else codes
                kv.append(_value64(raw[ids[at // page], h, at % page].view(codes.dtype),
                                   None if scale is None else scale[ids[at // page], h, at % page]))
            p = torch.softmax(s["q"][h].double() @ kv[0].T / D ** 0.5, -1)
            out[h] = p @ kv[1]
        return out
    out = torch.zeros(s["rows"], H * G, D, dtype=torch.float64, device=s["q"].device)
    row = 0
    for i, (n, kv) in enumerate(lens):
        K, V = _one_sequence(s, i, kv)
        pos = torch.arange(kv - n, kv, device=K.device)
        seen = torch.arange(kv, device=K.device)[None, :] <= (pos[:, None] if case["causal"] else kv)
        for hq in range(H * G):
            x = s["q"][row:row + n, hq].double() @ K[hq // G].T / D ** 0.5
            x = torch.where(seen, x, torch.full_like(x, float("-inf")))
            out[row:row + n, hq] = torch.softmax(x, -1) @ V[hq // G]
        row += n
    return out
