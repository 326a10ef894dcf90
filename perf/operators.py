"""Measured cases of the paged key/value cache operators: the write (per-head
norms, rotation, quantisation, one pass over the projected rows), the read
back into contiguous rows, and the attention over the pages for single
tokens, chunks, whole prompts and another sequence's states.

A cache pool holds pages of ``page`` tokens; a batch is ``q_start`` (first
new row of each sequence), ``kv_len`` (positions in the cache, the new rows
included) and the page table.  Row i of a sequence with n new rows stands at
position kv_len - n + i.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16,
          "int8": torch.int8, "e4m3": torch.float8_e4m3fn}
SIZES = {"f32": 4, "f16": 2, "bf16": 2, "int8": 1, "e4m3": 1}
LARGEST = {"int8": 127.0, "e4m3": 448.0}
EPS = 1e-6

# (query heads, kv heads, head_dim): the shapes of this repository.
HEADS = ((14, 2, 64), (28, 4, 128), (12, 2, 128), (8, 4, 128), (6, 2, 64), (4, 4, 64), (8, 1, 64), (4, 2, 128))


def _write(name, heads, n_seq, q, ctx, x, cache, page, norm, rotary, layout, mix):
    return {"name": name, "op": "write", "nh": heads[0], "nkv": heads[1], "hd": heads[2], "n_seq": n_seq,
            "q_min": q[0], "q_max": q[1], "ctx_min": ctx[0], "ctx_max": ctx[1], "x": x, "cache": cache,
            "page": page, "norm": norm, "rotary": rotary, "interleaved": layout == "interleaved", "mix": mix}


def _read(name, heads, n_seq, ctx, x, cache, page, mix):
    return {"name": name, "op": "read", "nh": heads[0], "nkv": heads[1], "hd": heads[2], "n_seq": n_seq,
            "q_min": 0, "q_max": 0, "ctx_min": ctx[0], "ctx_max": ctx[1], "x": x, "cache": cache, "page": page,
            "mix": mix}


def _attend(name, heads, n_seq, q, ctx, x, cache, page, causal, mix):
    return {"name": name, "op": "attend", "nh": heads[0], "nkv": heads[1], "hd": heads[2], "n_seq": n_seq,
            "q_min": q[0], "q_max": q[1], "ctx_min": ctx[0], "ctx_max": ctx[1], "x": x, "cache": cache,
            "page": page, "causal": causal, "mix": mix}


def listed():
    return [
        # One decode step of a small batch: one new row a sequence, f32 projections, f16 pages.
        _write("write step 8", (14, 2, 64), 8, (1, 1), (100, 4000), "f32", "f16", 16, False, 64, "half", 1),
        # A prompt chunk of several requests, per-head norms, a quarter of the head rotated, 8-bit pages.
        _write("write chunk int8", (28, 4, 128), 5, (200, 700), (0, 0), "bf16", "int8", 32, True, 32,
               "interleaved", 2),
        # Prompts of a whole batch in one pass.
        _write("write prompts e4m3", (28, 4, 128), 9, (1000, 2100), (0, 0), "bf16", "e4m3", 64, True, 128, "half", 3),
        # One conversation's layer taken out of the pages as f32 rows.
        _read("read one", (14, 2, 64), 1, (1234, 1234), "f32", "f16", 16, 4),
        # Long conversations kept in 8 bits, read back for another engine.
        _read("read long int8", (28, 4, 128), 8, (9000, 33000), "bf16", "int8", 64, 5),
        # One user's next token.
        _attend("attend token 1", (14, 2, 64), 1, (1, 1), (999, 999), "f16", "f16", 16, True, 6),
        # The decode step of a ragged batch (the batch and lengths of the 32-sequence benchmark).
        _attend("attend token 32", (14, 2, 64), 32, (1, 1), (256, 4095), "f16", "f16", 64, True, 7),
        # Long conversations on an 8-bit cache, next token.
        _attend("attend token long int8", (28, 4, 128), 16, (1, 1), (8000, 32700), "bf16", "int8", 64, True, 8),
        # Chunks of prompts beside decoding sequences in one batch.
        _attend("attend mixed", (14, 2, 64), 12, (1, 300), (0, 3000), "f16", "f16", 32, True, 9),
        # A prompt in one pass.
        _attend("attend prompt", (28, 4, 128), 1, (5001, 5001), (0, 0), "bf16", "bf16", 64, True, 10),
        # A chunk of a long document over its 8-bit cache.
        _attend("attend chunk e4m3", (28, 4, 128), 1, (1024, 1024), (31000, 31000), "f16", "e4m3", 64, True, 11),
        # Rows of a decoder over an encoder's states.
        _attend("attend cross", (12, 2, 128), 6, (30, 200), (1500, 1500), "bf16", "bf16", 128, False, 12),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], uniform in its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    heads = rng.choice(HEADS)
    nh, nkv, hd = heads
    page = rng.choice((16, 32, 64, 128))
    mix = rng.randrange(1 << 20)
    op = rng.choice(("write", "read", "attend", "attend", "attend"))
    if op == "write":
        n_seq = _spread(rng, 1, 64)
        q_max = _spread(rng, 1, max(1, 16000 // n_seq))
        cache = rng.choice(("f16", "bf16", "int8", "e4m3"))
        ctx = 0 if cache in LARGEST else _spread(rng, 1, 8000)
        rotary = rng.choice((0, hd // 4, hd // 2, hd, hd))
        c = _write("", heads, n_seq, (max(1, q_max // 2), q_max), (ctx // 2, ctx), rng.choice(("f32", "f16", "bf16")),
                   cache, page, rng.random() < 0.5, rotary, rng.choice(("half", "interleaved")), mix)
    elif op == "read":
        n_seq = _spread(rng, 1, 32)
        ctx = _spread(rng, 1, min(40000, 240000 // n_seq))
        c = _read("", heads, n_seq, (max(1, ctx // 3), ctx), rng.choice(("f32", "f16", "bf16")),
                  rng.choice(("f16", "bf16", "int8", "e4m3")), page, mix)
    else:
        x = rng.choice(("f16", "bf16"))
        cache = rng.choice((x, x, "int8", "e4m3"))
        form = rng.choice(("token", "few", "chunk", "prompt", "cross"))
        n_seq = _spread(rng, 1, 48 if form in ("token", "few") else 8)
        if form in ("token", "few"):
            q_max = 1 if form == "token" else rng.randint(2, 8)
            ctx = _spread(rng, 1, min(32000, 500000 // n_seq))
        elif form == "prompt":
            q_max, ctx = _spread(rng, 2, 4500), 0
        else:
            q_max = _spread(rng, 8, 1024)
            ctx = _spread(rng, 1, 16000)
        # At most as many scores as the largest listed cases have.
        while n_seq * nh * q_max * (q_max + ctx) > 6e8:
            if n_seq > 1:
                n_seq = max(1, n_seq // 2)
            else:
                q_max, ctx = max(1, q_max * 2 // 3), ctx * 2 // 3
        lo = q_max if form in ("token", "prompt") else max(1, q_max // 3)
        c = _attend("", heads, n_seq, (lo, q_max), (ctx // 2, ctx), x, cache, page, form != "cross", mix)
        if form == "cross":
            c["ctx_min"] = c["ctx_max"] = max(1, ctx)
    del c["name"]
    return c


def _lengths(case):
    """(new rows, cached positions with the new rows) of each sequence."""
    rng = random.Random(case["mix"])
    q = [_spread(rng, max(1, case["q_min"]), case["q_max"]) if case["q_max"] else 0 for _ in range(case["n_seq"])]
    ctx = [rng.randint(case["ctx_min"], case["ctx_max"]) for _ in q]
    if case["op"] == "attend" and not case["causal"]:
        return q, ctx
    return q, [a + b for a, b in zip(q, ctx)]


def work(case):
    q, kv = _lengths(case)
    nh, nkv, hd = case["nh"], case["nkv"], case["hd"]
    rows, held = sum(q), sum(kv)
    xs, cs = SIZES[case["x"]], SIZES[case["cache"]]
    quant = case["cache"] in LARGEST
    entry = 2 * nkv * (hd * cs + (4 if quant else 0))    # one position's K and V
    if case["op"] == "write":
        b = rows * (nh + 2 * nkv) * hd * xs + rows * nh * hd * 2 + rows * entry + rows * case["rotary"] // 2 * 8
        if quant:   # and what is read back
            b += rows * (entry + 2 * nkv * hd * 2)
        return {"bytes": b, "flops": 12 * rows * (nh + 2 * nkv) * hd}
    if case["op"] == "read":
        return {"bytes": held * (entry + 2 * nkv * hd * xs), "flops": held * 2 * nkv * hd}
    pairs = sum(n * (k - n) + n * (n + 1) // 2 if case["causal"] else n * k for n, k in zip(q, kv))
    return {"bytes": held * entry + 2 * rows * nh * hd * 2, "flops": 4 * hd * nh * pairs}


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _pool(g, case, n_pages):
    """K and V pages with what an earlier use left in them, and their scales."""
    nkv, hd, page = case["nkv"], case["hd"], case["page"]
    shape = (n_pages, page, nkv, hd)
    kind = case["cache"]
    if kind not in LARGEST:
        gain = torch.exp(0.3 * _normal(g, (hd,), torch.float32))
        k = (torch.randn(shape, generator=g, device="cuda", dtype=DTYPES[kind]) * gain.to(DTYPES[kind]))
        v = torch.randn(shape, generator=g, device="cuda", dtype=DTYPES[kind]) * 0.5
        return k, v, None, None
    pools = []
    for spread in (1.0, 0.5):
        codes = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
        largest = codes.abs().amax(-1, keepdim=True)
        codes *= LARGEST[kind] / largest
        codes = codes.round_().clamp_(-127, 127).to(torch.int8) if kind == "int8" else codes.to(torch.float8_e4m3fn)
        scale = largest[..., 0].float().permute(0, 2, 1).contiguous() * (spread / LARGEST[kind])
        pools.append((codes, scale))
    return pools[0][0], pools[1][0], pools[0][1], pools[1][1]


def _table(n_pos, rotary):
    """(cos, sin) of position * 1e6^(-2i / rotary), angles in 64 bits."""
    inv = 1e6 ** (-2.0 * torch.arange(rotary // 2, device="cuda", dtype=torch.float64) / rotary)
    angle = torch.arange(n_pos, device="cuda", dtype=torch.float64)[:, None] * inv
    return torch.stack((angle.cos(), angle.sin()), -1).float()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, kv = _lengths(case)
    nh, nkv, hd, page = case["nh"], case["nkv"], case["hd"], case["page"]
    need = [-(-n // page) for n in kv]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    pages = torch.zeros((len(kv), max(need)), dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(need):
        pages[s, :n] = order[at:at + n]
        at += n
    starts = [0]
    for n in q:
        starts.append(starts[-1] + n)
    s = {"case": case, "max_q": max(q), "max_kv": max(kv), "rows": starts[-1],
         "q_start": torch.tensor(starts, dtype=torch.int32, device="cuda"),
         "kv_len": torch.tensor(kv, dtype=torch.int32, device="cuda"), "pages": pages}
    s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"] = _pool(g, case, n_pages)
    x = DTYPES[case["x"]]
    if case["op"] == "write":
        # The fused projection's rows: q heads, then k, then v.
        qkv = _normal(g, (starts[-1], nh + 2 * nkv, hd), x)
        s["q"], s["k"], s["v"] = qkv[:, :nh], qkv[:, nh:nh + nkv], qkv[:, nh + nkv:]
        if case["norm"]:
            s["q_norm"] = 1 + 0.1 * _normal(g, (hd,), torch.float32)
            s["k_norm"] = 1 + 0.1 * _normal(g, (hd,), torch.float32)
        s["rope"] = _table(max(kv), case["rotary"]) if case["rotary"] else None
    if case["op"] == "attend":
        s["q"] = _normal(g, (starts[-1], nh, hd), x)
    if case["op"] == "read" or case["cache"] in LARGEST:
        s["held"] = sum(kv)
        ends = [0]
        for n in kv:
            ends.append(ends[-1] + n)
        s["out_start"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    if own:
        import qwen2_decoder_forward_gb300 as q2
        s["kv"] = q2.PagedKV(s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"])
        s["batch"] = q2.PagedBatch(s["q_start"], s["kv_len"], pages, max(1, max(q)))
    return s


def _place_rows(s):
    """(sequence, position) of each new row."""
    row = torch.arange(s["rows"], device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["q_start"][1:], row, right=True)
    length = (s["q_start"][1:] - s["q_start"][:-1])[seq]
    return seq, s["kv_len"][seq] - length + row - s["q_start"][seq]


def _norm_and_turn(x, weight, turn, interleaved):
    """The heads' norm and the rotation of their first dims, in 32 bits."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
    if turn is None:
        return x
    half = turn.shape[-2]
    c, d = turn[:, None, :, 0], turn[:, None, :, 1]
    a, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        lo, hi = a[..., 0::2], a[..., 1::2]
        a = torch.stack((lo * c - hi * d, hi * c + lo * d), -1).flatten(-2)
    else:
        lo, hi = a[..., :half], a[..., half:]
        a = torch.cat((lo * c - hi * d, hi * c + lo * d), -1)
    return torch.cat((a, rest), -1)


def _codes(x, kind):
    """8-bit codes and the scale of each (token, head)."""
    largest = x.abs().amax(-1)
    scale = torch.where(largest == 0, torch.ones_like(largest), largest / LARGEST[kind])
    y = x / scale[..., None]
    if kind == "e4m3":
        return y.clamp(-448, 448).to(torch.float8_e4m3fn), scale
    return (torch.sign(y) * torch.floor(y.abs() + 0.5)).clamp(-127, 127).to(torch.int8), scale


def _store(pool, scales, x, kind, page_of, slot_of):
    if kind not in LARGEST:
        pool[page_of, slot_of] = x.to(pool.dtype)
        return
    codes, scale = _codes(x, kind)
    pool.view(torch.int8)[page_of, slot_of] = codes.view(torch.int8)
    scales[page_of, :, slot_of] = scale


def _fetch(pool, scales, page_of, slot_of):
    """Cached values in 32 bits."""
    x = pool.view(torch.int8)[page_of, slot_of].view(pool.dtype) if pool.element_size() == 1 else pool[page_of, slot_of]
    x = x.float()
    return x if scales is None else x * scales[page_of, :, slot_of][..., None]


def _read_plain(s, dtype):
    page = s["case"]["page"]
    row = torch.arange(s["held"], device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["out_start"][1:], row, right=True)
    pos = row - s["out_start"][seq]
    page_of, slot_of = s["pages"][seq, pos // page].long(), (pos % page).long()
    return (_fetch(s["k_pool"], s["k_scale"], page_of, slot_of).to(dtype),
            _fetch(s["v_pool"], s["v_scale"], page_of, slot_of).to(dtype))


def _write_plain(s):
    case = s["case"]
    page, kind = case["page"], case["cache"]
    seq, pos = _place_rows(s)
    turn = s["rope"][pos.long()] if s["rope"] is not None else None
    q = _norm_and_turn(s["q"], s.get("q_norm"), turn, case["interleaved"])
    k = _norm_and_turn(s["k"], s.get("k_norm"), turn, case["interleaved"])
    page_of, slot_of = s["pages"][seq, pos // page].long(), (pos % page).long()
    _store(s["k_pool"], s["k_scale"], k, kind, page_of, slot_of)
    _store(s["v_pool"], s["v_scale"], s["v"].float(), kind, page_of, slot_of)
    return q.to(_q_type(case))


def _q_type(case):
    """The 16-bit type that the attention over this cache takes its queries in."""
    if case["cache"] not in LARGEST:
        return DTYPES[case["cache"]]
    return DTYPES[case["x"]] if case["x"] != "f32" else torch.float16


def _attend_plain(s):
    case = s["case"]
    nh, nkv, hd, page = case["nh"], case["nkv"], case["hd"], case["page"]
    n, group = case["n_seq"], nh // nkv
    j = torch.arange(s["max_kv"], device="cuda")
    page_of, slot_of = s["pages"][:, j // page].long(), (j % page).expand(n, -1)
    k = _fetch(s["k_pool"], s["k_scale"], page_of, slot_of).permute(0, 2, 1, 3)     # [n, nkv, keys, hd]
    v = _fetch(s["v_pool"], s["v_scale"], page_of, slot_of).permute(0, 2, 1, 3)
    i = torch.arange(s["max_q"], device="cuda")
    first, length = s["q_start"][:-1, None], (s["q_start"][1:] - s["q_start"][:-1])[:, None]
    rows = (first + i).clamp(max=s["rows"] - 1).long()
    q = s["q"].float()[rows].view(n, s["max_q"], nkv, group, hd).permute(0, 2, 3, 1, 4)
    scores = torch.matmul(q.reshape(n, nkv, -1, hd), k.transpose(-1, -2)).view(n, nkv, group, s["max_q"], -1)
    scores *= 1 / math.sqrt(hd)
    last = s["kv_len"][:, None] - 1
    if case["causal"]:
        last = torch.minimum(last, s["kv_len"][:, None] - length + i)
    else:
        last = last.expand(n, s["max_q"])
    scores.masked_fill_((j > last[..., None])[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(n, nkv, -1, s["max_kv"]), v).view(n, nkv, group, s["max_q"], hd)
    o = torch.where(total == 0, 0.0, o / total).permute(0, 3, 1, 2, 4).reshape(n, s["max_q"], nh, hd)
    row = torch.arange(s["rows"], device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["q_start"][1:], row, right=True)
    return o[seq, (row - s["q_start"][seq]).long()].to(s["q"].dtype)


def run(s):
    case = s["case"]
    quant = case["cache"] in LARGEST
    if own:
        import qwen2_decoder_forward_gb300 as q2
        if case["op"] == "attend":
            return {"o": q2.paged_attention(s["kv"], s["batch"], s["q"], causal=case["causal"])}
        if case["op"] == "read":
            k, v = q2.paged_read(s["kv"], s["batch"], s["out_start"], s["held"], dtype=DTYPES[case["x"]])
            return {"k": k, "v": v}
        q = q2.paged_write(s["kv"], s["batch"], s["k"], s["v"], q=s["q"], q_dtype=_q_type(case),
                           q_norm=s.get("q_norm"), k_norm=s.get("k_norm"), norm_eps=EPS, rope=s["rope"],
                           interleaved=case["interleaved"])
        if quant:
            k, v = q2.paged_read(s["kv"], s["batch"], s["out_start"], s["held"], dtype=_q_type(case))
            return {"q": q, "k": k, "v": v}
        return {"q": q, "k": s["k_pool"], "v": s["v_pool"]}
    if case["op"] == "attend":
        return {"o": _attend_plain(s)}
    if case["op"] == "read":
        k, v = _read_plain(s, DTYPES[case["x"]])
        return {"k": k, "v": v}
    q = _write_plain(s)
    if quant:
        k, v = _read_plain(s, _q_type(case))
        return {"q": q, "k": k, "v": v}
    return {"q": q, "k": s["k_pool"], "v": s["v_pool"]}


# ---- the definitions in 64 bits, one sequence and head at a time ----------------------------------


def _held64(s, which, seq, length):
    """Positions 0 .. length - 1 of one sequence: [length, nkv, hd]."""
    page = s["case"]["page"]
    pool, scale = s[which + "_pool"], s[which + "_scale"]
    need = -(-length // page)
    ids = s["pages"][seq, :need].tolist()
    values = torch.cat([pool[i:i + 1].to(torch.float32) for i in ids], 0).double()
    if scale is not None:
        values = values * torch.cat([scale[i:i + 1] for i in ids], 0).double().transpose(1, 2)[..., None]
    return values.reshape(need * page, *values.shape[2:])[:length]


def _turn64(x, weight, case, first):
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * weight.double()
    r = case["rotary"]
    if not r:
        return x
    pos = torch.arange(first, first + x.shape[0], device="cuda", dtype=torch.float64)
    out = x.clone()
    for i in range(r // 2):
        angle = pos * 1e6 ** (-2.0 * i / r)
        # The rotation goes by the 32-bit table that the operator is given.
        c, d = angle.cos().float().double()[:, None], angle.sin().float().double()[:, None]
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + r // 2)
        out[..., a] = x[..., a] * c - x[..., b] * d
        out[..., b] = x[..., b] * c + x[..., a] * d
    return out


def _coded64(x, kind):
    """What the 8-bit codes of x stand for."""
    largest = x.abs().amax(-1, keepdim=True)
    unit = torch.where(largest == 0, torch.ones_like(largest), largest / LARGEST[kind])
    y = x / unit
    if kind == "e4m3":
        y = y.float().to(torch.float8_e4m3fn).double()
    else:
        down = torch.floor(y.abs())
        y = torch.sign(y) * (down + (y.abs() - down >= 0.5))
    return y * unit


def exact(case, seed):
    s = prepare(case, seed)
    q_len, kv_len = _lengths(case)
    nh, nkv, hd, page = case["nh"], case["nkv"], case["hd"], case["page"]
    if case["op"] == "read":
        ks, vs = ([_held64(s, w, i, n) for i, n in enumerate(kv_len)] for w in ("k", "v"))
        return {"k": torch.cat(ks), "v": torch.cat(vs)}
    starts = s["q_start"].tolist()
    if case["op"] == "attend":
        out = torch.zeros((s["rows"], nh, hd), dtype=torch.float64, device="cuda")
        for i, (n, m) in enumerate(zip(q_len, kv_len)):
            k, v = _held64(s, "k", i, m), _held64(s, "v", i, m)
            rows = s["q"][starts[i]:starts[i + 1]].double()
            late = torch.arange(m, device="cuda")[None] > torch.arange(n, device="cuda")[:, None] + (m - n)
            for h in range(nh):
                a = rows[:, h] @ k[:, h * nkv // nh].T / math.sqrt(hd)
                if case["causal"]:
                    a = a.masked_fill(late, -math.inf)
                out[starts[i]:starts[i + 1], h] = torch.softmax(a, -1) @ v[:, h * nkv // nh]
        return {"o": out}
    q, k = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda"), []
    for i, (n, m) in enumerate(zip(q_len, kv_len)):
        at = slice(starts[i], starts[i + 1])
        q[at] = _turn64(s["q"][at], s.get("q_norm"), case, m - n)
        k.append(_turn64(s["k"][at], s.get("k_norm"), case, m - n))
    if case["cache"] in LARGEST:
        return {"q": q, "k": _coded64(torch.cat(k), case["cache"]), "v": _coded64(s["v"].double(), case["cache"])}
    k_all, v_all = s["k_pool"].double(), s["v_pool"].double()
    for i, (n, m) in enumerate(zip(q_len, kv_len)):
        table = s["pages"][i].long()
        pos = torch.arange(m - n, m, device="cuda")
        k_all[table[pos // page], pos % page] = k[i]
        v_all[table[pos // page], pos % page] = s["v"][starts[i]:starts[i + 1]].double()
    return {"q": q, "k": k_all, "v": v_all}
