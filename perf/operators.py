"""The KV-cache operators beside the PIVOT indexer, as they are measured: one pass each.

  append    kv_append: new keys and values rotated by position and written into the paged 8-bit
            cache (one power-of-two scale for each block of 16 tokens and head), the queries rotated
  attend    kv_attention: attention of each sequence's newest rows over its cached tokens, whole, or
            the last `window` tokens and the first `sinks`
  select    kv_attention_selected: attention of each row over its own list of positions, as the
            indexer returns it

`own` chooses between the plain torch form of each operator and the library's call.
"""
import math
import random

import torch

own = False

BLOCK = 16            # tokens under one scale
E_MIN, E_MAX = -60, 60  # exponents of a scale
E4M3_MAX = 448.0

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _case(op, name, batch, rows, len_min, len_max, q_heads, kv_heads, d, page, dtype="bf16", ragged=False, pad=0,
          rot=0, interleaved=False, window=0, sinks=0, topk=0):
    c = {"op": op, "batch": batch, "rows": rows, "len_min": len_min, "len_max": len_max, "q_heads": q_heads,
         "kv_heads": kv_heads, "d": d, "page": page, "dtype": dtype, "ragged": ragged, "pad": pad, "rot": rot,
         "interleaved": interleaved, "window": window, "sinks": sinks, "topk": topk}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # a decode step's append: one new token for each sequence, in the middle of its block
        _case("append", "append_decode_b32", 32, 1, 512, 4096, 64, 8, 128, 64, rot=128),
        # drafts of several tokens, fp32, a partial rotation of pairs, small pages, a padded batch
        _case("append", "append_drafts_f32", 64, 4, 16, 2000, 16, 2, 64, 16, dtype="f32", ragged=True, pad=5, rot=32,
              interleaved=True),
        # a prompt of 8192 tokens behind a cached start that ends inside a block
        _case("append", "append_prompt_8192", 1, 8192, 8203, 8203, 64, 8, 128, 64, rot=128),
        # several prompts of different lengths in one call
        _case("append", "append_ragged_prompts", 9, 1900, 1900, 4001, 24, 3, 128, 32, ragged=True, rot=64),
        # one token of one short sequence: latency
        _case("attend", "attend_one_512", 1, 1, 512, 512, 32, 8, 128, 64),
        # the repository's decode batch: 32 sequences of 16K to 200K tokens, the current token and three drafts
        _case("attend", "attend_drafts_b32_16k_200k", 32, 4, 16384, 200000, 32, 2, 128, 64),
        # local layers: the last 1024 tokens and the first 4, many sequences
        _case("attend", "attend_window_sinks_b48", 48, 1, 1, 32768, 64, 8, 64, 16, window=1024, sinks=4),
        # a chunk of a prompt against the cache that already holds it: the second half of 8192 tokens
        _case("attend", "attend_chunk_4096_of_8192", 1, 4096, 8192, 8192, 32, 4, 128, 64),
        # fp32 queries, three heads to a key head, ragged rows, short and empty sequences
        _case("attend", "attend_ragged_f32", 7, 6, 0, 3001, 12, 4, 64, 32, dtype="f32", ragged=True, pad=3),
        # a few rows with short lists, fp32, five heads to a key head
        _case("select", "select_small_f32", 3, 4, 1, 2000, 10, 2, 64, 16, dtype="f32", ragged=True, topk=97),
        # the repository's decode batch with its 2048 selected keys for each row
        _case("select", "select_drafts_b32_k2048", 32, 4, 16384, 200000, 32, 2, 128, 64, topk=2048),
        # a prompt's last 1024 rows of 8192, 2048 keys each
        _case("select", "select_prompt_1024_of_8192", 1, 1024, 8192, 8192, 64, 4, 128, 64, topk=2048),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "select"])
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    group = rng.choice([1, 2, 3, 4, 5, 8, 16])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    batch = _log_int(rng, 1, 48)
    ragged = rng.random() < 0.5
    pad = rng.choice([0, 0, 1, 7])
    if op == "append":
        rows = _log_int(rng, 1, max(1, 8192 // batch))
        cap = max(rows, (1 << 26) // (batch * kv_heads * d))  # values the cache holds in all
        len_max = _log_int(rng, rows, max(rows, min(8192, cap)))
        rot = rng.choice([0, d // 2, d])
        return _case(op, "", batch, rows, rng.choice([rows, len_max]), len_max, group * kv_heads, kv_heads, d, page,
                     dtype, ragged, pad, rot=rot, interleaved=rng.random() < 0.5)
    if op == "attend":
        rows = _log_int(rng, 1, 512 if rng.random() < 0.3 else 8)
        cap = min(200000, (1 << 29) // (batch * kv_heads * d), (1 << 28) // (batch * rows * group * kv_heads))
        len_max = _log_int(rng, rows, max(rows, cap))
        window = rng.choice([0, 0, _log_int(rng, 1, 4096)])
        return _case(op, "", batch, rows, rng.choice([0, len_max // 3, len_max]), len_max, group * kv_heads, kv_heads,
                     d, page, dtype, ragged, pad, window=window, sinks=rng.choice([0, 4, 33]) if window else 0)
    rows = _log_int(rng, 1, 8)
    topk = _log_int(rng, 1, min(2048, max(1, (1 << 28) // (batch * rows * kv_heads * d))))
    len_max = _log_int(rng, max(rows, topk // 2), min(200000, max(4096, (1 << 29) // (batch * kv_heads * d))))
    return _case(op, "", batch, rows, rng.choice([1, len_max // 2, len_max]), len_max, group * kv_heads, kv_heads, d,
                 page, dtype, ragged, pad, topk=topk)


def _shape(c):
    """(new rows, length) of each sequence: a function of the case alone."""
    r = random.Random(str(sorted((k, v) for k, v in c.items() if k != "name")))
    n = [r.randint(1, c["rows"]) if c["ragged"] else c["rows"] for _ in range(c["batch"])]
    lens = [r.randint(c["len_min"], c["len_max"]) for _ in range(c["batch"])]
    if c["batch"] > 1:
        lens[0], lens[-1] = c["len_max"], c["len_min"]
    return n, [max(a, b) if c["len_min"] else b for a, b in zip(n, lens)]


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    f = dict(device="cuda", generator=g)
    n, lens = _shape(c)
    dt, B, hq, hk, d, page = _DTYPES[c["dtype"]], c["batch"], c["q_heads"], c["kv_heads"], c["d"], c["page"]
    rows = sum(n) + c["pad"]
    pages_of = [-(-x // page) for x in lens]
    wide = max(1, max(pages_of)) + 1
    pages = sum(pages_of) + 3
    order = torch.randperm(pages, **f).to(torch.int32)
    table = torch.full((B, wide), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, m in enumerate(pages_of):
        table[b, :m] = order[at:at + m]
        at += m
    s = {"case": c, "n": n, "lens_host": lens, "table": table,
         "off": torch.tensor([sum(n[:i]) for i in range(B + 1)], dtype=torch.int64, device="cuda"),
         "lens": torch.tensor(lens, dtype=torch.int64, device="cuda")}

    def payload():  # blocks as a cache holds them: normal values that use most of e4m3's range
        p = torch.empty((pages, hk, page, d), dtype=torch.float8_e4m3fn, device="cuda")
        step = max(1, (1 << 26) // (hk * page * d))
        for i in range(0, pages, step):
            m = min(step, pages - i)
            p[i:i + m] = (torch.randn((m, hk, page, d), **f) * 110.0).clamp_(-E4M3_MAX, E4M3_MAX)
        return p

    s["k"], s["v"] = payload(), payload()
    s["k_exp"], s["v_exp"] = (torch.randint(-8, -5, (pages, hk, page // BLOCK), dtype=torch.int8, **f) for _ in "kv")
    s["q"] = torch.randn((rows, hq, d), **f).to(dt)
    if c["op"] == "append":
        # keys with a few large channels, as rotated keys have them; values of mixed size from token to token
        big = 1.0 + 7.0 * (torch.rand((1, hk, d), **f) < 0.05)
        s["new_k"] = (torch.randn((rows, hk, d), **f) * big).to(dt)
        s["new_v"] = (torch.randn((rows, hk, d), **f) * torch.exp(torch.randn((rows, 1, 1), **f))).to(dt)
        s["q_out"] = torch.zeros((rows, hq, d), dtype=dt, device="cuda")
        s["cos"] = s["sin"] = None
        if c["rot"]:
            inv = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda") / c["rot"])
            a = torch.arange(wide * page, dtype=torch.float64, device="cuda")[:, None] * inv
            s["cos"], s["sin"] = a.cos().float(), a.sin().float()
    else:
        s["out"] = torch.zeros((rows, hq, d), dtype=dt, device="cuda")
        s["lse"] = torch.zeros((rows, hq), dtype=torch.float32, device="cuda")
    if c["op"] == "select":
        idx = torch.full((rows, c["topk"]), -1, dtype=torch.int32, device="cuda")
        r = 0
        for b in range(B):  # each row: that many different positions up to its own, then -1
            pos = torch.arange(lens[b] - n[b], lens[b], device="cuda")[:, None]
            score = torch.rand((n[b], lens[b]), **f)
            score.masked_fill_(torch.arange(lens[b], device="cuda") > pos, -1.0)
            top = score.topk(min(c["topk"], lens[b]), dim=1)
            idx[r:r + n[b], :top.indices.shape[1]] = torch.where(top.values >= 0, top.indices, -1).to(torch.int32)
            r += n[b]
        s["indices"] = idx
    if own:
        import top_token_selection_proxy_b200 as P

        s["cache"] = P.KVCache(s["k"], s["v"], s["k_exp"], s["v_exp"])
    return s


# ---------------------------------------------------------------- plain forms


def _rows_of(s):
    """(sequence, position) of each row that belongs to a sequence."""
    total = sum(s["n"])
    r = torch.arange(total, device="cuda")
    seq = torch.searchsorted(s["off"][1:], r, right=True)
    return seq, s["lens"][seq] - s["off"][seq + 1] + r


def _rotate(x, cos, sin, interleaved):
    """x [rows, heads, d] in 64 bits; cos, sin [rows, rot/2]."""
    half = cos.shape[1]
    c, t = cos[:, None, :], sin[:, None, :]
    y = x.clone()
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    u, w = a * c - b * t, b * c + a * t
    if interleaved:
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = u, w
    else:
        y[..., :half], y[..., half:2 * half] = u, w
    return y


def _pow2(e):
    """2^e in 64 bits, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3(x):
    """x (64 bits) rounded to nearest even in e4m3."""
    ulp = _pow2(torch.frexp(x)[1].clamp(min=-5) - 4)
    return (torch.round(x / ulp) * ulp).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float32).to(torch.float8_e4m3fn)


def _exponent(amax):
    """The least e with amax <= 448 * 2^e, within its range."""
    m, e = torch.frexp(amax / E4M3_MAX)
    return torch.where(amax > 0, e - (m == 0.5).to(e.dtype), E_MIN).clamp(E_MIN, E_MAX)


def _append_one(s, new, cache, exps):
    c = s["case"]
    pages, hk, page, d = cache.shape
    seq, pos = _rows_of(s)
    slot = (s["table"][seq, pos // page].long() * (page // BLOCK) + pos % page // BLOCK)
    blocks = pages * (page // BLOCK)
    amax = torch.zeros((blocks, hk), dtype=torch.float64, device="cuda")
    amax.scatter_reduce_(0, slot[:, None].expand(-1, hk), new.abs().amax(2), "amax")
    fresh = torch.zeros(blocks, dtype=torch.bool, device="cuda").index_fill_(0, slot, True)
    old = exps.permute(0, 2, 1).reshape(blocks, hk).int()
    first = s["lens"] - (s["off"][1:] - s["off"][:-1])
    held = (first % BLOCK > 0) & (s["off"][1:] > s["off"][:-1])
    head = (s["table"].gather(1, (first // page)[:, None])[:, 0].long() * (page // BLOCK) + first % page // BLOCK)
    mixed = torch.zeros(blocks, dtype=torch.int32, device="cuda").index_add_(0, head.clamp(min=0), held.int()) > 0
    e = _exponent(amax)
    e = torch.where(mixed[:, None], torch.maximum(e, old), e)
    e = torch.where(fresh[:, None], e, old)
    # the tokens that the blocks of the first new tokens held before
    where = torch.arange(BLOCK, device="cuda")
    h = head.clamp(min=0)
    p, o = h // (page // BLOCK), (h % (page // BLOCK) * BLOCK)[:, None] + where
    rows = cache.view(torch.uint8)[p[:, None], :, o]  # [batch, BLOCK, hk, d]
    again = rows.view(torch.float8_e4m3fn).double() * _pow2(old[h] - e[h])[:, None, :, None]
    keep = held[:, None] & (where < (first % BLOCK)[:, None])
    value = torch.where(keep[:, :, None, None], _e4m3(again).view(torch.uint8), rows)
    live = held.nonzero()[:, 0]
    cache.view(torch.uint8)[p[live][:, None], :, o[live]] = value[live]
    y = _e4m3(new * _pow2(-e[slot])[:, :, None])
    cache.view(torch.uint8)[s["table"][seq, pos // page].long(), :, pos % page] = y.view(torch.uint8)
    exps.copy_(e.view(pages, page // BLOCK, hk).permute(0, 2, 1))


def _plain_append(s):
    c, total = s["case"], sum(s["n"])
    _, pos = _rows_of(s)
    q, k, v = (s[x][:total].double() for x in ("q", "new_k", "new_v"))
    if c["rot"]:
        cos, sin = s["cos"][pos].double(), s["sin"][pos].double()
        q, k = _rotate(q, cos, sin, c["interleaved"]), _rotate(k, cos, sin, c["interleaved"])
    _append_one(s, k, s["k"], s["k_exp"])
    _append_one(s, v, s["v"], s["v_exp"])
    s["q_out"][:total] = q.to(s["q"].dtype)
    return {"q": s["q_out"], "k": s["k"], "v": s["v"], "k_exp": s["k_exp"], "v_exp": s["v_exp"]}


def _gathered(s, x, exps, pages):
    """[batch, hk, tokens, d] in 32 bits: the pages of each sequence one behind another."""
    x = x.view(torch.uint8)[pages].view(torch.float8_e4m3fn).float()
    x *= _pow2(exps[pages]).float().repeat_interleave(BLOCK, 3)[..., None]
    b, m, hk, page, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(b, hk, m * page, d)


def _softmax(score, seen):
    """(weights that sum to one, their log-sum-exp); a row that sees nothing has no weight."""
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top.clamp(min=torch.finfo(score.dtype).min))
    total = p.sum(-1, keepdim=True)
    return p / total.clamp(min=torch.finfo(score.dtype).tiny), (top + torch.log(total))[..., 0]


def _plain_attend(s):
    c = s["case"]
    B, hq, hk, d = c["batch"], c["q_heads"], c["kv_heads"], c["d"]
    total, most = sum(s["n"]), max(s["n"])
    seq, pos = _rows_of(s)
    at = torch.arange(total, device="cuda") - s["off"][seq]
    pages = s["table"].long().clamp(min=0)
    k, v = _gathered(s, s["k"], s["k_exp"], pages), _gathered(s, s["v"], s["v_exp"], pages)
    q = torch.zeros((B, most, hq, d), device="cuda")
    q[seq, at] = s["q"][:total].float()
    where = torch.full((B, most), -1, device="cuda")
    where[seq, at] = pos
    t = torch.arange(k.shape[2], device="cuda")
    seen = (t <= where[..., None]) & (s["table"] >= 0).repeat_interleave(c["page"], 1)[:, None]
    if c["window"]:
        seen &= (t > where[..., None] - c["window"]) | (t < c["sinks"])
    q = q.view(B, most, hk, hq // hk, d).permute(0, 2, 1, 3, 4).reshape(B, hk, -1, d)
    score = (torch.matmul(q, k.transpose(2, 3)) * d ** -0.5).view(B, hk, most, hq // hk, -1)
    p, lse = _softmax(score, seen[:, None, :, None])
    o = torch.matmul(p.view(B, hk, -1, k.shape[2]), v).view(B, hk, most, hq // hk, d)
    s["out"][:total] = o.permute(0, 2, 1, 3, 4).reshape(B, most, hq, d)[seq, at].to(s["out"].dtype)
    s["lse"][:total] = lse.permute(0, 2, 1, 3).reshape(B, most, hq)[seq, at]
    return {"out": s["out"], "lse": s["lse"]}


def _plain_select(s):
    c, total = s["case"], sum(s["n"])
    hq, hk, d, page = c["q_heads"], c["kv_heads"], c["d"], c["page"]
    seq, pos = _rows_of(s)
    idx = s["indices"][:total].long()
    seen = (idx >= 0) & (idx <= pos[:, None])
    t = torch.where(seen, idx, 0)
    page_of = s["table"][seq[:, None], t // page].long()
    seen &= page_of >= 0
    page_of = page_of.clamp(min=0)

    def rows(x, exps):  # [rows, topk, hk, d] in 32 bits
        y = x.view(torch.uint8)[page_of, :, t % page].view(torch.float8_e4m3fn).float()
        return y.mul_(_pow2(exps[page_of, :, t % page // BLOCK]).float()[..., None])

    q = s["q"][:total].float().view(total, hk, hq // hk, d)
    score = torch.matmul(q, rows(s["k"], s["k_exp"]).permute(0, 2, 3, 1)) * d ** -0.5
    p, lse = _softmax(score, seen[:, None, None])
    o = torch.matmul(p, rows(s["v"], s["v_exp"]).permute(0, 2, 1, 3))
    s["out"][:total] = o.reshape(total, hq, d).to(s["out"].dtype)
    s["lse"][:total] = lse.reshape(total, hq)
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------- the library's calls


def _own_append(s):
    import top_token_selection_proxy_b200 as P

    P.kv_append(s["cache"], s["new_k"], s["new_v"], s["table"], s["off"], s["lens"], cos=s["cos"], sin=s["sin"],
                interleaved=s["case"]["interleaved"], q=s["q"], q_out=s["q_out"])
    return {"q": s["q_out"], "k": s["k"], "v": s["v"], "k_exp": s["k_exp"], "v_exp": s["v_exp"]}


def _own_attend(s):
    import top_token_selection_proxy_b200 as P

    out, lse = P.kv_attention(s["q"], s["cache"], s["table"], s["off"], s["lens"], window=s["case"]["window"],
                              sinks=s["case"]["sinks"], lse=s["lse"], out=s["out"])
    return {"out": out, "lse": lse}


def _own_select(s):
    import top_token_selection_proxy_b200 as P

    out, lse = P.kv_attention_selected(s["q"], s["cache"], s["indices"], s["table"], s["off"], s["lens"],
                                       lse=s["lse"], out=s["out"])
    return {"out": out, "lse": lse}


def run(s):
    op = s["case"]["op"]
    if op == "append":
        return _own_append(s) if own else _plain_append(s)
    if op == "attend":
        return _own_attend(s) if own else _plain_attend(s)
    return _own_select(s) if own else _plain_select(s)


# ---------------------------------------------------------------- work and the definition in 64 bits


def _visible(c, pos):
    """How many tokens the row at `pos` sees."""
    if pos < 0:
        return 0
    if not c["window"] or c["window"] > pos:
        return pos + 1
    return c["window"] + min(c["sinks"], pos + 1 - c["window"])


def work(c):
    n, lens = _shape(c)
    size, hq, hk, d = (2 if c["dtype"] == "bf16" else 4), c["q_heads"], c["kv_heads"], c["d"]
    rows = sum(n)
    if c["op"] == "append":
        moved = rows * hk * d * (2 * size + 2) + rows * hq * d * 2 * size + rows * c["rot"] * 4
        return {"bytes": moved, "flops": rows * (hq + hk) * c["rot"] * 3 + rows * hk * d * 4}
    seen = keys = 0
    for a, m in zip(n, lens):
        each = [min(c["topk"], p + 1) if c["op"] == "select" else _visible(c, p) for p in range(max(0, m - a), m)]
        seen += sum(each)
        if c["op"] == "select":
            keys += min(m, sum(each))
        elif not c["window"]:
            keys += m
        else:
            first = max(0, m - a) - c["window"] + 1
            keys += m - max(0, first) + min(c["sinks"], max(0, first))
    moved = keys * hk * (2 * d + 2 / BLOCK) + rows * hq * (2 * d * size + 4) + rows * 4 * c["topk"]
    return {"bytes": moved, "flops": 4 * d * hq * seen}


def _exact_tokens(s, name, b, pos, head):
    """Values of one sequence's positions and head in 64 bits."""
    c = s["case"]
    pg = s["table"][b].long()[pos // c["page"]]
    x = s[name].view(torch.uint8)[pg, head, pos % c["page"]].view(torch.float8_e4m3fn).double()
    return x * _exact_power(s[name + "_exp"][pg, head, pos % c["page"] // BLOCK])[:, None]


def _exact_rows(s):
    """Attention of each sequence and key head by its definition."""
    c = s["case"]
    hq, hk, d = c["q_heads"], c["kv_heads"], c["d"]
    group = hq // hk
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for b, (a, m) in enumerate(zip(s["n"], s["lens_host"])):
        if not m:
            lse[row:row + a] = -math.inf
        for h in range(hk if m else 0):
            heads = slice(h * group, (h + 1) * group)
            if c["op"] == "attend":
                t = torch.arange(m, device="cuda")
                k, v = _exact_tokens(s, "k", b, t, h), _exact_tokens(s, "v", b, t, h)
            step = max(1, (1 << 27) // (m * group)) if c["op"] == "attend" else 1
            for i in range(0, a, step):
                r = range(row + i, row + min(i + step, a))
                pos = torch.tensor([m - a + x - row for x in r], device="cuda")
                if c["op"] == "select":
                    t = s["indices"][r[0]].long()
                    t = t[(t >= 0) & (t <= pos[0])]
                    k, v = _exact_tokens(s, "k", b, t, h), _exact_tokens(s, "v", b, t, h)
                z = torch.einsum("rgd,sd->rgs", s["q"][r[0]:r[-1] + 1, heads].double(), k) / math.sqrt(d)
                hide = t[None] > pos[:, None]
                if c["window"]:
                    hide = hide | ((t[None] <= pos[:, None] - c["window"]) & (t[None] >= c["sinks"]))
                z = z.masked_fill(hide[:, None], -math.inf)
                total = torch.logsumexp(z, 2)
                w = torch.nan_to_num(torch.exp(z - total[..., None]), nan=0.0)
                out[r[0]:r[-1] + 1, heads] = torch.einsum("rgs,sd->rgd", w, v)
                lse[r[0]:r[-1] + 1, heads] = total
        row += a
    return {"out": out, "lse": lse}


def _exact_power(e):
    """2^e of whole numbers, from Python's own."""
    table = torch.tensor([2.0 ** i for i in range(-256, 257)], dtype=torch.float64, device="cuda")
    return table[e.long() + 256]


def _exact_round(x):
    """To the nearest e4m3 value, ties to the even one, by the table of all of them."""
    table = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()  # 0 .. 448
    a = x.abs().clamp(max=E4M3_MAX)
    hi = torch.searchsorted(table, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    below, above = a - table[lo], table[hi] - a
    pick = torch.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    return torch.copysign(table[pick], x)


def _exact_append(s):
    c, page, nb = s["case"], s["case"]["page"], s["case"]["page"] // BLOCK
    got = {"q": torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")}
    new = {}
    pos = torch.cat([torch.arange(m - a, m, device="cuda") for a, m in zip(s["n"], s["lens_host"])])
    for name, src in (("q", "q"), ("k", "new_k"), ("v", "new_v")):
        x = s[src][:len(pos)].double()
        if c["rot"] and name != "v":
            h = c["rot"] // 2
            i = torch.arange(h, device="cuda")
            i, j = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + h)
            z = torch.complex(x[..., i], x[..., j]) * torch.complex(s["cos"].double(), s["sin"].double())[pos][:, None]
            x = x.index_copy(2, i, z.real).index_copy(2, j, z.imag)
        if name == "q":
            got["q"][:len(pos)] = x
        new[name] = x
    for name in "kv":
        got[name], got[name + "_exp"] = s[name].double(), s[name + "_exp"].clone()
        row = 0
        for b, (a, m) in enumerate(zip(s["n"], s["lens_host"])):
            first, p = m - a, m - a
            while p < m:  # one block of the sequence after another
                q = min(m, (p // BLOCK + 1) * BLOCK)
                pg, blk, base = int(s["table"][b, p // page]), p % page // BLOCK, p // BLOCK * BLOCK
                x = new[name][row + p - first:row + q - first]
                top = x.abs().amax((0, 2)).clamp(min=1e-300)
                e = torch.ceil(torch.log2(top / E4M3_MAX)).clamp(E_MIN - 1, E_MAX + 1)
                e = e + (top > E4M3_MAX * _exact_power(e)).double() - (top <= E4M3_MAX * _exact_power(e - 1)).double()
                e = e.clamp(E_MIN, E_MAX)
                if p > base:
                    was = s[name + "_exp"][pg, :, blk].double()
                    e = torch.maximum(e, was)
                    held = got[name][pg, :, base % page:p - base + base % page]
                    held.copy_(_exact_round(held * _exact_power(was - e)[:, None, None]))
                got[name][pg, :, p % page:p % page + q - p] = _exact_round(x.transpose(0, 1) * _exact_power(-e)[:, None, None])
                got[name + "_exp"][pg, :, blk] = e.to(torch.int8)
                p = q
            row += a
    return got


def exact(c, seed):
    global own
    was, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = was
    return _exact_append(s) if c["op"] == "append" else _exact_rows(s)
