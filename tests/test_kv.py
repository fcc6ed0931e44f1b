"""The paged 8-bit key/value cache on the GPU: kv_append, kv_attention and kv_attention_selected against the 64-bit
forms of kv_reference.py, alone and as they are used together with the indexer."""
import math

import numpy as np
import pytest
import torch

import kv_reference as R
import top_token_selection_proxy_b200 as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from top_token_selection_proxy_b200 import build

    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def host(t):
    return None if t is None else t.detach().cpu().double().numpy()


def make_cache(pages, hk, page, d, seed):
    """A cache whose every byte is a finite payload."""
    g = gen(seed)
    pay = [(torch.randn((pages, hk, page, d), device="cuda", generator=g) * 110).clamp(-448, 448)
           .to(torch.float8_e4m3fn) for _ in "kv"]
    exps = [torch.randint(-9, -4, (pages, hk, page // 16), dtype=torch.int8, device="cuda", generator=g)
            for _ in "kv"]
    return P.KVCache(*pay, *exps)


def make_step(lens, new, page, seed, spare=2, wide=1):
    """(block table, row offsets, lens, number of pages): every sequence's pages in random order."""
    need = [-(-n // page) for n in lens]
    order = np.random.default_rng(seed).permutation(sum(need) + spare)
    table = np.full((len(lens), max(1, max(need)) + wide), -1, np.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
    return (torch.from_numpy(table).cuda(), torch.from_numpy(off).cuda(),
            torch.tensor(lens, dtype=torch.int64, device="cuda"), sum(need) + spare)


def angles(n, rot, seed=0):
    a = torch.arange(n, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, rot, 2).double() / rot) + seed
    return a.cos().float().cuda(), a.sin().float().cuda()


def payload(t):
    return t.cpu().view(torch.uint8).numpy()


def close(got, want, tol, what=""):
    got = host(got)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), f"{what}: NaN in other places"
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), f"{what}: infinities differ"
    ok = ~nan & ~inf
    bad = np.abs(got[ok] - want[ok]) > tol[ok]
    worst = np.max(np.abs(got[ok] - want[ok]) / np.maximum(tol[ok], 1e-300)) if ok.any() else 0
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, the worst by {worst:.3g} of its bound"


def check_attention(q, cache, table, off, lens, dtype, scale=None, window=0, sinks=0, indices=None, run=None):
    """A call against the 64-bit form, on rows that belong to a sequence; the other rows stay as they were."""
    rows, hq, d = q.shape
    out = torch.full((rows, hq, d), 77.0, dtype=dtype, device="cuda")
    lse = torch.full((rows, hq), 77.0, device="cuda")
    sc = d ** -0.5 if scale is None else scale
    if run is not None:
        run(out, lse)
    elif indices is None:
        P.kv_attention(q, cache, table, off, lens, scale=scale, window=window, sinks=sinks, lse=lse, out=out)
    else:
        P.kv_attention_selected(q, cache, indices, table, off, lens, scale=scale, lse=lse, out=out)
    torch.cuda.synchronize()
    want, want_lse, tol, lse_tol = R.attention(
        host(q), host(cache.k), host(cache.v), cache.k_exp.cpu().numpy(), cache.v_exp.cpu().numpy(),
        table.cpu().numpy(), off.cpu().tolist(), lens.cpu().tolist(), sc, dtype, window, sinks,
        None if indices is None else indices.cpu().numpy())
    mine = off.cpu().tolist()[-1]
    close(out[:mine], want[:mine], tol[:mine], "out")
    close(lse[:mine], want_lse[:mine], lse_tol[:mine], "lse")
    assert (out[mine:] == 77).all() and (lse[mine:] == 77).all(), "rows behind the last sequence were written"


# ---------------------------------------------------------------- append

APPENDS = [
    # lens, new, hq, hk, d, page, dtype, rot, interleaved, pad
    ([1], [1], 1, 1, 64, 16, "bf16", 64, False, 0),
    ([17], [17], 2, 1, 128, 16, "bf16", 128, False, 0),
    ([5, 16, 33, 64], [1, 1, 1, 1], 8, 2, 128, 64, "bf16", 128, True, 3),
    ([100, 3, 47, 0, 16], [37, 3, 1, 0, 16], 3, 3, 64, 48, "f32", 32, True, 1),
    ([61, 200], [60, 130], 0, 2, 128, 32, "f32", 64, False, 2),
    ([40], [40], 5, 5, 64, 128, "bf16", 0, False, 0),
    ([2, 9], [5, 4], 4, 2, 128, 16, "bf16", 16, False, 0),   # more rows than tokens: the first belong to none
    ([300], [283], 2, 1, 64, 16, "f32", 48, False, 0),
]


def run_append(lens, new, hq, hk, d, page, dtype, rot, interleaved, pad, seed=0, spoil=None):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    table, off, ln, pages = make_step(lens, new, page, seed)
    cache = make_cache(pages, hk, page, d, seed + 1)
    rows = sum(new) + pad
    # q, k and v as slices of one projection
    fused = torch.randn((rows, hq + 2 * hk, d), device="cuda", generator=gen(seed + 2)) * 3
    fused *= torch.exp2(torch.randint(-9, 9, (rows, 1, 1), device="cuda", generator=gen(seed + 3)).float())
    fused = fused.to(dt)
    if spoil is not None:
        spoil(fused)
    q, k, v = fused[:, :hq], fused[:, hq:hq + hk], fused[:, hq + hk:]
    cos, sin = angles(table.shape[1] * page, rot) if rot else (None, None)
    before = {n: payload(getattr(cache, n)).copy() for n in "kv"}
    exps = {n: getattr(cache, n + "_exp").cpu().numpy().astype(np.int64) for n in "kv"}
    pay = {n: host(getattr(cache, n)) for n in "kv"}
    q_out = torch.full((rows, hq, d), 55.0, dtype=dt, device="cuda") if hq else None
    got = P.kv_append(cache, k, v, table, off, ln, cos=cos, sin=sin, interleaved=interleaved,
                      q=q if hq else None, q_out=q_out)
    torch.cuda.synchronize()
    assert got is q_out
    tb, of, le = table.cpu().numpy(), off.cpu().tolist(), ln.cpu().tolist()
    c64, s64 = (host(cos), host(sin)) if rot else (None, None)
    for n, x in (("k", k), ("v", v)):
        old = pay[n].copy()
        exact = R.append(pay[n], exps[n], tb, of, le, host(x), c64 if n == "k" else None, s64, interleaved)
        assert np.array_equal(getattr(cache, n + "_exp").cpu().numpy(), exps[n]), f"{n}: exponents"
        now = host(getattr(cache, n))
        fresh = np.zeros(now.shape, bool)
        for at, (y, du) in exact.items():
            fresh[at] = True
            lo, hi = R.round_e4m3(y - du), R.round_e4m3(y + du)
            ok = (now[at] >= lo) & (now[at] <= hi) | (np.isnan(now[at]) & np.isnan(y))
            assert ok.all(), f"{n} {at}: {now[at][~ok][:3]} for {y[~ok][:3]}"
        same = (now == pay[n]) | (np.isnan(now) & np.isnan(pay[n]))
        assert same[~fresh].all(), f"{n}: tokens held before"
        untouched = ~fresh & ((old == pay[n]) | np.isnan(old))
        assert np.array_equal(payload(getattr(cache, n))[untouched], before[n][untouched])
    if hq:
        x = host(q)
        for r in range(rows):
            hit = [t for t in R.rows_of(of, le, rows) if t[0] == r and t[2] >= 0]
            if not hit:
                assert (q_out[r] == 55).all()
                continue
            y, mag = x[r], np.abs(x[r]) * 0
            if rot:
                y = R.rotate(x[r], c64[hit[0][2]], s64[hit[0][2]], interleaved)
                mag = np.abs(x[r]).max() * 4 * 2.0 ** -24 * np.ones_like(y)
            tol = mag + np.abs(y) * (2.0 ** -8 if dt == torch.bfloat16 else 2.0 ** -24) * 1.01
            close(q_out[r], y, tol, f"q row {r}")
    return cache


@pytest.mark.parametrize("case", APPENDS)
def test_append_matches_the_definition(case):
    run_append(*case)


def test_append_large_prompt_matches_the_definition():
    run_append([1037, 600], [1024, 590], 3, 2, 128, 64, "bf16", 128, False, 0, seed=5)


def test_append_zeros_tiny_huge_and_non_finite_values():
    def spoil(x):
        x[0] = 0
        x[1] = 1e-30
        x[17] = 3e38
        x[18, :, 3] = float("inf")
        x[19, :, 5] = float("nan")
        x[20] = 448.0 * 2.0 ** 3     # at a step between two exponents
        x[36] = 448.0 * 2.0 ** -5

    for dtype in ("bf16", "f32"):
        # unrotated, so that what each value becomes is known; a whole block of zeros at the end
        run_append([70], [70], 0, 2, 64, 16, dtype, 0, False, 0, seed=9, spoil=spoil)

        def zeros(x):
            x.zero_()

        c = run_append([20], [20], 0, 1, 128, 32, dtype, 0, False, 0, seed=9, spoil=zeros)
        assert (c.k[:, :, :].float() == 0).any()


@pytest.mark.parametrize("e", [-20, 0, 7])
def test_append_exponent_at_a_step_after_rotation(e):
    """A rotation by exact angles (cos 1, sin 0, and cos 0, sin 1) of values at, just under and just over
    448 * 2^e: the exponent is the definition's."""
    top = 448.0 * 2.0 ** e
    x = torch.zeros((6, 1, 64), device="cuda")
    for i, t in enumerate((top, np.nextafter(np.float32(top), np.float32(0)),
                           np.nextafter(np.float32(top), np.float32(1e30)))):
        x[i, 0, 7], x[i + 3, 0, 9] = float(t), -float(t)
    cos, sin = torch.ones((96, 32), device="cuda"), torch.zeros((96, 32), device="cuda")
    cos[:, 9], sin[:, 9] = 0, 1
    for row, want in enumerate((e, e, e + 1, e, e, e + 1)):
        cache = P.KVCache.empty(6, 1, 16, 64)
        step = [torch.tensor([[0, 1, 2, 3, 4, 5]], dtype=torch.int32, device="cuda"),
                torch.tensor([0, 1], device="cuda"), torch.tensor([1 + 16 * (row % 3)], device="cuda")]
        P.kv_append(cache, x[row:row + 1], x[row:row + 1], *step, cos=cos, sin=sin)
        assert int(cache.k_exp[row % 3, 0, 0]) == want


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_token_by_token_keeps_scales_and_stays_close_to_one_call(dtype):
    """61 tokens in calls of 1, 2, 3 ... rows: a block's exponent never falls, and equals that of one call; the
    payload is within the roundings that rising scales cost."""
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    hk, d, page, n = 2, 128, 32, 61
    x = torch.randn((n, hk, d), device="cuda", generator=gen(1)) * torch.exp2(torch.arange(n, device="cuda") % 9.0)[:, None, None]
    x = x.to(dt)
    table = torch.tensor([[3, 1, -1]], dtype=torch.int32, device="cuda")
    a, b = P.KVCache.empty(4, hk, page, d), P.KVCache.empty(4, hk, page, d)
    P.kv_append(a, x, x, table, [0, n], [n])
    at, i = 0, 1
    while at < n:
        m = min(i, n - at)
        was = b.k_exp.clone()
        P.kv_append(b, x[at:at + m], x[at:at + m], table, [0, m], [at + m])
        if at % 16:
            assert (b.k_exp[3 if at < 32 else 1, :, at % 32 // 16] >= was[3 if at < 32 else 1, :, at % 32 // 16]).all()
        at, i = at + m, i % 3 + 1
    assert torch.equal(a.k_exp, b.k_exp) and torch.equal(a.v_exp, b.v_exp)
    av, bv = host(a.k), host(b.k)
    # each rise rounds again only what leaves the normal range (steps of 2^-9), at most 9 rises a block
    tol = np.abs(av) * 2.0 ** -3 + 9 * 2.0 ** -10
    assert (np.abs(av - bv) <= tol).all()


def test_append_absent_pages_and_rows_behind_leave_the_cache_alone():
    hk, d, page = 1, 64, 16
    cache = make_cache(4, hk, page, d, 3)
    before = payload(cache.k).copy(), payload(cache.v).copy(), cache.k_exp.clone()
    x = torch.randn((40, hk, d), device="cuda", generator=gen(4))
    table = torch.tensor([[-1, 99, 2]], dtype=torch.int32, device="cuda")
    # positions 0-15 and 16-31 have no page, 32 .. 36 do; rows 37 .. 39 belong to no sequence
    P.kv_append(cache, x, x, table, [0, 37], [37])
    got = payload(cache.k)
    assert np.array_equal(got[[0, 1, 3]], before[0][[0, 1, 3]])
    assert np.array_equal(got[2, :, 5:], before[0][2, :, 5:])
    assert not np.array_equal(got[2, :, :5], before[0][2, :, :5])
    assert torch.equal(cache.k_exp[[0, 1, 3]], before[2][[0, 1, 3]])
    # past the table's width, and lengths that no table holds
    for n in (49, 2 ** 40):
        snap = payload(cache.k).copy()
        P.kv_append(cache, x[:1], x[:1], table, [0, 1], [n])
        assert np.array_equal(payload(cache.k), snap)


def test_append_rotates_q_in_place():
    hk, d, page, n = 1, 128, 16, 30
    table, off, lens, pages = make_step([n], [n], page, 0)
    x = torch.randn((n, 5 + 2 * hk, d), device="cuda", generator=gen(2)).to(torch.bfloat16)
    cos, sin = angles(table.shape[1] * page, 128)
    a, b = make_cache(pages, hk, page, d, 1), make_cache(pages, hk, page, d, 1)
    want = P.kv_append(a, x[:, 5:6], x[:, 6:], table, off, lens, cos=cos, sin=sin, q=x[:, :5])
    keep = x[:, 5:].clone()
    got = P.kv_append(b, x[:, 5:6], x[:, 6:], table, off, lens, cos=cos, sin=sin, q=x[:, :5], q_out=x[:, :5])
    assert torch.equal(got, want) and got.data_ptr() == x.data_ptr() and torch.equal(x[:, 5:], keep)
    assert np.array_equal(payload(a.k), payload(b.k))


# ---------------------------------------------------------------- attention

ATTENDS = [
    # lens, new, hq, hk, d, page, dtype, window, sinks, pad
    ([1], [1], 1, 1, 128, 16, "bf16", 0, 0, 0),
    ([0, 1, 2, 15, 16, 17], [1, 1, 2, 3, 4, 5], 4, 2, 64, 16, "bf16", 0, 0, 2),
    ([63, 64, 65, 129], [1, 1, 1, 1], 8, 1, 128, 64, "bf16", 0, 0, 0),
    ([500, 31], [4, 4], 32, 2, 128, 32, "bf16", 0, 0, 1),          # 64 rows for a key head
    ([700], [7], 10, 2, 128, 64, "f32", 0, 0, 0),
    ([257, 0, 90], [3, 2, 33], 6, 2, 64, 48, "f32", 0, 0, 3),
    ([900, 40], [2, 2], 8, 2, 64, 16, "bf16", 100, 4, 0),
    ([900, 1], [5, 1], 16, 1, 128, 128, "bf16", 1, 0, 0),          # each row sees itself alone
    ([400, 333], [40, 9], 6, 3, 128, 16, "f32", 33, 17, 0),
    ([260], [200], 4, 1, 128, 64, "bf16", 0, 0, 0),                # a chunk of a prompt: 800 rows for a key head
    ([260, 150], [200, 150], 6, 2, 64, 32, "bf16", 70, 3, 0),
    ([333], [333], 8, 1, 128, 16, "bf16", 50, 20, 5),
    ([1000, 3, 129], [130, 3, 128], 16, 1, 128, 64, "bf16", 0, 0, 1),
    ([2100], [1], 4, 4, 128, 64, "bf16", 5000, 4, 0),              # a window longer than the sequence
    ([40], [40], 3, 1, 128, 16, "bf16", 8, 100, 0),                # more sinks than tokens
]


def make_q(rows, hq, d, dtype, seed, factor=2.0):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    return (torch.randn((rows, hq, d), device="cuda", generator=gen(seed)) * factor).to(dt)


@pytest.mark.parametrize("case", ATTENDS)
def test_attention_matches_the_definition(case):
    lens, new, hq, hk, d, page, dtype, window, sinks, pad = case
    table, off, ln, pages = make_step(lens, new, page, 1)
    cache = make_cache(pages, hk, page, d, 2)
    q = make_q(sum(new) + pad, hq, d, dtype, 3)
    check_attention(q, cache, table, off, ln, q.dtype, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group,n", [(1, 1), (5, 1), (16, 1), (16, 4), (3, 50)])
def test_attention_peaked_scores_scales_far_apart_and_strided_rows(dtype, group, n):
    """Scores up to several hundred, blocks whose scales differ by 2^30, q a slice of a wider tensor, a scale of
    its own."""
    lens, hk, d, page = [300, 77], 2, 128, 32
    table, off, ln, pages = make_step(lens, [n, n], page, 4)
    cache = make_cache(pages, hk, page, d, 5)
    cache.v_exp.copy_(torch.randint(-25, 6, cache.v_exp.shape, device="cuda", generator=gen(6)).to(torch.int8))
    cache.k_exp.copy_(torch.randint(-9, -2, cache.k_exp.shape, device="cuda", generator=gen(7)).to(torch.int8))
    wide = make_q(2 * n, hk * group + 3, d, dtype, 8, 6.0)
    check_attention(wide[:, 3:], cache, table, off, ln, wide.dtype, scale=0.21)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new", [1, 5, 90])
def test_attention_ignores_what_masked_places_hold(dtype, new):
    """NaN payloads in every place that no row, or only some rows, may see; exponents of untouched blocks at 127."""
    lens, hk, d, page, group = [210], 1, 128, 32, 4
    table, off, ln, pages = make_step(lens, [new], page, 7)
    cache = make_cache(pages, hk, page, d, 8)
    t = table.cpu().tolist()[0]
    raw = [cache.k.view(torch.uint8), cache.v.view(torch.uint8)]
    used = set(x for x in t if x >= 0)
    for x in raw:
        for pg in range(pages):
            if pg not in used:
                x[pg] = 0x7F
        x[t[6], :, 210 - 192:] = 0xFF  # behind the last token
        x[t[6], :, 209 - 192] = 0x7F   # the last token itself: only the last row sees it
        x[t[1], :, 5] = 0xFF           # outside the window of every row but the first ones
    for pg in range(pages):
        if pg not in used:
            cache.k_exp[pg] = 127
            cache.v_exp[pg] = 127
    table[0, 2] = -1                   # an absent page in the middle
    q = make_q(new, group, d, dtype, 9)
    check_attention(q, cache, table, off, ln, q.dtype)
    check_attention(q, cache, table, off, ln, q.dtype, window=100, sinks=9)
    # NaN in V alone: the weights stay finite, and only the dims that hold NaN are NaN
    for x in (raw[0][t[6]], raw[0][t[1]]):
        x.fill_(0x38)
    raw[1][t[6], :, 209 - 192] = 0x30
    raw[1][t[6], :, 209 - 192, ::3] = 0x7F
    check_attention(q, cache, table, off, ln, q.dtype, window=100, sinks=9)


def test_attention_a_row_of_non_finite_queries_touches_no_other():
    table, off, ln, pages = make_step([130, 20], [3, 2], 16, 1)
    cache = make_cache(pages, 1, 16, 128, 2)
    q = make_q(5, 4, 128, "bf16", 3)
    clean, _ = P.kv_attention(q, cache, table, off, ln)
    q[1, 2] = float("nan")
    got, _ = P.kv_attention(q, cache, table, off, ln)
    assert torch.isnan(got[1, 2]).all()
    keep = torch.ones((5, 4), dtype=torch.bool, device="cuda")
    keep[1, 2] = False
    assert torch.equal(got[keep], clean[keep])


def test_attention_offsets_past_32_bits():
    """Pages more than 2^32 bytes into the cache."""
    hk, page, d = 4, 64, 128
    pages = (1 << 32) // (hk * page * d) + 8
    k, v = (torch.zeros((pages, hk, page, d), dtype=torch.float8_e4m3fn, device="cuda") for _ in "kv")
    exps = [torch.full((pages, hk, page // 16), -7, dtype=torch.int8, device="cuda") for _ in "kv"]
    cache = P.KVCache(k, v, *exps)
    small = make_cache(3, hk, page, d, 3)
    x = make_q(70, hk, d, "bf16", 11)
    q = make_q(70, hk * 2, d, "bf16", 12)
    far = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32, device="cuda")
    near = torch.tensor([[0, 2]], dtype=torch.int32, device="cuda")
    idx = torch.randint(0, 130, (70, 33), dtype=torch.int32, device="cuda", generator=gen(13))
    got = []
    for c, t in ((cache, far), (small, near)):
        P.kv_append(c, x[:58], x[:58], t, [0, 58], [58])  # in order: a block's earlier tokens are those of the cache
        P.kv_append(c, x, x, t, [0, 70], [128])
        got.append(P.kv_attention(q, c, t, [0, 70], [128]) + P.kv_attention_selected(q, c, idx, t, [0, 70], [128]))
        got[-1] += tuple(P.kv_attention(q[:2], c, t, [0, 2], [128]))
    for a, b in zip(*got):
        assert a is None or torch.equal(a, b)


# ---------------------------------------------------------------- selected

SELECTS = [
    # lens, new, hq, hk, d, page, dtype, topk, pad
    ([1], [1], 1, 1, 64, 16, "bf16", 1, 0),
    ([30, 1, 0, 200], [3, 1, 2, 4], 4, 2, 128, 16, "bf16", 7, 1),
    ([900], [5], 16, 1, 128, 64, "bf16", 257, 0),
    ([900, 20], [4, 4], 10, 2, 64, 48, "f32", 64, 2),
    ([600], [9], 40, 2, 128, 32, "bf16", 130, 0),     # 20 heads for a key head
    ([600], [2], 64, 1, 128, 128, "f32", 500, 0),
    ([5000, 3000 + 7], [1, 1], 8, 8, 128, 64, "bf16", 2048, 0),
]


@pytest.mark.parametrize("case", SELECTS)
def test_selected_matches_the_definition(case):
    """Lists in any order with -1 among them, entries behind the row's position and past every length, doubles."""
    lens, new, hq, hk, d, page, dtype, topk, pad = case
    table, off, ln, pages = make_step(lens, new, page, 1)
    cache = make_cache(pages, hk, page, d, 2)
    rows = sum(new) + pad
    q = make_q(rows, hq, d, dtype, 3)
    rng = np.random.default_rng(5)
    idx = np.full((rows, topk + 3), -1, np.int32)
    for r, b, p in R.rows_of(off.cpu().tolist(), lens, rows):
        idx[r] = rng.integers(-2, max(1, p + 3), topk + 3)
        idx[r, 0] = max(p, 0)
        if topk > 2:
            idx[r, 1], idx[r, 2] = 2 ** 31 - 1, -2 ** 31
    wide = torch.from_numpy(idx).cuda()
    check_attention(q, cache, table, off, ln, q.dtype, indices=wide[:, :topk])  # a strided list


def test_selected_empty_lists_give_zero_rows_and_absent_pages_do_not_count():
    table, off, ln, pages = make_step([100], [4], 16, 1)
    table[0, 3] = -1
    cache = make_cache(pages, 2, 16, 64, 2)
    q = make_q(4, 6, 64, "bf16", 3)
    idx = torch.full((4, 20), -1, dtype=torch.int32, device="cuda")
    idx[1, 5] = 50  # on the absent page
    idx[2, :8] = torch.arange(44, 52, dtype=torch.int32)
    idx[3, 19] = 99
    check_attention(q, cache, table, off, ln, q.dtype, indices=idx)


def test_selected_of_every_position_is_attention():
    table, off, ln, pages = make_step([333, 50], [4, 4], 32, 1)
    cache = make_cache(pages, 2, 32, 128, 2)
    for dtype, tol in (("bf16", 2.0 ** -6), ("f32", 2.0 ** -17)):
        q = make_q(8, 8, 128, dtype, 3)
        idx = torch.arange(333, dtype=torch.int32, device="cuda").flip(0).expand(8, 333).contiguous()
        a, la = P.kv_attention(q, cache, table, off, ln, lse=True)
        b, lb = P.kv_attention_selected(q, cache, idx, table, off, ln, lse=True)
        assert (a.float() - b.float()).abs().max() <= tol * a.float().abs().max()
        assert (la - lb).abs().max() <= 2.0 ** -10


def test_selected_ignores_what_unlisted_places_hold():
    table, off, ln, pages = make_step([210], [3], 32, 7)
    cache = make_cache(pages, 1, 32, 128, 8)
    kept = torch.tensor([0, 3, 50, 100, 207], device="cuda")
    for x in (cache.k, cache.v):
        raw, was = x.view(torch.uint8), x.view(torch.uint8).clone()
        raw.fill_(0x7F)
        for s in kept.tolist():
            pg = int(table[0, s // 32])
            raw[pg, :, s % 32] = was[pg, :, s % 32]
    q = make_q(3, 4, 128, "bf16", 9)
    idx = torch.full((3, 9), -1, dtype=torch.int32, device="cuda")
    idx[:, 2:7] = kept.to(torch.int32)
    idx[0, 0] = 209  # behind row 0's position
    check_attention(q, cache, table, off, ln, q.dtype, indices=idx)


# ---------------------------------------------------------------- as a program uses them


def test_decode_step_of_indexer_append_and_attention():
    """A batch of draft groups: the step's keys appended, the indexer's Refine rows over the index keys, attention
    over them; against the 64-bit form of each."""
    from top_token_selection_proxy_b200 import inputs

    g, H, d, topk, c = 4, 64, 128, 64, 128
    lens = [300, 70, 1000]
    rng = np.random.default_rng(3)
    total = sum(lens)
    iq = torch.from_numpy(rng.standard_normal((3 * g, H, d), dtype=np.float32)).cuda().to(torch.bfloat16)
    iw = torch.from_numpy(rng.standard_normal((3 * g, H), dtype=np.float32)).cuda()
    ik = torch.from_numpy(rng.standard_normal((total, d), dtype=np.float32)).cuda().to(torch.bfloat16)
    rows, _, _, _ = P.refine_varlen(iq, iw, ik, np.cumsum([0] + lens), topk, c, g)
    hq, hk, page = 8, 2, 64
    table, off, ln, pages = make_step(lens, [g] * 3, page, 1)
    cache = P.KVCache.empty(pages, hk, page, d)
    cos, sin = angles(table.shape[1] * page, d)
    x = torch.randn((total, hq + 2 * hk, d), device="cuda", generator=gen(1)).to(torch.bfloat16)
    first = torch.tensor([n - g for n in lens], device="cuda")
    starts = np.cumsum([0] + lens)
    old = torch.cat([x[starts[b]:starts[b] + lens[b] - g] for b in range(3)])
    P.kv_append(cache, old[:, hq:hq + hk], old[:, hq + hk:], table, np.cumsum([0] + [n - g for n in lens]), first,
                cos=cos, sin=sin)
    new = torch.cat([x[starts[b] + lens[b] - g:starts[b + 1]] for b in range(3)])
    q = P.kv_append(cache, new[:, hq:hq + hk], new[:, hq + hk:], table, off, ln, cos=cos, sin=sin, q=new[:, :hq])
    check_attention(q, cache, table, off, ln, torch.bfloat16, indices=rows)
    check_attention(q, cache, table, off, ln, torch.bfloat16)
    # Reuse rows of a prompt's range, as the prefill form returns them
    pre, _ = P.reuse(iq.repeat(25, 1, 1), iw.repeat(25, 1), ik[:300].contiguous(), topk, g)
    check_attention(q[:4].repeat(5, 1, 1)[:20], cache, table[:1], torch.tensor([0, 20], device="cuda"), ln[:1],
                    torch.bfloat16, indices=pre[280:300])


def test_calls_on_another_stream_and_captured_calls_follow_the_tensors():
    """A step captured once and replayed with other lengths, tokens and lists; two such graphs replayed on two
    streams at once; and the plain calls on a side stream.  All give what an eager call gives."""
    hq, hk, d, page = 8, 2, 128, 16
    lens = [200, 40, 3]
    table, off, ln, pages = make_step([400, 400, 400], [2, 2, 2], page, 1)
    cos, sin = angles(table.shape[1] * page, d)

    class Step:
        def __init__(self, seed):
            self.cache = make_cache(pages, hk, page, d, seed)
            self.ln = torch.tensor(lens, device="cuda")
            self.x = torch.randn((6, hq + 2 * hk, d), device="cuda", generator=gen(seed)).to(torch.bfloat16)
            self.idx = torch.randint(-1, 200, (6, 50), dtype=torch.int32, device="cuda", generator=gen(seed + 1))

        def __call__(self, stream=None):
            q = P.kv_append(self.cache, self.x[:, hq:hq + hk], self.x[:, hq + hk:], table, off, self.ln, cos=cos,
                            sin=sin, q=self.x[:, :hq], stream=stream)
            a, _ = P.kv_attention(q, self.cache, table, off, self.ln, stream=stream)
            w, _ = P.kv_attention(q, self.cache, table, off, self.ln, window=20, sinks=2, stream=stream)
            s, _ = P.kv_attention_selected(q, self.cache, self.idx, table, off, self.ln, stream=stream)
            return a, w, s

    steps = [Step(3), Step(30)]
    for s in steps:
        s()  # eager once: whatever is set up on first use
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(s())
        graphs.append(g)
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    for trial in range(3):
        for s in steps:
            s.ln.copy_(torch.tensor([390 - trial, 17 + trial, 2 + trial]))
            s.x.copy_(torch.randn(s.x.shape, device="cuda", generator=gen(trial + 50)))
            s.idx.copy_(torch.randint(-1, 300, s.idx.shape, dtype=torch.int32, device="cuda", generator=gen(trial)))
        torch.cuda.synchronize()
        for g, st in zip(graphs, sides):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for s, o in zip(steps, outs):
            want = s()
            with torch.cuda.stream(sides[0]):
                third = s()
            fourth = s(stream=sides[1])
            torch.cuda.synchronize()
            for w, x, y, z in zip(want, o, third, fourth):
                assert torch.equal(w, x) and torch.equal(w, y) and torch.equal(w, z)


def test_results_do_not_change_from_call_to_call():
    table, off, ln, pages = make_step([3001, 500, 64], [3, 3, 3], 64, 1)
    cache = make_cache(pages, 2, 64, 128, 2)
    q = make_q(9, 16, 128, "bf16", 3)
    idx = torch.randint(0, 500, (9, 300), dtype=torch.int32, device="cuda", generator=gen(4))
    a = P.kv_attention(q, cache, table, off, ln, lse=True) + P.kv_attention_selected(q, cache, idx, table, off, ln, lse=True)
    for _ in range(5):
        b = P.kv_attention(q, cache, table, off, ln, lse=True) + P.kv_attention_selected(q, cache, idx, table, off, ln, lse=True)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("d", [64, 128])
def test_attention_fp32_small_weights_keep_their_bits(d):
    """Half of the dims come from tokens of weight 1024.5 * 2^-26 alone: the heavy tokens' values are 0 there.  The weight
    stands between two fp16 values of 4 times it, so that what one of them leaves must not be lost."""
    table, off, ln, pages = make_step([300], [2], 32, 1)
    cache = make_cache(pages, 1, 32, d, 2)
    cache.k_exp.zero_(), cache.v_exp.zero_()
    k, v = cache.k.float().zero_(), cache.v.float().abs()
    for page in table[0, :4].tolist():  # a heavy token in each 32, so that every warp's reference is one's score
        k[page, 0, 3, 0] = 11.0
        v[page, 0, 3, : d // 2], v[page, 0, 3, d // 2:] = 448.0, 0.0
    cache.k.copy_(k.to(cache.k.dtype)), cache.v.copy_(v.to(cache.v.dtype))
    q = torch.zeros((2, 3, d), device="cuda")
    q[..., 0] = math.log(2.0 ** 26 / 1024.5) / 11
    check_attention(q, cache, table, off, ln, q.dtype, scale=1.0)
    idx = torch.arange(300, dtype=torch.int32, device="cuda").flip(0).repeat(2, 1).contiguous()
    check_attention(q, cache, table, off, ln, q.dtype, scale=1.0, indices=idx)


def test_arguments_past_64_bits_and_a_workspace_elsewhere():
    table, off, ln, pages = make_step([200], [3], 32, 1)
    cache = make_cache(pages, 1, 32, 64, 2)
    q = make_q(3, 4, 64, "bf16", 3)
    for far in (2 ** 63 - 1, 2 ** 64 + 1):
        for window in (far, 5):  # either way every row sees all
            check_attention(q, cache, table, off, ln, q.dtype, run=lambda out, lse: P.kv_attention(
                q, cache, table, off, ln, window=window, sinks=far, out=out, lse=lse))
    with pytest.raises(ValueError, match="workspace"):
        P.kv_attention(q, cache, table, off, ln, ws=P.Workspace("cpu"))
    with pytest.raises(P.PivotError):
        P.kv_attention(q, cache, table, off, ln, out=q)


def test_calls_without_rows_and_host_offsets():
    cache = make_cache(3, 2, 16, 64, 1)
    table = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    none = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = P.kv_attention(none, cache, table, [0, 0], [5], lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    assert P.kv_append(cache, none[:, :2], none[:, :2], table, [0, 0], [5], q=none).shape == (0, 4, 64)
    off = P.DeviceOffsets([0, 2], "cuda")
    lens = P.DeviceOffsets([20], "cuda")
    q = make_q(2, 4, 64, "bf16", 2)
    a, _ = P.kv_attention(q, cache, table, off, lens)
    b, _ = P.kv_attention(q, cache, table, [0, 2], [20], ws=P.Workspace("cuda"))
    assert torch.equal(a, b)


# ---------------------------------------------------------------- calls large enough for the tcgen05 kernel
# (more than 16 query rows for a key head on average, d = 128, bf16, and a table whose capacity promises enough work:
# the sequences themselves may be short)

WIDE = [
    # lens, new, hq, hk, page, window, sinks, pad
    ([1], [1], 17, 1, 16, 0, 0, 0),
    ([0, 1, 128, 129], [5, 5, 5, 5], 5, 1, 64, 0, 0, 2),            # the first rows of the first two belong to none
    ([127, 400], [7, 3], 48, 2, 48, 0, 0, 0),
    ([700], [300], 6, 2, 16, 0, 0, 1),                              # 900 rows for a key head: 8 items
    ([515, 260], [515, 260], 3, 1, 128, 0, 0, 0),                   # whole prompts
    ([900, 333], [90, 40], 4, 1, 32, 200, 5, 0),
    ([650], [400], 5, 1, 64, 1, 0, 0),                              # each row sees itself alone
    ([650, 1], [400, 1], 2, 1, 16, 129, 300, 3),                    # more first tokens than the window has
    ([1300], [20], 16, 1, 64, 100000, 4, 0),
    ([40, 30], [40, 30], 1, 1, 16, 8, 3, 0),
]


def wide_step(lens, new, hq, hk, page, seed):
    """make_step with room for 200,000 tokens a sequence, as a slice of a wider table."""
    table, off, ln, pages = make_step(lens, new, page, seed)
    wide = torch.full((len(lens), 200_000 // page + 7), -1, dtype=torch.int32, device="cuda")
    wide[:, 3:3 + table.shape[1]] = table
    return wide[:, 3:], off, ln, pages


@pytest.mark.parametrize("scale", [None, -0.21, 0.0])
@pytest.mark.parametrize("case", WIDE)
def test_attention_of_many_rows_matches_the_definition(case, scale):
    lens, new, hq, hk, page, window, sinks, pad = case
    table, off, ln, pages = wide_step(lens, new, hq, hk, page, 1)
    cache = make_cache(pages, hk, page, 128, 2)
    q = make_q(sum(new) + pad, hq + 1, 128, "bf16", 3)[:, 1:]
    ws = P.Workspace("cuda")

    def run(out, lse):
        P.kv_attention(q, cache, table, off, ln, scale=scale, window=window, sinks=sinks, lse=lse, out=out, ws=ws)
        assert P.last_device_status(ws) == 0

    check_attention(q, cache, table, off, ln, q.dtype, scale=scale, window=window, sinks=sinks, run=run)


@pytest.mark.parametrize("new,group", [(5, 16), (90, 4)])
def test_attention_of_many_rows_peaked_scores_and_scales_far_apart(new, group):
    """Rows whose largest score comes late and high: the rows' reference has to follow it."""
    lens, hk, page = [900, 300], 2, 32
    table, off, ln, pages = wide_step(lens, [new, new], hk * group, hk, page, 4)
    cache = make_cache(pages, hk, page, 128, 5)
    cache.v_exp.copy_(torch.randint(-25, 6, cache.v_exp.shape, device="cuda", generator=gen(6)).to(torch.int8))
    # scores grow along the sequence
    tab = table.cpu().numpy()
    for b, n in enumerate(lens):
        for s in range(0, n, 16):
            cache.k_exp[tab[b, s // page], :, s % page // 16] = -12 + s * 9 // n
    q = make_q(2 * new, hk * group, 128, "bf16", 8, 4.0)
    check_attention(q, cache, table, off, ln, q.dtype, scale=0.21)


@pytest.mark.parametrize("new", [20, 90])
def test_attention_of_many_rows_ignores_what_masked_places_hold(new):
    """As for few rows: NaN payloads where no row, or only some rows, may look."""
    lens, hk, page, group = [210], 1, 32, 4
    table, off, ln, pages = wide_step(lens, [new], group, hk, page, 7)
    cache = make_cache(pages, hk, page, 128, 8)
    t = table.cpu().tolist()[0]
    raw = [cache.k.view(torch.uint8), cache.v.view(torch.uint8)]
    used = set(x for x in t if x >= 0)
    for pg in range(pages):
        if pg not in used:
            for x in raw:
                x[pg] = 0x7F
            cache.k_exp[pg] = 127
            cache.v_exp[pg] = 127
    for x in raw:
        x[t[6], :, 210 - 192:] = 0xFF
    table[0, 2] = -1
    q = make_q(new, group, 128, "bf16", 9)
    check_attention(q, cache, table, off, ln, q.dtype)  # nothing but zeroed places
    for x in raw:
        x[t[6], :, 209 - 192] = 0x7F
        x[t[1], :, 5] = 0xFF
    check_attention(q, cache, table, off, ln, q.dtype)
    check_attention(q, cache, table, off, ln, q.dtype, window=100, sinks=9)
    for x in (raw[0][t[6]], raw[0][t[1]]):
        x.fill_(0x38)
    raw[1][t[6], :, 209 - 192] = 0x30
    raw[1][t[6], :, 209 - 192, ::3] = 0x7F
    check_attention(q, cache, table, off, ln, q.dtype, window=100, sinks=9)


def test_attention_of_many_rows_a_row_of_non_finite_queries_touches_no_other():
    table, off, ln, pages = wide_step([330, 20], [30, 20], 4, 1, 16, 1)
    cache = make_cache(pages, 1, 16, 128, 2)
    q = make_q(50, 4, 128, "bf16", 3)
    clean, _ = P.kv_attention(q, cache, table, off, ln)
    for bad in (float("nan"), float("inf")):
        spoilt = q.clone()
        spoilt[7, 2, 5] = bad
        got, _ = P.kv_attention(spoilt, cache, table, off, ln)
        assert torch.isnan(got[7, 2]).all()
        keep = torch.ones((50, 4), dtype=torch.bool, device="cuda")
        keep[7, 2] = False
        assert torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 9)])
def test_long_sequences_rows_together_and_alone(window, sinks):
    """Lengths of thousands, where a call's items are cut into many parts: a group of rows in one call (tcgen05) and
    each row in a call of its own (the few-row kernel) agree within their roundings, and so do ragged lengths."""
    lens, n, hq, hk, page = [20_011, 1, 7_000, 130], 4, 16, 2, 64
    table, off, ln, pages = make_step(lens, [n if x >= n else 1 for x in lens], page, 1)
    cache = make_cache(pages, hk, page, 128, 2)
    rows = int(off[-1])
    q = make_q(rows, hq, 128, "bf16", 3)
    q32 = q.float()
    together, lse = P.kv_attention(q, cache, table, off, ln, window=window, sinks=sinks, lse=True)
    exact, lse32 = P.kv_attention(q32, cache, table, off, ln, window=window, sinks=sinks, lse=True)
    # A = sum p|v| / sum p <= 448 * 2^-4 of this cache's values; random signs keep the sum's error far below
    assert (together.float() - exact).abs().max() <= 2.0 ** -7 * exact.abs().max() + 2.0 ** -8
    assert (lse - lse32).abs().max() <= 2.0 ** -11 * lse32.abs().max()
    of = off.tolist()
    for b in range(len(lens)):
        for r in range(of[b], of[b + 1]):
            at = torch.tensor([lens[b] - of[b + 1] + r + 1], device="cuda")
            one, one_lse = P.kv_attention(q32[r:r + 1], cache, table[b:b + 1], [0, 1], at, window=window, sinks=sinks,
                                          lse=True)
            assert (one[0] - exact[r]).abs().max() <= 2.0 ** -15 * exact[r].abs().max()
            assert (one_lse[0] - lse32[r]).abs().max() <= 2.0 ** -18 * lse32[r].abs().max()


def test_attention_of_many_rows_weights_that_fall_by_more_than_fp16_holds():
    """Tokens 128 to 159 give the tile's half a reference of -16; token 170, at -3.5, weighs 2^12.5 by it; token 2, at
    7.5, lowers all of that by 2^-23.5.  What is left of token 170, 2^-11, must keep its bits."""
    B, hk = 12, 8  # so many that a CTA takes an item's tiles together
    table, off, ln, pages = wide_step([300] * B, [100] * B, 4 * hk, hk, 64, 1)
    cache = make_cache(pages, hk, 64, 128, 2)
    cache.k_exp.zero_(), cache.v_exp.zero_()
    k, v = torch.zeros(cache.k.shape, device="cuda"), torch.zeros(cache.v.shape, device="cuda")
    k[..., 0] = -16.0
    for s, z, half in ((2, 7.5, 0), (170, -3.5, 1)):
        for page in table[:, s // 64].tolist():
            k[page, :, s % 64, 0] = z
            v[page, :, s % 64, 64 * half:64 * half + 64] = 1.0
    cache.k.copy_(k.to(cache.k.dtype)), cache.v.copy_(v.to(cache.v.dtype))
    q = torch.zeros((B * 100, 4 * hk, 128), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    out, _ = P.kv_attention(q, cache, table, off, ln, scale=math.log(2.0))
    w = 2.0 ** -11 / (1 + 2.0 ** -11 + 298 * 2.0 ** -23.5)
    # the output's rounding, the weight's two, and the scores' and exponentials' errors, which are far smaller
    assert ((out[..., 64:].double() / w - 1).abs() <= 2.0 ** -8 + 2 * 2.0 ** -11 + 2.0 ** -16).all()
    assert ((out[..., :64].double() - 1).abs() <= 2.0 ** -8).all()


@pytest.mark.parametrize("B,length,new,hq,hk,window", [
    (4, 8000, 4, 64, 8, 0),      # items of 32 rows: warps without rows beside one that has them
    (2, 8000, 4, 40, 8, 0),      # of 20
    (1, 9000, 8, 128, 8, 0),     # of 128
    (3, 2000, 300, 32, 2, 256),  # a window; several items a sequence, the last of fewer rows
])
def test_attention_of_many_rows_over_many_tiles_is_right_every_time(B, length, new, hq, hk, window):
    table, off, ln, pages = make_step([length] * B, [new] * B, 64, 1)
    cache = make_cache(pages, hk, 64, 128, 2)
    q = make_q(B * new, hq, 128, "bf16", 3)
    check_attention(q, cache, table, off, ln, q.dtype, window=window)
    want = P.kv_attention(q, cache, table, off, ln, window=window, lse=True)
    for _ in range(20):
        got = P.kv_attention(q, cache, table, off, ln, window=window, lse=True)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attention_of_many_rows_captured_and_on_two_streams():
    hq, hk, page = 16, 1, 16
    table, off, _, pages = wide_step([600, 600], [3, 3], hq, hk, page, 1)
    cache = make_cache(pages, hk, page, 128, 2)
    sets = []
    for s in range(2):
        q = make_q(6, hq, 128, "bf16", 3 + s)
        ln = torch.tensor([300, 20], device="cuda")
        P.kv_attention(q, cache, table, off, ln)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out, _ = P.kv_attention(q, cache, table, off, ln)
        sets.append((q, ln, g, out))
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    for trial in range(3):
        for s, (q, ln, _, _) in enumerate(sets):
            ln.copy_(torch.tensor([600 - 37 * trial, 3 + 100 * s + trial]))
            q.copy_(make_q(6, hq, 128, "bf16", 60 + trial + 7 * s))
        torch.cuda.synchronize()
        for (_, _, g, _), st in zip(sets, sides):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for (q, ln, _, out), st in zip(sets, sides):
            want, _ = P.kv_attention(q, cache, table, off, ln)
            other, _ = P.kv_attention(q, cache, table, off, ln, stream=st)
            torch.cuda.synchronize()
            assert torch.equal(out, want) and torch.equal(other, want)


@pytest.mark.parametrize("scale", [-0.4, 0.0])
def test_attention_of_few_rows_takes_any_scale(scale):
    table, off, ln, pages = make_step([300, 40], [2, 3], 32, 1)
    for d, dtype in ((64, "f32"), (128, "bf16")):
        cache = make_cache(pages, 2, 32, d, 2)
        q = make_q(5, 6, d, dtype, 3)
        check_attention(q, cache, table, off, ln, q.dtype, scale=scale)
        idx = torch.randint(-1, 300, (5, 70), dtype=torch.int32, device="cuda", generator=gen(5))
        check_attention(q, cache, table, off, ln, q.dtype, scale=scale, indices=idx)
