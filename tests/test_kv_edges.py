"""Edges of the key/value cache calls: values that are not finite or leave fp32, arguments at the ends of their types,
caches and queries that a call must not take, and waits that run out."""
import ctypes
import math

import numpy as np
import pytest
import torch

import kv_reference as R
import top_token_selection_proxy_b200 as P
from test_kv import angles, check_attention, gen, host, make_cache, make_q, make_step, payload, wide_step


@pytest.fixture(scope="module", autouse=True)
def _built():
    from top_token_selection_proxy_b200 import build

    build.build()


gpu = pytest.mark.gpu


# ---------------------------------------------------------------- append


def append_bit_for_bit(x, cos, sin, interleaved, rot, page=16):
    """Appends x [tokens, heads, d] as one sequence's keys and values; payload and exponents are the definition's."""
    n, hk, d = x.shape
    table, off, lens, pages = make_step([n], [n], page, 1)
    cache = make_cache(pages, hk, page, d, 2)
    want, exps = host(cache.k), cache.k_exp.cpu().numpy().astype(np.int64)
    P.kv_append(cache, x, x, table, off, lens, cos=cos, sin=sin, interleaved=interleaved)
    c64, s64 = (host(cos), host(sin)) if rot else (None, None)
    with np.errstate(all="ignore"):
        R.append(want, exps, table.cpu().numpy(), [0, n], [n], host(x), c64, s64, interleaved)
    assert np.array_equal(cache.k_exp.cpu().numpy(), exps)
    got = host(cache.k)
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    assert same.all(), f"{(~same).sum()} differ: {got[~same][:4]} for {want[~same][:4]}"
    return cache


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rot", [64, 32])
def test_append_rotated_keys_that_are_not_finite_or_leave_fp32(dtype, interleaved, rot):
    """Infinities stay infinite through the rotation (payload +-448, no part in the scale), NaN stays NaN, and a finite
    pair whose rotated value no fp32 holds counts as the finite value that it is (exponent 60, payload +-448)."""
    x = torch.randn((90, 2, 64), device="cuda", generator=gen(1)).to(dtype)
    inf, nan = float("inf"), float("nan")
    x[1, 0, 3], x[2, 1, 5], x[3, 0, 7] = inf, -inf, nan
    x[20, :, 0:40] = inf                # both of a pair: inf - inf is NaN in one of them
    x[37] = 3e38                        # rotated: 0.2 and 1.4 times that
    x[50, 0] = -3e38
    x[50, 1, 9] = nan                   # beside finite values only
    x[66, 0, 11], x[67, 0, 12] = 3e38, inf
    cos, sin = torch.full((128, rot // 2), 0.8, device="cuda"), torch.full((128, rot // 2), 0.6, device="cuda")
    cos[60:, 5], sin[60:, 5] = 0.0, 1.0
    sin[70:] = -0.6
    append_bit_for_bit(x, cos, sin, interleaved, rot)
    # angles with a gain, as long-context tables have them: both products leave fp32, their difference need not
    x = torch.randn((20, 1, 64), device="cuda", generator=gen(3)).to(dtype)
    x[4], x[18, :, 2] = 3e38, -3e38
    append_bit_for_bit(x, cos * 2, sin * 2.5, interleaved, rot)
    append_bit_for_bit(x, torch.full_like(cos, 1.5), torch.full_like(sin, 1.5), interleaved, rot)


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 128), (128, 48)])
def test_append_rotated_payload_is_the_exact_value_rounded_once(d, rot, dtype, interleaved):
    x = torch.randn((400, 3, d), device="cuda", generator=gen(5))
    x *= torch.exp2(torch.randint(-9, 9, (400, 1, 1), device="cuda", generator=gen(6)).float())
    append_bit_for_bit(x.to(dtype), *angles(26 * 16, rot, 0.3), interleaved, rot)


def beside(points, rng, dtype):
    """(a, b, c, s) with a c - b s just beside each of the points, on both sides: a and b of the rows' type."""
    a, b = (torch.from_numpy(rng.uniform(1, 2, points.shape) * np.abs(points) * f).to(dtype).double().numpy()
            for f in (1.0, 0.7))
    c = rng.uniform(0.3, 1.0, points.shape).astype(np.float32).astype(float)
    s = ((a * c - points) / b).astype(np.float32).astype(float)
    y = a * c - b * s
    s = np.where(np.abs(y - points) < 2.0 ** -45 * np.abs(points), np.nextafter(s.astype(np.float32), np.float32(9)), s)
    return a, b, c, s


def in_fp32(a, b, c, s):
    """The same in plain fp32: product, product, sum; and with the second product fused into the sum."""
    f = np.float32
    p = (a.astype(f) * c.astype(f)).astype(f)
    return p - (b.astype(f) * s.astype(f)).astype(f), (p.astype(float) - b * s).astype(f)


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_rotated_values_beside_e4m3_ties_fall_as_the_exact_ones(dtype, interleaved):
    """Rotated values so near to the middle between two e4m3 values that fp32 arithmetic lands on it or behind it."""
    rng = np.random.default_rng(3)
    n, half = 512, 32
    ties = (rng.integers(8, 16, (n, half)) + 0.5) / 8 * 2.0 ** rng.integers(-4, 5, (n, half))
    a, b, c, s = beside(ties, rng, dtype)
    a[:, -1], b[:, -1], c[:, -1], s[:, -1] = 448.0, 0.0, 1.0, 0.0  # every block's exponent is 0
    exact = a * c - b * s
    wrong = [(R.round_e4m3(y.astype(float)) != R.round_e4m3(exact))[:, :-1].mean() for y in in_fp32(a, b, c, s)]
    assert min(wrong) > 0.05  # what this test is for
    x = np.zeros((n, 1, 64))
    i = np.arange(half)
    x[:, 0, 2 * i if interleaved else i], x[:, 0, 2 * i + 1 if interleaved else i + half] = a, b
    cos, sin = np.ones((n + 16, half)), np.zeros((n + 16, half))
    cos[:n], sin[:n] = c, s
    cache = append_bit_for_bit(torch.from_numpy(x).cuda().to(dtype), torch.from_numpy(cos).float().cuda(),
                               torch.from_numpy(sin).float().cuda(), interleaved, 64)
    assert int((cache.k_exp == 0).sum()) >= n // 16


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_exponent_of_rotated_values_beside_a_step(dtype):
    """Largest values so near to 448 * 2^e, on either side, that fp32 arithmetic cannot tell."""
    rng = np.random.default_rng(4)
    steps = 448.0 * 2.0 ** rng.integers(-20, 20, 256)
    a, b, c, s = beside(steps, rng, dtype)
    exact = a * c - b * s
    assert min(((y > steps) != (exact > steps)).mean() for y in in_fp32(a, b, c, s)) > 0.05
    n = 16 * len(steps)  # a block for each
    x = np.zeros((n, 1, 64))
    cos, sin = np.ones((n + 16, 32)), np.zeros((n + 16, 32))
    at = 16 * np.arange(len(steps)) + rng.integers(0, 16, len(steps))
    x[at, 0, 3], x[at, 0, 35], cos[at, 3] = a, b, c
    sin[at, 3] = s
    # the pair's other value must not be the larger one: its sign and size come from b c + a s
    small = np.abs(b * c + a * s) < 0.9 * steps
    x[at[~small]] = 0.0
    assert small.sum() > 40
    append_bit_for_bit(torch.from_numpy(x).cuda().to(dtype), torch.from_numpy(cos).float().cuda(),
                       torch.from_numpy(sin).float().cuda(), False, 64)


# ---------------------------------------------------------------- attention of many rows: waits that run out


@gpu
@pytest.mark.parametrize("lens", [[1900, 300, 40], [5000]])
def test_attention_of_many_rows_whose_wait_runs_out_ends_and_says_so(lens):
    table, off, ln, pages = wide_step(lens, [30] * len(lens), 8, 2, 64, 1)
    cache = make_cache(pages, 2, 64, 128, 2)
    q = make_q(30 * len(lens), 16, 128, "bf16", 3)
    ws = P.Workspace("cuda")
    want = P.kv_attention(q, cache, table, off, ln, lse=True, ws=ws)
    assert P.last_device_status(ws) == 0
    try:
        P.set_device_timeout_ns(50_000_000)
        P.set_debug_flags(1)
        P.kv_attention(q, cache, table, off, ln, lse=True, ws=ws)
        assert P.last_device_status(ws) == 5  # PIVOT_ERR_DEVICE_TIMEOUT
        # its rows are right all the same, also for a caller who keeps no workspace to ask
        check_attention(q, cache, table, off, ln, q.dtype)
    finally:
        P.set_debug_flags(0)
        P.set_device_timeout_ns(2_000_000_000)
    got = P.kv_attention(q, cache, table, off, ln, lse=True, ws=ws)
    assert P.last_device_status(ws) == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ---------------------------------------------------------------- arguments


def c_attention(q, cache, table, off, lens, window, sinks):
    """pivot_kv_attention itself, with arguments that the binding would have made smaller."""
    out = torch.full(q.shape, 77.0, dtype=q.dtype, device="cuda")
    step, _keep = P._kv_step(cache, table, off, lens, q.shape[0])
    dt = P._KV_TYPES[q.dtype]
    size = P.lib().pivot_kv_workspace_size(q.shape[0], step.B, q.shape[1], cache.kv_heads, cache.d, 0, dt)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    st = P.lib().pivot_kv_attention(cache._ref, ctypes.byref(step), q.data_ptr(), q.stride(0), q.shape[1], dt,
                                    cache.d ** -0.5, window, sinks, out.data_ptr(), None, ws.data_ptr(), size,
                                    torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    return out


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_largest_window_is_no_window(dtype):
    """Also for sequences of more rows than tokens, whose first rows stand at positions below 0."""
    table, off, ln, pages = wide_step([300, 5], [305, 20], 4, 1, 32, 1)  # bf16: the kernel for many rows
    cache = make_cache(pages, 1, 32, 128, 2)
    q = make_q(325, 4, 128, dtype, 3)
    want, _ = P.kv_attention(q, cache, table, off, ln)
    for window in (2 ** 63 - 1, 2 ** 63 - 4, 2 ** 62 + 1):
        for sinks in (0, 2 ** 63 - 1):
            assert torch.equal(c_attention(q, cache, table, off, ln, window, sinks), want)
    # a window with more first tokens than there are
    assert torch.equal(c_attention(q, cache, table, off, ln, 7, 2 ** 63 - 1), want)


def test_a_cache_keeps_the_tensors_that_its_calls_write():
    """The calls go by pointers taken once: an attribute that pointed elsewhere would not be what they write."""
    cache = P.KVCache.__new__(P.KVCache)
    for name in ("k", "v", "k_exp", "v_exp", "device", "num_pages", "kv_heads", "page_size", "d", "_c", "_ref"):
        with pytest.raises(AttributeError):
            setattr(cache, name, torch.zeros(1))
        with pytest.raises(AttributeError):
            delattr(cache, name)
    cache.owner = "a caller's own attribute"
    assert cache.owner and not hasattr(cache, "k")


@gpu
def test_rows_that_require_a_gradient_are_refused():
    table, off, ln, pages = make_step([20], [2], 16, 1)
    cache = make_cache(pages, 2, 16, 64, 2)
    q, k, v = make_q(2, 4, 64, "f32", 3), make_q(2, 2, 64, "f32", 4), make_q(2, 2, 64, "f32", 5)
    idx = torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    before = payload(cache.k).copy()
    want, _ = P.kv_attention(q, cache, table, off, ln)
    grown = q.clone().requires_grad_(True)
    calls = [lambda x: P.kv_attention(x, cache, table, off, ln)[0],
             lambda x: P.kv_attention_selected(x, cache, idx, table, off, ln)[0],
             lambda x: P.kv_append(cache, k, v, table, off, ln, q=x),
             lambda x: P.kv_append(cache, x[:, :2], v, table, off, ln),
             lambda x: P.kv_append(cache, k, x[:, 2:], table, off, ln),
             lambda x: P.kv_attention(q, cache, table, off, ln, out=x)[0],
             lambda x: P.kv_append(cache, k, v, table, off, ln, q=q, q_out=x)]
    for call in calls:
        with pytest.raises(ValueError, match="gradient"):
            call(grown)
    assert np.array_equal(payload(cache.k), before)
    with torch.no_grad():
        assert torch.equal(calls[0](grown), want)
    assert torch.equal(calls[0](grown.detach()), want)


# ---------------------------------------------------------------- attention: values' scales at the ends of their range


@gpu
@pytest.mark.parametrize("heavy", [0, 700, 1400])
@pytest.mark.parametrize("form", ["f32", "bf16", "bf16 d 64", "selected", "cut f32", "many rows", "cut many rows"])
def test_tokens_of_small_values_count_in_the_sum_of_weights(form, heavy):
    """16 tokens with values of 2^60 and more at score 0, all others with values of 2^-60 at score -9 (in units of log 2):
    the others' values do not show beside the heavy ones, but their weights, 2^-9 each, are a sixth of the sum."""
    many, cut = "many" in form, "cut" in form
    d = 64 if form.endswith("64") else 128
    B, hk, group = (1, 1, 4) if cut or not many else (40, 4, 4)
    n = 1600 if not cut else 12_800  # cut: one sequence's tiles shared by many CTAs
    new = (20 if cut else 90) if many else 2
    step = wide_step([n] * B, [new] * B, hk * group, hk, 64, 1) if many else make_step([n] * B, [new] * B, 64, 1)
    table, off, ln, pages = step
    cache = make_cache(pages, hk, 64, d, 2)
    cache.v_exp.fill_(-60), cache.k_exp.zero_()
    k = torch.zeros(cache.k.shape, device="cuda")
    k[..., 0] = -9.0
    at = heavy * n // 1600 // 16 * 16
    for page in table[:, at // 64].tolist():
        cache.v_exp[page, :, at % 64 // 16] = 60
        k[page, :, at % 64:at % 64 + 16, 0] = 0.0
    cache.k.copy_(k.to(cache.k.dtype))
    q = torch.zeros((B * new, hk * group, d), dtype=torch.float32 if "f32" in form else torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    idx = None
    if form == "selected":
        idx = torch.arange(n, dtype=torch.int32, device="cuda").repeat(new, 1).contiguous()
    check_attention(q[:new] if B > 1 else q, cache, table[:1] if B > 1 else table, off[:2] if B > 1 else off,
                    ln[:1] if B > 1 else ln, q.dtype, scale=math.log(2.0), indices=idx)
    if B > 1:  # the batch, whose items are not cut: as the sequence alone
        one = P.kv_attention(q[:new], cache, table[:1], off[:2], ln[:1], scale=math.log(2.0), lse=True)
        for b in range(B):
            assert torch.equal(cache.v_exp[table[b, :n // 64].long()], cache.v_exp[table[0, :n // 64].long()])
        got = P.kv_attention(q, cache, table, off, ln, scale=math.log(2.0), lse=True)
        assert ((got[1].view(B, new, -1) - one[1]).abs() <= 2.0 ** -12).all()  # 1600 additions in fp32


@gpu
def test_attention_of_many_rows_rescaled_weights_are_not_biased():
    """Tokens 0 .. 95 set a tile's reference; token 127 stands 13 + 1 - 0.98 * 2^-11 / ln 2 above it, so that what was
    weighed before is scaled by a factor just below the middle between two fp16 values.  Half of the dims hold the first
    tokens' values alone: on average over many independent values their error is the factor's."""
    B, hk = 4, 8
    table, off, ln, pages = wide_step([228] * B, [100] * B, 4 * hk, hk, 64, 1)
    cache = make_cache(pages, hk, 64, 128, 2)
    cache.k_exp.zero_()
    cache.v_exp.fill_(-8)
    k = torch.zeros(cache.k.shape, device="cuda")
    v = cache.v.float().abs()
    rise = 14 - 0.98 * 2.0 ** -11 / math.log(2.0)
    spread = torch.randint(-14, 1, cache.k.shape[:3], device="cuda", generator=gen(9)).float() / 8  # 0 .. -1.75 rises / 16
    k[..., 0] = spread
    v[..., 64:] = v[..., 64:] + 1.0
    tab = table.cpu().numpy()
    for b in range(B):
        page = lambda s: int(tab[b, s // 64])
        for c in (0, 32, 64):
            k[page(c), :, c % 64, 0] = 0.0     # the largest of the first tokens: the reference
        for s in range(96, 228):
            k[page(s), :, s % 64, 0] = -448.0
            v[page(s), :, s % 64, 64:] = 0.0
        k[page(127), :, 63, 0] = 16.0
    cache.k.copy_(k.to(cache.k.dtype)), cache.v.copy_(v.to(cache.v.dtype))
    q = torch.zeros((B * 100, 4 * hk, 128), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    scale = rise / 16 * math.log(2.0)
    out, _ = P.kv_attention(q, cache, table, off, ln, scale=scale)
    errors = []
    for b in range(B):
        for h in range(hk):
            pages_b = table[b, :4].long()
            kk = (cache.k[pages_b, h].double()).reshape(256, 128)[:128, 0]
            vv = (cache.v[pages_b, h].double() * 2.0 ** -8).reshape(256, 128)[:128]
            p = torch.exp(kk * scale)
            want = (p @ vv / p.sum())[64:]
            errors.append(out[b * 100, 4 * h, 64:].double() / want - 1)
    errors = torch.cat(errors)
    # 2048 roundings to bf16 (2^-9 at most each, evenly spread: 2^-9 / sqrt(3 * 2048) for the mean, four times that here),
    # and the weights' own, 96 to a sum and 32 independent sums (2^-12 / sqrt(3 * 96 * 32) and less)
    assert abs(float(errors.mean())) <= 4 * 2.0 ** -9 / math.sqrt(3 * 2048) + 2.0 ** -18
    assert float(errors.abs().max()) <= 2.0 ** -8 + 2.0 ** -10


@pytest.mark.parametrize("call", ["attend", "select"])
def test_attention_refuses_a_log_sum_over_the_queries_or_the_outputs(call):
    import test_kv_abi as A

    run, lib = getattr(A, call), P.lib()
    rows = 3 * 1024 * 2  # bytes of q, and of out
    far = A.PTR + 2 * rows
    for lse in (A.PTR, A.PTR + rows - 4, A.PTR + rows, A.PTR + 2 * rows - 4):  # q, then out
        assert run(lib, A.cache(), A.step(), q=A.PTR, out=A.PTR + rows, lse=lse) == 1, lse - A.PTR
    for lse in (far - 3 * 8 * 4 + 4, far - 4, far + rows - 4):
        assert run(lib, A.cache(), A.step(), q=A.PTR, out=far, lse=lse) == 1, lse - far


def test_the_largest_cache_that_is_documented_is_taken():
    """num_pages * kv_heads * page_size up to 2^31 - 1, for a page size that does not divide 2^31 too."""
    import test_kv_abi as A

    lib = P.lib()
    for page, heads, pages in ((48, 1, 44_739_242), (16, 1, 134_217_727), (64, 7, 4_793_490), (48, 5, 8_947_848)):
        slots = page * heads * pages
        assert slots < 2 ** 31 <= slots + page * heads
        for more, want in ((0, 0), (1, 2)):
            c = A.cache(page_size=page, kv_heads=heads, num_pages=pages + more)
            none = A.step(rows=0)
            assert A.attend(lib, c, none, hq=heads, qs=1024) == want
            assert A.append(lib, c, none, ks=1024, vs=1024, n_pos=4 * page) == want


# ---------------------------------------------------------------- attention: the precision that pivot.h states


def check_stated_precision(q, cache, table, off, lens, out, query=0.0, indices=None):
    """out of a bf16 call against the definition, with the bounds that pivot.h states and no more: scores in fp32 (d
    products, (d + 8) 2^-24 of sum |q k|; `query` times the row's largest |q| for each element where the query is held
    in two parts), weights rounded to fp16 (2^-11, and 2^-25 of the row's largest p 2^e), fp32 sums, bf16 outputs."""
    d, group = cache.d, q.shape[1] // cache.kv_heads
    pay = {n: host(getattr(cache, n)) for n in "kv"}
    exp = {n: getattr(cache, n + "_exp").cpu().numpy().astype(float) for n in "kv"}
    tab, x, got, scale = table.cpu().numpy(), host(q), host(out), cache.d ** -0.5
    for r, b, p in R.rows_of(off.cpu().tolist(), lens.cpu().tolist(), q.shape[0]):
        s = np.arange(p + 1) if indices is None else indices[r].cpu().numpy().astype(np.int64)
        s = s[(s >= 0) & (s <= p)]
        pg, at = tab[b, s // cache.page_size], s % cache.page_size
        for j in range(q.shape[1]):
            h = j // group
            k = pay["k"][pg, h, at] * 2.0 ** exp["k"][pg, h, at // 16][:, None]
            e = 2.0 ** exp["v"][pg, h, at // 16][:, None]
            v = pay["v"][pg, h, at]
            z = k @ x[r, j] * scale
            w = np.exp(z - z.max())[:, None]
            total = w.sum()
            want = (w * e * v).sum(0) / total
            dz = (np.abs(k) @ np.abs(x[r, j])).max() * (d + 8) * 2.0 ** -24 * scale
            dz += query * np.abs(x[r, j]).max() * np.abs(k).sum(1).max() * scale
            size = (w * e * np.abs(v)).sum(0) / total
            far = 2.0 ** -25 * (w * e).max() * np.abs(v).sum(0) / total
            tol = (2 * dz + 2.0 ** -11 + (len(s) + 16) * 2.0 ** -24) * size + far + 2.0 ** -8 * np.abs(want) * 1.01
            worst = (np.abs(got[r, j] - want) / tol).max()
            assert worst <= 1, f"row {r} head {j}: {worst:.3g} of the bound"


@gpu
@pytest.mark.parametrize("outlier", [1.0, 2.0 ** 11])
@pytest.mark.parametrize("form", ["d 64", "d 128", "selected", "many rows"])
def test_attention_of_bf16_keeps_the_stated_precision(form, outlier):
    """Weights over many orders; and queries whose largest element, met by keys of 0, is 2^11 times the others: one fp16
    holds all of such a query, two e4m3 parts (many rows) hold 2^-17 of its largest."""
    d, hk, group, many = 64 if form == "d 64" else 128, 2, 4, form == "many rows"
    lens, new = [700, 90], [40, 40] if many else [2, 2]
    table, off, ln, pages = (wide_step if many else lambda l, n, _hq, _hk, page, seed: make_step(l, n, page, seed))(
        lens, new, hk * group, hk, 32, 1)
    cache = make_cache(pages, hk, 32, d, 2)
    cache.v_exp.copy_(torch.randint(-14, 1, cache.v_exp.shape, device="cuda", generator=gen(6)).to(torch.int8))
    k = cache.k.float()
    k[..., 5] = 0
    cache.k.copy_(k.to(cache.k.dtype))
    q = make_q(sum(new), hk * group, d, "bf16", 3, 5.0)
    q[..., 5] = 5.0 * outlier
    idx = None
    if form == "selected":
        idx = torch.randint(0, 700, (sum(new), 300), dtype=torch.int32, device="cuda", generator=gen(5))
        out, _ = P.kv_attention_selected(q, cache, idx, table, off, ln)
    else:
        out, _ = P.kv_attention(q, cache, table, off, ln)
    check_stated_precision(q, cache, table, off, ln, out, 2.0 ** -17 if many else 0.0, idx)
