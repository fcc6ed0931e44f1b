"""Host-side checks of the key/value cache calls: refusals need no GPU, since nothing is launched."""
import ctypes

import pytest
import torch

import top_token_selection_proxy_b200 as P


@pytest.fixture(scope="module")
def lib():
    from top_token_selection_proxy_b200 import build

    build.build()
    return P.lib()


BUF = ctypes.create_string_buffer(1 << 16)
PTR = (ctypes.addressof(BUF) + 255) // 256 * 256


def cache(**kw):
    c = dict(k=PTR, v=PTR, k_exp=PTR, v_exp=PTR, num_pages=4, kv_heads=2, page_size=32, d=128)
    c.update(kw)
    return P._CacheC(**c)


def step(**kw):
    s = dict(block_table=PTR, row_offsets=PTR, lens=PTR, table_stride=4, rows=3, table_width=4, B=2)
    s.update(kw)
    return P._StepC(**s)


def ref(x):
    return None if x is None else ctypes.byref(x)


def append(lib, c, s, **kw):
    a = dict(k=PTR, ks=256, v=PTR, vs=256, dt=P.BF16, cos=PTR, sin=PTR, n_pos=128, rot=128, inter=0, q=None, qs=0, hq=0,
             qo=None, qos=0)
    a.update(kw)
    return lib.pivot_kv_append(ref(c), ref(s), a["k"], a["ks"], a["v"], a["vs"], a["dt"], a["cos"], a["sin"], a["n_pos"],
                               a["rot"], a["inter"], a["q"], a["qs"], a["hq"], a["qo"], a["qos"], None)


def attend(lib, c, s, **kw):
    a = dict(q=PTR, qs=1024, hq=8, dt=P.BF16, scale=0.1, window=0, sinks=0, out=PTR, lse=None, ws=PTR, wsb=1 << 30)
    a.update(kw)
    return lib.pivot_kv_attention(ref(c), ref(s), a["q"], a["qs"], a["hq"], a["dt"], a["scale"], a["window"], a["sinks"],
                                  a["out"], a["lse"], a["ws"], a["wsb"], None)


def select(lib, c, s, **kw):
    a = dict(q=PTR, qs=1024, hq=8, dt=P.BF16, scale=0.1, idx=PTR, ist=5, topk=5, out=PTR, lse=None, ws=PTR, wsb=1 << 30)
    a.update(kw)
    return lib.pivot_kv_attention_selected(ref(c), ref(s), a["q"], a["qs"], a["hq"], a["dt"], a["scale"], a["idx"],
                                           a["ist"], a["topk"], a["out"], a["lse"], a["ws"], a["wsb"], None)


BAD_CACHE = [(dict(k=None), 1), (dict(v_exp=None), 1), (dict(k=PTR + 8), 1), (dict(num_pages=0), 1),
             (dict(kv_heads=0), 1), (dict(page_size=0), 1), (dict(page_size=24), 1), (dict(page_size=-16), 1),
             (dict(d=96), 2), (dict(d=0), 2), (dict(kv_heads=1025), 2), (dict(num_pages=1 << 25, page_size=64), 2)]
BAD_STEP = [(dict(block_table=None), 1), (dict(row_offsets=None), 1), (dict(lens=None), 1), (dict(B=0), 1),
            (dict(rows=-1), 1), (dict(table_width=0), 1), (dict(table_stride=3), 1), (dict(rows=2 ** 31 - 1), 2),
            (dict(table_width=1 << 26, table_stride=1 << 26), 2)]


@pytest.mark.parametrize("call", [append, attend, select])
def test_every_call_refuses_a_bad_cache_or_step(lib, call):
    assert call(lib, None, step()) == 1 and call(lib, cache(), None) == 1
    for kw, want in BAD_CACHE:
        assert call(lib, cache(**kw), step()) == want, kw
    for kw, want in BAD_STEP:
        assert call(lib, cache(), step(**kw)) == want, kw


def test_append_refusals(lib):
    for kw in (dict(k=None), dict(v=None), dict(ks=255), dict(ks=250), dict(vs=260 + 2), dict(k=PTR + 2), dict(dt=2),
               dict(rot=8), dict(rot=144), dict(rot=-16), dict(inter=2), dict(cos=None), dict(sin=PTR + 4),
               dict(n_pos=127), dict(q=PTR, qs=1024, hq=8, qo=None, qos=1024),
               dict(q=PTR, qs=1024, hq=0, qo=PTR, qos=1024), dict(q=PTR, qs=1000, hq=8, qo=PTR, qos=1024),
               dict(q=PTR, qs=1032, hq=8, qo=PTR, qos=1024), dict(q=PTR + 8, qs=1024, hq=8, qo=PTR, qos=1024)):
        assert append(lib, cache(), step(), **kw) == 1, kw
    assert append(lib, cache(), step(rows=0)) == 0  # nothing to do, nothing launched


@pytest.mark.parametrize("call", [attend, select])
def test_attention_refusals(lib, call):
    for kw in (dict(q=None), dict(q=PTR + 8), dict(qs=1000), dict(qs=1028), dict(hq=0), dict(hq=7), dict(dt=5),
               dict(out=None), dict(out=PTR + 8), dict(ws=None), dict(ws=PTR + 16), dict(scale=float("nan")),
               dict(scale=float("inf"))):
        assert call(lib, cache(), step(), **kw) == 1, kw
    assert call(lib, cache(), step(), hq=1026, qs=1026 * 128) == 2
    assert call(lib, cache(), step(), wsb=0) == 3
    assert call(lib, cache(), step(rows=0)) == 0


@pytest.mark.parametrize("call", [attend, select])
def test_attention_refuses_a_scale_past_fp32_and_outputs_over_the_queries(lib, call):
    far = PTR + 3 * 1024 * 2
    assert call(lib, cache(), step(rows=0), out=far, scale=3e38) == 1   # times log2(e) it is infinite
    assert call(lib, cache(), step(rows=0), out=far, scale=2e38) == 0
    for at in (0, 16, 3 * 1024 * 2 - 16):                               # 3 rows of 1024 bf16 values
        assert call(lib, cache(), step(), q=PTR, out=PTR + at) == 1, at
        assert call(lib, cache(), step(), q=PTR + at, out=PTR) == 1, at
    # rows further apart: the last one counts whole
    assert call(lib, cache(), step(), q=PTR, qs=2048, out=PTR + (2 * 2048 + 1024) * 2 - 16) == 1


def test_window_and_list_refusals(lib):
    assert attend(lib, cache(), step(), window=-1) == 1
    assert attend(lib, cache(), step(), sinks=-1) == 1
    for kw in (dict(idx=None), dict(topk=0), dict(topk=-1), dict(ist=4)):
        assert select(lib, cache(), step(), **kw) == 1, kw
    assert select(lib, cache(), step(), topk=65537, ist=65537) == 2


def test_workspace_size(lib):
    size = lib.pivot_kv_workspace_size
    assert size(4, 2, 8, 2, 128, 0, P.BF16) >= 256
    for bad in ((-1, 2, 8, 2, 128, 0, 0), (4, 0, 8, 2, 128, 0, 0), (4, 2, 8, 3, 128, 0, 0), (4, 2, 8, 2, 32, 0, 0),
                (4, 2, 8, 2, 128, -1, 0), (4, 2, 8, 2, 128, 0, 7), (4, 2, 2048, 2, 128, 0, 0),
                (2 ** 31, 2, 8, 2, 128, 0, 0), (4, 2, 8, 2, 128, 65537, 0)):
        assert size(*bad) == 0, bad


def test_binding_refuses_what_is_no_cache():
    k = torch.zeros((2, 1, 16, 64), dtype=torch.float8_e4m3fn)
    e = torch.zeros((2, 1, 1), dtype=torch.int8)
    with pytest.raises(ValueError):
        P.KVCache(k, k, e, e)                              # not on a CUDA device
    with pytest.raises(ValueError):
        P.KVCache(k.view(torch.uint8), k, e, e)            # another type
    with pytest.raises(ValueError):
        P.KVCache(torch.zeros((2, 1, 24, 64), dtype=torch.float8_e4m3fn), k, e, e)
    with pytest.raises(ValueError):
        P.KVCache(k, k, e, torch.zeros((2, 1, 2), dtype=torch.int8))
    with pytest.raises(ValueError):
        P.KVCache(k, k, e, e.int())
