"""Paged key-value cache, without a GPU: what the library and the binding
refuse before anything is enqueued, and the plain implementations that the GPU
tests compare with, against independent statements of the same rules."""
import ctypes
import math

import pytest
import torch

from mixture_value_routing_b200 import _lib, api, build
from tests import _paged as P

FAKE = 4096  # an address that no call below gets to use


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def pages(**kw):
    f = dict(k=FAKE, v=FAKE, dtype=_lib.BF16, num_pages=10, kv_heads=8, page_size=64, k_page_stride=0, v_page_stride=0,
             k_scale=0, v_scale=0)
    f.update(kw)
    return _lib.Pages(**f)


BIG = 1 << 40


def test_workspace_size(lib):
    size = lib.mova_page_workspace_size
    assert size(8, 100, 8, 32) > 0 and size(8, 100, 8, 32) % 256 == 0
    assert size(0, 1, 1, 1) >= 256
    assert size(4096, 100, 8, 32) > 4096 * 8 * 100 * 8
    for bad in ((-1, 1, 1, 1), (1, 0, 1, 1), (1, 1, 0, 1), (1, 1, 1, 0), (4097, 1, 1, 1), (1, 1, 2, 3), (1, 1, 1, 17),
                (4096, 1 << 20, 8, 8)):
        assert size(*bad) == 0, bad


def call_map(lib, **kw):
    a = dict(cached=FAKE, added=FAKE, B=4, table=FAKE, stride=0, max_pages=8, free=FAKE, n_free=5, taken=FAKE, page=64,
             num=10, T=9, lens=FAKE, starts=FAKE, slots=FAKE, positions=FAKE, out=FAKE, ws=FAKE, ws_bytes=256)
    a.update(kw)
    return lib.mova_page_map(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), "INVALID_ARG"), (dict(B=4097), "UNSUPPORTED"), (dict(T=-1), "INVALID_ARG"),
    (dict(n_free=-1), "INVALID_ARG"), (dict(page=48), "UNSUPPORTED"), (dict(page=0), "INVALID_ARG"),
    (dict(page=8), "UNSUPPORTED"), (dict(page=512), "UNSUPPORTED"), (dict(num=0), "INVALID_ARG"),
    (dict(num=1 << 26), "UNSUPPORTED"), (dict(max_pages=0), "INVALID_ARG"), (dict(max_pages=1 << 25), "UNSUPPORTED"),
    (dict(stride=7), "INVALID_ARG"), (dict(cached=None), "INVALID_ARG"), (dict(added=FAKE + 2), "INVALID_ARG"),
    (dict(free=None), "INVALID_ARG"), (dict(taken=None), "INVALID_ARG"), (dict(out=None), "INVALID_ARG"),
    (dict(slots=None), "INVALID_ARG"), (dict(lens=None), "INVALID_ARG"), (dict(starts=None), "INVALID_ARG"),
    (dict(ws=None), "INVALID_ARG"), (dict(ws=FAKE + 16), "INVALID_ARG"), (dict(ws_bytes=255), "INVALID_ARG"),
])
def test_map_refuses(lib, kw, want):
    assert _lib.STATUS_NAMES[call_map(lib, **kw)] == "MOVA_ERR_" + want


PAGES_REFUSED = [
    (dict(dtype=_lib.F16), "UNSUPPORTED"), (dict(dtype=77), "UNSUPPORTED"), (dict(num_pages=0), "INVALID_ARG"),
    (dict(kv_heads=0), "INVALID_ARG"), (dict(page_size=96), "UNSUPPORTED"), (dict(page_size=-64), "INVALID_ARG"),
    (dict(num_pages=1 << 25), "UNSUPPORTED"), (dict(k_page_stride=8 * 64 * 128 - 8), "INVALID_ARG"),
    (dict(k_page_stride=-1), "INVALID_ARG"), (dict(k=FAKE + 8), "INVALID_ARG"), (dict(k=0), "INVALID_ARG"),
    (dict(k_page_stride=8 * 64 * 128 + 4), "INVALID_ARG"), (dict(k_scale=FAKE + 1), "INVALID_ARG"),
]


def call_write(lib, desc, **kw):
    a = dict(k=FAKE, v=FAKE, dt=_lib.BF16, ks=0, vs=0, slots=FAKE, T=3, p=ctypes.addressof(desc), ws=FAKE, ws_bytes=256)
    a.update(kw)
    return lib.mova_page_write(*a.values(), None)


@pytest.mark.parametrize("kw,want", PAGES_REFUSED + [(dict(v=0), "INVALID_ARG"), (dict(v_page_stride=64), "INVALID_ARG")])
def test_write_refuses_pages(lib, kw, want):
    assert _lib.STATUS_NAMES[call_write(lib, pages(**kw))] == "MOVA_ERR_" + want


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), "INVALID_ARG"), (dict(v=FAKE + 8), "INVALID_ARG"), (dict(dt=_lib.F32), "UNSUPPORTED"),
    (dict(dt=_lib.F16), "UNSUPPORTED"), (dict(ks=1023), "INVALID_ARG"), (dict(vs=1028), "INVALID_ARG"),
    (dict(slots=None), "INVALID_ARG"), (dict(T=-1), "INVALID_ARG"), (dict(p=None), "INVALID_ARG"),
    (dict(ws=None), "INVALID_ARG"), (dict(ws_bytes=0), "INVALID_ARG"),
])
def test_write_refuses(lib, kw, want):
    assert _lib.STATUS_NAMES[call_write(lib, pages(), **kw)] == "MOVA_ERR_" + want


def test_no_tokens_or_requests_is_a_no_op(lib):
    before = lib.mova_launch_count()
    assert call_write(lib, pages(), T=0, k=None, v=None, slots=None, ws=None) == _lib.OK
    assert call_bounds(lib, pages(), B=0, ws=None, table=None) == _lib.OK
    assert call_attend(lib, pages(), B=0, ws=None, q=None) == _lib.OK
    assert call_select(lib, pages(), B=0, ws=None, q=None) == _lib.OK
    assert lib.mova_launch_count() == before


def call_bounds(lib, p, **kw):
    a = dict(p=ctypes.addressof(p), table=FAKE, stride=0, max_pages=8, cached=FAKE, lens=FAKE, B=4, lo=FAKE, hi=FAKE,
             ws=FAKE, ws_bytes=256)
    a.update(kw)
    return lib.mova_page_bounds(*a.values(), None)


@pytest.mark.parametrize("kw,want", PAGES_REFUSED)
def test_bounds_refuses_pages(lib, kw, want):
    assert _lib.STATUS_NAMES[call_bounds(lib, pages(**kw))] == "MOVA_ERR_" + want


def call_attend(lib, p, **kw):
    a = dict(q=FAKE, dt=_lib.BF16, qs=0, H=32, p=ctypes.addressof(p), table=FAKE, stride=0, max_pages=8, lens=FAKE, B=4,
             scale=1.0, picked=None, top=0, o=FAKE, lse=None, ws=FAKE, ws_bytes=BIG)
    a.update(kw)
    return lib.mova_page_attend(*a.values(), None)


TABLE_REFUSED = [
    (dict(table=None), "INVALID_ARG"), (dict(lens=None), "INVALID_ARG"), (dict(max_pages=0), "INVALID_ARG"),
    (dict(stride=7), "INVALID_ARG"), (dict(B=-1), "INVALID_ARG"), (dict(B=5000), "UNSUPPORTED"),
    (dict(max_pages=1 << 25), "UNSUPPORTED"), (dict(B=4096, max_pages=1 << 16), "UNSUPPORTED"),
    (dict(ws=None), "INVALID_ARG"), (dict(ws=FAKE + 128), "INVALID_ARG"), (dict(ws_bytes=255), "INVALID_ARG"),
]


@pytest.mark.parametrize("kw,want", TABLE_REFUSED + [(dict(cached=None), "INVALID_ARG"), (dict(lo=None), "INVALID_ARG"),
                                                     (dict(hi=FAKE + 8), "INVALID_ARG")])
def test_bounds_refuses(lib, kw, want):
    assert _lib.STATUS_NAMES[call_bounds(lib, pages(), **kw)] == "MOVA_ERR_" + want


HEADS_REFUSED = [
    (dict(H=0), "INVALID_ARG"), (dict(H=12), "UNSUPPORTED"), (dict(H=136), "UNSUPPORTED"),
    (dict(dt=_lib.F32), "UNSUPPORTED"), (dict(dt=_lib.E4M3), "UNSUPPORTED"), (dict(qs=4095), "INVALID_ARG"),
    (dict(qs=4100), "INVALID_ARG"), (dict(q=None), "INVALID_ARG"), (dict(q=FAKE + 2), "INVALID_ARG"),
]


@pytest.mark.parametrize("kw,want", PAGES_REFUSED + [(dict(v=0), "INVALID_ARG")])
def test_attend_refuses_pages(lib, kw, want):
    assert _lib.STATUS_NAMES[call_attend(lib, pages(**kw))] == "MOVA_ERR_" + want


@pytest.mark.parametrize("kw,want", TABLE_REFUSED + HEADS_REFUSED + [
    (dict(o=None), "INVALID_ARG"), (dict(o=FAKE + 8), "INVALID_ARG"), (dict(lse=FAKE + 2), "INVALID_ARG"),
    (dict(top=3), "INVALID_ARG"), (dict(picked=FAKE), "INVALID_ARG"), (dict(picked=FAKE + 2, top=3), "INVALID_ARG"),
])
def test_attend_refuses(lib, kw, want):
    assert _lib.STATUS_NAMES[call_attend(lib, pages(), **kw)] == "MOVA_ERR_" + want


def call_select(lib, p, **kw):
    a = dict(q=FAKE, dt=_lib.BF16, qs=0, H=32, p=ctypes.addressof(p), lo=FAKE, hi=FAKE, table=FAKE, stride=0,
             max_pages=8, lens=FAKE, B=4, top=3, picked=FAKE, ws=FAKE, ws_bytes=BIG)
    a.update(kw)
    return lib.mova_page_select(*a.values(), None)


@pytest.mark.parametrize("kw,want", TABLE_REFUSED + HEADS_REFUSED + [
    (dict(lo=None), "INVALID_ARG"), (dict(hi=FAKE + 8), "INVALID_ARG"), (dict(picked=None), "INVALID_ARG"),
    (dict(top=0), "INVALID_ARG"), (dict(top=-1), "INVALID_ARG"),
])
def test_select_refuses(lib, kw, want):
    assert _lib.STATUS_NAMES[call_select(lib, pages(k=0, v=0), **kw)] == "MOVA_ERR_" + want


def test_empty_calls_refuse_a_workspace_that_cannot_hold_their_status(lib):
    for ws in (dict(ws=FAKE + 16), dict(ws_bytes=255)):
        assert _lib.STATUS_NAMES[call_write(lib, pages(), T=0, **ws)] == "MOVA_ERR_INVALID_ARG"
        for call in (call_bounds, call_attend, call_select):
            assert _lib.STATUS_NAMES[call(lib, pages(), B=0, **ws)] == "MOVA_ERR_INVALID_ARG"


# ---- The binding ----------------------------------------------------------------

def test_row_stride():
    t = torch.zeros(4, 12, 128)
    assert api._row_stride(t, "t", 12 * 128) == 12 * 128
    assert api._row_stride(t[:, 2:5], "t", 3 * 128) == 12 * 128
    assert api._row_stride(t[:1, 2:5], "t", 3 * 128) == 3 * 128  # one row: its stride says nothing
    assert api._row_stride(t[:, :1], "t", 128) == 12 * 128
    assert api._row_stride(t.view(4, -1)[:, 128:256], "t", 128) == 12 * 128
    for bad, width in ((t[:, ::2], 6 * 128), (t[:, :, :64], 12 * 64), (t, 128), (t[:1].expand(4, 12, 128), 12 * 128),
                       (t.transpose(0, 1), 4 * 128)):
        with pytest.raises(ValueError):
            api._row_stride(bad, "t", width)


def _state(**kw):
    s = P.make("bf16", [70, 3], 2, 4, 16, device="cpu")
    s.update(kw)
    return s


@pytest.fixture
def host(monkeypatch):
    """The binding's own checks with host tensors: a call that passes them all
    ends at the library, which is replaced."""
    class Reached(Exception):
        pass

    class Lib:
        def __getattr__(self, name):
            def call(*a):
                raise Reached(name)
            return call

    monkeypatch.setattr(api, "_elsewhere", lambda t: False)
    monkeypatch.setattr(api, "_page_ws", lambda ws, n, dev: (0, 0, 0))
    monkeypatch.setattr(api, "page_workspace_size", lambda *a: 0)
    monkeypatch.setattr(api._lib, "load", Lib)
    return Reached


def _attend(s, **kw):
    return api.page_attend(s["q"], s["k"], s["v"], s["table"], s["lens"], k_scale=s["ks"], v_scale=s["vs"], **kw)


def test_binding_passes_good_calls(host):
    s = _state()
    picked = torch.zeros(2, 2, 3, dtype=torch.int32)
    lo = torch.zeros(s["k"].shape[0], 2, 128, dtype=torch.bfloat16)
    vec = torch.zeros(2, dtype=torch.int32)
    one = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: _attend(s), lambda: _attend(s, picked=picked, return_lse=True),
                 lambda: api.page_select(s["q"], lo, lo, s["table"], s["lens"], 16, 3),
                 lambda: api.page_bounds(s["k"], s["table"], vec, s["lens"], lo, lo),
                 lambda: api.page_write(torch.zeros(3, 2, 128, dtype=torch.bfloat16),
                                        torch.zeros(3, 256, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32),
                                        s["k"], s["v"]),
                 lambda: api.page_map(vec, vec, s["table"], vec, one, 16, 9, 5, taken_out=one)):
        with pytest.raises(host):
            call()


@pytest.mark.parametrize("kw", [
    dict(q=torch.zeros(2, 8, 64, dtype=torch.bfloat16)), dict(q=torch.zeros(2, 8, 128)),
    dict(q=torch.zeros(3, 8, 128, dtype=torch.bfloat16)), dict(lens=torch.zeros(2)),
    dict(lens=torch.zeros(3, dtype=torch.int32)), dict(table=torch.zeros(2, 5)),
    dict(table=torch.zeros(5, 2, dtype=torch.int32).T), dict(table=torch.zeros(1, 5, dtype=torch.int32).expand(2, 5)),
    dict(k=torch.zeros(9, 2, 16, 128)), dict(k=torch.zeros(9, 16, 2, 128, dtype=torch.bfloat16).transpose(1, 2)),
    dict(k=torch.zeros(9, 2, 16, 128, dtype=torch.float16)), dict(ks=torch.ones(2), vs=torch.ones(2)),
    dict(v=torch.zeros(2, 2, 16, 128, dtype=torch.bfloat16)),
])
def test_binding_refuses(host, kw):
    with pytest.raises(ValueError):
        _attend(_state(**kw))


def test_binding_refuses_more(host):
    s = _state()
    lo = torch.zeros(s["k"].shape[0], 2, 128, dtype=torch.bfloat16)
    vec, one = torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    k = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    i3 = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: _attend(s, picked=torch.zeros(2, 1, 3, dtype=torch.int32)),
                 lambda: _attend(s, picked=torch.zeros(2, 2, 3)),
                 lambda: _attend(s, out=torch.zeros(2, 8, 128)),
                 lambda: api.page_select(s["q"], lo, lo[1:], s["table"], s["lens"], 16, 3),
                 lambda: api.page_select(s["q"], lo.float(), lo.float(), s["table"], s["lens"], 16, 3),
                 lambda: api.page_bounds(s["k"], s["table"], vec, s["lens"], lo, lo.float()),
                 lambda: api.page_bounds(s["k"], s["table"], one, s["lens"], lo, lo),
                 lambda: api.page_write(k, k[:2], i3, s["k"], s["v"]),
                 lambda: api.page_write(k.float(), k.float(), i3, s["k"], s["v"]),
                 lambda: api.page_write(k, k, i3.long(), s["k"], s["v"]),
                 lambda: api.page_write(k[:, :1], k[:, :1], i3, s["k"], s["v"]),
                 lambda: api.page_map(vec, one, s["table"], vec, one, 16, 9, 5),
                 lambda: api.page_map(vec, vec, s["table"], vec, vec, 16, 9, 5),
                 lambda: api.page_map(vec, vec, s["table"][:1], vec, one, 16, 9, 5)):
        with pytest.raises(ValueError):
            call()


def test_calls_run_on_their_tensors_device(monkeypatch):
    """Tensors on another device than the current one: the call is made with
    that device current, so that its stream and workspace are used."""
    seen = []

    class Guard:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            seen.append(self.dev)

        def __exit__(self, *a):
            seen.append("out")

    monkeypatch.setattr(api, "_elsewhere", lambda t: not seen)
    monkeypatch.setattr(api.torch.cuda, "device", Guard)
    s = _state(lens=torch.zeros(9, dtype=torch.int32))
    with pytest.raises(ValueError):
        _attend(s)
    assert seen == [s["q"].device, "out"]


def test_the_value_path_knows_no_8_bit_floats(lib):
    """E4M3 is a type of cache pages alone."""
    assert api.auto_path(100, torch.bfloat16) == "tensor"
    with pytest.raises(KeyError):
        api.auto_path(100, torch.float8_e4m3fn)


def test_packed_pages_are_the_struct():
    p = _lib.Pages(1, 2, 3, 4, 5, 6, 7, 8, 9, 10)
    assert bytes(p) == api._PAGES.pack(1, 2, 3, 4, 5, 6, 7, 8, 9, 10)


# ---- The plain implementations -----------------------------------------------------

def test_e4m3_rounding_agrees_with_torch():
    x = torch.cat([torch.linspace(-500, 500, 20001), torch.logspace(-12, 2, 5000, base=2.0)]).double()
    got = x.float().clamp(-448, 448).to(torch.float8_e4m3fn).double()
    assert torch.equal(P.e4m3(x.float().double()), got)


def test_attend_of_one_token_is_its_value():
    s = P.make("f32", [1, 0, 33], 2, 3, 16, device="cpu")
    o, lse, _, _ = P.attend(s["q"], s["k"], s["v"], s["table"], s["lens"], dtype="f32")
    v = s["v"][s["table"][0, 0], :, 0].double()
    assert torch.equal(o[0], v.repeat_interleave(3, 0))
    assert (o[1] == 0).all() and (lse[1] == -math.inf).all()
    assert torch.isfinite(o).all()  # NaN in places that no token fills


def test_plain_map_by_hand():
    #       grows into a page | new, two pages | no growth needed | refused: too long | padding
    table = [[7, -1, -1], [-1] * 3, [4, -1, -1], [-1] * 3, [-1] * 3]
    got = P.page_map([16, 0, 3, 0, 0], [2, 20, 1, 49, 0], table, [9, 8, 2, 1], 0, 16, 10, 75)
    table, lens, starts, slots, positions, taken, bad = got
    assert table == [[7, 9, -1], [8, 2, -1], [4, -1, -1], [-1] * 3, [-1] * 3]
    assert lens == [18, 20, 4, 0, 0] and starts == [0, 2, 22, 23, 72, 72] and taken == 3 and bad == 3
    assert slots[:3] == [144, 145, 128] and slots[17:19] == [143, 32] and slots[22] == 67
    assert slots[23:] == [-1] * 52 and positions[:3] == [16, 17, 0] and positions[22:24] == [3, -1]
