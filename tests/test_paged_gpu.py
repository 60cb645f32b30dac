"""Paged key-value cache on the GPU, against the plain implementations and
bounds of tests/_paged.py."""
import math

import pytest
import torch

from tests import _paged as P

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module")
def api():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from mixture_value_routing_b200 import build
    build.build()
    from mixture_value_routing_b200 import api as A
    return A


def ints(v):
    return torch.tensor(v, dtype=I32, device="cuda")


def ok(api, want=("MOVA_OK", 0)):
    assert api.get_status() == want


# ---- Tables and slots --------------------------------------------------------------

def check_map(api, cached, added, table, free, taken, page, num, T, alias=False, wide=0):
    want = P.page_map(cached, added, table, free, taken, page, num, T)
    t = torch.full((len(table), len(table[0]) + wide if table else 1), -7, dtype=I32, device="cuda")
    if table:
        t[:, :len(table[0])] = ints(table)
    view = t[:, :len(table[0])] if table else t
    tk = ints([taken])
    got = api.page_map(ints(cached), ints(added), view, ints(free), tk, page, num, T, taken_out=tk if alias else None)
    status = api.get_status()
    names = ("lens", "starts", "slots", "positions")
    for name, g, w in zip(names, got, want[1:5]):
        assert g.tolist() == w, name
    assert view.tolist() == want[0] or not table
    assert (t[:, len(table[0]):] == -7).all() if table else True
    assert got[4].tolist() == [want[5]]
    assert tk.tolist() == ([want[5]] if alias else [taken])
    assert status == (("MOVA_OK", 0) if want[6] is None else ("MOVA_ERR_DEVICE_CHECK", want[6]))


def test_map_by_hand(api):
    table = [[7, -1, -1], [-1] * 3, [4, -1, -1], [-1] * 3, [-1] * 3]
    for alias in (False, True):
        check_map(api, [16, 0, 3, 0, 0], [2, 20, 1, 49, 0], table, [9, 8, 2, 1], 0, 16, 10, 75, alias)


@pytest.mark.parametrize("B,page,longest,T_extra,seed", [
    (1, 16, 1, 0, 0), (1, 256, 5000, 3, 1), (7, 16, 100, 0, 2), (64, 64, 40, 9, 3), (300, 32, 200, 100, 4),
    (1025, 16, 3, 0, 5), (4096, 128, 9, 17, 6), (40, 64, 1700, 5, 7),
])
def test_map_random(api, B, page, longest, T_extra, seed):
    g = torch.Generator().manual_seed(seed)
    cached = (torch.randint(0, longest + 1, (B,), generator=g)).tolist()
    added = (torch.randint(0, longest + 1, (B,), generator=g) * (torch.rand(B, generator=g) < 0.8)).tolist()
    width = P.ceil_div(2 * longest, page) + 1
    num = B * width + 20
    order = torch.randperm(num, generator=g).tolist()
    table = [[order.pop() if j < P.ceil_div(c, page) else -1 for j in range(width)] for c in cached]
    check_map(api, cached, added, table, order, 3, page, num, sum(added) + T_extra, alias=seed % 2 == 0, wide=seed)


@pytest.mark.parametrize("what", ["no pages left", "bad taken", "negative taken", "negative counts", "bad old page",
                                  "bad free page", "tokens past T", "outgrows its row", "huge counts"])
def test_map_refusals(api, what):
    cached, added, free, taken, T, num = [5, 16, 0, 30], [3, 1, 40, 2], [1, 2, 3, 4, 5, 6], 0, 60, 10
    table = [[7, -1, -1], [8, -1, -1], [-1] * 3, [9, 0, -1]]
    if what == "no pages left":
        taken = 4  # row 1 takes the fifth; row 2 wants three; row 3 wants none
    elif what == "bad taken":
        taken = 7
    elif what == "negative taken":
        taken = -1
    elif what == "negative counts":
        cached, added = [-5, 16, 0, 30], [3, -1, 40, 2]
    elif what == "bad old page":
        table[0][0] = 10
    elif what == "bad free page":
        free[0] = -1
    elif what == "tokens past T":
        T = 5
    elif what == "outgrows its row":
        added[1] = 40
    else:
        added = [2 ** 31 - 1, 2 ** 31 - 1, 40, 2]
        cached[1] = 2 ** 31 - 1
    check_map(api, cached, added, table, free, taken, 16, num, T)


def test_map_sums_past_32_bits(api):
    """Forty requests of 2^30 tokens each want 40 * 2^26 pages: none has room, and
    none is taken for one that needs no page once the sum has passed 32 bits."""
    B, width = 40, 1 << 26
    table = torch.empty(B, width, dtype=I32, device="cuda")
    added = ints([1 << 30] * (B - 1) + [17])
    lens, starts, slots, positions, taken = api.page_map(ints([0] * B), added, table, ints([3, 4, 5]), ints([1]), 16, 10, 50)
    assert api.get_status() == ("MOVA_ERR_DEVICE_CHECK", 0)
    assert lens.tolist() == [0] * B and taken.tolist() == [1]
    assert starts.tolist() == [0, 1 << 30] + [2 ** 31 - 1] * (B - 1)
    assert slots.tolist() == positions.tolist() == [-1] * 50


def test_map_without_requests_or_tokens(api):
    check_map(api, [], [], [], [1], 0, 16, 10, 5)
    check_map(api, [3], [0], [[1]], [], 0, 16, 10, 0)


# ---- Writing -----------------------------------------------------------------------

def check_write(api, dtype, T, kv, page, seed=0, stride_pages=0, combined=False):
    g = torch.Generator().manual_seed(seed)
    num = P.ceil_div(T, page) + 4
    io, ct = P.IO[dtype], P.CACHE[dtype]
    slots = torch.randperm(num * page, generator=g)[:T].to(I32)
    if T > 2:
        slots[torch.randperm(T, generator=g)[:T // 3]] = -1
    k = torch.randn(T, 3 + kv, 128, generator=g).to(io)[:, 2:2 + kv]
    v = torch.randn(T, kv * 128, generator=g).to(io)
    if T:
        k[0, 0, :6] = torch.tensor([math.nan, math.inf, -math.inf, 1e30, 0.0, -0.0]).to(io)
    ks = 0.01 * (1 + torch.rand(kv, generator=g)) if dtype == "e4m3" else None
    vs = 0.02 * (1 + torch.rand(kv, generator=g)) if dtype == "e4m3" else None
    if combined:  # keys and values of a page side by side in one tensor
        both = torch.randn(num, 2, kv, page, 128, generator=g).to(io).to(ct).cuda()
        kc, vc = both[:, 0], both[:, 1]
    else:
        kc, vc = (torch.randn(num, kv, page, 128, generator=g).to(io).to(ct).cuda() for _ in range(2))
    want = []
    for cache, new, scale in ((kc, k, ks), (vc, v.view(T, kv, 128), vs)):
        w = cache.cpu().clone()
        for t in range(T):
            if slots[t] >= 0:
                x = new[t]
                if scale is not None:
                    x = (x.float() / scale[:, None]).clamp(-448, 448).to(ct)  # IEEE fp32 division; NaN stays
                w[int(slots[t]) // page, :, int(slots[t]) % page] = x
        want.append(w)
    dev = [t.cuda() if t is not None else None for t in (ks, vs)]
    kd = torch.empty(T, 3 + kv, 128, dtype=io, device="cuda")[:, 2:2 + kv].copy_(k)
    api.page_write(kd, v.cuda(), slots.cuda(), kc, vc, *dev)
    ok(api)
    for cache, w in ((kc, want[0]), (vc, want[1])):
        got = cache.cpu()
        bits = torch.uint8 if ct == torch.float8_e4m3fn else (torch.int32 if ct == torch.float32 else torch.int16)
        same = (got.contiguous().view(bits) == w.contiguous().view(bits)) | (got.float().isnan() & w.float().isnan())
        assert same.all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("T,kv,page", [(1, 8, 64), (2, 1, 16), (65, 3, 32), (301, 8, 128), (700, 2, 256), (33, 13, 16)])
def test_write(api, dtype, T, kv, page):
    check_write(api, dtype, T, kv, page, seed=T, combined=T % 2 == 1)


@pytest.mark.parametrize("low,high", [(-126, 126), (-12, 3)])
def test_write_e4m3_divides_exactly(api, low, high):
    """Every bf16 number over scales of many sizes: the stored E4M3 number is that
    of the IEEE fp32 quotient, clamped."""
    kv, page = 8, 64
    every = torch.arange(65536, dtype=torch.int32).to(torch.uint16).view(torch.bfloat16).view(64, kv, 128)
    every = every.repeat(kv, 1, 1)  # each number under each head's scale
    for h in range(kv):
        every[64 * h:64 * h + 64] = every[64 * h:64 * h + 64].roll(h, 1)
    g = torch.Generator().manual_seed(low)
    for _ in range(4):
        scale = (torch.rand(kv, generator=g) + 1) * 2.0 ** torch.randint(low, high, (kv,), generator=g)
        kc, vc = (torch.zeros(8, kv, page, 128).to(torch.float8_e4m3fn).cuda() for _ in range(2))
        dev, ds = every.cuda(), scale.cuda()
        api.page_write(dev, dev, ints(list(range(512))), kc, vc, ds, ds)
        ok(api)
        want = (every.float() / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        got = kc.cpu().transpose(1, 2).reshape(512, kv, 128)
        same = (got.view(torch.uint8) == want.view(torch.uint8)) | (got.float().isnan() & want.float().isnan())
        assert same.all(), (every[~same][:5], scale)


def test_write_reports_bad_slots(api):
    kc, vc = (torch.zeros(3, 2, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k = torch.ones(5, 2, 128, dtype=torch.bfloat16, device="cuda")
    api.page_write(k, k, ints([0, -1, 48, -2, 47]), kc, vc)
    ok(api, ("MOVA_ERR_DEVICE_CHECK", 2))
    for c in (kc, vc):
        assert c.sum().item() == 2 * 2 * 128 and (c[0, :, 0] == 1).all() and (c[2, :, 15] == 1).all()
    api.page_write(k, k, ints([0, 1, 2, 3, 4]), kc, vc)
    ok(api)


# ---- Bounds ------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("lens,cached,kv,page", [
    ([64], [0], 8, 64), ([15, 16, 17, 0, 33], [0, 0, 0, 0, 16], 2, 16), ([1000, 128, 127, 300], [500, 127, 0, 299], 3, 128),
    ([256, 700], [0, 256], 1, 256), ([40] * 70, list(range(70)), 2, 32),
])
def test_bounds(api, dtype, lens, cached, kv, page):
    s = P.make(dtype, lens, kv, 1, page, seed=len(lens))
    if lens[0] > 60:
        s["k"][s["table"][0, 0].item(), 0, 3, 5] = math.nan
    lo = torch.full((s["k"].shape[0], kv, 128), 3.0).to(s["k"].dtype).cuda()
    hi = lo.clone()
    api.page_bounds(s["k"], s["table"], ints(cached), s["lens"], lo, hi)
    ok(api)
    want_lo, want_hi = torch.full(lo.shape, 3.0), torch.full(lo.shape, 3.0)
    k = s["k"].cpu().float()
    for b, (c, n) in enumerate(zip(cached, lens)):
        for j in range(c // page, n // page):
            at = s["table"][b, j].item()
            want_lo[at], want_hi[at] = k[at].amin(1), k[at].amax(1)  # NaN where a key is NaN
    assert torch.equal(lo.cpu().float().nan_to_num(99.0), want_lo.nan_to_num(99.0))
    assert torch.equal(hi.cpu().float().nan_to_num(99.0), want_hi.nan_to_num(99.0))
    assert not want_hi.isnan().all()


def test_bounds_reports_bad_pages_and_lengths(api):
    s = P.make("bf16", [64, 64, 64], 2, 1, 16)
    lo = torch.zeros(s["k"].shape[0], 2, 128, dtype=torch.bfloat16, device="cuda")
    hi = lo.clone()
    s["table"][1, 2] = s["k"].shape[0]
    s["table"][2, 0] = -1
    api.page_bounds(s["k"], s["table"], ints([0, 0, 0]), s["lens"], lo, hi)
    ok(api, ("MOVA_ERR_DEVICE_CHECK", 1))
    assert (hi.float().abs().sum((1, 2)) > 0).sum().item() == 10
    s = P.make("bf16", [64, 64], 2, 1, 16)
    lo, hi = (torch.zeros(s["k"].shape[0], 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    s["lens"][1] = 1000
    api.page_bounds(s["k"], s["table"], ints([0, 0]), s["lens"], lo, hi)
    ok(api, ("MOVA_ERR_DEVICE_CHECK", 1))


# ---- Attention ---------------------------------------------------------------------

def check_attend(api, s, dtype, scale=None, picked=None, status=("MOVA_OK", 0), **kw):
    o, lse = api.page_attend(s["q"], s["k"], s["v"], s["table"], s["lens"], scale=scale, picked=picked, k_scale=s["ks"],
                             v_scale=s["vs"], return_lse=True, **kw)
    ok(api, status)
    wo, wl, to, tl = P.attend(s["q"], s["k"], s["v"], s["table"], s["lens"], scale, None if picked is None else picked.cpu(),
                              None if s["ks"] is None else s["ks"].cpu(), None if s["vs"] is None else s["vs"].cpu(), dtype)
    err = (P.f64(o) - wo).abs()
    assert torch.isfinite(o.float()).all()
    assert (err <= to).all(), (err - to).max()
    empty = wl == -math.inf
    assert torch.equal(P.f64(lse) == -math.inf, empty)
    assert ((P.f64(lse) - wl).abs()[~empty] <= tl[~empty]).all()
    assert (o.cpu()[empty] == 0).all()
    return o, lse


EDGES = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 257, 500]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("kv,G,page", [(1, 1, 16), (2, 4, 64), (8, 4, 32), (3, 7, 128), (1, 16, 16), (2, 13, 256), (4, 8, 64),
                                       (5, 2, 16)])
def test_attend_edges(api, dtype, kv, G, page):
    check_attend(api, P.make(dtype, EDGES, kv, G, page, seed=kv + G), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("lens,kv,G,page", [
    ([1], 8, 4, 64), ([7, 0, 0], 8, 4, 16), ([20011], 2, 4, 64), ([9000, 1, 3500, 0, 12], 4, 5, 32), ([2049] * 3, 8, 1, 128),
    ([30] * 600, 2, 3, 16), ([5] * 300 + [3000, 0, 700], 4, 9, 32), ([17] * 1100 + [2500], 1, 6, 16), ([1] * 1030, 1, 1, 256),
])
def test_attend_lengths(api, dtype, lens, kv, G, page):
    check_attend(api, P.make(dtype, lens, kv, G, page, seed=len(lens)), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("kv,G,page", [(1, 1, 16), (8, 4, 32), (3, 7, 128), (2, 16, 256), (5, 2, 16)])
@pytest.mark.parametrize("tokens", [512, 4096, 100000])
def test_attend_table_widths(api, dtype, kv, G, page, tokens):
    """The same short rows, where the table could hold few tokens each, and many."""
    lens = EDGES[::2] if kv < 4 else [500, 0, 64]
    check_attend(api, P.make(dtype, lens, kv, G, page, seed=kv + G, width=tokens // page), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("kv,G,page", [(1, 16, 16), (7, 4, 32), (2, 9, 64)])
@pytest.mark.parametrize("tokens", [256, 40000])
def test_attend_many_short_rows(api, dtype, kv, G, page, tokens):
    """More rows than CTAs fit, some empty, where the table could hold few tokens each, and many."""
    lens = [(37 * i) % 131 if i % 5 else 0 for i in range(1203 // kv)]
    check_attend(api, P.make(dtype, lens, kv, G, page, seed=kv, width=tokens // page), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "e4m3"])
def test_attend_many_rows_of_picked_pages(api, dtype):
    s = P.make(dtype, [(41 * i) % 190 for i in range(600)], 2, 4, 16, seed=8)
    picked = (torch.arange(600 * 2 * 4).view(600, 2, 4) * 7 % 13).to(I32)
    picked[::9] = -1
    check_attend(api, s, dtype, picked=picked.cuda())


@pytest.mark.parametrize("dtype", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("tokens", [512, 60000])
@pytest.mark.parametrize("pick", [False, True])
@pytest.mark.parametrize("rows", [40, 700])
def test_attend_reports_the_first_bad_request(api, dtype, tokens, pick, rows):
    s = P.make(dtype, [130] * 40 + [3] * (rows - 40), 2, 4, 16, width=(tokens if rows == 40 else tokens // 2) // 16)
    picked = torch.arange(1, 9, dtype=I32).repeat(rows, 2, 1).cuda() if pick else None  # not page 0
    s["table"][35, 4], s["table"][21, 8], s["table"][9, 0] = -1, s["k"].shape[0], 1 << 30
    want = 21 if pick else 9
    check_attend(api, s, dtype, picked=picked, status=("MOVA_ERR_DEVICE_CHECK", want))
    s["lens"][3] = 1 << 30
    api.page_attend(s["q"], s["k"], s["v"], s["table"], s["lens"], picked=picked, k_scale=s["ks"], v_scale=s["vs"])
    ok(api, ("MOVA_ERR_DEVICE_CHECK", 3))
    s["lens"][3] = -1
    api.page_attend(s["q"], s["k"], s["v"], s["table"], s["lens"], picked=picked, k_scale=s["ks"], v_scale=s["vs"])
    ok(api, ("MOVA_ERR_DEVICE_CHECK", 3))
    s["lens"][3] = 130
    s["table"][[35, 21, 9], [4, 8, 0]] = 0
    api.page_attend(s["q"], s["k"], s["v"], s["table"], s["lens"], picked=picked, k_scale=s["ks"], v_scale=s["vs"])
    ok(api)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("lens,kv,G", [([30011], 1, 16), ([30011], 1, 1), ([20000, 0, 777], 1, 5), ([9000, 8000], 2, 8)])
def test_attend_rows_of_many_parts(api, dtype, lens, kv, G):
    check_attend(api, P.make(dtype, lens, kv, G, 64, seed=G), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("G", [1, 7, 16])
@pytest.mark.parametrize("seed", range(4))
def test_attend_uneven_rows_of_a_wide_table(api, dtype, G, seed):
    """Shares that begin and end at, before and after a row's end."""
    g = torch.Generator().manual_seed(seed)
    lens = (torch.randint(400, (50 + 7 * seed,), generator=g) * torch.randint(2, (50 + 7 * seed,), generator=g)).tolist()
    lens[3] = 2500
    check_attend(api, P.make(dtype, lens, 3 + seed, G, 32, seed=seed, width=1500), dtype)


@pytest.mark.parametrize("dtype,G", [("f32", 4), ("f32", 8), ("bf16", 4), ("bf16", 16), ("e4m3", 8), ("e4m3", 16)])
@pytest.mark.parametrize("rows", [16, 33, 36, 48, 51, 72, 105, 300, 440])
def test_attend_rows_about_what_is_resident(api, dtype, G, rows):
    lens = [(61 * i) % 203 for i in range(rows)]
    check_attend(api, P.make(dtype, lens, 1, G, 16, seed=rows, width=13), dtype)


def test_attend_takes_clusters_that_are_all_resident(api):
    """36 rows and the status in clusters of 8, two CTAs an SM, would have to fill 148
    SMs without a gap, but clusters lie in groups of SMs: two launches."""
    for rows, launches in ((8, 1), (36, 2)):
        s = P.make("bf16", [100] * rows, 1, 4, 32, width=125)
        before = api.launch_count()
        check_attend(api, s, "bf16")
        assert api.launch_count() - before == launches


def test_attend_many_requests(api):
    lens = [(7 * i) % 23 for i in range(4096)]
    check_attend(api, P.make("bf16", lens, 1, 2, 16), "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "e4m3"])
def test_attend_all_rows_empty(api, dtype):
    s = P.make(dtype, [0, 0, 0], 2, 4, 16)
    check_attend(api, s, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "e4m3"])
def test_attend_layouts(api, dtype):
    """Pages further apart than dense (keys and values in one tensor), table rows
    of a longer table, dense q, a given output, another scale."""
    s = P.make(dtype, [300, 77, 0, 1029], 4, 4, 64, seed=3, fused=False)
    both = torch.stack([s["k"].view(torch.uint8), s["v"].view(torch.uint8)], 1).view(s["k"].dtype)
    s["k"], s["v"] = both[:, 0], both[:, 1]
    wide = torch.full((4, 50), -5, dtype=I32, device="cuda")
    wide[:, 20:20 + s["table"].shape[1]] = s["table"]
    s["table"] = wide[:, 20:20 + s["table"].shape[1]]
    out = torch.empty_like(s["q"])
    o, _ = check_attend(api, s, dtype, scale=0.31, out=out)
    assert o is out


@pytest.mark.parametrize("dtype", ["f32", "bf16", "e4m3"])
def test_attend_large_scores(api, dtype):
    """Scores of a few hundred: the softmax is close to picking one token, and the
    running maximum moves."""
    s = P.make(dtype, [1, 900, 64, 333], 2, 4, 32, seed=9)
    s["q"] = (s["q"] * torch.linspace(1, 20, 8, device="cuda")[:, None]).to(s["q"].dtype)
    check_attend(api, s, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "e4m3"])
def test_attend_growing_scores(api, dtype):
    """The maximum grows from token to token, so every tile rescales."""
    s = P.make(dtype, [700, 350], 1, 4, 16, seed=2)
    s["q"] = torch.ones_like(s["q"]) / 16
    for b, n in enumerate((700, 350)):
        for i in range(n):
            s["k"][s["table"][b, i // 16].item(), :, i % 16] = torch.tensor(i / n).to(s["k"].dtype)
    check_attend(api, s, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "e4m3"])
def test_attend_q_of_any_size(api, dtype):
    """Rows of q from 2^-100 to 2^100, and a row of zeros: scores stay products."""
    s = P.make(dtype, [130, 65], 2, 4, 16, seed=4, fused=False)
    size = torch.tensor([2.0 ** -100, 2.0 ** -20, 0.0, 1.0, 2.0 ** -130, 3.0, 2.0 ** -7, 0.5], device="cuda")
    s["q"] = (s["q"].float() * size[:, None]).to(s["q"].dtype)
    check_attend(api, s, dtype)
    s["q"] = torch.full_like(s["q"], 2.0 ** 100)
    s["k"] = torch.zeros_like(s["k"])
    check_attend(api, s, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("gap", [12.0, 16.0, 17.0, 18.5, 20.0])
@pytest.mark.parametrize("lens,kv,G,page,width", [
    ([32, 20, 700], 2, 4, 16, None), ([700, 32], 1, 16, 64, 600), ([30] * 300, 4, 1, 16, None), ([30] * 700, 2, 2, 16, 2000),
])
def test_attend_sink_without_a_value(api, dtype, gap, lens, kv, G, page, width):
    """A first token that outscores all others, which weigh alike, by `gap` and whose
    value is zero: the output is the others', however small their weights.  Values
    are not negative and weights alike, so the error is relative to the output:
    scores off by es (tests/_paged.py; q and keys are whole numbers of every type),
    2^-21 for the exponential and its argument, one weight's rounding (SPLIT; all
    are above 2^-29 of the first), fp32 sums of n terms, the output's rounding."""
    s = P.make(dtype, lens, kv, G, page, seed=int(gap), width=width, fused=False)
    s["q"], s["ks"] = torch.ones_like(s["q"]), None if s["ks"] is None else torch.ones_like(s["ks"])
    s["k"] = torch.zeros(s["k"].shape).to(s["k"].dtype).cuda()
    s["v"] = s["v"].float().nan_to_num(0.0).abs().to(s["v"].dtype)
    first = s["table"][:, 0].long()
    s["k"].view(torch.uint8 if dtype == "e4m3" else s["k"].dtype)[first, :, 0] = (
        torch.ones(1).to(s["k"].dtype).view(torch.uint8).item() if dtype == "e4m3" else 1.0)
    s["v"].view(torch.uint8 if dtype == "e4m3" else s["v"].dtype)[first, :, 0] = 0
    scale = gap / 128
    o, lse = api.page_attend(s["q"], s["k"], s["v"], s["table"], s["lens"], scale=scale, k_scale=s["ks"], v_scale=s["vs"],
                             return_lse=True)
    ok(api)
    wo, wl, _, tl = P.attend(s["q"], s["k"], s["v"], s["table"], s["lens"], scale, None,
                             None if s["ks"] is None else s["ks"].cpu(), None if s["vs"] is None else s["vs"].cpu(), dtype)
    es = 2 * 130 * P.U * gap
    tol = P.OUT[dtype] + P.SPLIT[dtype] + 2 * es + 2.0 ** -20 + 4 * max(lens) * P.U
    err = (P.f64(o) - wo).abs()
    assert (wo > 0).any() and (err <= tol * wo).all(), (err / wo).nan_to_num(0.0).max()
    assert ((P.f64(lse) - wl).abs() <= tl).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attend_nan_and_infinities_show(api, dtype):
    """A NaN or infinite key or value that is attended shows in its heads' outputs,
    as in the formula, and nowhere else."""
    s = P.make(dtype, [40, 40, 40], 2, 2, 16, seed=5)
    s["k"][s["table"][0, 1].item(), 0, 3, 0] = math.nan
    s["v"][s["table"][1, 0].item(), 1, 2, 7] = math.inf
    s["k"][s["table"][2, 0].item(), 0, 1] = math.inf  # q . k infinite or NaN
    o, lse = api.page_attend(s["q"], s["k"], s["v"], s["table"], s["lens"], return_lse=True)
    ok(api)
    assert o[0, :2].isnan().all() and lse[0, :2].isnan().all() and torch.isfinite(o[0, 2:]).all()
    assert o[1, 2:, 7].isinf().all() and torch.isfinite(o[1, :, :7]).all() and torch.isfinite(o[1, :, 8:]).all()
    assert not torch.isfinite(o[2, :2]).any() and torch.isfinite(o[2, 2:]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width", [None, 3000])
@pytest.mark.parametrize("rows", [4, 1100])
def test_attend_scores_of_minus_infinity(api, dtype, width, rows):
    """A token whose score is -inf has no weight; a row of such tokens counts as one
    without tokens."""
    s = P.make(dtype, [1, 17, 40, 33] * (rows // 4), 1, 3, 16, seed=5, width=width, fused=False)
    s["q"] = s["q"].abs() + 0.5
    want = api.page_attend(s["q"], s["k"], s["v"], s["table"], s["lens"], return_lse=True)
    for b in range(0, rows, 4):
        s["k"][s["table"][b, 0].item(), 0, 0, 7] = -math.inf
        s["k"][s["table"][b + 1, :2].long(), :, :, 9] = -math.inf
    s["k"][s["table"][2, 2].item(), 0, :8, 0] = -math.inf  # the last eight of 40
    o, lse = api.page_attend(s["q"], s["k"], s["v"], s["table"], s["lens"], return_lse=True)
    ok(api)
    for b in (0, 1, rows - 4, rows - 3):
        assert (o[b] == 0).all() and (lse[b] == -math.inf).all()
    assert torch.equal(o[3], want[0][3]) and torch.equal(lse[3], want[1][3])
    s["lens"][2] = 32
    few = api.page_attend(s["q"], s["k"], s["v"], s["table"], s["lens"], return_lse=True)
    # The same sums of 32 terms, in another order: 2 * 32 u of them, with |v| below 6, and both outputs' rounding.
    assert ((o[2] - few[0][2]).abs() <= 2 * P.OUT[dtype] * few[0][2].abs() + 2 * 2 * 32 * P.U * 6).all()
    assert ((lse[2] - few[1][2]).abs() <= 2 * 2 * 32 * P.U + 2.0 ** -20).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [5, 300])
def test_attend_infinite_value_of_little_weight(api, dtype, n):
    """A weight of 2^-90 of the greatest, and an infinite value: as in the formula."""
    s = P.make(dtype, [n], 1, 2, 16, seed=5, fused=False)
    s["q"] = torch.ones_like(s["q"])
    s["k"].zero_()
    s["v"].fill_(1.0)
    s["k"][s["table"][0, 0].item(), 0, 0, 0] = 90.0
    s["v"][s["table"][0, (n - 1) // 16].item(), 0, (n - 1) % 16, 3] = -math.inf
    o = api.page_attend(s["q"], s["k"], s["v"], s["table"], s["lens"], scale=math.log(2.0))
    ok(api)
    assert (o[..., 3] == -math.inf).all() and torch.isfinite(o[..., :3]).all() and torch.isfinite(o[..., 4:]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "e4m3"])
def test_attend_bad_pages_count_as_absent(api, dtype):
    s = P.make(dtype, [100, 64, 48], 2, 4, 16, seed=6)
    s["table"][1, 1] = s["k"].shape[0]
    s["table"][2] = -1
    check_attend(api, s, dtype, status=("MOVA_ERR_DEVICE_CHECK", 1))


def test_attend_bad_lengths(api):
    s = P.make("bf16", [100, 64, 48], 2, 4, 16, seed=6)
    s["lens"][1] = -3
    check_attend(api, s, "bf16", status=("MOVA_ERR_DEVICE_CHECK", 1))
    s = P.make("bf16", [100, 112], 2, 4, 16, seed=6)
    s["lens"][1] = 2 ** 31 - 1
    check_attend(api, s, "bf16", status=("MOVA_ERR_DEVICE_CHECK", 1))


def test_attend_far_pages(api):
    """Pages whose element offsets pass 32 bits."""
    num, kv, page = 9000, 8, 64
    k = torch.empty(num, 2, kv, page, 128, dtype=torch.bfloat16, device="cuda")
    assert k[:, 0].stride(0) * (num - 1) > 2 ** 30 and k.numel() > 2 ** 30
    s = P.make("bf16", [200, 130], kv, 4, page, seed=8)
    small = s["table"].clone()
    far = torch.where((small >= 0) & (small < s["k"].shape[0]), num - 1 - small, small)
    for x in range(s["k"].shape[0]):
        k[num - 1 - x, 0], k[num - 1 - x, 1] = s["k"][x], s["v"][x]
    a = api.page_attend(s["q"], s["k"], s["v"], small, s["lens"])
    b = api.page_attend(s["q"], k[:, 0], k[:, 1], far, s["lens"])
    ok(api)
    assert torch.equal(a, b)
    del k
    num = 140000  # fp32 pages of one head: byte offsets past 2^32, element offsets past 2^31
    k = torch.empty(num, 1, 128, 128, dtype=torch.float32, device="cuda")
    assert k.numel() > 2 ** 31
    s = P.make("f32", [200, 300], 1, 4, 128, seed=8)
    small = s["table"].clone()
    inside = (small >= 0) & (small < s["k"].shape[0])
    far = torch.where(inside, num - 1 - small, small)
    for x in range(s["k"].shape[0]):
        k[num - 1 - x] = s["k"][x]
    a = api.page_attend(s["q"], s["k"], s["k"], small, s["lens"])
    b = api.page_attend(s["q"], k, k, far, s["lens"])
    new = torch.randn(2, 1, 128, device="cuda")
    api.page_write(new, new, ints([num * 128 - 1, num * 128 - 129]), k, k)
    ok(api)
    assert torch.equal(a, b)
    assert torch.equal(k[-1, 0, 127], new[0, 0]) and torch.equal(k[-2, 0, 127], new[1, 0])


# ---- Selected pages ----------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16", "e4m3"])
def test_attend_given_pages(api, dtype):
    s = P.make(dtype, [200, 33, 0, 130], 2, 4, 16, seed=11)
    picked = torch.full((4, 2, 9), -1, dtype=I32)
    picked[0, 0] = torch.tensor([12, 0, 5, -1, 3, 3, 11, 99, 1])  # out of order, one twice, holes, one too high
    picked[0, 1, 4] = 7
    picked[1, 0, :3] = torch.tensor([2, 1, 0])
    picked[3] = torch.arange(9)
    check_attend(api, s, dtype, picked=picked.cuda())


def bounds_of(s, page):
    k = s["k"].float().cpu()
    lo = k.nan_to_num(0.0).amin(2).to(s["q"].dtype).to(s["k"].dtype).cuda()
    return lo, k.nan_to_num(0.0).amax(2).to(s["q"].dtype).to(s["k"].dtype).cuda()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("lens,kv,G,page,top", [
    ([500], 2, 4, 16, 5), ([500, 16, 0, 17, 81, 1], 2, 4, 16, 1), ([500, 16, 0, 17, 81, 1], 3, 7, 16, 5),
    ([3000, 2999, 100, 1], 1, 16, 32, 40), ([12000, 700], 2, 1, 16, 64), ([900] * 40, 2, 2, 128, 3),
    ([33000], 1, 8, 16, 1000), ([140000, 300000], 1, 2, 16, 50),
])
def test_select(api, dtype, lens, kv, G, page, top):
    s = P.make(dtype, lens, kv, G, page, seed=top)
    lo, hi = bounds_of(s, page)
    picked = api.page_select(s["q"], lo, hi, s["table"], s["lens"], page, top)
    ok(api)
    assert torch.equal(picked.cpu(), P.select(s["q"], lo, hi, s["table"], s["lens"], page, top))
    if sum(lens) < 5000:
        check_attend(api, s, dtype, picked=picked)


def test_select_ties_go_to_the_lower_page(api):
    s = P.make("bf16", [16 * 100, 16 * 50], 2, 4, 16)
    lo = torch.zeros(s["k"].shape[0], 2, 128, dtype=torch.bfloat16, device="cuda")
    picked = api.page_select(s["q"], lo, lo, s["table"], s["lens"], 16, 7)
    ok(api)
    assert (picked[0].cpu() == torch.tensor([0, 1, 2, 3, 4, 5, 99])).all()
    assert (picked[1].cpu() == torch.tensor([0, 1, 2, 3, 4, 5, 49])).all()
    # Two values only: those with the greater, lowest first, then the others.
    hi = lo.clone()
    s["q"] = s["q"].abs()
    for j in (90, 20, 30):
        hi[s["table"][0, j].item()] = 1.0
    picked = api.page_select(s["q"], lo, hi, s["table"], s["lens"], 16, 6)
    assert (picked[0].cpu() == torch.tensor([0, 1, 20, 30, 90, 99])).all()
    picked = api.page_select(s["q"], lo, hi, s["table"], s["lens"], 16, 3)
    assert (picked[0].cpu() == torch.tensor([20, 30, 99])).all()


def test_select_zero_signs_and_nan(api):
    s = P.make("f32", [16 * 20], 1, 1, 16, fused=False)
    n = s["k"].shape[0]
    lo = torch.zeros(n, 1, 128, device="cuda")
    hi = lo.clone()
    hi[s["table"][0, 4].item()] = -0.0
    s["q"] = torch.ones_like(s["q"])
    assert api.page_select(s["q"], lo, hi, s["table"], s["lens"], 16, 6).tolist() == [[[0, 1, 2, 3, 4, 19]]]
    lo[s["table"][0, 9].item(), 0, 3] = hi[s["table"][0, 9].item(), 0, 3] = math.nan
    hi[s["table"][0, 7].item(), 0, 3] = math.inf
    lo[s["table"][0, 2].item()], hi[s["table"][0, 2].item()] = -math.inf, -math.inf
    assert api.page_select(s["q"], lo, hi, s["table"], s["lens"], 16, 3).tolist() == [[[7, 9, 19]]]
    assert api.page_select(s["q"], lo, hi, s["table"], s["lens"], 16, 2).tolist() == [[[9, 19]]]
    assert 2 not in api.page_select(s["q"], lo, hi, s["table"], s["lens"], 16, 19).tolist()[0][0]
    ok(api)


def test_select_reports_bad_pages(api):
    s = P.make("bf16", [500, 300], 2, 4, 16)
    lo, hi = bounds_of(s, 16)
    s["table"][1, 3] = -9
    picked = api.page_select(s["q"], lo, hi, s["table"], s["lens"], 16, 18)
    ok(api, ("MOVA_ERR_DEVICE_CHECK", 1))
    assert picked.cpu()[1].tolist() == [[j for j in range(19) if j != 3]] * 2  # counts below every other


def repeated(dtype, G, logical, physical, seed=0, kv=2):
    """One request of `logical` full pages and a last one, over `physical` pages of random bounds."""
    g = torch.Generator().manual_seed(seed)
    qt = torch.float32 if dtype == "f32" else torch.bfloat16
    kt = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[dtype]
    hi = torch.randn(physical, kv, 128, generator=g).to(qt).to(kt)
    lo = (hi.float() - torch.rand(physical, kv, 128, generator=g)).to(qt).to(kt)
    q = torch.randn(1, kv * G, 128, generator=g).to(qt)
    table = torch.randint(physical, (1, logical + 1), generator=g, dtype=I32)
    return q.cuda(), lo.cuda(), hi.cuda(), table.cuda(), torch.tensor([16 * logical + 1], dtype=I32).cuda()


def check_select(api, args, top, status=None):
    picked = api.page_select(*args, 16, top)
    ok(api, *([] if status is None else [status]))
    assert torch.equal(picked.cpu(), P.select(*args, 16, top))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("logical,physical,top", [
    (3000, 1, 9), (3000, 1, 2900), (600, 500, 200), (40000, 700, 100), (70000, 900, 40000), (33000, 3, 30000),
])
def test_select_pages_that_repeat(api, dtype, logical, physical, top):
    check_select(api, repeated(dtype, 4, logical, physical, seed=top), top)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("G", [1, 5, 16])
def test_select_scores_that_nearly_agree(api, dtype, G):
    # Pages that differ by one step in one element, the smallest of the query's: the scores differ
    # by far less than the rounding of a sum in fp32, and by far more than one in fp64.
    q, lo, hi, table, lens = repeated(dtype, G, 400, 300, seed=G)
    q[..., 5] *= 2.0 ** -14
    lo[:], hi[:] = lo[:1].clone(), hi[:1].clone()
    raw = {4: torch.int32, 2: torch.int16, 1: torch.int8}[lo.element_size()]
    for x in (lo, hi):
        x[:, :, 5] = 1.0
        x.view(raw)[1::3, :, 5] += 1
        x.view(raw)[2::3, :, 5] -= 1
    check_select(api, (q, lo, hi, table, lens), 150)
    check_select(api, (q, lo, hi, table, lens), 30)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "e4m3"])
def test_select_bounds_that_are_not_finite(api, dtype):
    q, lo, hi, table, lens = repeated(dtype, 1, 900, 901, seed=3, kv=1)
    table[0] = torch.randperm(901, generator=torch.Generator().manual_seed(4)).to(I32)
    up, down = (q[0, 0] > 0).nonzero()[:, 0].tolist(), (q[0, 0] < 0).nonzero()[:, 0].tolist()
    at = table[0].tolist()
    hi[at[100], 0, up[3]] = math.nan     # a score that is NaN: before all others
    hi[at[101], 0, down[3]] = math.nan   # an upper bound that the query does not use
    lo[at[102], 0, up[0]] = math.nan     # and a lower one
    check_select(api, (q, lo, hi, table, lens), 60)
    if dtype == "e4m3":
        return  # no infinities
    hi[at[200], 0, up[5]] = math.inf     # the greatest
    lo[at[201], 0, down[5]] = -math.inf  # as great
    hi[at[202], 0, up[5]] = -math.inf    # the least
    lo[at[203], 0, up[5]] = -math.inf    # not used
    check_select(api, (q, lo, hi, table, lens), 60)
    check_select(api, (q, lo, hi, table, lens), 4)
    check_select(api, (q, lo, hi, table, lens), 900)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "e4m3"])
def test_select_ranges(api, dtype):
    q, lo, hi, table, lens = repeated(dtype, 4, 2000, 1500, seed=5)
    check_select(api, (q * 0, lo, hi, table, lens), 50)                    # all scores are zero
    check_select(api, (q * 2.0 ** -130, lo, hi, table, lens), 50)          # subnormal products
    check_select(api, (q * 2.0 ** 124, lo, hi, table, lens), 50)           # sums beyond fp32's range
    q[:, 1] *= 2.0 ** 20                                                   # heads of unlike size
    check_select(api, (q, lo, hi, table, lens), 50)
    hi[table[0, 77].item()] = (hi[table[0, 77].item()].float() * 0).to(hi.dtype)
    lo[table[0, 77].item()] = (lo[table[0, 77].item()].float() * 0).to(lo.dtype)
    hi[table[0, 78].item()] = (hi[table[0, 78].item()].float() * 64).to(hi.dtype)  # one page far above
    check_select(api, (q, lo, hi, table, lens), 2)
    check_select(api, (q, lo, hi, table, lens), 500)


def test_select_sums_past_32_bit_floats(api):
    """Scores that fp32 holds, of sums that it does not: a head whose negative products
    alone pass 2^128 beside one of a lower, finite score."""
    lo, hi = torch.zeros(21, 1, 128), torch.zeros(21, 1, 128)
    j = torch.arange(21.0)[:, None, None] / 256
    lo[..., :64], hi[..., :64] = (0.5 + j) * 2.0 ** 62, (0.75 + j) * 2.0 ** 62
    lo[..., 64:] = hi[..., 64:] = 1.0625 * 2.0 ** 62
    q = torch.zeros(1, 2, 128)
    q[0, 0, :64], q[0, 0, 64:], q[0, 1, :64] = 2.0 ** 60, -2.0 ** 60, -2.0 ** 60
    table, lens = ints([list(range(21))]), ints([16 * 20 + 1])
    q, lo, hi = (x.bfloat16().cuda() for x in (q, lo, hi))
    want = P.select(q, lo, hi, table, lens, 16, 4)
    assert want.tolist() == [[[17, 18, 19, 20]]]
    check_select(api, (q, lo, hi, table, lens), 4)


def test_select_scores_next_to_the_greatest_32_bit_float(api):
    """Equal scores less than their error bound below 2^128."""
    hi = torch.full((21, 1, 128), 0.99609375 * 2.0 ** 61)
    q = torch.full((1, 1, 128), 2.0 ** 60)
    q[..., 5] *= 1.5
    assert 0.9999 * 2.0 ** 128 < float((q.double() * hi[0].double()).sum()) < 2.0 ** 128
    q, hi = q.bfloat16().cuda(), hi.bfloat16().cuda()
    check_select(api, (q, hi, hi, ints([list(range(21))]), ints([16 * 20 + 1])), 4)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "e4m3"])
def test_select_more_pages_than_are_there(api, dtype):
    q, lo, hi, table, lens = repeated(dtype, 4, 50, 40, kv=1)
    table[0, [7, 13, 30, 31]] = torch.tensor([-1, 40, -5, 1 << 30], dtype=I32).cuda()
    picked = api.page_select(q, lo, hi, table, lens, 16, 49)
    ok(api, ("MOVA_ERR_DEVICE_CHECK", 0))
    assert picked[0, 0].tolist() == [j for j in range(51) if j not in (30, 31)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "e4m3"])
def test_select_more_heads_than_warps(api, dtype):
    q, lo, hi, table, lens = repeated(dtype, 1, 5, 4, kv=3001)
    check_select(api, (q, lo, hi, table, lens), 3)


def test_empty_calls_report_themselves(api):
    """A call of no tokens or requests leaves its own status, not the one before's:
    in a workspace that has just been made, too, and when a graph replays it."""
    s, e = P.make("bf16", [20, 70], 2, 4, 16), P.make("bf16", [], 2, 4, 16, width=3)
    assert e["q"].shape[0] == e["table"].shape[0] == 0
    lo, hi = bounds_of(s, 16)
    k = torch.zeros(1, 2, 128, dtype=torch.bfloat16, device="cuda")
    none = ints([])
    for empty in (lambda ws: api.page_write(k[:0], k[:0], none, s["k"], s["v"], ws=ws),
                  lambda ws: api.page_bounds(s["k"], e["table"], none, none, lo, hi, ws=ws),
                  lambda ws: api.page_select(e["q"], lo, hi, e["table"], none, 16, 3, ws=ws),
                  lambda ws: api.page_attend(e["q"], s["k"], s["v"], e["table"], none, ws=ws)):
        api.page_write(k, k, ints([-7]), s["k"], s["v"])
        ok(api, ("MOVA_ERR_DEVICE_CHECK", 0))
        empty(None)
        ok(api)
        ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
        empty(ws)
        assert api.get_status(ws) == ("MOVA_OK", 0)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            empty(ws)
        ws.fill_(255)
        graph.replay()
        assert api.get_status(ws) == ("MOVA_OK", 0)


# ---- Streams, graphs, repetition -----------------------------------------------------

def test_repeated_calls_are_bit_identical(api):
    s = P.make("bf16", [5000, 100, 0, 2222, 64], 8, 4, 64, seed=1)
    lo, hi = bounds_of(s, 64)
    ws = torch.full((api.page_workspace_size(5, s["table"].shape[1], 8, 32),), 255, dtype=torch.uint8, device="cuda")
    first = api.page_attend(s["q"], s["k"], s["v"], s["table"], s["lens"], return_lse=True)
    for _ in range(3):
        picked = api.page_select(s["q"], lo, hi, s["table"], s["lens"], 64, 9, ws=ws)  # leaves the workspace changed
        again = api.page_attend(s["q"], s["k"], s["v"], s["table"], s["lens"], return_lse=True, ws=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
        assert torch.equal(picked, api.page_select(s["q"], lo, hi, s["table"], s["lens"], 64, 9))
    assert api.get_status(ws) == ("MOVA_OK", 0)


def test_calls_on_two_streams(api):
    states = [P.make("bf16", [4000, 1, 300], 8, 4, 64, seed=x) for x in range(2)]
    alone = [api.page_attend(s["q"], s["k"], s["v"], s["table"], s["lens"]) for s in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    got = [[], []]
    for _ in range(20):
        for x, s in enumerate(states):
            with torch.cuda.stream(streams[x]):
                got[x].append(api.page_attend(s["q"], s["k"], s["v"], s["table"], s["lens"]))
    torch.cuda.synchronize()
    for x in range(2):
        assert all(torch.equal(g, alone[x]) for g in got[x])


def test_captured_step_follows_its_inputs(api):
    """One decode step captured in a graph -- page_map, page_write, page_bounds,
    page_select and both attentions -- and replayed as the lengths grow: each
    replay equals the step run call by call on a copy of the state."""
    B, kv, G, page, num, width = 5, 2, 4, 16, 80, 12
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *shape: torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)

    def state():
        return dict(cached=ints([0, 15, 16, 100, 0]), added=ints([1, 1, 1, 1, 0]), table=torch.zeros(B, width, dtype=I32, device="cuda"),
                    taken=ints([10]), kc=torch.zeros(num, kv, page, 128, dtype=torch.bfloat16, device="cuda"),
                    vc=torch.zeros(num, kv, page, 128, dtype=torch.bfloat16, device="cuda"),
                    lo=torch.zeros(num, kv, 128, dtype=torch.bfloat16, device="cuda"),
                    hi=torch.zeros(num, kv, 128, dtype=torch.bfloat16, device="cuda"))

    free = torch.randperm(num, generator=g, device="cuda").to(I32)
    k0, v0 = rnd(num, kv, page, 128), rnd(num, kv, page, 128)

    def start(s):
        # The requests' first pages: entries 0..9 of the free list.
        at = 0
        for b, n in enumerate([0, 15, 16, 100, 0]):
            for j in range(P.ceil_div(n, page)):
                s["table"][b, j] = free[at]
                at += 1
        s["kc"].copy_(k0)
        s["vc"].copy_(v0)
        for x, f in ((s["lo"], k0.amin(2)), (s["hi"], k0.amax(2))):
            x.copy_(f)
        assert at <= 10
        return s

    q, k, v = rnd(B, kv * G, 128), rnd(B, kv, 128), rnd(B, kv * 128)

    def step(s):
        lens, starts, slots, positions, _ = api.page_map(s["cached"], s["added"], s["table"], free, s["taken"], page,
                                                         num, B, taken_out=s["taken"])
        api.page_write(k, v, slots, s["kc"], s["vc"])
        api.page_bounds(s["kc"], s["table"], s["cached"], lens, s["lo"], s["hi"])
        picked = api.page_select(q, s["lo"], s["hi"], s["table"], lens, page, 3)
        o = api.page_attend(q, s["kc"], s["vc"], s["table"], lens)
        sparse = api.page_attend(q, s["kc"], s["vc"], s["table"], lens, picked=picked)
        s["cached"].copy_(lens)
        return lens, slots, picked, o, sparse

    warm = start(state())
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(warm)
    torch.cuda.synchronize()
    a, b = start(state()), start(state())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(a)
    start(a)
    a["cached"].copy_(ints([0, 15, 16, 100, 0]))
    a["taken"].copy_(ints([10]))
    for i in range(40):
        for t, seed in ((q, 1), (k, 2), (v, 3)):
            t.copy_(torch.randn(t.shape, generator=torch.Generator(device="cuda").manual_seed(100 * i + seed), device="cuda"))
        graph.replay()
        want = step(b)
        for x, y in zip(captured, want):
            assert torch.equal(x, y), i
        for name in a:
            assert torch.equal(a[name], b[name]), (i, name)
    assert a["cached"].tolist() == [40, 55, 56, 140, 0]
    wo, _, to, _ = P.attend(q, a["kc"], a["vc"], a["table"], a["cached"], dtype="bf16")
    assert ((P.f64(captured[3]) - wo).abs() <= to).all()


def test_captured_calls_have_their_own_workspaces(api):
    """Two graphs captured on one stream, replayed at once on two, and again after
    the stream's own workspace has been replaced by a larger one."""
    states = [P.make("bf16", [3000 + 500 * x, 1, 300], 8, 4, 64, seed=x) for x in range(2)]
    alone = [api.page_attend(s["q"], s["k"], s["v"], s["table"], s["lens"]) for s in states]
    side = torch.cuda.Stream()
    graphs, outs = [], []
    for s in states:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(api.page_attend(s["q"], s["k"], s["v"], s["table"], s["lens"]))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in states]
    for _ in range(30):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for o, want in zip(outs, alone):
        assert torch.equal(o, want)
    big = P.make("bf16", [40] * 64, 8, 16, 16, seed=5)
    with torch.cuda.stream(side):
        api.page_attend(big["q"], big["k"], big["v"], big["table"], big["lens"])
        filler = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for o, want in zip(outs, alone):
        assert torch.equal(o, want)
    assert (filler == 255).all()


def test_captured_value_call_keeps_its_workspace(api):
    """value_routed in a graph, after a call that needed a larger workspace on the
    capturing stream and work that takes whatever memory is free."""
    d, E, n = 256, 8, 256
    g = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *shape: torch.randn(*shape, generator=g, device="cuda")
    x, Wr, br, Wv = rnd(40, d).bfloat16(), 0.1 * rnd(E, d), 0.01 * rnd(E), (rnd(E, n, d) / 16).bfloat16()
    want = api.value_routed(x, Wr, br, Wv, 2)
    big = P.make("bf16", [40] * 64, 8, 16, 16, seed=5)
    assert api.page_workspace_size(64, 3, 8, 128) > api.workspace_size(40, d, E, 2, n)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        api.value_routed(x, Wr, br, Wv, 2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        v = api.value_routed(x, Wr, br, Wv, 2)
    with torch.cuda.stream(side):
        api.page_attend(big["q"], big["k"], big["v"], big["table"], big["lens"])
        filler = [torch.full((1 << k,), 255, dtype=torch.uint8, device="cuda") for k in range(12, 22) for _ in range(8)]
        for _ in range(3):
            graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(v, want) and all((f == 255).all() for f in filler)


# ---- With the value path ----------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16", "e4m3"])
def test_serving_steps(api, dtype):
    """A prefill step and decode steps as a server runs them: v from value_routed,
    page_map, page_write, page_bounds, then attention over all pages and over
    selected ones; the cache's content and both outputs against plain ones."""
    d, E, n, kv, G, page, num = 256, 8, 512, 4, 4, 16, 60
    io = P.IO[dtype]
    g = torch.Generator(device="cuda").manual_seed(7)
    rnd = lambda *shape: torch.randn(*shape, generator=g, device="cuda")
    Wr, br, Wv = 0.1 * rnd(E, d), 0.01 * rnd(E), (rnd(E, n, d) / 16).to(io)
    Wq, Wk = rnd(kv * G * 128, d) / 16, rnd(kv * 128, d) / 16
    kc, vc = (torch.full((num, kv, page, 128), math.nan).to(io).to(P.CACHE[dtype]).cuda() for _ in range(2))
    lo, hi = (torch.zeros(num, kv, 128).to(io).to(P.CACHE[dtype]).cuda() for _ in range(2))
    ks = vs = None
    if dtype == "e4m3":
        ks, vs = 0.02 + 0.01 * torch.rand(kv, device="cuda"), 0.01 + 0.01 * torch.rand(kv, device="cuda")
    table = torch.full((4, 14), -1, dtype=I32, device="cuda")
    free, taken = torch.randperm(num, generator=g, device="cuda").to(I32), ints([0])
    cached = ints([0, 0, 0, 0])
    history = [[], [], [], []]
    for step, added in enumerate([[50, 1, 0, 130], [1, 1, 17, 1], [1, 1, 1, 1], [1, 1, 1, 1], [0, 1, 0, 1]]):
        T = sum(added) + 2
        x = rnd(T, d).to(io)
        q = (x.float() @ Wq.T).to(io).view(T, kv * G, 128)
        k = (x.float() @ Wk.T).to(io).view(T, kv, 128)
        v = api.value_routed(x, Wr, br, Wv, 2)
        lens, starts, slots, positions, taken = api.page_map(cached, ints(added), table, free, taken, page, num, T)
        ok(api)
        api.page_write(k, v, slots, kc, vc, ks, vs)
        ok(api)
        api.page_bounds(kc, table, cached, lens, lo, hi)
        ok(api)
        at = 0
        for b, a in enumerate(added):
            assert positions[at:at + a].tolist() == list(range(len(history[b]), len(history[b]) + a))
            history[b] += [(k[at + i].cpu(), v[at + i].view(kv, 128).cpu()) for i in range(a)]
            at += a
        assert slots[at:].tolist() == [-1, -1]
        for b in range(4):  # what the cache holds is what was written
            for i, (kk, vv) in enumerate(history[b]):
                at_k = kc[table[b, i // page].item(), :, i % page].cpu()
                at_v = vc[table[b, i // page].item(), :, i % page].cpu()
                if dtype == "e4m3":
                    kk = (kk.float() / ks.cpu()[:, None]).clamp(-448, 448).to(kc.dtype)
                    vv = (vv.float() / vs.cpu()[:, None]).clamp(-448, 448).to(vc.dtype)
                assert torch.equal(at_k.float(), kk.float()) and torch.equal(at_v.float(), vv.float())
        last = (starts[1:] - 1).clamp(min=0).long()
        s = dict(q=q[last].contiguous(), k=kc, v=vc, ks=ks, vs=vs, table=table, lens=lens)
        check_attend(api, s, dtype)
        picked = api.page_select(s["q"], lo, hi, table, lens, page, 3)
        ok(api)
        assert torch.equal(picked.cpu(), P.select(s["q"], lo, hi, table, lens, page, 3))
        check_attend(api, s, dtype, picked=picked)
        cached = lens
    assert taken.item() == sum(P.ceil_div(len(h), page) for h in history)
