"""Cases of the paged key-value cache operators: page tables and slot maps from
request lengths (page_map), writing new tokens' keys and values (page_write),
per-page key bounds (page_bounds), attention of one new token per request over
its pages (page_attend), and the same over the few pages that a bound on the
scores selects (page_select, then page_attend).

run(state) computes an operator in plain torch (fp32, or fp64 where a border is
decided), or, with `own` true, through mixture_value_routing_b200.api.

Layouts: caches (pages, KV heads, page size, 128); a request's tokens fill the
pages of its row of `table` in order; slot = page * page_size + place in it.
"""
import math
import random

import torch

own = False

HD = 128  # values and keys per head
_T = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
_SIZE = {"f32": 4, "bf16": 2, "e4m3": 1}
E4M3_MAX = 448.0


# ---- cases ------------------------------------------------------------------

def _case(op, name=None, dtype="bf16", rows=1, length=1, kv=8, group=4, page=64, top=0, pad=0, even=False):
    c = dict(op=op, dtype=dtype, rows=rows, length=length, kv=kv, group=group, page=page, top=top, pad=pad, even=even)
    return c if name is None else dict(c, name=name)


def listed():
    return [
        # One decode step of 64 running requests: each gets one token, a few of them a new page.
        _case("map", "map decode 64 rows", rows=64, length=8192),
        # Chunked prefill mixed with decode: 256 requests, about 32768 new tokens in one step.
        _case("map", "map prefill 256 rows", rows=256, length=512, top=1, pad=77),
        # The keys and values of one decode step, 64 tokens and 8 rows of padding.
        _case("write", "write decode 64 tokens", rows=64, pad=8),
        # A prefill step of 16384 tokens.
        _case("write", "write prefill 16384 tokens", rows=16384, top=1, pad=5),
        # Decode: the few pages that the step's tokens have just filled.
        _case("bounds", "bounds decode 64 rows", rows=64, length=4096),
        # Prefill: every page of long prompts.
        _case("bounds", "bounds prefill 8 rows", rows=8, length=16384, top=1),
        # A small decode batch with short contexts: latency.
        _case("attend", "attend 8 rows to 500", rows=8, length=500, page=16),
        # A large decode batch of ordinary contexts, one row of padding.
        _case("attend", "attend 64 rows e4m3 to 8192", dtype="e4m3", rows=64, length=8192),
        # Long contexts, ragged.
        _case("attend", "attend 16 rows to 32768", rows=16, length=32768),
        # The fp32 layer, 7 query heads for each KV head.
        _case("attend", "attend f32 5 rows to 3001", dtype="f32", rows=5, length=3001, kv=4, group=7, page=32),
        # One request with a long context, 64 of its pages for each KV head.
        _case("sparse", "sparse 1 row of 100000", rows=1, length=100000, top=64),
        # Long contexts in a batch, one head-parallel rank's share of the heads.
        _case("sparse", "sparse 4 rows of 262144", rows=4, length=262144, kv=4, top=128, even=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["map", "write", "bounds", "attend", "attend", "sparse"])
    kv = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "e4m3", "f32"])
    if op == "map":
        rows = _log(rng, 1, 512)
        return _case("map", rows=rows, length=_log(rng, 1, max(1, 60000 // rows)), page=page, top=rng.randrange(2),
                     pad=rng.randrange(100))
    if op == "write":
        return _case("write", dtype=dtype, rows=_log(rng, 1, 12000), kv=kv, page=page, top=rng.randrange(2),
                     pad=rng.randrange(9))
    if op == "bounds":
        rows = _log(rng, 1, 128)
        return _case("bounds", dtype=dtype, rows=rows, length=_log(rng, 1, max(1, 120000 // rows)), kv=kv, page=page,
                     top=rng.randrange(2))
    group = rng.choice([1, 2, 3, 4, 6, 8, 13, 16])
    if op == "attend":
        rows = _log(rng, 1, 256)
        return _case("attend", dtype=dtype, rows=rows, length=_log(rng, 1, min(65536, 1800000 // (rows * kv))), kv=kv,
                     group=group, page=page, even=rng.random() < 0.3)
    rows = _log(rng, 1, 16)
    return _case("sparse", dtype=dtype, rows=rows, length=_log(rng, 200, min(200000, 1500000 // (rows * kv))), kv=kv,
                 group=group, page=page, top=rng.choice([1, 5, 16, 64, 100]))


def _lens(c):
    """Context lengths after the step: the longest first; in larger ragged
    batches also a row of padding (0) and one of a single token."""
    rng = random.Random("lens %(op)s %(rows)d %(length)d %(kv)d %(page)d" % c)
    n, top = c["rows"], c["length"]
    if c["even"]:
        return [top] * n
    out = [max(1, int(top * math.exp(-2.0 * rng.random()))) for _ in range(n)]
    out[0] = top
    if n >= 8:
        out[n // 2], out[n - 2] = 0, 1
    return out


def _added(c):
    """New tokens of each row in this step: one each for decode; with top = 1
    whole prompts, pieces of prompts and decode rows mixed."""
    rng = random.Random("added %(op)s %(rows)d %(length)d" % c)
    out = []
    for n in _lens(c):
        if not c["top"]:
            out.append(min(n, 1))
        else:
            out.append(n if rng.random() < 0.6 else rng.randint(0, n))
    return out


def _filled(c):
    """Full pages that the step's tokens complete, over all rows."""
    return sum(n // c["page"] - (n - a) // c["page"] for n, a in zip(_lens(c), _added(c)))


def work(case):
    c = case
    p, kv, es = c["page"], c["kv"], _SIZE[c["dtype"]]
    io = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "map":
        lens, added = _lens(c), _added(c)
        new = sum(-(-n // p) - -(-(n - a) // p) for n, a in zip(lens, added))
        return {"bytes": 4 * (4 * len(lens) + 2) + 8 * new + 8 * (sum(added) + c["pad"]), "flops": 0}
    if c["op"] == "write":
        return {"bytes": 2 * c["rows"] * kv * HD * (io + es) + 4 * (c["rows"] + c["pad"]), "flops": 0}
    if c["op"] == "bounds":
        return {"bytes": _filled(c) * kv * HD * es * (p + 2) + 8 * c["rows"] + 4 * _filled(c), "flops": 0}
    lens, heads = _lens(c), kv * c["group"]
    rows = 2 * len(lens) * heads * HD * io + 4 * len(lens) * (heads + 1)
    if c["op"] == "attend":
        tokens = sum(lens)
        return {"bytes": tokens * kv * HD * 2 * es + 4 * sum(-(-n // p) for n in lens) + rows,
                "flops": 4 * tokens * heads * HD}
    tokens = scored = 0
    for n in lens:
        pages = -(-n // p)
        if pages > c["top"]:
            scored += pages - 1
            tokens += (c["top"] - 1) * p + (n - (pages - 1) * p)
        else:
            tokens += n
    picked = 4 * len(lens) * kv * c["top"]
    return {"bytes": (tokens + scored) * kv * HD * 2 * es + picked + rows,
            "flops": 4 * (tokens + scored) * heads * HD}


# ---- inputs -----------------------------------------------------------------

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _caches(c, pages, g, values=True):
    """Key and value pages of recycled memory: every place holds numbers. Keys of one page share a part."""
    shape = (pages, c["kv"], c["page"], HD)
    dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    k = torch.randn(shape, generator=g, device="cuda", dtype=dt)
    k += 0.7 * torch.randn((pages, c["kv"], 1, HD), generator=g, device="cuda", dtype=dt)
    v = torch.randn(shape, generator=g, device="cuda", dtype=dt) if values else None
    return k.to(_T[c["dtype"]]), v.to(_T[c["dtype"]]) if values else None


def _scales(c, g):
    if c["dtype"] != "e4m3":
        return None, None
    return tuple(0.5 + torch.rand(c["kv"], generator=g, device="cuda") for _ in range(2))


def _pages_of(lens, page, width, total, g):
    """Each row's pages in the order of a shuffled pool, and the pool's rest."""
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32).tolist()
    table, at = [], 0
    for n in lens:
        need = -(-n // page)
        table.append(order[at:at + need] + [0] * (width - need))
        at += need
    return table, order[at:]


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    io = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    p, kv, heads = c["page"], c["kv"], c["kv"] * c["group"]
    s = {"case": c}
    if c["op"] == "write":
        T = c["rows"]
        run = p if c["top"] else 1  # tokens that follow one another in a page
        pages = -(-T // run) + 3
        order = torch.randperm(pages, generator=g, device="cuda")
        i = torch.arange(T, device="cuda")
        place = i % run if c["top"] else torch.randint(0, p, (T,), generator=g, device="cuda")
        slots = order[i // run] * p + place
        s["slots"] = torch.cat([slots, torch.full((c["pad"],), -1, device="cuda")]).to(torch.int32)
        n = T + c["pad"]
        # Keys are a part of the fused query-key projection's rows; values come from the value projection.
        s["k"] = torch.randn((n, heads + kv, HD), generator=g, device="cuda", dtype=io)[:, heads:]
        s["v"] = torch.randn((n, kv * HD), generator=g, device="cuda", dtype=io)
        s["k_cache"], s["v_cache"] = _caches(c, pages, g)
        s["k_scale"], s["v_scale"] = _scales(c, g)
        if s["k_scale"] is not None:
            s["k_scale"], s["v_scale"] = s["k_scale"] / 64, s["v_scale"] / 64
        return s
    lens = _lens(c)
    width = -(-max(lens) // p) + 1
    used = sum(-(-n // p) for n in lens)
    if c["op"] == "map":
        added = _added(c)
        cached = [n - a for n, a in zip(lens, added)]
        s["num_pages"] = used + 61
        table, rest = _pages_of(cached, p, width, s["num_pages"], g)
        s["table"], s["free"] = _ints(table), _ints([0] * 5 + rest)
        s["cached"], s["added"], s["taken"] = _ints(cached), _ints(added), _ints([5])
        s["tokens"] = sum(added) + c["pad"]
        return s
    table, _ = _pages_of(lens, p, width, used + 3, g)
    s["table"], s["lens"] = _ints(table), _ints(lens)
    if c["op"] == "bounds":
        s["cached"] = _ints([n - a for n, a in zip(lens, _added(c))])
        s["k_cache"], _ = _caches(c, used + 3, g, values=False)
        s["k_lo"], s["k_hi"] = (torch.randn((used + 3, kv, HD), generator=g, device="cuda", dtype=io).to(_T[c["dtype"]])
                                for _ in range(2))
        return s
    s["k_cache"], s["v_cache"] = _caches(c, used + 3, g)
    s["k_scale"], s["v_scale"] = _scales(c, g)
    s["q"] = torch.randn((len(lens), heads + kv, HD), generator=g, device="cuda", dtype=io)[:, :heads]
    if c["op"] == "sparse":
        dt = io if c["dtype"] == "e4m3" else s["k_cache"].dtype
        lo, hi = [], []
        for part in s["k_cache"].split(256):
            lo.append(part.to(dt).amin(2))
            hi.append(part.to(dt).amax(2))
        s["k_lo"], s["k_hi"] = torch.cat(lo).to(_T[c["dtype"]]), torch.cat(hi).to(_T[c["dtype"]])
    return s


# ---- the operators ----------------------------------------------------------

def _values(t):
    """What is held in 8 bits as the numbers it stands for."""
    return t.to(torch.bfloat16) if t.dtype == torch.float8_e4m3fn else t


def run(state):
    return _RUN[state["case"]["op"]](state)


def _run_map(s):
    p, table = s["case"]["page"], s["table"]
    if own:
        from mixture_value_routing_b200 import api
        lens, starts, slots, positions, taken = api.page_map(s["cached"], s["added"], table, s["free"], s["taken"], p,
                                                             s["num_pages"], s["tokens"])
        return dict(table=table, lens=lens, starts=starts, slots=slots, positions=positions, taken=taken)
    cached, added = s["cached"].long(), s["added"].long()
    lens = cached + added
    have = (cached + p - 1) // p
    need = (lens + p - 1) // p - have
    base = s["taken"].long() + need.cumsum(0) - need
    j = torch.arange(table.shape[1], device="cuda")[None, :] - have[:, None]
    new = (j >= 0) & (j < need[:, None])
    source = (base[:, None] + j).clamp(0, s["free"].numel() - 1)
    table.copy_(torch.where(new, s["free"][source], table))
    ends = added.cumsum(0)
    starts = torch.cat([ends.new_zeros(1), ends])
    i = torch.arange(s["tokens"], device="cuda")
    row = (i[:, None] >= ends[None, :]).sum(1)
    live = row < lens.numel()
    row = row.clamp(max=lens.numel() - 1)
    pos = cached[row] + i - starts[row]
    page = table[row, (pos // p).clamp(0, table.shape[1] - 1)].long()
    slots = torch.where(live, page * p + pos % p, -1)
    return dict(table=table, lens=lens.int(), starts=starts.int(), slots=slots.int(),
                positions=torch.where(live, pos, -1).int(), taken=(s["taken"] + need.sum()).int())


def _run_write(s):
    k, v, kc, vc = s["k"], s["v"], s["k_cache"], s["v_cache"]
    if own:
        from mixture_value_routing_b200 import api
        api.page_write(k, v, s["slots"], kc, vc, k_scale=s["k_scale"], v_scale=s["v_scale"])
        return dict(k=_values(kc), v=_values(vc))
    p = s["case"]["page"]
    keep = (s["slots"] >= 0).nonzero()[:, 0]
    slot = s["slots"][keep].long()
    for new, cache, scale in ((k, kc, s["k_scale"]), (v.view(k.shape), vc, s["v_scale"])):
        new = new[keep]
        if scale is not None:
            new = (new.float() / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(cache.dtype)
            cache, new = cache.view(torch.uint8), new.view(torch.uint8)
        cache[slot // p, :, slot % p] = new
    return dict(k=_values(kc), v=_values(vc))


def _run_bounds(s):
    kc, lo, hi = s["k_cache"], s["k_lo"], s["k_hi"]
    if own:
        from mixture_value_routing_b200 import api
        api.page_bounds(kc, s["table"], s["cached"], s["lens"], lo, hi)
        return dict(lo=_values(lo), hi=_values(hi))
    p, table = s["case"]["page"], s["table"]
    j = torch.arange(table.shape[1], device="cuda")
    done = (j >= (s["cached"] // p)[:, None]) & (j < (s["lens"] // p)[:, None])
    pages = table[done].long()
    keys = kc.view(torch.uint8)[pages].view(kc.dtype).float() if kc.dtype == torch.float8_e4m3fn else kc[pages].float()
    for t, of in ((lo, keys.amin(2)), (hi, keys.amax(2))):
        if t.dtype == torch.float8_e4m3fn:
            t.view(torch.uint8)[pages] = of.to(t.dtype).view(torch.uint8)
        else:
            t[pages] = of.to(t.dtype)
    return dict(lo=_values(lo), hi=_values(hi))


def _gather(cache, pages, scale):
    """Pages (B, n) of all heads as (B, KV, n * page, 128) in fp32."""
    raw = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
    x = raw[pages].transpose(1, 2)  # (B, KV, n, page, 128)
    x = x.reshape(x.shape[0], x.shape[1], -1, x.shape[4]).view(cache.dtype).float()
    return x if scale is None else x * scale[:, None, None]


def _softmax_pv(q, k, v, valid):
    """q (B, KV, G, 128), k and v (B, KV, n, 128), valid (B, 1 or KV, n): outputs and the logarithms of the sums."""
    x = (q @ k.transpose(2, 3)) * (1.0 / math.sqrt(HD))
    x = x.masked_fill(~valid[:, :, None, :], -math.inf)
    top = x.amax(3, keepdim=True)
    e = (x - torch.where(top == -math.inf, 0.0, top)).exp()
    total = e.sum(3, keepdim=True)
    o = (e @ v) / torch.where(total > 0, total, 1.0)
    return o, (top + total.log())[..., 0]


def _run_attend(s):
    q, lens, table = s["q"], s["lens"], s["table"]
    if own:
        from mixture_value_routing_b200 import api
        o, lse = api.page_attend(q, s["k_cache"], s["v_cache"], table, lens, k_scale=s["k_scale"], v_scale=s["v_scale"],
                                 return_lse=True)
        return dict(o=o, lse=lse)
    c = s["case"]
    B, kv = len(lens), c["kv"]
    pages = table.long()
    k, v = _gather(s["k_cache"], pages, s["k_scale"]), _gather(s["v_cache"], pages, s["v_scale"])
    valid = (torch.arange(k.shape[2], device="cuda")[None, :] < lens[:, None])[:, None, :]
    o, lse = _softmax_pv(q.float().view(B, kv, -1, HD), k, v, valid)
    return dict(o=o.view(B, -1, HD).to(q.dtype), lse=lse.reshape(B, -1))


def _run_sparse(s):
    q, lens, table, c = s["q"], s["lens"], s["table"], s["case"]
    if own:
        from mixture_value_routing_b200 import api
        picked = api.page_select(q, s["k_lo"], s["k_hi"], table, lens, c["page"], c["top"])
        o = api.page_attend(q, s["k_cache"], s["v_cache"], table, lens, picked=picked, k_scale=s["k_scale"],
                            v_scale=s["v_scale"])
        return dict(o=o, picked=picked)
    B, kv, p, top = len(lens), c["kv"], c["page"], c["top"]
    n = (lens.long() + p - 1) // p  # pages of each row
    j = torch.arange(table.shape[1], device="cuda")
    pages = table.long()
    # A page's score bounds every key's product with the query from above; the best head of a group counts.
    # In 64 bits: scores next to the border decide what is read.
    qd = q.double().view(B, kv, -1, HD)
    score = None
    for part, bound in ((qd.clamp(min=0), s["k_hi"]), (qd.clamp(max=0), s["k_lo"])):
        if bound.dtype == torch.float8_e4m3fn:
            bound = bound.to(torch.bfloat16)
        x = part @ bound[pages].permute(0, 2, 3, 1).double()
        score = x if score is None else score + x
    score = score.amax(2)
    last = j[None, :] == n[:, None] - 1
    score = torch.where(last[:, None], math.inf, score)
    score = torch.where((j[None, :] < n[:, None])[:, None], score, -math.inf)
    order = score.sort(dim=2, descending=True, stable=True).indices[:, :, :top]
    place = torch.arange(order.shape[2], device="cuda")
    order = torch.where(place < n[:, None, None], order, table.shape[1]).sort(dim=2).values
    picked = torch.full((B, kv, top), -1, device="cuda", dtype=torch.int32)
    picked[:, :, :order.shape[2]] = torch.where(order < table.shape[1], order, -1)
    at = pages[torch.arange(B, device="cuda")[:, None, None], picked.long().clamp(min=0)]  # (B, KV, top)
    head = torch.arange(kv, device="cuda")[None, :, None]
    k, v = (_picked(s[x + "_cache"], at, head, s[x + "_scale"]) for x in "kv")
    pos = picked.long()[..., None] * p + torch.arange(p, device="cuda")
    valid = ((picked >= 0)[..., None] & (pos < lens[:, None, None, None])).flatten(2)
    o, _ = _softmax_pv(q.float().view(B, kv, -1, HD), k, v, valid)
    return dict(o=o.view(B, -1, HD).to(q.dtype), picked=picked)


def _picked(cache, pages, head, scale):
    raw = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
    x = raw[pages, head].flatten(2, 3).view(cache.dtype).float()
    return x if scale is None else x * scale[:, None, None]


_RUN = {"map": _run_map, "write": _run_write, "bounds": _run_bounds, "attend": _run_attend, "sparse": _run_sparse}


# ---- in 64 bits, from the definitions ------------------------------------------

def _e4m3(x):
    """The nearest number of 1 sign, 4 exponent and 3 fraction bits (bias 7, largest 448), ties to even."""
    m, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
    return ((x / step).round() * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    p, kv, op = c["page"], c["kv"], c["op"]
    if op == "map":
        return None  # whole numbers only
    if op == "write":
        out = {}
        for x in "kv":
            cache = s[x + "_cache"].to(torch.bfloat16 if c["dtype"] == "e4m3" else _T[c["dtype"]]).double()
            new = s[x].double().reshape(-1, kv, HD)
            if c["dtype"] == "e4m3":
                # The quotient is an fp32 number: its rounding belongs to the definition.
                new = _e4m3((new / s[x + "_scale"].double()[:, None]).float().double())
            flat = cache.transpose(1, 2).reshape(-1, kv, HD)
            flat[s["slots"][:c["rows"]].long()] = new[:c["rows"]]
            out[x] = flat.view(-1, p, kv, HD).transpose(1, 2)
        return out
    if op == "bounds":
        lo, hi = s["k_lo"].float().double(), s["k_hi"].float().double()
        for row, n, a in zip(s["table"].tolist(), _lens(c), _added(c)):
            for page in row[(n - a) // p:n // p]:
                keys = s["k_cache"][page].float().double()
                lo[page], hi[page] = keys.min(1).values, keys.max(1).values
        return dict(lo=lo, hi=hi)
    o, lse = [], []
    for b, n in enumerate(_lens(c)):
        pages = s["table"][b].long()
        for h in range(kv):
            q = s["q"][b, h * c["group"]:(h + 1) * c["group"]].double()
            if n == 0:
                o.append(torch.zeros_like(q))
                lse.append(q.new_full((c["group"],), -math.inf))
                continue
            count = -(-n // p)
            if op == "sparse" and count > c["top"]:
                here = pages[:count - 1]
                lo, hi = (s[x][here, h].float().double() for x in ("k_lo", "k_hi"))
                score = torch.maximum(q[:, None] * lo, q[:, None] * hi).sum(2).max(0).values.tolist()
                best = sorted(range(count - 1), key=lambda i: (-score[i], i))[:c["top"] - 1]
                chosen = sorted(best) + [count - 1]
            else:
                chosen = list(range(count))
            at = pages[torch.tensor(chosen, device="cuda")]
            pos = (torch.tensor(chosen, device="cuda")[:, None] * p + torch.arange(p, device="cuda")).reshape(-1)
            k, v = (s[x + "_cache"].view(torch.uint8 if c["dtype"] == "e4m3" else _T[c["dtype"]])[at, h]
                    .view(_T[c["dtype"]]).float().double().reshape(-1, HD)[pos < n] for x in "kv")
            if c["dtype"] == "e4m3":
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            x = q @ k.T / math.sqrt(HD)
            lse.append(torch.logsumexp(x, 1))
            o.append(torch.softmax(x, 1) @ v)
    B = c["rows"]
    o = torch.stack(o).view(B, -1, HD)
    return dict(o=o, lse=torch.stack(lse).view(B, -1)) if op == "attend" else dict(o=o, picked=None)
