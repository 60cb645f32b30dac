"""Plain implementations of the paged cache operators (Python and fp64 torch on
the CPU), and the error bounds their GPU counterparts are held to.

Bounds, from the arithmetic of the kernels (u = 2^-24, fp32's half step; the
tensor cores' fp32 sums may truncate, so a sum's step counts 2u):
  scores    128 products summed in fp32, scaled, against Q = max sum_d |q_d k_d|:
            es = 2 * 130 u * scale * Q; with E4M3 pages q is held in fp16 relative
            to its row's largest element: + 128 * 2^-25 * scale * max|q| max|k|
  weights   relative: es, 2^-21 for the exponential and its argument's rounding
            at scores up to 32 in base 2, and the split or rounding of P
            (bf16 pages: 2^-16; E4M3: 2^-11; fp32: none): ep
  outputs   a weighted mean of v with weights off by ep relative, and fp32 sums
            over n tokens: (2 ep + 2 n u) max|v|, and the output's rounding
            (bf16: 2^-8 |o|)
  lse       es + 2^-21 + 2 n u + 2^-22 |lse|
"""
import math

import torch

U = 2.0 ** -24
IO = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.bfloat16}
CACHE = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SPLIT = {"f32": 0.0, "bf16": 2.0 ** -16, "e4m3": 2.0 ** -11}
OUT = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -8}


def f64(t):
    return t.detach().cpu().float().double()


def ceil_div(a, b):
    return -(-a // b)


def attend(q, k_cache, v_cache, table, lens, scale=None, picked=None, k_scale=None, v_scale=None, dtype="bf16"):
    """(o, lse, tolerance of o, tolerance of lse), all fp64 on the CPU."""
    scale = 1 / math.sqrt(128) if scale is None else scale
    k_cache, v_cache, q = f64(k_cache), f64(v_cache), f64(q)
    table, lens = table.cpu().tolist(), lens.cpu().tolist()
    num, kv, p, _ = k_cache.shape
    B, H, _ = q.shape
    G = H // kv
    o, lse = torch.zeros(B, H, 128, dtype=torch.float64), torch.full((B, H), -math.inf, dtype=torch.float64)
    to, tl = torch.zeros(B, H, 1, dtype=torch.float64), torch.zeros(B, H, dtype=torch.float64)
    for b in range(B):
        n = min(max(lens[b], 0), len(table[b]) * p)
        pages = ceil_div(n, p)
        for h in range(kv):
            if picked is None:
                chosen = list(range(pages))
            else:
                chosen = [j for j in picked[b, h].tolist()[:pages] if 0 <= j < pages]
            ks, vs = [], []
            for j in chosen:
                if 0 <= table[b][j] < num:
                    m = min(p, n - j * p)
                    ks.append(k_cache[table[b][j], h, :m])
                    vs.append(v_cache[table[b][j], h, :m])
            if not ks:
                continue
            k, v = torch.cat(ks), torch.cat(vs)
            if k_scale is not None:
                k, v = k * float(k_scale[h]), v * float(v_scale[h])
            qs = q[b, h * G:(h + 1) * G]
            s = qs @ k.T * scale
            lse[b, h * G:(h + 1) * G] = torch.logsumexp(s, 1)
            o[b, h * G:(h + 1) * G] = torch.softmax(s, 1) @ v
            es = 2 * 130 * U * scale * float((qs.abs() @ k.abs().T).max())
            if dtype == "e4m3":
                es += 128 * 2.0 ** -25 * scale * float(qs.abs().max() * k.abs().max())
            ep = es + 2.0 ** -21 + SPLIT[dtype]
            tokens = k.shape[0]
            to[b, h * G:(h + 1) * G] = (2 * ep + 2 * tokens * U) * float(v.abs().max())
            tl[b, h * G:(h + 1) * G] = es + 2.0 ** -21 + 2 * tokens * U
    return o, lse, to + OUT[dtype] * o.abs(), tl + 2.0 ** -22 * torch.where(lse.isinf(), 0.0, lse.abs())


def select(q, k_lo, k_hi, table, lens, page, top):
    """picked (B, KV, top), by a full sort of fp64 scores."""
    q, lo, hi = f64(q), f64(k_lo), f64(k_hi)
    B, H, _ = q.shape
    kv = lo.shape[1]
    G = H // kv
    out = torch.full((B, kv, top), -1, dtype=torch.int32)
    for b, n in enumerate(lens.cpu().tolist()):
        pages = ceil_div(n, page)
        for h in range(kv):
            chosen = list(range(pages))
            if pages > top:
                ids = table[b, :pages - 1].cpu().long()
                qs = q[b, h * G:(h + 1) * G]
                s = (qs[:, None] * torch.where(qs[:, None] < 0, lo[ids, h][None], hi[ids, h][None])).sum(2)
                s = torch.where(s.isnan(), math.inf, s).amax(0).tolist()
                chosen = sorted(sorted(range(pages - 1), key=lambda j: (-s[j], j))[:top - 1]) + [pages - 1]
            out[b, h, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
    return out


def page_map(cached, added, table, free, taken, page, num_pages, T):
    """(table, lens, starts, slots, positions, taken, first bad request or None), plain lists."""
    table = [list(r) for r in table]
    width = len(table[0]) if table else 0
    lens, starts, slots, positions = [], [0], [-1] * T, [-1] * T
    avail = len(free) - taken if 0 <= taken <= len(free) else 0
    asked = used = at = 0
    bad = []
    for b, (c, n) in enumerate(zip(cached, added)):
        ok = c >= 0 and n >= 0 and c + n <= width * page
        need = ceil_div(c + n, page) - ceil_div(c, page) if ok else 0
        asked += need
        ok = ok and (need == 0 or asked <= avail)
        if ok and need:
            have = ceil_div(c, page)
            table[b][have:have + need] = free[taken + asked - need:taken + asked]
            used = asked
        count = max(n, 0)
        if not ok or at + count > T:
            bad.append(b)
        for i in range(at, min(at + count, T)):
            if ok:
                positions[i] = c + i - at
                entry = table[b][positions[i] // page]
                if 0 <= entry < num_pages:
                    slots[i] = entry * page + positions[i] % page
                else:
                    bad.append(b)
        lens.append(c + n if ok else max(c, 0))
        at += count
        starts.append(min(at, 2 ** 31 - 1))
    return table, lens, starts, slots, positions, taken + used, min(bad) if bad else None


def e4m3(x):
    """Nearest E4M3 value, ties to even, clamped to +-448, fp64 in and out."""
    m, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
    return ((x / step).round() * step).clamp(-448.0, 448.0)


def make(dtype, lens, kv, G, page, seed=0, spare=3, width=None, device="cuda", fused=True, nan_tail=True):
    """q, caches, scales, table, lens of a batch; every place that no token fills
    holds NaN, and table entries past a row's pages are out of range."""
    g = torch.Generator().manual_seed(seed)
    used = sum(ceil_div(max(n, 0), page) for n in lens)
    num = used + spare
    order = torch.randperm(num, generator=g).tolist()
    width = max([ceil_div(max(n, 0), page) for n in lens] + [1]) if width is None else width
    k = torch.full((num, kv, page, 128), math.nan if nan_tail else 0.0)
    v = k.clone()
    table = torch.full((len(lens), width), 2 ** 30, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        for j in range(ceil_div(max(n, 0), page)):
            page_id = order[at]
            at += 1
            table[b, j] = page_id
            m = min(page, n - j * page)
            k[page_id, :, :m] = torch.randn(kv, m, 128, generator=g)
            v[page_id, :, :m] = torch.randn(kv, m, 128, generator=g)
    H = kv * G
    q = torch.randn(len(lens), H + (2 * kv if fused else 0), 128, generator=g).to(IO[dtype]).to(device)[:, :H]
    k, v = (t.to(IO[dtype]).to(CACHE[dtype]).to(device) for t in (k, v))
    ks = vs = None
    if dtype == "e4m3":
        ks, vs = (0.5 + torch.rand(kv, generator=g) for _ in range(2))
        ks, vs = ks.to(device), vs.to(device)
    return dict(q=q, k=k, v=v, ks=ks, vs=vs, table=table.to(device),
                lens=torch.tensor(lens, dtype=torch.int32, device=device))
