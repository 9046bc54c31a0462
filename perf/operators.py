"""The operators of the paged FP4 cache, as measured cases: their plain forms in
elementary torch operations and the same calls through the package.

Operators
  qk_norm_rope  RMS norm of queries and cache entries with the rotary embedding in the
                same pass; the entries are quantised (E2M1 codes, one E4M3 scale per 16
                channels) into rows of a paged cache
  paged_attn    attention of each sequence's newest queries over its pages: every visible
                entry, or a list of selected ones; an entry is both key and value
  branch        sequences forked from others (pages shared) and grown by a few entries
                (the shared, partly filled last page is copied, new pages are taken)
  compact       a fragmented pool's pages moved to the lowest places, tables rewritten

A paged cache is rows uint8 [P][page][D/2 + D/16], table int32 [S][M] (pages of each
sequence, -1 past the last), len int32 [S] and refs int32 [P] (0: the page is free).
"""
import math

import numpy as np
import torch

own = False

D_ATTN = 512


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one token of one sequence at a short context, few heads: latency alone
        dict(name="attn_1x1000", op="paged_attn", B=1, Tq=1, H=16, lo=1000, hi=1000, page=16, K=0),
        # the 128K decode's batch and lengths, every entry attended
        dict(name="attn_32x32768", op="paged_attn", B=32, Tq=1, H=64, lo=16384, hi=32768, page=64, K=0),
        # four sequences of a million tokens at 4 tokens per entry
        dict(name="attn_4x262144", op="paged_attn", B=4, Tq=1, H=64, lo=262144, hi=262144, page=64, K=0),
        # drafted tokens checked together: three queries per sequence, odd lengths from empty on
        dict(name="attn_draft_19x4999", op="paged_attn", B=19, Tq=3, H=40, lo=0, hi=4999, page=32, K=0),
        # the 128K decode's selected entries, read from pages
        dict(name="attn_top2048_32", op="paged_attn", B=32, Tq=1, H=64, lo=16384, hi=32768, page=64, K=2048),
        # one decoded token of one sequence
        dict(name="rope_1", op="qk_norm_rope", T=1, H=64, E=1, D=512, R=64, half=0, begin=448, wide=0, scaled=0),
        # a decode step of a batch, queries and entries straight from fp32 projections
        dict(name="rope_129", op="qk_norm_rope", T=129, H=40, E=129, D=256, R=128, half=1, begin=0, wide=1, scaled=1),
        # a prefill chunk, four tokens per entry
        dict(name="rope_4096", op="qk_norm_rope", T=4096, H=64, E=1024, D=512, R=64, half=0, begin=448, wide=0, scaled=1),
        # parallel sampling: seven continuations of one prompt
        dict(name="branch_7", op="branch", src=1, dst=7, lo=1000, hi=1000, grow=1, page=16, D=512, spare=512),
        # a batch of searches over long prompts, four continuations each
        dict(name="branch_256", op="branch", src=64, dst=256, lo=30001, hi=65521, grow=5, page=16, D=512, spare=8192),
        # a small pool after many requests came and went
        dict(name="compact_509", op="compact", S=13, lo=0, hi=900, page=16, D=512, P=1024),
        # a large one, half full
        dict(name="compact_65536", op="compact", S=64, lo=16384, hi=49152, page=64, D=512, P=65536),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["paged_attn", "paged_attn", "paged_attn", "qk_norm_rope", "qk_norm_rope", "branch", "compact"])
    if op == "paged_attn":
        page = rng.choice([16, 32, 64, 128])
        H = rng.choice([1, 8, 16, 24, 40, 64, 64, 64, 128])
        B, Tq = _log(rng, 1, 48), rng.choice([1, 1, 1, 2, 3, 4])
        # at most the largest listed case's entries and products
        top = min(131072, 2 ** 26 // (H * Tq * B), 2 ** 20 // B)
        hi = _log(rng, 1, max(2, top))
        lo = rng.randint(0, hi)
        K = _log(rng, 1, 2048) if rng.random() < 0.3 and B * Tq <= 64 else 0
        return dict(op=op, B=B, Tq=Tq, H=H, lo=lo, hi=hi, page=page, K=K)
    if op == "qk_norm_rope":
        D = rng.choice([128, 256, 512, 512, 640, 1024])
        H = rng.choice([1, 3, 8, 40, 64])
        T = _log(rng, 1, max(2, min(4096, 4096 * 64 * 512 // (2 * H * D))))
        R = 2 * rng.randint(0, D // 2)
        begin = rng.choice([0, D - R, 2 * rng.randint(0, (D - R) // 2)])
        return dict(op=op, T=T, H=H, E=rng.randint(0, T), D=D, R=R, half=rng.randint(0, 1), begin=begin,
                    wide=rng.randint(0, 1), scaled=rng.randint(0, 1))
    if op == "branch":
        src = _log(rng, 1, 64)
        hi = _log(rng, 1, 65000)
        page = rng.choice([16, 32, 64, 128])
        return dict(op=op, src=src, dst=src * rng.randint(1, 4), lo=rng.randint(0, hi), hi=hi, grow=_log(rng, 1, 200), page=page,
                    D=rng.choice([128, 512]), spare=_log(rng, 2048, 16384))
    S, hi = _log(rng, 1, 64), _log(rng, 1, 16384)
    page = rng.choice([16, 32, 64, 128])
    used = S * (hi // page + 1)
    return dict(op=op, S=S, lo=rng.randint(0, hi), hi=hi, page=page, D=rng.choice([128, 512]), P=used + _log(rng, 1, 2 * used + 1))


# ---------------------------------------------------------------- inputs
def _lens(n, lo, hi):
    """n lengths from lo to hi, evenly spread: what a case reads does not depend on its seed."""
    return [lo + (hi - lo) * i // max(1, n - 1) if n > 1 else hi for i in range(n)]


def _pages_of(n, page):
    return -(-n // page)


def _row_bytes(D):
    return D // 2 + D // 16


def _rows(P, page, D, gen):
    """Random entries: E2M1 codes, and E4M3 scales between 0.17 and 0.63, as of values near N(0, 1)."""
    rows = torch.randint(0, 256, (P, page, _row_bytes(D)), dtype=torch.uint8, device="cuda", generator=gen)
    rows[:, :, D // 2:] = 0x23 + (rows[:, :, D // 2:] & 15)
    return rows


def _cache(lens, P, page, D, M, gen):
    """A paged cache whose sequences hold scattered pages."""
    S = len(lens)
    pages = torch.tensor([_pages_of(n, page) for n in lens], device="cuda")
    order = torch.randperm(P, device="cuda", generator=gen).to(torch.int32)
    start = torch.cumsum(pages, 0) - pages
    j = torch.arange(M, device="cuda")
    held = j[None] < pages[:, None]
    table = torch.where(held, order[(start[:, None] + j[None]).clamp(max=P - 1)], -1).to(torch.int32).contiguous()
    refs = torch.zeros(P, dtype=torch.int32, device="cuda")
    refs[table[held].long()] = 1
    return dict(rows=_rows(P, page, D, gen), table=table, len=torch.tensor(lens, dtype=torch.int32, device="cuda"), refs=refs,
                page=page, D=D)


def _turns(R, base, factor):
    """Turns of each channel pair per position, as 64-bit binary fractions; positions interpolated by `factor`."""
    theta = base ** (-np.arange(0, R, 2, dtype=np.float64) / max(R, 1)) / factor
    fixed = [int(t * 2.0 ** 64) for t in theta / (2.0 * math.pi)]
    return torch.tensor([f - 2 ** 64 if f >= 2 ** 63 else f for f in fixed], dtype=torch.int64)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 17)
    host = np.random.RandomState((int(seed) * 31 + 5) % (1 << 31))
    s = dict(case=c)
    if c["op"] == "paged_attn":
        lens = list(host.permutation(_lens(c["B"], c["lo"], c["hi"])))
        lens = [int(n) for n in lens]
        M = _pages_of(max(lens + [1]), c["page"])
        P = sum(_pages_of(n, c["page"]) for n in lens) + 3
        s.update(_cache(lens, P, c["page"], D_ATTN, M, gen))
        s["seq"] = torch.arange(c["B"], dtype=torch.int32, device="cuda")
        s["q"] = torch.randn((c["B"], c["Tq"], c["H"], D_ATTN), device="cuda", generator=gen).to(torch.bfloat16)
        # query t of a sequence sees the entries before it: the last sees all
        back = torch.arange(c["Tq"] - 1, -1, -1, dtype=torch.int32, device="cuda")
        s["nvalid"] = (s["len"][:, None] - back[None]).clamp(min=0).contiguous()
        s["topk"] = None
        if c["K"]:
            # the selected ids, ascending, -1 behind the last: one out of every stretch of the visible range
            k = torch.arange(c["K"], device="cuda")
            nv = s["nvalid"].double()[:, :, None]
            lo, hi = torch.floor(k * nv / c["K"]), torch.floor((k + 1) * nv / c["K"])
            pick = lo + torch.floor(torch.rand(lo.shape, device="cuda", generator=gen).double() * (hi - lo))
            ids = torch.where(hi > lo, pick.clamp(max=hi - 1), torch.inf)
            ids = torch.sort(ids, dim=-1).values
            s["topk"] = torch.where(torch.isinf(ids), -1.0, ids).to(torch.int32).contiguous()
        s["scale"] = 1.0 / math.sqrt(D_ATTN)
    elif c["op"] == "qk_norm_rope":
        kind = torch.float32 if c["wide"] else torch.bfloat16
        S, page = 8, 64
        each = _pages_of(c["E"], S) + 70
        s.update(_cache([each] * S, S * _pages_of(each, page) + 1, page, c["D"], _pages_of(each, page), gen))
        # queries and entries are slices of one projection's output
        width = c["H"] * c["D"] + c["D"]
        s["proj"] = (torch.randn((c["T"], width), device="cuda", generator=gen) * 1.7).to(kind)
        s["q"] = s["proj"][:, : c["H"] * c["D"]].view(c["T"], c["H"], c["D"])
        s["kv"] = s["proj"][: c["E"], c["H"] * c["D"]:]
        s["q_weight"] = 1.0 + 0.2 * torch.randn(c["D"], device="cuda", generator=gen)
        s["kv_weight"] = 1.0 + 0.2 * torch.randn(c["D"], device="cuda", generator=gen)
        # positions far into a context of a million tokens
        first = int(host.randint(0, 1 << 20))
        s["pos"] = (first + torch.arange(c["T"], device="cuda")).to(torch.int32)
        s["kv_pos"] = (first + 4 * torch.arange(c["E"], device="cuda")).to(torch.int32)
        e = torch.arange(c["E"], device="cuda")
        s["seq"] = (e % S).to(torch.int32)
        s["entry"] = (e // S + 33).to(torch.int32)
        s["turns"] = _turns(c["R"], 10000.0, 16.0 if c["scaled"] else 1.0).cuda()
        s["rot_scale"] = 0.1 * math.log(16.0) + 1.0 if c["scaled"] else 1.0
        s["q_out"] = torch.empty((c["T"], c["H"], c["D"]), dtype=torch.bfloat16, device="cuda")
        s["kv_out"] = torch.empty((c["E"], c["D"]), dtype=torch.bfloat16, device="cuda")
    elif c["op"] == "branch":
        lens = [int(n) for n in host.permutation(_lens(c["src"], c["lo"], c["hi"]))]
        M = _pages_of(c["hi"] + c["grow"], c["page"])
        extra = c["dst"] * (_pages_of(c["grow"], c["page"]) + 2)
        P = sum(_pages_of(n, c["page"]) for n in lens) + extra + c["spare"]
        s.update(_cache(lens + [0] * c["dst"], P, c["page"], c["D"], M, gen))
        s["dst"] = torch.from_numpy(host.permutation(c["dst"]) + c["src"]).to(torch.int32).cuda()
        s["src"] = torch.from_numpy(np.arange(c["dst"]) % c["src"]).to(torch.int32).cuda()
        s["new_len"] = (s["len"][s["src"].long()] + c["grow"]).contiguous()
    else:
        lens = [int(n) for n in host.permutation(_lens(c["S"], c["lo"], c["hi"]))]
        s.update(_cache(lens, c["P"], c["page"], c["D"], _pages_of(c["hi"], c["page"]) + 1, gen))
        s["before"] = s["table"].clone(), s["refs"].clone()
        s["used"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------------- plain forms
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _values(rows, D):
    """uint8 [..., D/2 + D/16] -> float32 [..., D]."""
    grid = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=rows.device)
    codes = rows[..., : D // 2]
    v = torch.stack((grid[(codes & 15).int()], grid[(codes >> 4).int()]), dim=-1)
    scale = rows[..., D // 2:].contiguous().view(torch.float8_e4m3fn).float()
    return (v.reshape(*rows.shape[:-1], D // 16, 16) * scale[..., None]).reshape(*rows.shape[:-1], D)


def _plain_attn(s):
    q, page = s["q"].float(), s["page"]
    B, Tq, H, D = q.shape
    table = s["table"][s["seq"].long()]
    if s["topk"] is None:
        ids = torch.arange(table.shape[1] * page, device=q.device).expand(B, 1, -1)
        seen = ids < s["nvalid"][:, :, None]
    else:
        ids, seen = s["topk"].long(), s["topk"] >= 0
    at = ids.clamp(min=0)
    pages = torch.gather(table[:, None].expand(-1, at.shape[1], -1), 2, at // page).long().clamp(min=0)
    v = _values(s["rows"][pages, at % page], D)                       # [B, 1 | Tq, n, D]
    logits = torch.matmul(q.reshape(B, v.shape[1], -1, D), v.transpose(-1, -2)).reshape(B, Tq, H, -1) * s["scale"]
    logits = torch.where(seen[:, :, None], logits, -torch.inf)
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.reshape(B, v.shape[1], -1, p.shape[-1]), v).reshape(B, Tq, H, D) / torch.where(total == 0, 1.0, total)
    lse = (top + torch.log(total))[..., 0]
    return dict(out=out.to(torch.bfloat16), lse=lse)


def _normed(x, weight, eps):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight


def _rotated(x, pos, s):
    """x [n, ..., D] with channels [begin, begin + R) rotated by each row's position."""
    c = s["case"]
    a, R = c["begin"], c["R"]
    if not R:
        return x
    angle = (pos.long()[:, None] * s["turns"][None]).double() * (2.0 * math.pi / 2.0 ** 64)   # wraps at whole turns
    shape = (pos.shape[0],) + (1,) * (x.dim() - 2) + (R // 2,)
    cos, sin = ((f(angle) * s["rot_scale"]).to(x.dtype).reshape(shape) for f in (torch.cos, torch.sin))
    part = x[..., a: a + R]
    u, v = (part[..., : R // 2], part[..., R // 2:]) if c["half"] else (part[..., 0::2], part[..., 1::2])
    pair = (u * cos - v * sin, v * cos + u * sin)
    part = torch.cat(pair, -1) if c["half"] else torch.stack(pair, -1).flatten(-2)
    return torch.cat((x[..., :a], part, x[..., a + R:]), -1)


def _e4m3(x):
    """float64 >= 0 -> the nearest E4M3 value, ties to even, at most 448."""
    step = torch.exp2(torch.floor(torch.log2(x.clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(max=448.0)


def _codes(x, scale):
    """E2M1 codes of float64 x at its scales: nearest, ties to the even code."""
    y = x.abs() / torch.where(scale == 0, 1.0, scale)
    n = (y > 0.25).int() + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0)
    return torch.where(scale == 0, 0, n + 8 * torch.signbit(x).int())


def _plain_norm_rope(s):
    D = s["case"]["D"]
    q = _rotated(_normed(s["q"].float(), s["q_weight"], 1e-6), s["pos"], s)
    # in 64 bits: a value next to a border of the 4-bit grid falls to one side
    kv = _rotated(_normed(s["kv"].double(), s["kv_weight"].double(), 1e-6), s["kv_pos"], s)
    g = kv.reshape(-1, D // 16, 16)
    scale = _e4m3(g.abs().amax(-1, keepdim=True) / 6.0)
    code = _codes(g, scale)
    flat = code.reshape(-1, D).to(torch.uint8)
    held = scale[..., 0].float().to(torch.float8_e4m3fn).view(torch.uint8)
    at = s["entry"].long()
    s["rows"][s["table"][s["seq"].long(), at // s["page"]].long(), at % s["page"]] = torch.cat(
        (flat[:, 0::2] | flat[:, 1::2] << 4, held), -1)
    grid = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=q.device, dtype=torch.float64)
    stored = (grid[code] * scale).reshape(-1, D).to(torch.bfloat16)
    return dict(q=q.to(torch.bfloat16), kv=stored, rows=s["rows"].view(torch.int32))


def _plain_fork(s, src, dst):
    table, refs = s["table"], s["refs"]
    new, old = table[src], table[dst]
    refs += torch.bincount(new.flatten() + 1, minlength=refs.shape[0] + 1)[1:].int()
    refs -= torch.bincount(old.flatten() + 1, minlength=refs.shape[0] + 1)[1:].int()
    table[dst] = new
    s["len"][dst] = s["len"][src]


def _plain_resize(s, seq, new_len):
    table, refs, page, P = s["table"], s["refs"], s["page"], s["refs"].shape[0]
    cur, new = s["len"][seq].long(), new_len.long()
    have, want = (cur + page - 1) // page, (new + page - 1) // page
    tail = torch.gather(table[seq], 1, (have - 1).clamp(min=0)[:, None])[:, 0].long()
    cow = (new > cur) & (cur % page != 0) & (refs[tail.clamp(min=0)] > 1)
    need = (want - have).clamp(min=0) + cow
    start = torch.cumsum(need, 0) - need
    free = torch.argsort((refs != 0).to(torch.int8), stable=True)       # free pages first, lowest first
    fits = (need == 0) | (start + need <= (refs == 0).sum())
    j = torch.arange(table.shape[1], device=table.device)[None]
    first = (have - cow.long())[:, None]                               # the copied tail's place comes first
    taken = fits[:, None] & (j >= first) & (j < want[:, None])
    row = torch.where(taken, free[(start[:, None] + j - first).clamp(0, P - 1)].int(), table[seq])
    row = torch.where(fits[:, None] & (j >= want[:, None]), -1, row)
    lost = fits[:, None] & (table[seq] >= 0) & (table[seq] != row)
    refs -= torch.bincount(torch.where(lost, table[seq] + 1, 0).flatten(), minlength=P + 1)[1:].int()
    refs += torch.bincount(torch.where(taken, row + 1, 0).flatten(), minlength=P + 1)[1:].int()
    cow = cow & fits
    to = torch.gather(row, 1, (have - 1).clamp(min=0)[:, None])[:, 0].long()[cow]
    filled = torch.arange(page, device=table.device)[None] < (cur % page)[cow][:, None]
    s["rows"][to] = torch.where(filled[..., None], s["rows"][tail[cow]], s["rows"][to])
    table[seq] = row
    s["len"][seq] = torch.where(fits, new, cur).int()


def _plain_compact(s):
    table, refs, P = s["table"], s["refs"], s["refs"].shape[0]
    used = (refs > 0).sum()
    at = torch.arange(P, device=refs.device)
    src, dst = ((refs > 0) & (at >= used)).nonzero()[:, 0], ((refs == 0) & (at < used)).nonzero()[:, 0]
    s["rows"][dst] = s["rows"][src]
    place = at.int()
    place[src] = dst.int()
    refs[dst] = refs[src]
    refs[src] = 0
    table.copy_(torch.where(table >= 0, place[table.clamp(min=0).long()], -1))
    s["used"].copy_(used[None])


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        from fp4_kv_cache_step_b200 import csa2

        if "pages" not in s:        # the handle that a program keeps beside its tensors
            s["pages"] = csa2.Fp4Pages(s["rows"], s["table"], s["len"], s["refs"])
        pages = s["pages"]
    if op == "paged_attn":
        if not own:
            return _plain_attn(s)
        out, lse = csa2.csa2_paged_attn(s["q"], pages, s["scale"], seq=s["seq"], nvalid=s["nvalid"], topk_idx=s["topk"])
        return dict(out=out, lse=lse)
    if op == "qk_norm_rope":
        if not own:
            return _plain_norm_rope(s)
        c = s["case"]
        q, kv = csa2.csa2_qk_norm_rope(s["turns"], rot_begin=c["begin"], interleaved=not c["half"], rot_scale=s["rot_scale"],
                                       q=s["q"], pos=s["pos"], q_weight=s["q_weight"], q_out=s["q_out"],
                                       kv=s["kv"], kv_pos=s["kv_pos"], kv_weight=s["kv_weight"], pages=pages, seq=s["seq"],
                                       entry=s["entry"], kv_out=s["kv_out"])
        return dict(q=q, kv=kv, rows=s["rows"].view(torch.int32))
    if op == "branch":
        if own:
            csa2.fp4_kv_pages_fork(pages, s["src"], s["dst"])
            csa2.fp4_kv_pages_resize(pages, s["dst"], s["new_len"])
        else:
            _plain_fork(s, s["src"].long(), s["dst"].long())
            _plain_resize(s, s["dst"].long(), s["new_len"])
        return dict(table=s["table"], len=s["len"], refs=s["refs"], rows=s["rows"].view(torch.int32))
    # the pool as it was: the pages that a pass moved are still where they were
    s["table"].copy_(s["before"][0])
    s["refs"].copy_(s["before"][1])
    if own:
        csa2.fp4_kv_pages_compact(pages, used=s["used"])
    else:
        _plain_compact(s)
    return dict(table=s["table"], refs=s["refs"], used=s["used"], rows=s["rows"].view(torch.int32))


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "paged_attn":
        lens = _lens(c["B"], c["lo"], c["hi"])
        io = c["B"] * c["Tq"] * c["H"] * (4 * D_ATTN + 4)
        seen = [[max(0, n - t) for t in range(c["Tq"])] for n in lens]
        pairs = sum(min(n, c["K"]) if c["K"] else n for r in seen for n in r)
        entries = pairs if c["K"] else sum(lens)
        index = 4 * pairs if c["K"] else 4 * sum(_pages_of(n, c["page"]) for n in lens)
        return dict(bytes=io + entries * _row_bytes(D_ATTN) + index, flops=4 * D_ATTN * c["H"] * pairs)
    if c["op"] == "qk_norm_rope":
        size = 4 if c["wide"] else 2
        n, e = c["T"] * c["H"] * c["D"], c["E"] * c["D"]
        return dict(bytes=n * (size + 2) + e * (size + 2) + c["E"] * _row_bytes(c["D"]), flops=6 * (n + e))
    if c["op"] == "branch":
        lens = _lens(c["src"], c["lo"], c["hi"])
        lens = [lens[i % c["src"]] for i in range(c["dst"])]
        held = [_pages_of(n, c["page"]) for n in lens]
        # table rows read and written, each reference taken and given back, the copied part of the last pages
        copied = sum(n % c["page"] for n in lens) * _row_bytes(c["D"])
        return dict(bytes=sum(held) * (8 + 16) + 2 * copied, flops=0)
    pages = sum(_pages_of(n, c["page"]) for n in _lens(c["S"], c["lo"], c["hi"]))
    moved = pages * (1 - pages / c["P"])                                # the pages above the used count, on average
    return dict(bytes=2 * moved * c["page"] * _row_bytes(c["D"]) + 8 * pages + 8 * c["P"], flops=0)


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    c = case
    if c["op"] in ("branch", "compact"):
        return None
    s = prepare(case, seed)
    if c["op"] == "paged_attn":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device="cuda")
        grid = torch.tensor(_E2M1, dtype=torch.float64, device="cuda")
        length, table = s["nvalid"].cpu(), s["table"]
        for b in range(c["B"]):
            n = int(s["len"][b])
            every = s["rows"][table[b, : _pages_of(n, c["page"])].long()].flatten(0, 1)[:n]
            for t in range(c["Tq"]):
                row = every[: int(length[b, t])]
                if c["K"]:
                    ids = s["topk"][b, t]
                    row = every[ids[ids >= 0].long()]
                if not row.shape[0]:
                    continue
                code = torch.empty((row.shape[0], D_ATTN), dtype=torch.uint8, device="cuda")
                code[:, 0::2], code[:, 1::2] = row[:, : D_ATTN // 2] % 16, row[:, : D_ATTN // 2] // 16
                byte = row[:, D_ATTN // 2:].int()
                e, m = (byte >> 3) & 15, (byte & 7).double()
                scale = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2((e - 7).double()))
                v = grid[(code % 8).long()] * (1.0 - 2.0 * (code // 8).double()) * scale.repeat_interleave(16, dim=1)
                x = s["q"][b, t].double() @ v.T * s["scale"]
                lse[b, t] = torch.logsumexp(x, -1)
                out[b, t] = torch.softmax(x, -1) @ v
        return dict(out=out, lse=lse)
    R, a, D = c["R"], c["begin"], c["D"]
    # channel pairs (first[i], second[i])
    i = torch.arange(R // 2, device="cuda")
    first, second = (a + i, a + R // 2 + i) if c["half"] else (a + 2 * i, a + 2 * i + 1)
    theta = 10000.0 ** (-2.0 * i.double() / max(R, 1)) / (16.0 if c["scaled"] else 1.0)

    def turned(x, weight, pos):
        y = x.double() / torch.sqrt(x.double().square().sum(-1, keepdim=True) / D + 1e-6) * weight.double()
        z = y.clone()
        phi = (pos.double()[:, None] * theta).reshape((-1,) + (1,) * (x.dim() - 2) + (R // 2,))
        z[..., first] = s["rot_scale"] * (y[..., first] * torch.cos(phi) - y[..., second] * torch.sin(phi))
        z[..., second] = s["rot_scale"] * (y[..., first] * torch.sin(phi) + y[..., second] * torch.cos(phi))
        return z

    kv = turned(s["kv"], s["kv_weight"], s["kv_pos"]).reshape(-1, D // 16, 16)
    # the E4M3 numbers from 0 to 448, and the nearest one (of two equally near, the one with an even code)
    codes = torch.arange(127, device="cuda")
    e4m3 = torch.where(codes < 8, codes * 2.0 ** -9, (1 + (codes % 8) / 8.0) * torch.exp2((codes // 8 - 7).double())).double()

    def nearest(x, table):
        hi = torch.searchsorted(table, x.contiguous()).clamp(1, len(table) - 1)
        lo = hi - 1
        d = (x - table[lo]) - (table[hi] - x)
        return table[torch.where((d < 0) | ((d == 0) & (lo % 2 == 0)), lo, hi)]

    scale = nearest(kv.abs().amax(-1, keepdim=True) / 6.0, e4m3)
    ratio = torch.where(scale > 0, kv.abs() / torch.where(scale > 0, scale, 1.0), 0.0)
    grid = torch.tensor(_E2M1, dtype=torch.float64, device="cuda")
    stored = nearest(ratio, grid) * torch.sign(kv) * scale
    return dict(q=turned(s["q"], s["q_weight"], s["pos"]), kv=stored.reshape(-1, D), rows=None)
