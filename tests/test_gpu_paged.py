"""The paged FP4 cache on the GPU, against the numpy model in paged_model.py:
upkeep (resize, fork, compact: every number equal), norm + rotation + append
(stored bytes equal, queries within half a bf16 step), attention over pages
(dense and over lists), and a run of all of them as a decode loop uses them."""
import math

import numpy as np
import pytest
import torch

from fp4_kv_cache_step_b200 import csa2
from tests import paged_model as pm
from tests.parity_utils import bf16_ulp

pytestmark = pytest.mark.gpu


def dev(a, dtype=None, device="cuda"):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).to(device)


def i32(a):
    return dev(np.asarray(a, np.int32))


def caches(P, page, D, S, M, seed=0):
    """The model and the library's cache over the same random rows."""
    r = np.random.RandomState(seed)
    rows = r.randint(0, 256, (P, page, D // 2 + D // 16)).astype(np.uint8)
    rows[..., D // 2:] = r.randint(0x23, 0x33, rows[..., D // 2:].shape)
    m = pm.Cache(rows.copy(), S, M)
    g = csa2.Fp4Pages(dev(rows), dev(m.table), dev(m.length), dev(m.refs))
    return m, g


def same(m, g):
    np.testing.assert_array_equal(g.table.cpu().numpy(), m.table)
    np.testing.assert_array_equal(g.length.cpu().numpy(), m.length)
    np.testing.assert_array_equal(g.refs.cpu().numpy(), m.refs)
    np.testing.assert_array_equal(g.rows.cpu().numpy(), m.rows)


def errors():
    try:
        csa2.check_device_errors()
    except csa2.Csa2Error as e:
        return csa2.STATUS[e.status]
    return "OK"


def resize(m, g, seq, new_len):
    m.resize(seq, new_len)
    csa2.fp4_kv_pages_resize(g, i32(seq), i32(new_len))


def fork(m, g, src, dst):
    m.fork(src, dst)
    csa2.fp4_kv_pages_fork(g, i32(src), i32(dst))


# ---------------------------------------------------------------- upkeep
@pytest.mark.parametrize("page,D,P", [(8, 128, 300), (16, 512, 257), (64, 256, 1000)])
def test_random_upkeep(page, D, P):
    S, M = 11, 9
    m, g = caches(P, page, D, S, M, seed=page)
    r = np.random.RandomState(page + 1)
    for step in range(40):
        what = r.randint(0, 4)
        n = r.randint(1, S + 1)
        slots = r.permutation(S)[:n]
        if what == 0:
            resize(m, g, slots, r.randint(0, M * page + 1, n))
        elif what == 1:                              # grow a little: copies of shared last pages
            resize(m, g, slots, np.minimum(m.length[slots] + r.randint(0, 3, n), M * page))
        elif what == 2:
            fork(m, g, r.randint(0, S, n), slots)    # sources repeat, and may be destinations
        else:
            used = torch.zeros(1, dtype=torch.int32, device="cuda")
            csa2.fp4_kv_pages_compact(g, used)
            assert int(used) == m.compact()
        same(m, g)
    assert errors() == "OK" and not m.no_pages and not m.bad


def test_permuted_slots_and_a_slot_onto_itself():
    m, g = caches(64, 8, 128, 5, 4)
    resize(m, g, [0, 1, 2, 3], [5, 17, 0, 32])
    fork(m, g, [1, 2, 3, 0, 4], [0, 1, 2, 3, 4])
    same(m, g)
    assert errors() == "OK"


def test_lowest_free_pages_first_and_none_left():
    m, g = caches(10, 8, 128, 6, 4)
    resize(m, g, [0, 1, 2], [24, 24, 24])            # nine of ten pages
    resize(m, g, [1], [0])                           # three back, in the middle
    # 2 + 1 fit (3 and 4 are listed in order), 3 more do not; a shrinking one still goes
    resize(m, g, [3, 4, 5, 0], [16, 8, 24, 3])
    same(m, g)
    assert m.no_pages and errors() == "NO_PAGES"
    resize(m, g, [5], [24])                          # the pages that came back
    same(m, g)
    assert errors() == "OK"


def test_two_sharers_of_a_last_page_both_grow():
    m, g = caches(32, 16, 512, 4, 4)
    resize(m, g, [0], [21])
    fork(m, g, [0, 0], [1, 2])
    resize(m, g, [0, 1, 2], [22, 30, 40])            # three copies; the shared page is free again
    same(m, g)
    fork(m, g, [2], [3])
    resize(m, g, [3], [17])                          # shrunk inside the shared page
    resize(m, g, [3], [18])                          # one row to copy
    resize(m, g, [2, 3], [0, 0])
    same(m, g)
    assert errors() == "OK"


@pytest.mark.parametrize("seq,new", [([0, 7], [8, 8]), ([-1, 1], [8, 8]), ([1, 1], [8, 16]),
                                     ([0, 1], [-1, 9]), ([2, 0], [33, 4])])
def test_bad_requests_are_recorded_and_skipped(seq, new):
    m, g = caches(32, 8, 128, 4, 4)
    resize(m, g, [0, 1], [10, 20])
    resize(m, g, seq, new)
    same(m, g)
    assert m.bad and errors() == "DEVICE_INDEX"
    assert errors() == "OK"


@pytest.mark.parametrize("src,dst", [([0, 1], [2, 2]), ([4, 0], [3, 1]), ([0, 0], [-1, 2])])
def test_bad_forks_are_recorded_and_skipped(src, dst):
    m, g = caches(32, 8, 128, 4, 4)
    resize(m, g, [0, 1, 2], [10, 20, 3])
    fork(m, g, src, dst)
    same(m, g)
    assert m.bad and errors() == "DEVICE_INDEX"


def test_empty_lists_and_an_empty_cache():
    m, g = caches(16, 8, 128, 3, 2)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    csa2.fp4_kv_pages_resize(g, none, none)
    csa2.fp4_kv_pages_fork(g, none, none)
    csa2.fp4_kv_pages_compact(g)
    same(m, g)
    fork(m, g, [0], [1])
    resize(m, g, [0, 1], [0, 0])
    same(m, g)
    assert errors() == "OK"


def test_large_pool_and_many_slots():
    """Stretches of many pages per warp, lists longer than a CTA."""
    S, M, P, page = 3000, 5, 40001, 8
    m, g = caches(P, page, 128, S, M)
    r = np.random.RandomState(5)
    lens = r.randint(0, M * page + 1, S)
    # the model one sequence at a time is slow here: the same numbers by hand
    need = -(-lens // page)
    start = np.cumsum(need) - need
    order = r.permutation(S)
    csa2.fp4_kv_pages_resize(g, i32(order), i32(lens))
    table = np.full((S, M), -1, np.int32)
    for i, s in enumerate(order):
        table[s, : need[i]] = start[i] + np.arange(need[i])
    np.testing.assert_array_equal(g.table.cpu().numpy(), table)
    assert int(g.refs.sum()) == need.sum() and int(g.refs[: need.sum()].min()) == 1
    # every other slot freed, then compacted: the rows follow their tables
    g.rows.copy_(torch.arange(P, device="cuda")[:, None, None].to(torch.uint8).expand_as(g.rows))
    odd = np.arange(1, S, 2)
    csa2.fp4_kv_pages_resize(g, i32(odd), i32(np.zeros(len(odd))))
    table[odd] = -1
    left = np.unique(table[table >= 0])
    csa2.fp4_kv_pages_compact(g)
    U = len(left)
    place = np.arange(P)
    place[left[left >= U]] = np.setdiff1d(np.arange(U), left)
    want = np.where(table >= 0, place[np.maximum(table, 0)], -1)
    np.testing.assert_array_equal(g.table.cpu().numpy(), want)
    held = want >= 0
    got = g.rows[torch.from_numpy(want[held]).cuda().long(), 0, 0].cpu().numpy()
    np.testing.assert_array_equal(got, table[held].astype(np.uint8))
    assert int(g.refs[:U].min()) == 1 and int(g.refs[U:].sum()) == 0
    assert errors() == "OK"


@pytest.mark.parametrize("page,D,S,M", [(64, 512, 9, 7), (128, 512, 5, 4), (8, 128, 300, 100),
                                        (16, 640, 40, 700)])
def test_large_pages_and_long_tables(page, D, S, M):
    """Copies in several pieces, and lists too long for one cluster's launch."""
    r = np.random.RandomState(page)
    P = S * M // 2 + 40
    m, g = caches(P, page, D, S, M, seed=7)
    half = S // 2
    resize(m, g, np.arange(half), r.randint(0, M * page // 2, half))
    dst = half + r.permutation(S - half)
    fork(m, g, r.randint(0, half, S - half), dst)
    same(m, g)
    every = r.permutation(S)
    resize(m, g, every, np.minimum(m.length[every] + r.randint(0, 4, S), M * page))
    same(m, g)
    fork(m, g, r.randint(0, S, half), np.arange(half))      # some places keep their page
    resize(m, g, r.permutation(S)[: S // 3], r.randint(0, page, S // 3))
    same(m, g)
    csa2.fp4_kv_pages_compact(g)
    m.compact()
    same(m, g)
    assert errors() == "OK" and not m.no_pages


def test_upkeep_in_a_graph():
    """A captured fork + resize replayed: the second replay gives back what the first took."""
    m, g = caches(64, 8, 128, 4, 4)
    resize(m, g, [0], [13])
    src, dst, new = i32([0, 0]), i32([1, 2]), i32([14, 20])
    ws = [torch.empty(1 << 16, dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        csa2.fp4_kv_pages_fork(g, src, dst, workspace=ws[0])
        csa2.fp4_kv_pages_resize(g, dst, new, workspace=ws[1])
    for _ in range(3):
        graph.replay()
        m.fork([0, 0], [1, 2])
        m.resize([1, 2], [14, 20])
        same(m, g)
    assert errors() == "OK"


# ---------------------------------------------------------------- norm, rotation, append
def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)


@pytest.mark.parametrize("D,H,T,E,R,begin,inter,wide,norm,weight,inverse", [
    (512, 64, 1, 1, 64, 448, True, False, True, True, False),
    (512, 5, 7, 3, 64, 448, False, True, True, False, False),
    (128, 3, 9, 9, 128, 0, True, False, True, True, False),
    (128, 1, 2, 2, 126, 1, False, False, True, True, True),
    (256, 9, 33, 17, 30, 77, True, True, False, False, True),
    (640, 2, 3, 4, 640, 0, False, False, True, True, False),
    (1024, 4, 5, 5, 1024, 0, True, True, True, True, False),
    (768, 2, 3, 1, 0, 0, True, False, True, True, False),
    (256, 40, 200, 0, 128, 128, False, False, True, False, False),
    (512, 1, 0, 6, 64, 448, True, False, True, True, False),
    # few heads: several tokens share a CTA, the last one fewer
    (1024, 1, 9, 6, 1024, 0, False, False, True, True, False),
    (512, 1, 19, 9, 78, 434, False, False, True, True, False),
    (512, 4, 7, 2, 184, 52, True, True, True, False, True),
    (128, 3, 5, 5, 70, 2, True, False, True, True, False),
    (256, 2, 9, 300, 64, 61, True, False, True, True, False),
    (384, 8, 9, 160, 64, 316, False, True, True, True, False),
    (512, 64, 5, 3, 70, 442, False, False, True, True, False)])
def test_norm_rope_append(D, H, T, E, R, begin, inter, wide, norm, weight, inverse):
    r = np.random.RandomState(D + H + T)
    S, page, M = 3, 16, 4 if E <= 84 else 8
    m, g = caches(S * M + 2, page, D, S, M, seed=3)
    resize(m, g, range(S), [40, 64, 33] if M == 4 else [105, 128, 110])
    # queries and entries are slices of one projection
    n = max(T, E, 1)
    x = (r.standard_normal((n, (H + 1) * D + 8)) * 2).astype(np.float32)
    t = dev(x) if wide else bf16(x).cuda()
    x = t.double().cpu().numpy()
    q = t[:T, : H * D].unflatten(1, (H, D))
    kv = t[:E, H * D: (H + 1) * D]
    first = [0, 12345, 1048575, 2 ** 31 - 1 - n][T % 4]
    pos, kv_pos = first + np.arange(T), first + 2 ** 10 * 0 + np.arange(E)
    qw = r.standard_normal(D).astype(np.float32) if weight else None
    kw = r.standard_normal(D).astype(np.float32) if weight else None
    turns = csa2.csa2_rope_turns(R, 10000.0, "linear", factor=4.0)
    fixed = turns.cpu().numpy().view(np.uint64)
    seq = np.arange(E) % S
    entry = 5 + np.arange(E) // S
    kv_out = torch.empty((E, D), dtype=torch.bfloat16, device="cuda")
    got, kv_out = csa2.csa2_qk_norm_rope(
        turns, begin, interleaved=inter, inverse=inverse, rot_scale=1.25, eps=1e-5,
        q=q if T else None, pos=i32(pos) if T else None, q_norm=norm,
        q_weight=None if qw is None else dev(qw), kv=kv if E else None, kv_pos=i32(kv_pos) if E else None,
        kv_norm=norm, kv_weight=None if kw is None else dev(kw), pages=g, seq=i32(seq),
        entry=i32(entry), kv_out=kv_out if E else None) if (T or E) else (None, None)
    args = dict(fixed=fixed, begin=begin, interleaved=inter, inverse=inverse, rot_scale=1.25,
                eps=float(np.float32(1e-5)), norm=norm)
    if T:
        want = pm.norm_rope(x[:T, : H * D].reshape(T, H, D), pos, weight=qw, **args)
        # fp32: a sum of D squares (relative D 2^-24 at most), a dozen roundings, the
        # angle's fraction to 2^-24 of a half turn: under (D + 64) 2^-24 of the row's largest
        # value; then half a bf16 step
        e = (D + 64) * 2.0 ** -24 * np.abs(want).max(-1, keepdims=True) * 2
        err = np.abs(got.double().cpu().numpy() - want)
        assert np.all(err <= 0.5 * bf16_ulp(np.abs(want) + e) + e)
    if E:
        ent = pm.norm_rope(x[:E, H * D: (H + 1) * D], kv_pos, weight=kw, **args)
        rows, vals = pm.quantise(ent)
        for i in range(E):
            m.rows[m.table[seq[i], entry[i] // page], entry[i] % page] = rows[i]
        np.testing.assert_array_equal(kv_out.double().cpu().numpy(), vals)
    same(m, g)
    assert errors() == "OK"


def test_rotation_in_place_and_back():
    r = np.random.RandomState(0)
    x = bf16(r.standard_normal((6, 4, 512))).cuda()
    turns = csa2.csa2_rope_turns(64)
    pos = i32([0, 1, 77, 4096, 999999, 2 ** 31 - 1])
    y = x.clone()
    out, _ = csa2.csa2_qk_norm_rope(turns, 448, q=y, pos=pos, q_norm=False, q_out=y)
    assert out is y
    want = pm.norm_rope(x.double().cpu().numpy(), pos.cpu().numpy(),
                        turns.cpu().numpy().view(np.uint64), 448, True, norm=False)
    err = np.abs(y.double().cpu().numpy() - want)
    e = 2.0 ** -20 * np.abs(want).max(-1, keepdims=True)
    assert np.all(err <= 0.5 * bf16_ulp(np.abs(want) + e) + e)
    assert torch.equal(y[..., :448], x[..., :448])          # the other channels pass unchanged
    csa2.csa2_qk_norm_rope(turns, 448, q=y, pos=pos, q_norm=False, inverse=True, q_out=y)
    # two roundings to bf16 of values within sqrt(2) of the row's largest
    assert float((y.float() - x.float()).abs().max()) <= 2 * 2.0 ** -8 * 1.5 * float(x.abs().max())


def test_entries_on_grid_borders_and_zeros():
    """Exact ties of the scale and the codes, signed zeros, a zero row."""
    m, g = caches(4, 8, 128, 1, 2)
    resize(m, g, [0], [8])
    x = np.zeros((5, 128), np.float32)
    x[0, :16] = [6, -6, 5, -5, 2.5, 3.5, 1.75, 1.25, 0.75, 0.25, -0.25, -0.0, 0.0, 4.5, 0.3, -3]
    x[1] = 1.0
    x[2, 16:32] = np.linspace(-2700, 3000, 16)              # beyond 6 * 448
    x[3, ::16] = 6 * (2.0 ** -9) * (np.arange(8) + 0.5)     # subnormal scales, at their ties
    kv_out = torch.empty((5, 128), dtype=torch.bfloat16, device="cuda")
    csa2.csa2_qk_norm_rope(csa2.csa2_rope_turns(0), 0, kv=dev(x), kv_pos=i32([0] * 5),
                           kv_norm=False, pages=g, seq=i32([0] * 5), entry=i32(range(5)),
                           kv_out=kv_out)
    rows, vals = pm.quantise(x.astype(np.float64))
    m.rows[m.table[0, 0], :5] = rows
    same(m, g)
    np.testing.assert_array_equal(kv_out.double().cpu().numpy(), vals)
    assert errors() == "OK"
    # the same bytes as the library's own pack
    np.testing.assert_array_equal(csa2.fp4_kv_pack_g16(dev(x[None]))[0].cpu().numpy(), rows)


def test_bad_entries_are_recorded_and_skipped():
    m, g = caches(16, 8, 128, 4, 2)
    resize(m, g, [0, 1], [16, 5])
    fork(m, g, [1], [2])                                    # a shared page is not written
    x = np.random.RandomState(1).standard_normal((6, 128)).astype(np.float32)
    seq, entry = [0, 0, 1, 2, 9, -1], [3, 16, 4, 0, 0, 0]
    kv_out = torch.zeros((6, 128), dtype=torch.bfloat16, device="cuda")
    csa2.csa2_qk_norm_rope(csa2.csa2_rope_turns(0), 0, kv=dev(x), kv_pos=i32([0] * 6),
                           kv_norm=False, pages=g, seq=i32(seq), entry=i32(entry), kv_out=kv_out)
    rows, vals = pm.quantise(x.astype(np.float64))
    m.rows[m.table[0, 0], 3] = rows[0]
    same(m, g)
    np.testing.assert_array_equal(kv_out.double().cpu().numpy(), vals)
    assert errors() == "DEVICE_INDEX"
    x[0, 7] = np.nan
    csa2.csa2_qk_norm_rope(csa2.csa2_rope_turns(0), 0, kv=dev(x[:1]), kv_pos=i32([0]),
                           kv_norm=False, pages=g, seq=i32([0]), entry=i32([3]))
    assert errors() == "NONFINITE"


# ---------------------------------------------------------------- attention
def attn_case(B, Tq, H, lens, page, seed=0, spare=3, D=512):
    S = B + 2
    M = -(-max(max(lens), 1) // page) + 1
    P = sum(-(-n // page) for n in lens) + spare
    m, g = caches(P, page, D, S, M, seed=seed)
    slots = np.random.RandomState(seed + 1).permutation(S)[:B]
    # scattered pages, dealt out at random as a long-lived pool has them
    order = np.random.RandomState(seed + 2).permutation(P)
    at = 0
    for b, n in enumerate(lens):
        k = -(-n // page)
        m.table[slots[b], :k] = order[at: at + k]
        m.refs[order[at: at + k]] = 1
        m.length[slots[b]] = n
        at += k
    for t, a in ((g.table, m.table), (g.length, m.length), (g.refs, m.refs)):
        t.copy_(dev(a))
    q = bf16(np.random.RandomState(seed + 3).standard_normal((B, Tq, H, D))).cuda()
    return m, g, slots, q


def check_attn(m, slots, q, got, lse, scale, nvalid=None, ids=None):
    q = q.double().cpu().numpy()
    B, Tq, H, D = q.shape
    got, lse = got.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(B):
        v = pm.values(m.entries(slots[b]), D)
        for t in range(Tq):
            n = len(v) if nvalid is None else int(nvalid[b, t])
            sel = v[:n] if ids is None else v[[i for i in ids[b, t] if i >= 0]]
            want, wl = pm.attention(q[b, t], sel, scale)
            vmax = np.abs(sel).max() if len(sel) else 0.0
            # fp16 probabilities: relative 2^-11 each, moving a weighted mean of values by at
            # most 2^-11 vmax; partials rounded to fp16 in a cluster's merge as much again;
            # fp32 sums and exp2 below 2^-16 vmax; then half a bf16 step
            e = 2.0 ** -9 * vmax
            err = np.abs(got[b, t] - want)
            assert np.all(err <= 0.5 * bf16_ulp(np.abs(want) + e) + e), (b, t, err.max())
            if len(sel) == 0:
                assert np.all(got[b, t] == 0) and np.all(np.isneginf(lse[b, t]))
            else:
                # logits: 512 exact products added in fp32 (2^-24 of the sum of magnitudes per
                # addition, a few dozen of them deep), exp2 and log2 to 2^-22
                mag = np.abs(q[b, t]).dot(np.abs(sel).T).max() * abs(scale)
                assert np.all(np.abs(lse[b, t] - wl) <= 2.0 ** -18 * (1 + mag)), (b, t)


@pytest.mark.parametrize("B,Tq,H,lens,page", [
    (1, 1, 1, [1], 8), (1, 1, 16, [1000], 16), (1, 1, 64, [95], 16), (1, 1, 64, [96], 32),
    (1, 1, 64, [97], 64), (2, 1, 64, [0, 193], 8), (3, 2, 24, [1, 2, 500], 32),
    (2, 3, 40, [0, 777], 16), (1, 1, 128, [640], 128), (5, 1, 8, [64, 128, 192, 63, 65], 64),
    (1, 4, 64, [2049], 256), (1, 1, 64, [20000], 64), (40, 1, 64, [300 + 7 * i for i in range(40)], 16),
    (3, 1, 200, [130, 0, 5], 8),
    # short pairs, dealt out whole: one, two and four to an SM of 148; and one that is long
    (36, 2, 70, [(37 * i) % 161 for i in range(36)], 16),
    (98, 3, 64, [81 + (i * 7) % 80 for i in range(98)], 32),
    (590, 1, 8, [(i * 11) % 81 for i in range(590)], 8),
    (36, 2, 70, [(37 * i) % 161 + 2000 * (i == 20) for i in range(36)], 16)])
def test_dense(B, Tq, H, lens, page):
    m, g, slots, q = attn_case(B, Tq, H, lens, page)
    scale = 1 / math.sqrt(512)
    out, lse = csa2.csa2_paged_attn(q, g, scale, seq=i32(slots))
    check_attn(m, slots, q, out, lse, scale)
    # each query its own visible length
    nv = np.maximum(np.array(lens)[:, None] - np.arange(Tq)[::-1][None] * 3, 0)
    out, lse = csa2.csa2_paged_attn(q, g, scale, seq=i32(slots), nvalid=i32(nv))
    check_attn(m, slots, q, out, lse, scale, nvalid=nv)
    assert errors() == "OK"


@pytest.mark.parametrize("scale", [1.0, 8.0])
def test_dense_with_sharp_softmax(scale):
    """Logits far apart: the running maximum rises in the middle of a row."""
    m, g, slots, q = attn_case(2, 1, 64, [1500, 700], 16, seed=9)
    out, lse = csa2.csa2_paged_attn(q, g, scale, seq=i32(slots))
    check_attn(m, slots, q, out, lse, scale)
    assert errors() == "OK"


@pytest.mark.parametrize("lens,K", [([200, 70], 0), ([9000, 5000], 0), ([300, 300], 100)])
def test_queries_of_any_magnitude(lens, K):
    """Logits of 2^100 and of 2^-100: differences, not the logits themselves, are rounded.
    A NaN or an infinity in a row of q fills that row, if it sees an entry, and no other."""
    m, g, slots, q = attn_case(2, 2, 16, lens, 16, seed=12)
    factor = 2.0 ** torch.tensor([0, 100, -100, 20, 40, 0, 0, 0, 64, -130, 26, 0, 10, 80, 100, 5.0])
    q = (q.float() * factor.cuda()[:, None]).to(torch.bfloat16)
    clean = q.clone()
    q[:, :, 5, 77] = float("nan")
    q[:, :, 6, 500] = float("inf")
    q[:, :, 7, 0] = -float("inf")
    nv = np.array([[lens[0], 0], [0, lens[1] - 3]])
    ids = None
    if K:
        r = np.random.RandomState(5)
        ids = np.stack([[r.permutation(max(K, n))[:K] if n else np.full(K, -1) for n in row]
                        for row in nv]).astype(np.int64)
        ids[ids >= nv[:, :, None]] = -1
    out, lse = csa2.csa2_paged_attn(q, g, 0.05, seq=i32(slots), nvalid=i32(nv),
                                    topk_idx=None if ids is None else i32(ids))
    for b, t in ((0, 0), (1, 1)):
        assert torch.isnan(out[b, t, 5:8]).all() and torch.isnan(lse[b, t, 5:8]).all()
    # the other rows, and those that see nothing, as without them
    want, want_lse = csa2.csa2_paged_attn(clean, g, 0.05, seq=i32(slots), nvalid=i32(nv),
                                          topk_idx=None if ids is None else i32(ids))
    rest = [h for h in range(16) if not 5 <= h <= 7]
    assert torch.equal(out[:, :, rest], want[:, :, rest])
    assert torch.equal(lse[:, :, rest], want_lse[:, :, rest])
    for b, t in ((0, 1), (1, 0)):
        assert torch.equal(out[b, t], want[b, t]) and torch.equal(lse[b, t], want_lse[b, t])
    check_attn(m, slots, clean, want, want_lse, 0.05, nvalid=nv, ids=ids)
    assert errors() == "OK"


@pytest.mark.parametrize("scale", [0.0, -0.3])
def test_scales_that_are_not_positive(scale):
    """Scale 0: the mean of the visible values; a negative one turns the order round."""
    m, g, slots, q = attn_case(2, 2, 40, [400, 81], 16, seed=6)
    nv = np.array([[399, 400], [3, 81]])
    out, lse = csa2.csa2_paged_attn(q, g, scale, seq=i32(slots), nvalid=i32(nv))
    check_attn(m, slots, q, out, lse, scale, nvalid=nv)
    assert errors() == "OK"


def test_rows_behind_the_length_are_not_read():
    """Free pages and the places behind a sequence's end hold NaN scales."""
    m, g, slots, q = attn_case(3, 1, 64, [100, 1, 165], 16, seed=12)
    held = np.zeros((m.P, m.page), bool)
    for s in slots:
        at = np.arange(m.length[s])
        held[m.table[s, at // m.page], at % m.page] = True
    m.rows[~held] = 0xff
    g.rows.copy_(dev(m.rows))
    out, lse = csa2.csa2_paged_attn(q, g, 0.05, seq=i32(slots))
    check_attn(m, slots, q, out, lse, 0.05)
    ids = np.array([[[0, 99, -1]], [[-1, 0, -1]], [[5, 6, 164]]])
    out, lse = csa2.csa2_paged_attn(q, g, 0.05, seq=i32(slots), topk_idx=i32(ids))
    check_attn(m, slots, q, out, lse, 0.05, ids=ids)
    assert errors() == "OK"


def test_pools_beyond_four_gigabytes():
    """Pages whose bytes lie past 2^32: written, read, copied and moved."""
    P, page, D, M = 240000, 64, 512, 3                      # 4.4 GB
    if torch.cuda.get_device_properties(0).total_memory < 16 << 30:
        pytest.skip("needs 16 GB")
    g = csa2.Fp4Pages(torch.empty((P, page, 288), dtype=torch.uint8, device="cuda"),
                      torch.full((2, M), -1, dtype=torch.int32, device="cuda"),
                      torch.zeros(2, dtype=torch.int32, device="cuda"),
                      torch.ones(P, dtype=torch.int32, device="cuda"))
    g.refs[P - 5:] = 0                                      # the only free pages
    csa2.fp4_kv_pages_resize(g, i32([0]), i32([100]))
    assert g.table[0].tolist() == [P - 5, P - 4, -1]
    x = bf16(np.random.RandomState(0).standard_normal((100, D)))
    csa2.csa2_qk_norm_rope(csa2.csa2_rope_turns(0), 0, kv=x.cuda(), kv_pos=i32([0] * 100),
                           kv_norm=False, pages=g, seq=i32([0] * 100), entry=i32(range(100)))
    rows, vals = pm.quantise(x.double().numpy())
    np.testing.assert_array_equal(g.rows[P - 5].cpu().numpy(), rows[:64])
    q = bf16(np.random.RandomState(1).standard_normal((1, 1, 16, D))).cuda()
    want, _ = pm.attention(q[0, 0].double().cpu().numpy(), vals, 0.05)
    bound = 2.0 ** -9 * np.abs(vals).max()
    for ids in (None, i32([[list(range(100))]])):
        out, _ = csa2.csa2_paged_attn(q, g, 0.05, seq=i32([0]), topk_idx=ids)
        err = np.abs(out[0, 0].double().cpu().numpy() - want)
        assert np.all(err <= 0.5 * bf16_ulp(np.abs(want) + bound) + bound)
    csa2.fp4_kv_pages_fork(g, i32([0]), i32([1]))
    csa2.fp4_kv_pages_resize(g, i32([1]), i32([101]))       # 36 rows to page P - 3
    assert g.table[1].tolist() == [P - 5, P - 3, -1]
    np.testing.assert_array_equal(g.rows[P - 3, :36].cpu().numpy(), rows[64:])
    g.refs[: P - 5] = 0                                     # three pages left in use
    csa2.fp4_kv_pages_compact(g)
    assert g.table.tolist() == [[0, 1, -1], [0, 2, -1]]
    np.testing.assert_array_equal(g.rows[:2].flatten(0, 1)[:100].cpu().numpy(), rows)
    assert errors() == "OK"


@pytest.mark.parametrize("B,Tq,H,lens,page,K", [(2, 1, 64, [900, 64], 16, 100),
                                                (3, 2, 16, [1, 700, 0], 32, 33),
                                                (1, 1, 1, [1], 8, 1), (1, 1, 64, [500], 8, 80),
                                                (2, 1, 130, [500, 90], 16, 81),
                                                (1, 5, 40, [3000], 64, 1999),
                                                (32, 1, 64, [1000] * 32, 64, 512)])
def test_listed_entries(B, Tq, H, lens, page, K):
    m, g, slots, q = attn_case(B, Tq, H, lens, page, seed=4)
    r = np.random.RandomState(8)
    ids = np.full((B, Tq, K), -1, np.int32)
    for b in range(B):
        for t in range(Tq):
            k = min(K, lens[b])
            ids[b, t, :k] = np.sort(r.permutation(lens[b])[:k])
    scale = 1 / math.sqrt(512)
    out, lse = csa2.csa2_paged_attn(q, g, scale, seq=i32(slots), topk_idx=i32(ids))
    check_attn(m, slots, q, out, lse, scale, ids=ids)
    assert errors() == "OK"


def test_lists_in_any_order_with_repeats():
    m, g, slots, q = attn_case(1, 1, 16, [300], 16, seed=5)
    ids = np.array([[[299, 7, 7, -1, 0, 150, 7, -1, 31, 32]]])
    out, lse = csa2.csa2_paged_attn(q, g, 0.05, seq=i32(slots), topk_idx=i32(ids))
    check_attn(m, slots, q, out, lse, 0.05, ids=ids)        # an id counts as often as listed
    assert errors() == "OK"


def test_slots_in_order_and_without_lse():
    m, g, slots, q = attn_case(2, 1, 16, [50, 130], 16)
    every = q[:1].expand(4, 1, 16, 512).contiguous()        # rows 0 .. 3 read slots 0 .. 3
    out, lse = csa2.csa2_paged_attn(every, g, 0.05)
    check_attn(m, range(4), every, out, lse, 0.05)
    out2, none = csa2.csa2_paged_attn(every, g, 0.05, want_lse=False)
    assert none is None and torch.equal(out, out2)


def test_bad_slots_lengths_and_places_are_recorded():
    m, g, slots, q = attn_case(2, 1, 16, [50, 130], 16)
    scale = 0.05
    seq = np.array([slots[0], 99])
    out, lse = csa2.csa2_paged_attn(q, g, scale, seq=i32(seq))
    check_attn(m, slots[:1], q[:1], out[:1], lse[:1], scale)
    assert not out[1].any() and torch.isneginf(lse[1]).all() and errors() == "DEVICE_INDEX"
    out, lse = csa2.csa2_paged_attn(q, g, scale, seq=i32(slots), nvalid=i32([[51], [-4]]))
    check_attn(m, slots, q, out, lse, scale, nvalid=np.array([[50], [0]]))
    assert errors() == "DEVICE_INDEX"
    # a place without a page: its entries are left out
    g.table[int(slots[1]), 3] = -1
    ids = np.array([[[i for i in range(130) if i // 16 != 3]], ] * 2)
    out, lse = csa2.csa2_paged_attn(q, g, scale, seq=i32(slots))
    check_attn(m, slots[1:], q[1:], out[1:], lse[1:], scale, ids=ids[1:])
    assert errors() == "DEVICE_INDEX"
    out, lse = csa2.csa2_paged_attn(q, g, scale, seq=i32(slots),
                                    topk_idx=i32([[[3, 50, -1]], [[0, 1, -2]]]))
    check_attn(m, slots, q, out, lse, scale, ids=np.array([[[3]], [[0, 1]]], object))
    assert errors() == "DEVICE_INDEX"


def test_attention_in_a_graph_and_on_another_stream():
    m, g, slots, q = attn_case(3, 1, 64, [700, 1, 333], 16)
    scale = 0.05
    seq = i32(slots)
    want, want_lse = csa2.csa2_paged_attn(q, g, scale, seq=seq)
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    need = csa2.load().csa2_paged_attn_workspace_bytes(g.ref, 3, 1, 64, 0)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        csa2.csa2_paged_attn(q, g, scale, seq=seq, out=out, lse=lse, workspace=ws)
    for _ in range(2):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = csa2.csa2_paged_attn(q, g, scale, seq=seq)[0]
    b = csa2.csa2_paged_attn(q, g, scale, seq=seq)[0]       # two calls at once
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)


def test_paged_agrees_with_contiguous():
    """Listed entries of a paged cache against csa2_sparse_attn_g16, whose kernel adds
    in another order: each is within e = 2^-9 vmax of the exact value before it is
    rounded (see check_attn), so they differ by at most 2 e and a bf16 step."""
    m, g, slots, q = attn_case(2, 1, 64, [640, 640], 64, seed=2)
    rows = dev(np.stack([m.entries(s) for s in slots]))
    idx = i32(np.broadcast_to(np.arange(0, 640, 2), (2, 1, 320)))
    want, wl = csa2.csa2_sparse_attn_g16(q, rows, idx, 0.05)
    out, lse = csa2.csa2_paged_attn(q, g, 0.05, seq=i32(slots), topk_idx=idx)
    want = want.double().cpu().numpy()
    vmax = np.abs(pm.values(rows.cpu().numpy(), 512)).max()
    err = np.abs(out.double().cpu().numpy() - want)
    assert np.all(err <= bf16_ulp(np.abs(want) + 2.0 ** -9 * vmax) + 2.0 ** -8 * vmax)
    assert float((lse - wl).abs().max()) <= 2.0 ** -17 * 64


# ---------------------------------------------------------------- together
def test_decode_loop():
    """Prefill, fork, decode with copies of shared pages, compaction and a freed
    slot between steps, a scored selection over the pages; against the model."""
    r = np.random.RandomState(0)
    D, H, page, S, M = 512, 16, 16, 4, 12
    m, g = caches(64, page, D, S, M)
    turns = csa2.csa2_rope_turns(64, 10000.0, "yarn", factor=4.0, context=4096.0)
    fixed = turns.cpu().numpy().view(np.uint64)
    w = (1 + 0.1 * r.standard_normal(D)).astype(np.float32)
    scale = 1 / math.sqrt(D)

    def append(slots, count):
        slots = np.asarray(slots)
        at = m.length[slots].copy()
        resize(m, g, slots, at + count)
        seq = np.repeat(slots, count)
        entry = (at[:, None] + np.arange(count)).reshape(-1)
        kv = bf16(r.standard_normal((len(seq), D)))
        q = bf16(r.standard_normal((len(seq), H, D)))
        out, _ = csa2.csa2_qk_norm_rope(turns, 448, q=q.cuda(), pos=i32(entry), q_weight=dev(w),
                                        kv=kv.cuda(), kv_pos=i32(entry), kv_weight=dev(w),
                                        pages=g, seq=i32(seq), entry=i32(entry))
        rows, _ = pm.quantise(pm.norm_rope(kv.double().numpy(), entry, fixed, 448, True, weight=w,
                                           eps=float(np.float32(1e-6))))
        for i, (s, e) in enumerate(zip(seq, entry)):
            m.rows[m.table[s, e // page], e % page] = rows[i]
        return out.view(len(slots), count, H, D)

    def attend(slots, q):
        nv = m.length[slots][:, None] - np.arange(q.shape[1])[::-1][None]
        out, lse = csa2.csa2_paged_attn(q, g, scale, seq=i32(slots), nvalid=i32(nv))
        check_attn(m, slots, q, out, lse, scale, nvalid=nv)
        pos = i32(nv.reshape(-1) - 1)
        back, _ = csa2.csa2_qk_norm_rope(turns, 448, q=out.flatten(0, 1), pos=pos, q_norm=False,
                                         inverse=True)
        assert torch.isfinite(back.float()).all()

    attend(np.array([0]), append([0], 37))
    fork(m, g, [0, 0], [1, 2])
    for step in range(4):
        attend(np.array([0, 1, 2]), append([0, 1, 2], 1 + step % 2))
        same(m, g)
        if step == 1:
            resize(m, g, [1], [0])
            fork(m, g, [2], [1])
        if step == 2:
            csa2.fp4_kv_pages_compact(g)
            m.compact()
            same(m, g)
    # a selection over the paged cache: scores of a contiguous indexer cache, top-K, attention
    slots = np.array([0, 1, 2])
    n = m.length[slots].astype(np.int32)
    idx_k = torch.randint(0x30, 0x3c, (3, 64, 64), dtype=torch.uint8, device="cuda")
    idx_q = torch.randint(0x30, 0x3c, (3, 1, 4, 64), dtype=torch.uint8, device="cuda")
    idx_w = torch.ones((3, 1, 4), device="cuda")
    nv = i32(n[:, None])
    ids = csa2.csa2_topk(csa2.csa2_index_score(idx_q, idx_w, idx_k, nv), 20, nv)
    q = bf16(r.standard_normal((3, 1, H, D))).cuda()
    out, lse = csa2.csa2_paged_attn(q, g, scale, seq=i32(slots), nvalid=nv, topk_idx=ids)
    check_attn(m, slots, q, out, lse, scale, ids=ids.cpu().numpy())
    resize(m, g, [0, 1, 2, 3], [0, 0, 0, 0])
    same(m, g)
    assert errors() == "OK" and not m.refs.any()


# ---------------------------------------------------------------- calls at once
@pytest.mark.parametrize("D,H,R,begin,inter", [(512, 3, 64, 448, True), (512, 5, 64, 448, False),
                                               (1024, 1, 1024, 0, False), (128, 40, 30, 97, True)])
def test_in_place_as_apart(D, H, R, begin, inter):
    """Runs of rows across tokens: in place gives the bytes that another output gets."""
    q = bf16(np.random.RandomState(1).standard_normal((997, H, D))).cuda()
    pos = torch.randint(0, 1 << 20, (997,), dtype=torch.int32, device="cuda")
    turns = csa2.csa2_rope_turns(R)
    w = torch.rand(D, device="cuda")
    want, _ = csa2.csa2_qk_norm_rope(turns, begin, interleaved=inter, q=q, pos=pos, q_weight=w)
    got, _ = csa2.csa2_qk_norm_rope(turns, begin, interleaved=inter, q=q, pos=pos, q_weight=w, q_out=q)
    assert got is q and torch.equal(got, want)
    assert errors() == "OK"


def test_two_streams_at_once():
    """Calls on two streams, each with its own outputs: the bytes of calls made alone."""
    # short pairs (whole to a piece), long ones (cut), and a list
    cases = [attn_case(40, 2, 64, [3 + 4 * i for i in range(40)], 16, seed=1),
             attn_case(3, 1, 64, [7000, 20, 12001], 64, seed=2)]
    ids = torch.randint(0, 20, (3, 1, 500), dtype=torch.int32, device="cuda")
    turns = csa2.csa2_rope_turns(64)
    pos = torch.arange(999, dtype=torch.int32, device="cuda")
    x = bf16(np.random.RandomState(3).standard_normal((999, 8, 512))).cuda()
    seqs = [i32(c[2]) for c in cases]

    def call(k):
        if k == 2:
            return csa2.csa2_paged_attn(cases[1][3], cases[1][1], 0.05, seq=seqs[1], topk_idx=ids)
        if k == 3:
            return csa2.csa2_qk_norm_rope(turns, 448, q=x, pos=pos)[:1]
        return csa2.csa2_paged_attn(cases[k][3], cases[k][1], 0.05, seq=seqs[k])

    alone = [call(k) for k in range(4)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    results = []
    for i in range(24):
        with torch.cuda.stream(streams[i % 2]):
            results.append((i // 2 % 4, call((i // 2) % 4)))
    torch.cuda.synchronize()
    for k, got in results:
        assert all(torch.equal(a, b) for a, b in zip(got, alone[k])), k
    assert errors() == "OK"
