"""Paged attention where one CTA goes through many entries: as many row blocks as SMs, so
that a piece holds whole long sequences. A few entries far above a long tail (a sink) show
what fp16 probabilities and long fp32 sums lose. Against the definition in 64 bits, here in
torch on the GPU, as the host would take minutes."""
import math

import pytest
import torch

from fp4_kv_cache_step_b200 import csa2

pytestmark = pytest.mark.gpu

D, PAGE = 512, 64
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def values(rows):
    """uint8 [n][288] -> float64 [n][512]."""
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=rows.device)
    code = rows[:, : D // 2]
    v = torch.stack((grid[(code & 15).int()], grid[(code >> 4).int()]), -1).flatten(1)
    scale = rows[:, D // 2:].contiguous().view(torch.float8_e4m3fn).double()
    return (v.unflatten(1, (D // 16, 16)) * scale[:, :, None]).flatten(1)


def cache(n, seed, positive):
    """One sequence of n entries in scattered pages, values up to 3 (all >= 0 if `positive`:
    what is lost of a tail then adds up); channels 0-15 are zero."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    M = -(-n // PAGE)
    rows = torch.randint(0, 256, (M + 2, PAGE, 288), dtype=torch.uint8, device="cuda", generator=gen)
    if positive:
        rows[..., : D // 2] &= 0x77
    rows[..., D // 2:] = 0x30                               # scale 1/2
    rows[..., :8] = 0
    table = torch.randperm(M + 2, device="cuda", generator=gen)[:M].to(torch.int32)
    refs = torch.zeros(M + 2, dtype=torch.int32, device="cuda")
    refs[table.long()] = 1
    g = csa2.Fp4Pages(rows, table[None].contiguous(),
                      torch.tensor([n], dtype=torch.int32, device="cuda"), refs)
    return g, gen


def entry(g, i):
    """Row i of the sequence, as a view."""
    return g.rows[int(g.table[0, i // PAGE]), i % PAGE]


def all_values(g, n):
    return values(g.rows[g.table[0].long()].flatten(0, 1)[:n])


def spoiled(g, *shape):
    """A workspace that holds something already."""
    need = csa2.load().csa2_paged_attn_workspace_bytes(g.ref, *shape)
    return torch.full((need,), 0x7f, dtype=torch.uint8, device="cuda")


def check(out, lse, q, v, scale, count=None):
    """out [R][512], lse [R] of the rows q [R][512] over the values v [n][512] (each `count`
    times, where given)."""
    x = q.double() @ v.T * scale
    if count is not None:
        x = x + torch.log(count.double())
    want_lse = torch.logsumexp(x, -1)
    want = torch.softmax(x, -1) @ v
    vmax = float(v.abs().max())
    # logits: 32 steps of 16 products, each off by a last place (2^-23) of at most the sum
    # of magnitudes, and the exponential
    off = 2.0 ** -18 * (1 + (q.double().abs() @ v.abs().T).amax(-1) * abs(scale))
    # probabilities in fp16: half a step, 2^-11, each; where they fall below its normal
    # range, half its least step is 2^-32 of the reference, 64000 times at most: 2^-16.
    # Sums in tensor memory: two last places, 2^-22 of the sum, for each step of 16 of a
    # segment's 64000 entries: 2^-10. Partials in fp16: 2^-11. Weights off by the logits'
    # part move a mean by twice that at most. Then half a bf16 step.
    e = (2.0 ** -11 + 2.0 ** -16 + 2.0 ** -10 + 2.0 ** -11 + 2 * off[:, None]) * vmax
    half_step = 2.0 ** -8 * torch.exp2(torch.floor(torch.log2(want.abs() + e)))
    err = (out.double() - want).abs() - half_step - e
    assert bool((err <= 0).all()), float(err.max()) / vmax
    # the row sum: 800 tiles' sums added in fp32, 2^-24 of it each
    err = (lse.double() - want_lse).abs() - off - 2.0 ** -14
    assert bool((err <= 0).all()), float(err.max())


@pytest.mark.parametrize("sink", [0x77, 0x11, 0x00])
@pytest.mark.parametrize("n,tokens", [(64000, 148), (262144, 148), (1 << 20, 148), (200001, 100)])
def test_a_sink_before_a_long_tail(n, tokens, sink):
    """Head h's sink is 14 + h / 3.5 log2 units above the other entries (14 to 32), which
    are alike to a few hundredths."""
    H = 64
    g, gen = cache(n, seed=n + sink, positive=True)
    first = entry(g, 0)
    first[: D // 2] = sink
    first[:8] = 0
    first[0] = 7                                            # channel 0 holds 3, only here
    q = 0.01 * torch.randn((1, tokens, H, D), device="cuda", generator=gen)
    q[..., 0] = 14 + torch.arange(H, device="cuda") / 3.5
    q = q.to(torch.bfloat16)
    scale = math.log(2) / 3
    out, lse = csa2.csa2_paged_attn(q, g, scale, workspace=spoiled(g, 1, tokens, H, 0))
    v = all_values(g, n)
    for t in (0, tokens // 2, tokens - 1):
        check(out[0, t], lse[0, t], q[0, t], v, scale)
    csa2.check_device_errors()


@pytest.mark.parametrize("tokens", [60, 100, 148, 149, 300])
def test_segments_and_what_each_query_sees(tokens):
    """Pieces of several segments, whole and cut, with lengths around the segments' borders;
    queries that see nothing, queries with a NaN, logits far apart."""
    n, H = 200001, 64
    g, gen = cache(n, seed=tokens, positive=False)
    q = torch.randn((1, tokens, H, D), device="cuda", generator=gen)
    q[..., :16, :] *= 20                                    # sharp rows: the maximum rises often
    q[..., 16, :] *= 2.0 ** 100
    q = q.to(torch.bfloat16)
    q[:, :, 40, 3] = float("nan")
    lens = [0, 1, 63999, 64000, 64001, 128000, 128079, 200000, n, 80, 81]
    nv = torch.tensor([lens[t % len(lens)] for t in range(tokens)], dtype=torch.int32, device="cuda")
    scale = 1 / math.sqrt(D)
    out, lse = csa2.csa2_paged_attn(q, g, scale, nvalid=nv[None], workspace=spoiled(g, 1, tokens, H, 0))
    again, again_lse = csa2.csa2_paged_attn(q, g, scale, nvalid=nv[None])
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    assert torch.equal(lse.view(torch.int32), again_lse.view(torch.int32))
    v = all_values(g, n)
    rest = [h for h in range(H) if h not in (16, 40)]
    for t in list(range(11)) + [tokens - 11 + i for i in range(11)]:
        seen = int(nv[t])
        if seen == 0:
            assert not out[0, t].any() and torch.isneginf(lse[0, t]).all()
            continue
        check(out[0, t, rest], lse[0, t, rest], q[0, t, rest], v[:seen], scale)
        assert torch.isnan(out[0, t, 40]).all() and torch.isnan(lse[0, t, 40])
        # 2^100 times the logits: the largest entry alone, up to its fp16 and bf16 rounding
        # (which of two within 2^-16 of each other is larger is not asked)
        x = q[0, t, 16].double() @ v[:seen].T
        top = torch.topk(x, min(2, seen))
        if seen == 1 or float(top.values[0] - top.values[1]) > 2.0 ** -16 * float(x.abs().max()):
            want = v[int(top.indices[0])]
            assert bool(((out[0, t, 16].double() - want).abs() <= 2.0 ** -8 * want.abs()).all())
    csa2.check_device_errors()


@pytest.mark.parametrize("tokens", [100, 148])
def test_long_lists(tokens):
    """Lists of 130001 places over 5000 entries: ids that repeat, places without one."""
    n, H, K = 5000, 64, 130001
    g, gen = cache(n, seed=3, positive=True)
    first = entry(g, 0)
    first[0] = 7
    q = 0.01 * torch.randn((1, tokens, H, D), device="cuda", generator=gen)
    q[..., 0] = 14 + torch.arange(H, device="cuda") / 3.5
    q = q.to(torch.bfloat16)
    scale = math.log(2) / 3
    ids = torch.randint(1, n, (1, tokens, K), dtype=torch.int32, device="cuda", generator=gen)
    ids[torch.rand(ids.shape, device="cuda", generator=gen) < 0.1] = -1
    ids[..., 0] = 0                                         # the sink, once
    out, lse = csa2.csa2_paged_attn(q, g, scale, topk_idx=ids, workspace=spoiled(g, 1, tokens, H, K))
    v = all_values(g, n)
    for t in (0, tokens // 2, tokens - 1):
        count = torch.bincount(ids[0, t][ids[0, t] >= 0].long(), minlength=n)
        check(out[0, t], lse[0, t], q[0, t], v, scale, count)
    csa2.check_device_errors()
