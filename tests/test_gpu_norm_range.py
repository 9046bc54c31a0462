"""The norm of queries at every magnitude that bf16 and fp32 hold: squares beyond fp32's
range, or below it, against the formula in 64 bits."""
import numpy as np
import pytest
import torch

from fp4_kv_cache_step_b200 import csa2
from tests import paged_model as pm

pytestmark = pytest.mark.gpu

# every way that channels rotate, and rows of one to four chunks a lane
SHAPES = [(512, 64, 448, True), (512, 0, 0, True), (512, 128, 0, False), (512, 512, 0, False),
          (512, 70, 442, True), (128, 128, 0, False), (256, 64, 192, True), (640, 64, 0, True),
          (1024, 1024, 0, False), (1024, 64, 8, True)]


def rows_of(T, H, D, wide, seed):
    """Rows of largest magnitudes from fp32's least step to its end, a few ordinary."""
    r = np.random.RandomState(seed)
    x = r.standard_normal((T, H, D)) / 4
    x = x / np.abs(x).max(-1, keepdims=True)               # the largest is 1
    k = np.linspace(-148 if wide else -132, 127.9, T * H)  # (no row rounds to zeros)
    r.shuffle(k)
    x *= 2.0 ** k.reshape(T, H, 1)
    x[::3, 0] = r.standard_normal((len(x[::3]), D))
    t = torch.from_numpy(x.astype(np.float32))
    return t if wide else t.to(torch.bfloat16)


def check(got, x, turns, begin, inter, w, eps, pos):
    want = pm.norm_rope(x.double().numpy(), pos.numpy(), turns.cpu().numpy().view(np.uint64), begin,
                        inter, weight=w.numpy().astype(np.float64), eps=float(np.float32(eps)))
    got = got.double().cpu().numpy()
    # fp32: a sum of D squares (D 2^-24 of it at most) and a dozen roundings of the row's
    # largest value; then half a bf16 step (the least is 2^-133)
    e = 2 * (x.shape[-1] + 64) * 2.0 ** -24 * np.abs(want).max(-1, keepdims=True)
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(want) + e, 2.0 ** -126))) - 7)
    assert np.isfinite(want).all()
    bad = ~(np.abs(got - want) <= 0.5 * step + e)          # a NaN too
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-33])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("D,R,begin,inter", SHAPES)
def test_rows_of_any_magnitude(D, R, begin, inter, wide, eps):
    T, H = 23, 9
    x = rows_of(T, H, D, wide, seed=D + R)
    turns = csa2.csa2_rope_turns(R)
    pos = torch.arange(T, dtype=torch.int32) * 1000
    w = 1 + 0.2 * torch.randn(D, generator=torch.Generator().manual_seed(1))
    kw = dict(interleaved=inter, eps=eps, pos=pos.cuda(), q_weight=w.cuda())
    q = x.cuda()
    got, _ = csa2.csa2_qk_norm_rope(turns, begin, q=q, **kw)
    check(got, x, turns, begin, inter, w, eps, pos)
    if not wide:                                            # the same in place
        csa2.csa2_qk_norm_rope(turns, begin, q=q, q_out=q, **kw)
        assert torch.equal(q.view(torch.int16), got.view(torch.int16))
    csa2.check_device_errors()


def test_strided_tokens_and_every_row_out_of_range():
    """Slices of a wider projection; CTAs whose rows all take the long way."""
    T, H, D = 300, 8, 512
    x = rows_of(T, H + 1, D, False, seed=5)
    x = (x.float().sign() * 2.0 ** 90 * (1 + x.float().abs().clamp(max=1))).to(torch.bfloat16)
    whole = x.flatten(1).cuda()
    turns = csa2.csa2_rope_turns(64)
    pos = torch.arange(T, dtype=torch.int32)
    w = torch.ones(D)
    got, _ = csa2.csa2_qk_norm_rope(turns, 448, q=whole[:, : H * D].unflatten(1, (H, D)), pos=pos.cuda(),
                                    q_weight=w.cuda())
    check(got, x[:, :H], turns, 448, True, w, 1e-6, pos)
    csa2.check_device_errors()


def test_rows_that_have_no_norm():
    """A NaN fills its row, an infinity gives zeros and a NaN; a row of zeros is zeros with
    eps, and NaN without; the rows beside them are as they were."""
    D = 512
    x = torch.randn((2, 6, D), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    clean = x.clone()
    x[0, 1, 77] = float("nan")
    x[1, 2, 3] = float("inf")
    x[:, 4] = 0
    turns = csa2.csa2_rope_turns(0)
    pos = torch.zeros(2, dtype=torch.int32).cuda()
    want, _ = csa2.csa2_qk_norm_rope(turns, 0, q=clean.cuda(), pos=pos)
    for eps in (1e-6, 0.0):
        got, _ = csa2.csa2_qk_norm_rope(turns, 0, q=x.cuda(), pos=pos, eps=eps)
        assert torch.isnan(got[0, 1]).all()
        assert torch.isnan(got[1, 2, 3]) and not got[1, 2, :3].any() and not got[1, 2, 4:].any()
        assert bool((got[:, 4] == 0).all() if eps else torch.isnan(got[:, 4]).all())
        if eps:
            for t, h in ((0, 0), (0, 2), (1, 1), (1, 3), (1, 5)):
                assert torch.equal(got[t, h], want[t, h])
    csa2.check_device_errors()


@pytest.mark.parametrize("D,R,inter,T,E", [(768, 768, True, 8003, 300), (768, 768, True, 20, 1),
                                           (512, 384, True, 33000, 0), (1024, 1024, True, 5, 200),
                                           (1024, 1024, False, 5, 200), (512, 512, False, 3000, 149),
                                           (384, 192, False, 29000, 0)])
def test_tables_as_large_as_they_get(D, R, inter, T, E):
    """One head: CTAs of as many tokens, and entries, as shared memory has tables for."""
    gen = torch.Generator().manual_seed(D + T)
    x = torch.randn((T, 1, D), generator=gen).to(torch.bfloat16)
    kv = torch.randn((E, D), generator=gen)
    turns = csa2.csa2_rope_turns(R)
    pos = torch.arange(T, dtype=torch.int32)
    kv_pos = torch.arange(E, dtype=torch.int32)
    kw = {}
    if E:
        g = csa2.Fp4Pages.empty(E // 8 + 1, 8, D, 1, E // 8 + 1)
        one = torch.zeros(1, dtype=torch.int32, device="cuda")
        csa2.fp4_kv_pages_resize(g, one, one + E)
        kw = dict(kv=kv.cuda(), kv_pos=kv_pos.cuda(), pages=g, entry=kv_pos.cuda(),
                  seq=torch.zeros(E, dtype=torch.int32, device="cuda"),
                  kv_out=torch.empty((E, D), dtype=torch.bfloat16, device="cuda"))
    got, stored = csa2.csa2_qk_norm_rope(turns, 0, interleaved=inter, q=x.cuda(), pos=pos.cuda(), **kw)
    some = list(range(0, T, max(1, T // 40))) + [T - 1]
    check(got[some], x[some], turns, 0, inter, torch.ones(D), 1e-6, pos[some])
    if E:
        fixed = turns.cpu().numpy().view(np.uint64)
        _, vals = pm.quantise(pm.norm_rope(kv.double().numpy(), kv_pos.numpy(), fixed, 0, inter,
                                           eps=float(np.float32(1e-6))))
        np.testing.assert_array_equal(stored.double().cpu().numpy(), vals)
    csa2.check_device_errors()
