"""Forks of thousands of pairs, by one cluster and by the wide launches: repeated
destinations near either end of the list, bad slots, sources that are destinations."""
import numpy as np
import pytest
import torch

from fp4_kv_cache_step_b200 import csa2
from tests import paged_model as pm

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


@pytest.mark.parametrize("n,M", [(2500, 3), (5000, 3), (2500, 9), (5000, 7)])
def test_forks_of_thousands(n, M):
    r = np.random.RandomState(n + M)
    page, D = 8, 128
    S = n + 900
    # the first third of the slots holds something, in scattered pages
    P = S * M // 2
    held = r.randint(0, M + 1, S)
    held[S // 3:] = 0
    order = r.permutation(P)
    m = pm.Cache(np.zeros((P, page, D // 2 + D // 16), np.uint8), S, M)
    at = 0
    for s in range(S // 3):
        k = int(held[s])
        m.table[s, :k] = order[at: at + k]
        m.length[s] = max(0, k * page - r.randint(0, page)) if k else 0
        at += k
    m.refs[order[:at]] = 1
    g = csa2.Fp4Pages(torch.from_numpy(m.rows).cuda(), i32(m.table), i32(m.length), i32(m.refs))
    src, dst = r.randint(0, S, n), r.permutation(S)[:n]
    dst[1], dst[n // 2], dst[n - 2] = dst[n - 1], dst[n // 2 - 300], dst[0]
    src[3], dst[n - 5] = S, -1
    m.fork(src, dst)
    csa2.fp4_kv_pages_fork(g, i32(src), i32(dst))
    np.testing.assert_array_equal(g.table.cpu().numpy(), m.table)
    np.testing.assert_array_equal(g.length.cpu().numpy(), m.length)
    np.testing.assert_array_equal(g.refs.cpu().numpy(), m.refs)
    with pytest.raises(csa2.Csa2Error, match="DEVICE_INDEX"):
        csa2.check_device_errors()
    # and again, sound: most places keep what they hold
    dst = r.permutation(S)[:n]
    m.fork(src % S, dst)
    csa2.fp4_kv_pages_fork(g, i32(src % S), i32(dst))
    np.testing.assert_array_equal(g.table.cpu().numpy(), m.table)
    np.testing.assert_array_equal(g.length.cpu().numpy(), m.length)
    np.testing.assert_array_equal(g.refs.cpu().numpy(), m.refs)
    csa2.check_device_errors()
