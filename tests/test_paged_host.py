"""The paged cache's calls without a GPU: refusals before anything is launched,
workspace sizes, the struct layouts and the rotation frequencies."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

from tests import paged_model as pm
from fp4_kv_cache_step_b200 import build as libbuild
from fp4_kv_cache_step_b200 import csa2

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return csa2.load()


A = 256          # an aligned address that no refused call reads


def pages(**kw):
    d = dict(rows=A, table=A, len=A, refs=A, P=64, page=16, D=512, S=4, M=8)
    d.update(kw)
    return csa2.PagesStruct(*(d[k] for k in ("rows", "table", "len", "refs", "P", "page", "D", "S",
                                             "M")))


def status(rc):
    return csa2.STATUS[rc]


@pytest.mark.parametrize("bad", [dict(rows=None), dict(table=A + 4), dict(len=None), dict(refs=8),
                                 dict(page=12), dict(page=4), dict(page=1 << 17), dict(D=96),
                                 dict(D=1152), dict(S=0), dict(S=65537), dict(M=0),
                                 dict(M=1 << 27), dict(P=0), dict(P=1 << 27)])
def test_bad_caches_are_refused_by_every_call(lib, bad):
    pg = ctypes.byref(pages(**bad))
    p, big = ctypes.c_void_p(A), 1 << 40
    assert status(lib.fp4_kv_pages_resize(pg, p, p, 1, p, big, None)) == "INVALID_ARG"
    assert status(lib.fp4_kv_pages_fork(pg, p, p, 1, p, big, None)) == "INVALID_ARG"
    assert status(lib.fp4_kv_pages_compact(pg, None, p, big, None)) == "INVALID_ARG"
    assert status(lib.csa2_paged_attn(p, pg, None, None, None, 1, 1, 8, 0, 1.0, p, None, p, big,
                                      None)) == "INVALID_ARG"
    a = rope_args()
    assert status(lib.csa2_qk_norm_rope(ctypes.byref(a), pg, None)) == "INVALID_ARG"


def rope_args(**kw):
    a = csa2.NormRopeArgs()
    d = dict(D=512, R=64, rot_begin=448, interleaved=1, rot_scale=1.0, eps=1e-6, turns=A, T=2,
             Hq=4, q_norm=1, q=1 << 20, q_stride=2048, pos=A, q_weight=A, q_out=1 << 24, E=2,
             kv_norm=1, kv=A, kv_stride=512, kv_pos=A, seq=A, entry=A, kv_out=A)
    d.update(kw)
    for k, v in d.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad", [
    dict(D=500), dict(D=0), dict(R=63), dict(R=-2), dict(rot_begin=449), dict(rot_begin=-1),
    dict(R=1024), dict(turns=None), dict(T=-1), dict(E=-1), dict(eps=-1.0), dict(Hq=0),
    dict(Hq=65536), dict(q=None), dict(q=8), dict(q_out=None), dict(pos=None), dict(pos=2),
    dict(q_stride=2040), dict(q_stride=2052), dict(q_out=(1 << 20) + 16),
    dict(q_out=1 << 20, q_stride=2056), dict(q_out=1 << 20, q_f32=1), dict(kv=None),
    dict(kv_stride=504), dict(kv_stride=516), dict(kv_pos=None), dict(seq=None), dict(entry=None),
    dict(kv_out=8), dict(D=256, rot_begin=0, kv_stride=512, Hq=2)])
def test_bad_norm_rope_arguments_are_refused(lib, bad):
    a = rope_args(**bad)
    rc = lib.csa2_qk_norm_rope(ctypes.byref(a), ctypes.byref(pages()), None)
    assert status(rc) == "INVALID_ARG", csa2.load().csa2_last_error()


def test_entries_need_pages_and_queries_do_not(lib):
    a = rope_args()
    assert status(lib.csa2_qk_norm_rope(ctypes.byref(a), None, None)) == "INVALID_ARG"
    assert status(lib.csa2_qk_norm_rope(None, ctypes.byref(pages()), None)) == "INVALID_ARG"


@pytest.mark.parametrize("bad,want", [
    (dict(q=None), "INVALID_ARG"), (dict(out=None), "INVALID_ARG"), (dict(out=8), "INVALID_ARG"),
    (dict(B=-1), "INVALID_ARG"), (dict(B=65536), "INVALID_ARG"), (dict(B=5), "INVALID_ARG"),
    (dict(Hq=0), "INVALID_ARG"), (dict(Hq=65535, Tq=2), "INVALID_ARG"),
    (dict(lse=2), "INVALID_ARG"), (dict(nvalid=2), "INVALID_ARG"),
    (dict(topk=A, K=0), "INVALID_ARG"), (dict(ws=None), "WORKSPACE"),
    (dict(size=0), "WORKSPACE"), (dict(ws=8), "WORKSPACE"), (dict(pg=pages(D=256)), "UNSUPPORTED")])
def test_bad_attention_arguments_are_refused(lib, bad, want):
    d = dict(q=A, pg=pages(), seq=None, nvalid=None, topk=None, B=2, Tq=1, Hq=8, K=0, out=A,
             lse=None, ws=A, size=1 << 40)
    d.update(bad)
    rc = lib.csa2_paged_attn(d["q"], ctypes.byref(d["pg"]), d["seq"], d["nvalid"], d["topk"],
                             d["B"], d["Tq"], d["Hq"], d["K"], 1.0, d["out"], d["lse"], d["ws"],
                             d["size"], None)
    assert status(rc) == want


def test_page_calls_check_their_lists_and_workspaces(lib):
    pg = ctypes.byref(pages())
    for call, size in ((lib.fp4_kv_pages_resize, lib.fp4_kv_pages_resize_workspace_bytes),
                       (lib.fp4_kv_pages_fork, lib.fp4_kv_pages_fork_workspace_bytes)):
        need = size(pg, 3)
        assert need > 0 and need % 256 == 0 and size(pg, 0) == 0
        assert status(call(pg, A, A, 3, A, need - 256, None)) == "WORKSPACE"
        assert status(call(pg, A, A, 3, None, need, None)) == "WORKSPACE"
        assert status(call(pg, A, A, 3, A + 8, need, None)) == "WORKSPACE"
        assert status(call(pg, None, A, 3, A, need, None)) == "INVALID_ARG"
        assert status(call(pg, A, A + 2, 3, A, need, None)) == "INVALID_ARG"
        assert status(call(pg, A, A, -1, A, need, None)) == "INVALID_ARG"
        assert status(call(pg, A, A, 65537, A, 1 << 40, None)) == "INVALID_ARG"
        assert status(call(pg, None, None, 0, None, 0, None)) == "OK"
    need = lib.fp4_kv_pages_compact_workspace_bytes(pg)
    assert status(lib.fp4_kv_pages_compact(pg, None, A, need - 256, None)) == "WORKSPACE"
    assert status(lib.fp4_kv_pages_compact(pg, 2, A, need, None)) == "INVALID_ARG"


@pytest.mark.parametrize("scaling,kw", [("plain", {}), ("linear", dict(factor=16.0)),
                                        ("ntk", dict(factor=8.0)),
                                        ("yarn", dict(factor=16.0, context=4096.0)),
                                        ("yarn", dict(factor=1.0, context=65536.0, fast=40.0,
                                                      slow=2.0))])
@pytest.mark.parametrize("R", [0, 4, 64, 126, 512])
def test_rope_turns(lib, scaling, kw, R):
    got = csa2.csa2_rope_turns(R, 10000.0, scaling, device="cpu", **kw).numpy().view(np.uint64)
    want = pm.turns(R, 10000.0, scaling, **kw)
    assert got.shape == (R // 2,)
    # a handful of double operations each, of at most 2 ulp (pow): 2^-53 * 32; and a
    # fraction is a multiple of 2^-64, so rounding to one adds up to 2^-65
    assert np.all(np.abs(got.astype(np.float64) * 2.0 ** -64 - want)
                  <= want * 2.0 ** -48 + 2.0 ** -65)


@pytest.mark.parametrize("kw", [dict(R=3), dict(R=-2), dict(R=1026), dict(base=1.0),
                                dict(base=math.nan), dict(factor=0.5), dict(scaling="yarn"),
                                dict(scaling="yarn", context=100.0, fast=1.0, slow=1.0),
                                dict(R=2, scaling="ntk", factor=2.0)])
def test_rope_turns_refuses(lib, kw):
    kw = dict(dict(R=64), **kw)
    with pytest.raises((csa2.Csa2Error, ValueError)):
        if kw["R"] % 2 or kw["R"] < 0:
            buf = (ctypes.c_uint64 * 4096)()
            csa2._check(lib.csa2_rope_turns(kw["R"], 1e4, 0, 1.0, 0.0, 32.0, 1.0, buf), "turns")
        csa2.csa2_rope_turns(kw.pop("R"), device="cpu", **kw)
    with pytest.raises(ValueError):
        csa2.csa2_rope_turns(64, scaling="other", device="cpu")


def test_structs_match_the_header(tmp_path):
    fields = {"fp4_kv_pages": csa2.PagesStruct, "csa2_norm_rope_args": csa2.NormRopeArgs}
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "csa2.h"', "int main(void) {"]
    want = []
    for name, struct in fields.items():
        lines.append('  printf("%%zu\\n", sizeof(%s));' % name)
        want.append(ctypes.sizeof(struct))
        for f, _ in struct._fields_:
            lines.append('  printf("%%zu\\n", offsetof(%s, %s));' % (name, f))
            want.append(getattr(struct, f).offset)
    lines += ["  return 0;", "}"]
    (tmp_path / "l.c").write_text("\n".join(lines))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(tmp_path / "l.c"), "-o",
                    str(tmp_path / "l")], check=True)
    got = subprocess.run([str(tmp_path / "l")], capture_output=True, text=True, check=True).stdout
    assert [int(x) for x in got.split()] == want


def test_binding_refuses_tensors_that_do_not_fit():
    cpu = dict(dtype=torch.int32)
    rows, table = torch.zeros((4, 16, 288), dtype=torch.uint8), torch.zeros((2, 3), **cpu)
    with pytest.raises(ValueError):                       # not on a GPU
        csa2.Fp4Pages(rows, table, torch.zeros(2, **cpu), torch.zeros(4, **cpu))
    with pytest.raises(ValueError):                       # 100 bytes are no row
        csa2.Fp4Pages(torch.zeros((4, 16, 100), dtype=torch.uint8), table, torch.zeros(2, **cpu),
                      torch.zeros(4, **cpu))
    with pytest.raises(ValueError):
        csa2.Fp4Pages(rows, table, torch.zeros(3, **cpu), torch.zeros(4, **cpu))
    with pytest.raises(TypeError):
        csa2.Fp4Pages(rows, table.long(), torch.zeros(2, **cpu), torch.zeros(4, **cpu))
    turns = torch.zeros(32, dtype=torch.int64)
    with pytest.raises(ValueError):
        csa2.csa2_qk_norm_rope(turns, 0)
    with pytest.raises(TypeError):
        csa2.csa2_qk_norm_rope(turns, 0, q=torch.zeros((1, 2, 128), dtype=torch.float16),
                               pos=torch.zeros(1, **cpu))
    with pytest.raises(ValueError):
        csa2.csa2_qk_norm_rope(turns, 0, q=torch.zeros((1, 2, 128)).transpose(1, 2),
                               pos=torch.zeros(1, **cpu))
    with pytest.raises(ValueError):                       # entries without pages
        csa2.csa2_qk_norm_rope(turns, 0, kv=torch.zeros((1, 128)))


def test_model_quantises_like_the_oracle():
    import oracle
    oracle.build()
    x = np.random.RandomState(3).standard_normal((1, 37, 512)).astype(np.float32)
    x[0, 5] = 0.0
    x[0, 6, :16] = np.array([6, -6, 5, 2.5, 1.75, 0.25, -0.25, 0.75, 3.5, 1.25] + [0.0] * 6)
    rows, vals = pm.quantise(x.astype(np.float64))
    want = oracle.fp4_kv_pack_g16(x)
    np.testing.assert_array_equal(pm.values(rows, 512), pm.values(want, 512))
    np.testing.assert_array_equal(vals, pm.values(rows, 512))
