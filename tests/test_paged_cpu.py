"""Host checks of rotary positions and the paged cache: refusals (nothing is
launched), the workspace's size, the angles' table.  No GPU needed."""
import ctypes
import math
import os

import pytest
import torch

from quantized_attention_gb300 import binding as qb
from quantized_attention_gb300 import build
from quantized_attention_gb300.pipeline import rope_table


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(qb.library_path()):
        build.build()
    return qb.lib()


vp = ctypes.c_void_p
FAKE, ODD = vp(1 << 20), vp((1 << 20) + 2)  # never dereferenced: validation fails first
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 5
ref = ctypes.byref


def rope(table=1 << 20, n=100, rot=64, layout=0, inverse=0):
    return qb.Rope(table, n, rot, layout, inverse)


def rotate(L, X=FAKE, st=None, dtype=qb.DT_BF16, dims=(2, 3, 5, 64), pos=None, r=None, Y=FAKE):
    return L.qattn_rotate(X, st, dtype, *dims, pos, ref(rope() if r is None else r), Y, None)


def test_rotate_refusals(L):
    assert rotate(L, X=None) == INVALID and rotate(L, X=ODD) == INVALID
    assert rotate(L, Y=None) == INVALID and rotate(L, Y=ODD) == INVALID
    assert rotate(L, pos=vp((1 << 20) + 1)) == INVALID
    assert rotate(L, dtype=qb.DT_I8) == INVALID
    assert L.qattn_rotate(FAKE, None, qb.DT_BF16, 2, 3, 5, 64, None, None, FAKE, None) == INVALID
    for bad in (rope(table=None), rope(table=(1 << 20) + 4), rope(rot=12), rope(rot=0), rope(rot=72), rope(layout=2),
                rope(inverse=2), rope(n=-1)):
        assert rotate(L, r=bad) == INVALID
    assert rotate(L, r=rope(n=1 << 31)) == UNSUPPORTED
    assert rotate(L, dims=(2, 3, 5, 96)) == UNSUPPORTED and rotate(L, dims=(2, 3, -1, 64)) == INVALID
    assert rotate(L, dims=(65535, 1, 65535, 64)) == UNSUPPORTED  # more tokens than 31 bits
    assert rotate(L, dims=(1, 70000, 1, 64)) == UNSUPPORTED
    odd = (ctypes.c_int64 * 4)(3 * 5 * 64, 5 * 64, 4, 1)
    assert rotate(L, st=odd) == INVALID
    token_major = (ctypes.c_int64 * 4)(3 * 5 * 64, 64, 3 * 64, 1)
    assert rotate(L, st=token_major) == INVALID  # in place needs a dense X
    for empty in ((0, 3, 5, 64), (2, 0, 5, 64), (2, 3, 0, 64)):
        assert rotate(L, dims=empty, X=None, Y=None) == OK


def paging(n=10, page=64, width=4, dt=qb.DT_I8):
    return qb.make_paging(n, page, width, dt)


SHAPE = (2, 8, 2, 4, 200, 128)


def append(L, shape=SHAPE, g=None, r=None, **kw):
    a = dict(Q=FAKE, K=FAKE, V=FAKE, lengths=FAKE, n_new=FAKE, positions=FAKE, page_table=FAKE, Q_out=vp(2 << 20),
             k_pages=FAKE, v_pages=FAKE, k_scales=FAKE, v_scales=FAKE, st=None)
    a.update(kw)
    return L.qattn_paged_append(a["Q"], None, a["K"], a["st"], a["V"], None, ref(qb.make_shape(*shape)), a["lengths"],
                                a["n_new"], a["positions"], ref(rope()) if r is None else r,
                                ref(paging() if g is None else g), a["page_table"], a["Q_out"], a["k_pages"],
                                a["v_pages"], a["k_scales"], a["v_scales"], None)


def fwd(L, shape=SHAPE, g=None, params=None, ws=1 << 30, **kw):
    a = dict(Q=FAKE, lengths=FAKE, n_new=FAKE, page_table=FAKE, k_pages=FAKE, v_pages=FAKE, k_scales=FAKE,
             v_scales=FAKE, O=FAKE, lse=FAKE, workspace=FAKE, st=None)
    a.update(kw)
    return L.qattn_paged_fwd(a["Q"], a["st"], ref(qb.make_shape(*shape)), ref(params or qb.make_params()), a["lengths"],
                             a["n_new"], ref(paging() if g is None else g), a["page_table"], a["k_pages"], a["v_pages"],
                             a["k_scales"], a["v_scales"], a["O"], a["lse"], a["workspace"], ws, None)


@pytest.mark.parametrize("call", [append, fwd])
def test_pool_and_shape_refusals(L, call):
    for g, want in ((paging(n=0), INVALID), (paging(n=-1), INVALID), (paging(page=16), UNSUPPORTED),
                    (paging(page=256), UNSUPPORTED), (paging(width=3), INVALID), (paging(width=-1), INVALID),
                    (paging(dt=qb.DT_BF16), INVALID), (paging(n=1 << 30), UNSUPPORTED)):
        assert call(L, g=g) == want
    assert call(L, shape=(2, 8, 2, 4, 200, 32)) == UNSUPPORTED
    assert call(L, shape=(2, 7, 2, 4, 200, 128)) == INVALID
    assert call(L, shape=(2, 8, 2, 4, -1, 128)) == INVALID
    for n in ("lengths", "page_table", "k_pages", "v_pages", "k_scales", "v_scales"):
        assert call(L, **{n: None}) == INVALID, n
        assert call(L, **{n: ODD}) == INVALID, n
    assert call(L, n_new=ODD) == INVALID
    bad = (ctypes.c_int64 * 4)(4 * 2 * 128, 4, 2 * 128, 1)  # rows not on 16-byte boundaries
    assert call(L, st=bad) == INVALID
    for empty in ((0, 8, 2, 4, 200, 128), (2, 8, 2, 0, 200, 128)):
        assert call(L, shape=empty) == OK


def test_append_refusals(L):
    for n in ("K", "V"):
        assert append(L, **{n: None}) == INVALID and append(L, **{n: ODD}) == INVALID
    assert append(L, Q=None) == INVALID and append(L, Q_out=None) == INVALID  # both or neither
    assert append(L, Q=ODD) == INVALID and append(L, Q_out=ODD) == INVALID
    assert append(L, positions=ODD) == INVALID
    assert append(L, r=ref(rope(rot=136))) == INVALID and append(L, r=ref(rope(table=None))) == INVALID
    assert append(L, shape=(1, 8, 2, 65535 * 32, 100, 128), g=paging(page=32)) == UNSUPPORTED


def test_fwd_refusals_and_workspace(L):
    for n in ("Q", "O"):
        assert fwd(L, **{n: None}) == INVALID and fwd(L, **{n: ODD}) == INVALID
    assert fwd(L, lse=ODD) == INVALID
    for p in (qb.make_params(q_pos0=3), qb.make_params(pv_mode=qb.PV_INT8), qb.make_params(kv_capacity=256)):
        assert fwd(L, params=p) == UNSUPPORTED
    assert fwd(L, params=qb.make_params(sm_scale=-1.0)) == INVALID
    long, g, p = (2, 8, 2, 1, 64 * 3000, 128), paging(n=9000, width=3000), qb.make_params(causal=True)
    need = qb.paged_workspace_size(qb.make_shape(*long), p, g)
    assert need > 0
    assert fwd(L, shape=long, g=g, params=p, workspace=None) == WORKSPACE
    assert fwd(L, shape=long, g=g, params=p, ws=need - 1) == WORKSPACE
    assert fwd(L, shape=long, g=g, params=p, workspace=ODD) == WORKSPACE
    assert qb.paged_workspace_size(qb.make_shape(0, 8, 2, 1, 64, 128), p, g) == 0
    assert qb.paged_workspace_size(qb.make_shape(2, 8, 2, 1, 64, 32), p, g) == 0
    sizes = [qb.paged_workspace_size(qb.make_shape(2, 8, 2, T, n, 128), p, g) for T in (1, 40)
             for n in (1, 500, 9000, 64 * 3000)]
    assert sizes[:4] == sorted(sizes[:4]) and sizes[4:] == sorted(sizes[4:])  # never shrinks as Nk grows


def test_binding_names_what_is_missing():
    with pytest.raises(ValueError, match="4-D"):
        qb.rotate(None, None, None)
    with pytest.raises(TypeError, match="bfloat16 or torch.float32"):
        qb.rotate(torch.zeros(1, 1, 1, 64, dtype=torch.float16), None, None)
    with pytest.raises(ValueError, match="rope is missing"):
        qb.rotate(torch.zeros(1, 1, 1, 64), None, None)
    with pytest.raises(ValueError, match="CUDA"):
        qb.make_rope(torch.zeros(4, 64))
    with pytest.raises(ValueError, match="K is missing"):
        qb._strided_ptr(0, "K", None, torch.bfloat16, (1, 2, 3, 64))
    with pytest.raises(ValueError, match="expected shape"):
        qb._strided_ptr(0, "K", torch.zeros(1, 2, 3, 64), torch.bfloat16, (1, 2, 4, 64))


def test_rope_table_angles():
    """Against the definition, in Python's own 64-bit functions: off by half a step of
    fp32 of the value, and by what 64 bits lose in an angle of up to 2^17 (2^-35)."""
    n, rot = 131072, 32
    for kw in ({}, dict(scaling="linear", factor=4.0), dict(scaling="base", factor=4.0), dict(base=5e5, mscale=1.3),
               dict(scaling="ramp", factor=8.0, trained=8192, slow=1.0, fast=4.0)):
        t = rope_table(n, rot, device="cpu", **kw)
        assert t.shape == (n, rot) and t.dtype == torch.float32
        base = kw.get("base", 10000.0)
        f = kw.get("factor", 1.0)
        if kw.get("scaling") == "base":
            base *= f ** (rot / (rot - 2))
        for i in range(rot // 2):
            w = base ** (-2 * i / rot)
            if kw.get("scaling") == "linear":
                w /= f
            if kw.get("scaling") == "ramp":
                turns = w * kw["trained"] / (2 * math.pi)
                keep = min(1.0, max(0.0, (turns - kw["slow"]) / (kw["fast"] - kw["slow"])))
                w = w * keep + w / f * (1 - keep)
            for p in (0, 1, 77, 131071):
                m = kw.get("mscale", 1.0)
                assert abs(float(t[p, i]) - m * math.cos(p * w)) <= 2.0 ** -25 * m * 2 + 2.0 ** -34
                assert abs(float(t[p, rot // 2 + i]) - m * math.sin(p * w)) <= 2.0 ** -25 * m * 2 + 2.0 ** -34
    for bad in (dict(rot_dim=12), dict(rot_dim=0), dict(rot_dim=32, scaling="other")):
        with pytest.raises(ValueError):
            rope_table(4, device="cpu", **bad)
