"""Host checks of the serving operators: refusals (nothing is launched), the
workspace's size and the ancestor words of a tree.  No GPU needed."""
import ctypes
import os

import numpy as np
import pytest
import torch

from quantized_attention_gb300 import binding as qb
from quantized_attention_gb300 import build
from quantized_attention_gb300.pipeline import tree_mask


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(qb.library_path()):
        build.build()
    return qb.lib()


vp = ctypes.c_void_p
FAKE, ODD = vp(1 << 20), vp((1 << 20) + 2)  # never dereferenced: validation fails first
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 5


def tree(L, shape=(2, 8, 2, 4, 100, 128), ws=1 << 30, params=None, **kw):
    names = ("q_codes", "q_scales", "k_codes", "v_codes", "k_chan_scale", "v_chan_scale", "k_mean", "lengths",
             "K_new", "k_strides", "V_new", "v_strides", "tree_mask")
    a = {n: FAKE for n in names}
    a.update(k_strides=None, v_strides=None, O=FAKE, lse=FAKE, workspace=FAKE)
    a.update(kw)
    s, p = qb.make_shape(*shape), params or qb.make_params(kv_capacity=128)
    return L.qattn_tree_decode(*[a[n] for n in names], ctypes.byref(s), ctypes.byref(p), a["O"], a["lse"],
                               a["workspace"], ws, None)


def test_tree_decode_refusals(L):
    for n in ("q_codes", "q_scales", "k_codes", "v_codes", "k_chan_scale", "v_chan_scale", "k_mean", "K_new", "V_new",
              "O"):
        assert tree(L, **{n: None}) == INVALID, n
    for n in ("q_codes", "k_codes", "v_codes", "O", "K_new", "V_new", "k_mean", "v_chan_scale", "lengths", "tree_mask",
              "lse", "q_scales"):
        assert tree(L, **{n: ODD}) == INVALID, n
    long = (2, 8, 2, 5, 128 * 1000, 128)  # long caches, 20 rows: shares in the workspace
    p = qb.make_params()
    assert tree(L, shape=long, params=p, workspace=None) == WORKSPACE
    assert tree(L, shape=long, params=p, ws=16) == WORKSPACE
    assert tree(L, shape=(2, 8, 2, 129, 100, 128)) == UNSUPPORTED  # more drafts than a mask holds
    assert tree(L, shape=(2, 8, 2, 4, 100, 32)) == UNSUPPORTED
    assert tree(L, shape=(2, 7, 2, 4, 100, 128)) == INVALID
    assert tree(L, params=qb.make_params(kv_capacity=99)) == INVALID
    assert tree(L, params=qb.make_params(kv_capacity=128, q_pos0=3)) == UNSUPPORTED
    assert tree(L, params=qb.make_params(kv_capacity=128, pv_mode=qb.PV_INT8)) == UNSUPPORTED
    assert tree(L, K_new=None, V_new=None) == INVALID  # a mask without drafts
    st = (ctypes.c_int64 * 4)(4 * 128, 4, 4 * 128, 1)  # rows not on 16-byte boundaries
    assert tree(L, k_strides=st) == INVALID
    for empty in ((0, 8, 2, 4, 100, 128), (2, 8, 2, 0, 100, 128)):
        assert tree(L, shape=empty) == OK


def test_tree_workspace(L):
    """None for short caches (a head's cluster joins itself); for long ones two shares
    of a row block per CTA, whatever the length."""
    p = qb.make_params()
    size = lambda *s: qb.tree_workspace_size(qb.make_shape(*s), p)  # noqa: E731
    assert size(0, 8, 2, 4, 100, 128) == 0 and size(1, 8, 2, 129, 100, 128) == 0
    assert size(1, 8, 2, 1, 100, 128) == 0  # short and few rows: joined inside a cluster
    assert size(1, 8, 2, 5, 100, 128) == 0 < size(1, 8, 2, 5, 100000, 128)
    assert 0 < size(1, 8, 2, 1, 100000, 128)
    assert size(1, 8, 2, 128, 10 ** 6, 128) == size(1, 8, 2, 128, 8 * 10 ** 6, 128) < 64 << 20


@pytest.mark.parametrize("B,Hq,Hkv,T", [(1, 8, 8, 1), (1, 8, 2, 8), (2, 16, 8, 4), (3, 20, 5, 40), (5, 12, 4, 128),
                                        (19, 32, 8, 16), (64, 8, 1, 2)])
def test_tree_workspace_grows_with_the_cache(L, B, Hq, Hkv, T):
    """A workspace for a cache's capacity serves every shorter one."""
    sizes = [qb.tree_workspace_size(qb.make_shape(B, Hq, Hkv, T, n, 128), qb.make_params())
             for n in list(range(0, 40000, 97)) + [10 ** 5, 10 ** 6]]
    assert sizes == sorted(sizes)


def commit(L, B=2, Hkv=2, T=4, d=64, cap=32, **kw):
    names = ("K_new", "k_strides", "V_new", "v_strides", "path", "n_accept")
    rest = ("k_chan_scale", "v_chan_scale", "lengths", "seen", "k_mean", "v_code_amax", "lengths_out", "seen_out",
            "k_mean_out", "v_code_amax_out", "weights", "k_codes", "v_codes")
    a = {n: FAKE for n in names + rest}
    a.update(k_strides=None, v_strides=None)
    a.update(kw)
    return L.qattn_tree_commit(*[a[n] for n in names], B, Hkv, T, d, cap, *[a[n] for n in rest], None)


def test_commit_refusals(L):
    for n in ("K_new", "V_new", "path", "n_accept", "k_chan_scale", "v_chan_scale", "lengths", "k_mean", "v_code_amax",
              "lengths_out", "k_mean_out", "v_code_amax_out", "k_codes", "v_codes", "seen", "seen_out"):
        assert commit(L, **{n: None}) == INVALID, n
    assert commit(L, path=ODD) == INVALID and commit(L, weights=ODD) == INVALID
    assert commit(L, d=1025) == INVALID and commit(L, cap=-1) == INVALID and commit(L, B=65536) == INVALID
    assert commit(L, cap=(1 << 24) + 1) == INVALID and commit(L, Hkv=0) == INVALID
    assert commit(L, B=0) == OK


def weights(L, shape=(2, 8, 2, 4, 100, 128), params=None, **kw):
    names = ("q_codes", "q_scales", "k_codes", "k_scales", "lse", "lengths")
    a = {n: FAKE for n in names}
    a.update(base=FAKE, weights=FAKE)
    a.update(kw)
    s, p = qb.make_shape(*shape), params or qb.make_params()
    return L.qattn_kv_weights(*[a[n] for n in names], ctypes.byref(s), ctypes.byref(p), a["base"], a["weights"], None)


def test_weights_refusals(L):
    for n in ("q_codes", "q_scales", "k_codes", "lse", "weights"):
        assert weights(L, **{n: None}) == INVALID, n
    for n in ("q_codes", "k_codes", "k_scales", "lse", "lengths", "base", "weights"):
        assert weights(L, **{n: ODD}) == INVALID, n
    assert weights(L, shape=(2, 8, 2, 4, 100, 32)) == UNSUPPORTED
    assert weights(L, shape=(2, 0, 40000, 4, 100, 128)) == UNSUPPORTED  # more KV heads than a grid holds
    assert weights(L, params=qb.make_params(kv_capacity=50)) == INVALID
    assert weights(L, params=qb.make_params(causal=True, q_pos0=1 << 40)) == UNSUPPORTED
    assert weights(L, shape=(0, 8, 2, 4, 100, 128)) == OK and weights(L, shape=(2, 8, 2, 4, 0, 128)) == OK


def evict(L, B=2, Hkv=2, Nk=100, d=64, cap=128, budget=10, sink=2, recent=3, ocap=16, **kw):
    ins = ("k_codes", "v_codes", "weights", "lengths")
    a = {n: FAKE for n in ins}
    a.update({n: vp(1 << 21) for n in ("k_out", "v_out", "weights_out", "kept", "lengths_out", "v_code_amax")})
    a.update(kw)
    return L.qattn_kv_evict(*[a[n] for n in ins], B, Hkv, Nk, d, cap, budget, sink, recent, a["k_out"], a["v_out"],
                            ocap, a["weights_out"], a["kept"], a["lengths_out"], a["v_code_amax"], None)


def test_evict_refusals(L):
    for n in ("k_codes", "v_codes", "weights", "k_out", "v_out", "weights_out", "kept", "lengths_out", "v_code_amax"):
        assert evict(L, **{n: None}) == INVALID, n
    assert evict(L, k_out=FAKE) == INVALID and evict(L, lengths_out=FAKE) == INVALID  # in place
    assert evict(L, budget=0) == INVALID and evict(L, budget=17) == INVALID
    assert evict(L, sink=8, recent=3) == INVALID and evict(L, sink=-1) == INVALID
    assert evict(L, Nk=129) == INVALID and evict(L, d=96) == UNSUPPORTED and evict(L, B=40000) == UNSUPPORTED
    assert evict(L, B=0) == OK


def test_tree_mask_words():
    """Each draft sees itself and its ancestors; padding sees nothing."""
    rng = np.random.default_rng(1)
    for T in (1, 5, 32, 33, 70, 128):
        parents = np.array([[int(rng.integers(-1, j)) if j else -1 for j in range(T)] for _ in range(2)])
        if T > 4:
            parents[1, T - 1] = -2
        w = tree_mask(torch.from_numpy(parents)).numpy().view(np.uint32)
        assert w.shape == (2, T, (T + 31) // 32)
        for b in range(2):
            for i in range(T):
                want, j = set(), i if parents[b, i] > -2 else -1
                while j >= 0:
                    want.add(j)
                    j = int(parents[b, j])
                assert {j for j in range(32 * w.shape[2]) if (int(w[b, i, j // 32]) >> (j % 32)) & 1} == want


@pytest.mark.parametrize("bad", [[[-1, 1]], [[-3, 0]], [[-1, 5]], [[-2, 0]]])
def test_tree_mask_refuses(bad):
    with pytest.raises(ValueError):
        tree_mask(torch.tensor(bad))
