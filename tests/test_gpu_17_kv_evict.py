"""The attention weight of cached rows (qattn_kv_weights) and the eviction by it
(qattn_kv_evict) against plain 64-bit forms, and the whole serving loop."""
import numpy as np
import pytest
import torch

from quantized_attention_gb300 import binding as qb
from quantized_attention_gb300.pipeline import Problem, TreeCache, tree_mask
from tests import tree_ref as R
from tests.gpu_common import ensure_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_library()


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def make(seed, B, Hq, Hkv, d, T, lens, q_gran, k_gran, cap=None, Nk=None):
    rng = np.random.default_rng(seed)
    Nk = max(lens) if Nk is None else Nk
    cap = Nk + 3 if cap is None else cap
    x = dict(B=B, Hq=Hq, Hkv=Hkv, d=d, T=T, lens=np.asarray(lens, np.int32), cap=cap, Nk=Nk, rng=rng)
    x["qc"] = rng.integers(-127, 128, (B, Hq, T, d)).astype(np.int8)
    x["kc"] = np.clip(np.rint(rng.normal(size=(B, Hkv, cap, d)) * 28), -127, 127).astype(np.int8)
    nq = {0: (1, 1, 1), 1: (B, Hq, 1), 2: (B, Hq, (T + 127) // 128)}[q_gran]
    nk = {0: (1, 1, 1), 1: (B, Hkv, 1), 2: (B, Hkv, (Nk + 127) // 128)}[k_gran]
    x["qs"] = (rng.uniform(0.5, 1.0, nq) * 2.0 / 74.0).astype(np.float32)
    x["ks"] = (rng.uniform(0.5, 1.0, nk) / 28.0).astype(np.float32)
    return x


def scales(s, H, N, B):
    """A scale per (b, h, token)."""
    s = np.broadcast_to(s, (B, H, s.shape[2]))
    return s[:, :, np.minimum(np.arange(N) // 128, s.shape[2] - 1)]


def see_of(T, L, causal, pos0):
    if not causal:
        return np.ones((T, L), bool)
    p = L - T if pos0 is None else pos0
    return np.arange(L)[None] <= (p + np.arange(T))[:, None]


CASES = [
    # B, Hq, Hkv, d, T, lengths, causal, pos0
    (1, 4, 1, 128, 1, [1000], False, None),
    (2, 6, 2, 64, 3, [0, 257], False, None),
    (3, 8, 2, 128, 5, [1, 33, 300], True, None),
    (1, 2, 2, 64, 130, [517], True, None),        # more than one Q scale block
    (1, 4, 2, 128, 300, [300], True, None),       # a whole causal prompt
    (1, 8, 1, 128, 64, [500], True, None),
    (1, 4, 1, 128, 200, [150], True, None),       # the first queries see nothing
    (1, 2, 1, 64, 20, [100], True, 40),           # tokens in the middle of the cache
    (1, 3, 1, 64, 9, [70], True, -4),
    (3, 8, 2, 128, 300, [985, 1500, 0], True, None),   # many tiles a unit, ragged
    (3, 16, 1, 64, 200, [700, 100, 1300], True, None),  # some sequences shorter than their queries
    (2, 6, 2, 128, 40, [1300, 513], False, None),       # one packed tile that stays for a run of units
    (4, 4, 4, 64, 400, [300, 900, 1, 650], False, None),  # the most tiles that stay
]


@pytest.mark.parametrize("case", CASES, ids=[f"H{c[1]}-{c[2]}-d{c[3]}-T{c[4]}-L{max(c[5])}-c{int(c[6])}-p{c[7]}"
                                             for c in CASES])
@pytest.mark.parametrize("q_gran,k_gran", [(2, 2), (0, 1), (1, None)])
def test_weights_match_fp64(case, q_gran, k_gran):
    """Per key, the sum of n positive terms: each off by e = ln 2 (2 roundings of
    the exponent's parts, at most 2 max|t| each, plus lse log2 e's own) 2^-24 +
    2^-22 (ex2), the additions by one rounding (2^-24) each: relative."""
    B, Hq, Hkv, d, T, lens, causal, pos0 = case
    x = make(31, B, Hq, Hkv, d, T, lens, q_gran, 1 if k_gran is None else k_gran)
    if k_gran is None:
        x["ks"][:] = 1.0
        x["qs"] /= 28.0
    sm = 1.0 / np.sqrt(d)
    G, qs, ks = Hq // Hkv, scales(x["qs"], Hq, T, B), scales(x["ks"], Hkv, x["Nk"], B)
    lse = np.full((B, Hq, T), -np.inf, np.float32)
    for b in range(B):
        L = lens[b]
        for h in range(Hq):
            s = (x["qc"][b, h].astype(np.float64) @ x["kc"][b, h // G, :L].astype(np.float64).T) * sm
            s = s * qs[b, h][:, None] * ks[b, h // G][None, :L]
            s = np.where(see_of(T, L, causal, pos0), s, -np.inf)
            m = s.max(axis=1, initial=-np.inf)
            ok = m > -np.inf
            lse[b, h, ok] = (m + np.log(np.exp(s - np.where(ok, m, 0)[:, None]).sum(axis=1).clip(1e-300)))[ok]
    if T > 2:
        lse[0, 0, 1] = -np.inf  # a query that does not count
    base = x["rng"].random((B, Hkv, x["cap"])).astype(np.float32)
    shape = qb.make_shape(B, Hq, Hkv, T, x["Nk"], d)
    params = qb.make_params(causal=causal, q_pos0=pos0, q_gran=q_gran, k_gran=1 if k_gran is None else k_gran,
                            kv_capacity=x["cap"])
    for use_base in (False, True):
        out = torch.full((B, Hkv, x["cap"]), -7.0, device="cuda")
        qb.kv_weights(dev(x["qc"]), dev(x["qs"]), dev(x["kc"]), None if k_gran is None else dev(x["ks"]),
                      dev(lse), shape, params, out, base=dev(base) if use_base else None, lengths=dev(x["lens"]))
        torch.cuda.synchronize()
        assert qb.get_error() == 0
        got = out.cpu().numpy().astype(np.float64)
        for b in range(B):
            L = lens[b]
            assert np.all(got[b, :, L:] == -7.0)
            for hk in range(Hkv):
                want, big = np.zeros(L), 0.0
                for h in range(hk * G, (hk + 1) * G):
                    wh, t = R.weight(x["qc"][b, h], qs[b, h], x["kc"][b, hk, :L], ks[b, hk][:L],
                                     lse[b, h].astype(np.float64), see_of(T, L, causal, pos0), sm)
                    want, big = want + wh, max(big, t)
                top = np.abs(lse[b][np.isfinite(lse[b])]).max(initial=0.0) / np.log(2)
                e = np.log(2) * (4 * big + 2 * top) * 2.0 ** -24 + 2.0 ** -22
                tol = want * (e + (G * T + 8) * 2.0 ** -24) + (2.0 ** -23 * (want + 1) if use_base else 0)
                np.testing.assert_array_less(np.abs(got[b, hk, :L] - want - (base[b, hk, :L] if use_base else 0)),
                                             tol + 1e-30)


def test_weights_in_place_and_repeatable():
    x = make(32, 1, 8, 2, 128, 40, [900], 2, 2)
    shape = qb.make_shape(1, 8, 2, 40, 900, 128)
    params = qb.make_params(kv_capacity=x["cap"])
    args = (dev(x["qc"]), dev(x["qs"]), dev(x["kc"]), dev(x["ks"]), torch.full((1, 8, 40), 9.0, device="cuda"))
    a = torch.zeros(1, 2, x["cap"], device="cuda")
    qb.kv_weights(*args, shape, params, a)
    b = torch.zeros_like(a)
    qb.kv_weights(*args, shape, params, b, base=b)
    assert torch.equal(a, b)
    qb.kv_weights(*args, shape, params, b, base=b)
    torch.cuda.synchronize()
    # fp32: x + x is exact
    assert torch.equal(b[:, :, :900], 2 * a[:, :, :900]) and qb.get_error() == 0


def test_weights_of_no_queries_and_bad_lengths():
    """No query: the base as it is.  Lengths outside the cache are clamped and
    reported, for few rows and for many."""
    base = torch.rand(2, 2, 70, device="cuda")
    for T in (0, 3, 70):
        x = make(33, 2, 4, 2, 64, T, [70, 20], 2, 2, cap=70)
        shape = qb.make_shape(2, 4, 2, T, 70, 64)
        lse = torch.full((2, 4, T), 5.0, device="cuda")
        args = (dev(x["qc"]), dev(x["qs"]), dev(x["kc"]), dev(x["ks"]), lse, shape, qb.make_params(kv_capacity=70))
        w, v = torch.zeros_like(base), torch.zeros_like(base)
        qb.kv_weights(*args, w, base=base, lengths=dev(x["lens"]))
        torch.cuda.synchronize()
        assert qb.get_error() == 0 and torch.all(w[1, :, 20:] == 0)
        if T == 0:
            assert torch.equal(w[0], base[0]) and torch.equal(w[1, :, :20], base[1, :, :20])
        qb.kv_weights(*args, v, base=base, lengths=dev(np.array([71, -5], np.int32)))
        torch.cuda.synchronize()
        assert qb.get_error() == qb.ERR_INVALID_ARG
        assert torch.equal(v[0], w[0]) and torch.all(v[1] == 0)


def test_a_prompts_weights_after_prefill():
    """qattn_fwd's own codes and lse: each query hands out 1 per head, up to its
    lse's rounding (|lse| 2^-24 and the kernels' fp32 sums, 2^-17 in all)."""
    B, Hq, Hkv, N, d = 1, 4, 2, 600, 128
    torch.manual_seed(3)
    P = Problem(B, Hq, Hkv, N, N, d, causal=True, want_lse=True)
    Q, K, V = (torch.randn(B, h, N, d, device="cuda", dtype=torch.bfloat16) for h in (Hq, Hkv, Hkv))
    P.run(Q, K, V)
    w = torch.zeros(B, Hkv, N, device="cuda")
    qb.kv_weights(P.q_codes, P.q_scales, P.k_codes, P.k_scales, P.lse, P.shape, P.params, w)
    torch.cuda.synchronize()
    assert qb.get_error() == 0
    total = w.double().sum(dim=2).cpu().numpy()
    np.testing.assert_allclose(total, N * Hq / Hkv, rtol=2.0 ** -17)


# ------------------------------------------------------------------ eviction
def evict(x, w, budget, n_sink, n_recent, lens, Nk, ocap):
    B, H, cap, d = x["k"].shape
    out = dict(k=torch.full((B, H, ocap, d), 77, dtype=torch.int8, device="cuda"),
               v=torch.full((B, H, ocap, d), 78, dtype=torch.int8, device="cuda"),
               w=torch.full((B, H, ocap), -3.0, device="cuda"),
               kept=torch.full((B, H, budget), -9, dtype=torch.int32, device="cuda"),
               n=torch.full((B,), -1, dtype=torch.int32, device="cuda"),
               am=torch.full((B, H, d), -1.0, device="cuda"))
    qb.kv_evict(dev(x["k"]), dev(x["v"]), dev(w), budget, out["k"], out["v"], out["w"], out["kept"], out["n"],
                out["am"], lengths=None if lens is None else dev(np.asarray(lens, np.int32)), Nk=Nk,
                n_sink=n_sink, n_recent=n_recent)
    torch.cuda.synchronize()
    assert qb.get_error() == 0
    return {k: t.cpu().numpy() for k, t in out.items()}


def check_evict(x, w, budget, n_sink, n_recent, lens, Nk, ocap):
    out = evict(x, w, budget, n_sink, n_recent, lens, Nk, ocap)
    B, H = x["k"].shape[:2]
    for b in range(B):
        L = Nk if lens is None else lens[b]
        n = min(L, budget)
        assert out["n"][b] == n
        for h in range(H):
            rows = R.keep(w[b, h], L, budget, n_sink, n_recent)
            assert np.array_equal(out["kept"][b, h, :n], rows)
            assert np.all(out["kept"][b, h, n:] == -9)
            assert np.array_equal(out["k"][b, h, :n], x["k"][b, h, rows])
            assert np.array_equal(out["v"][b, h, :n], x["v"][b, h, rows])
            assert np.array_equal(out["w"][b, h, :n].view(np.uint32), w[b, h, rows].view(np.uint32))
            assert np.all(out["k"][b, h, n:] == 77) and np.all(out["v"][b, h, n:] == 78)
            assert np.all(out["w"][b, h, n:] == -3.0)
            amax = np.abs(x["v"][b, h, rows].astype(np.int32)).max(axis=0, initial=0)
            assert np.array_equal(out["am"][b, h], amax.astype(np.float32))


def cache(rng, B, H, cap, d):
    return dict(k=rng.integers(-127, 128, (B, H, cap, d)).astype(np.int8),
                v=rng.integers(-127, 128, (B, H, cap, d)).astype(np.int8))


@pytest.mark.parametrize("B,H,d,lens,budget,sink,recent", [
    (1, 1, 64, [1], 1, 0, 0),
    (1, 2, 128, [1000], 100, 4, 16),
    (3, 2, 32, [0, 50, 333], 51, 1, 50),
    (2, 3, 64, [4097, 17], 4096, 0, 0),
    (1, 1, 128, [70000], 5000, 4, 100),
    (1, 1, 32, [9], 8, 8, 0),                 # everything protected but one
    (2, 1, 128, [130, 257], 300, 3, 7),       # below the budget: all kept
])
@pytest.mark.parametrize("kind", ["spread", "ties", "special"])
def test_evict_matches_a_full_sort(B, H, d, lens, budget, sink, recent, kind):
    rng = np.random.default_rng(41)
    cap, ocap = max(lens) + 7, budget + 3
    x = cache(rng, B, H, cap, d)
    w = np.exp(2 * rng.normal(size=(B, H, cap))).astype(np.float32)
    if kind == "ties":      # few values, most rows zero of either sign
        w = rng.choice(np.array([0.0, -0.0, 0.0, 0.25, 1.0], np.float32), size=w.shape)
    if kind == "special":   # NaN, infinities, negatives, denormals, the lowest value
        w[rng.random(w.shape) < 0.3] = np.nan
        w[rng.random(w.shape) < 0.1] = -np.inf
        w[rng.random(w.shape) < 0.1] = np.finfo(np.float32).min
        w[rng.random(w.shape) < 0.1] = 1e-42
        w[rng.random(w.shape) < 0.02] = np.inf
    check_evict(x, w, budget, sink, recent, lens, max(lens), ocap)


def test_evict_without_lengths_and_all_equal():
    rng = np.random.default_rng(42)
    x = cache(rng, 2, 2, 5000, 64)
    check_evict(x, np.full((2, 2, 5000), 0.5, np.float32), 777, 3, 11, None, 4999, 800)


def test_evict_more_rows_than_shared_memory_holds():
    """Slices past 40960 rows are read again from memory each round."""
    rng = np.random.default_rng(43)
    n = 8 * 40960 + 4321
    x = cache(rng, 1, 1, n, 32)
    w = np.exp(2 * rng.normal(size=(1, 1, n))).astype(np.float32)
    check_evict(x, w, 100001, 4, 1000, [n], n, 100001)


# ------------------------------------------------------------------ all together
def test_serving_loop():
    """Verify, weigh, commit and evict over several steps through TreeCache, each
    step against the plain forms run on the same state."""
    rng = np.random.default_rng(51)
    B, Hq, Hkv, d, T, cap = 2, 8, 2, 128, 12, 240
    G = Hq // Hkv
    lens = [150, 97]
    kc = np.zeros((B, Hkv, cap, d), np.int8)
    vc = np.zeros_like(kc)
    for b in range(B):
        kc[b, :, :lens[b]] = np.clip(np.rint(rng.normal(size=(Hkv, lens[b], d)) * 28), -127, 127)
        vc[b, :, :lens[b]] = np.clip(np.rint(rng.normal(size=(Hkv, lens[b], d)) * 28), -127, 127)
    ks = rng.uniform(0.02, 0.06, (B, Hkv, d)).astype(np.float32)
    vs = rng.uniform(0.02, 0.06, (B, Hkv, d)).astype(np.float32)
    mean = rng.normal(size=(B, Hkv, d)).astype(np.float32)
    amax = np.abs(vc.astype(np.float32)).max(axis=2)
    C = TreeCache(dev(kc), dev(vc), dev(ks), dev(vs), dev(mean), dev(amax), dev(np.asarray(lens, np.int32)), Hq, T,
                  out_dtype=qb.DT_F32)
    evicted = False
    for step in range(6):
        parents = torch.tensor([[int(rng.integers(-1, j)) if j else -1 for j in range(T)] for _ in range(B)])
        mask = tree_mask(parents).cuda()
        Q = torch.randn(B, Hq, T, d, device="cuda").to(torch.bfloat16)
        K = (dev(mean)[:, :, None] + 1.2 * torch.randn(B, Hkv, T, d, device="cuda")).to(torch.bfloat16)
        V = (1.2 * torch.randn(B, Hkv, T, d, device="cuda")).to(torch.bfloat16)
        before = {k: getattr(C, k).cpu().numpy().copy() for k in ("k_codes", "v_codes", "k_mean", "v_code_amax",
                                                                   "lengths", "seen", "weights")}
        C.verify(Q, K, V, mask)
        # accepted: a path from the root, as long as the tree allows
        path, n = np.zeros((B, T), np.int32), np.zeros(B, np.int32)
        for b in range(B):
            chain, j = [], int(rng.integers(0, T))
            while j >= 0:
                chain.append(j)
                j = int(parents[b, j])
            n[b] = len(chain)
            path[b, :n[b]] = chain[::-1]
        lse = C.lse.clone()
        counted = torch.zeros(B, T, dtype=torch.bool)
        for b in range(B):
            counted[b, path[b, :n[b]].tolist()] = True
        lse.masked_fill_(~counted[:, None].cuda(), -float("inf"))
        C.weigh(lse)
        C.commit(K, V, dev(path), dev(n))
        torch.cuda.synchronize()
        assert qb.get_error() == 0
        qc, qs = C.q_codes.cpu().numpy(), C.q_scales.cpu().numpy().reshape(B, Hq)
        Kf, Vf = K.float().cpu().numpy(), V.float().cpu().numpy()
        words = mask.cpu().numpy().view(np.uint32)[:, :, 0]
        for b in range(B):
            L = int(before["lengths"][b])
            see = ((words[b][:, None] >> np.arange(T, dtype=np.uint32)) & 1).astype(bool)
            for h in range(Hkv):
                dk, dv = R.draft_codes(Kf[b, h], Vf[b, h], before["k_mean"][b, h], ks[b, h], vs[b, h])
                kk = np.concatenate([before["k_codes"][b, h, :L], dk])
                vv = np.concatenate([before["v_codes"][b, h, :L], dv])
                total = before["weights"][b, h, :L].astype(np.float64)
                for hq in range(h * G, (h + 1) * G):
                    o, z, A, big = R.attend(qc[b, hq], float(qs[b, hq]) / np.sqrt(d), kk, vv, vs[b, h],
                                            R.visible(T, L, see, "tree"))
                    e_p = np.log(2) * 4 * big * 2.0 ** -24 + 2.0 ** -22
                    tol = A * (2.0 ** -11 + 2 * e_p + 2.0 ** -13) + 127 * vs[b, h].max() * len(kk) * 2.0 ** -25
                    np.testing.assert_array_less(np.abs(C.O[b, hq].double().cpu().numpy() - o), tol)
                    ztol = e_p + 2.0 ** -13 + 2.0 ** -22 * (np.abs(z) + 2 * big)
                    got_z = C.lse[b, hq].double().cpu().numpy()
                    np.testing.assert_array_less(np.abs(got_z - z), ztol)
                    wh, _ = R.weight(qc[b, hq], np.full(T, qs[b, hq]), kk[:L], np.ones(L),
                                     lse[b, hq].double().cpu().numpy(), np.ones((T, L), bool), 1 / np.sqrt(d))
                    total += wh
                # relative 2^-14 covers the exponent's 2^-24 (4 max|t| + 2 |lse|) ln 2 + 2^-22
                got = C.weights[b, h].cpu().numpy().astype(np.float64)
                np.testing.assert_allclose(got[:L], total, rtol=2.0 ** -14)
                assert np.all(got[L:L + n[b]] == 0)
            ck, cv = before["k_codes"][b].copy(), before["v_codes"][b].copy()
            m, am = R.commit(Kf[b], Vf[b], path[b], int(n[b]), L, int(before["seen"][b]), ks[b], vs[b],
                             before["k_mean"][b], before["v_code_amax"][b], ck, cv)
            assert np.array_equal(C.k_codes[b].cpu().numpy(), ck) and np.array_equal(C.v_codes[b].cpu().numpy(), cv)
            assert np.array_equal(C.k_mean[b].cpu().numpy(), m)
            assert np.array_equal(C.v_code_amax[b].cpu().numpy(), am)
            assert int(C.lengths[b]) == L + n[b]
        if step % 3 == 2:  # every third step: the cache cut to 120 rows
            old = {k: getattr(C, k).cpu().numpy().copy() for k in ("k_codes", "v_codes", "weights", "lengths")}
            cut = 120
            kept = C.evict(cut, n_sink=2, n_recent=8).cpu().numpy()
            torch.cuda.synchronize()
            evicted = True
            for b in range(B):
                m = min(int(old["lengths"][b]), cut)
                assert int(C.lengths[b]) == m
                for h in range(Hkv):
                    rows = R.keep(old["weights"][b, h], int(old["lengths"][b]), cut, 2, 8)
                    assert np.array_equal(kept[b, h, :m], rows)
                    assert np.array_equal(C.k_codes[b, h, :m].cpu().numpy(), old["k_codes"][b, h, rows])
                    assert np.array_equal(C.v_codes[b, h, :m].cpu().numpy(), old["v_codes"][b, h, rows])
    assert evicted and qb.get_error() == 0


def tree_cache(rng, B, Hq, Hkv, d, T, cap, lens):
    code = lambda: np.clip(np.rint(rng.normal(size=(B, Hkv, cap, d)) * 28), -127, 127).astype(np.int8)  # noqa: E731
    scale = lambda: rng.uniform(0.02, 0.06, (B, Hkv, d)).astype(np.float32)  # noqa: E731
    return TreeCache(dev(code()), dev(code()), dev(scale()), dev(scale()),
                     dev(rng.normal(size=(B, Hkv, d)).astype(np.float32)), torch.zeros(B, Hkv, d, device="cuda"),
                     dev(np.asarray(lens, np.int32)), Hq, T, out_dtype=qb.DT_F32)


@pytest.mark.parametrize("T", [3, 40])
def test_weigh_after_a_verify_without_drafts(T):
    """Queries whose rows are in the cache already see it causally, and so do their
    weights: each query hands out 1."""
    rng = np.random.default_rng(61)
    B, Hq, Hkv, d, cap, lens = 2, 4, 2, 64, 200, [200, 71]
    C = tree_cache(rng, B, Hq, Hkv, d, T, cap, lens)
    C.verify(torch.randn(B, Hq, T, d, device="cuda").to(torch.bfloat16))
    C.weigh()
    torch.cuda.synchronize()
    assert qb.get_error() == 0
    qc, qs, lse = C.q_codes.cpu().numpy(), C.q_scales.cpu().numpy().reshape(B, Hq), C.lse.double().cpu().numpy()
    for b, L in enumerate(lens):
        see = np.arange(L)[None, :] <= L - T + np.arange(T)[:, None]
        for h in range(Hkv):
            kk = C.k_codes[b, h, :L].cpu().numpy()
            want = sum(R.weight(qc[b, hq], np.full(T, qs[b, hq]), kk, np.ones(L), lse[b, hq], see, 1 / np.sqrt(d))[0]
                       for hq in range(2 * h, 2 * h + 2))
            got = C.weights[b, h].cpu().numpy().astype(np.float64)
            # as in the serving loop: relative 2^-14
            np.testing.assert_allclose(got[:L], want, rtol=2.0 ** -14)
            assert np.all(got[L:] == 0)


def test_steps_on_another_stream_and_in_a_graph():
    """A step of the loop (verify, weigh, commit, evict) on a side stream, its first
    eviction's second set allocated there, gives the bits of the same step on the
    current stream; so does a captured step replayed."""
    B, Hq, Hkv, d, T, cap, lens = 2, 8, 2, 128, 9, 400, [310, 180]
    gen = torch.Generator(device="cuda").manual_seed(5)
    Q, K, V = (torch.randn(B, h, T, d, device="cuda", generator=gen).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    path = dev(np.tile(np.arange(T, dtype=np.int32), (B, 1)))
    n = dev(np.array([4, 9], np.int32))

    def state(C):
        return [getattr(C, k).clone() for k in ("O", "lse", "k_mean", "v_code_amax", "lengths", "seen")] + [
            t[b, :, :int(C.lengths[b])].clone() for t in (C.k_codes, C.v_codes, C.weights) for b in range(B)]

    def step(C, evict, stream=None):
        C.verify(Q, K, V, stream=stream)
        C.weigh(stream=stream)
        C.commit(K, V, path, n, stream=stream)
        return C.evict(100, 2, 20, stream=stream) if evict else None

    fresh = lambda: tree_cache(np.random.default_rng(62), B, Hq, Hkv, d, T, cap, lens)  # noqa: E731
    A = fresh()
    kept = step(A, True)
    torch.cuda.synchronize()
    want = state(A)
    S, side = fresh(), torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.empty(1 << 28, device="cuda").fill_(1.0)  # the current stream is busy meanwhile
    kept_s = step(S, True, side)
    side.synchronize()
    assert torch.equal(kept, kept_s)
    torch.cuda.synchronize()
    for x, y in zip(want, state(S)):
        assert torch.equal(x, y)
    E, C = fresh(), fresh()
    step(E, False)
    step(E, False)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(C, False)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    for x, y in zip(state(E), state(C)):
        assert torch.equal(x, y)
    assert qb.get_error() == 0
