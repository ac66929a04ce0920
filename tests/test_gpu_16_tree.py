"""Tree attention over the int8 KV cache (qattn_tree_decode) and the commit of
the accepted path (qattn_tree_commit) against plain 64-bit forms."""
import numpy as np
import pytest
import torch

from quantized_attention_gb300 import binding as qb
from quantized_attention_gb300.pipeline import tree_mask
from tests import tree_ref as R
from tests.gpu_common import ensure_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_library()


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).float().numpy()


def random_mask(rng, B, T):
    """[B, T, T] ancestor masks of random trees, and their words."""
    parents = np.array([[int(rng.integers(-1, j)) if j else -1 for j in range(T)] for _ in range(B)])
    see = np.zeros((B, T, T), dtype=bool)
    for b in range(B):
        for j in range(T):
            if parents[b, j] >= 0:
                see[b, j] = see[b, parents[b, j]]
            see[b, j, j] = True
    return see, tree_mask(torch.from_numpy(parents))


def words_of(see):
    B, T, _ = see.shape
    W = (T + 31) // 32
    w = np.zeros((B, T, W), np.uint32)
    for j in range(T):
        w[:, :, j // 32] |= see[:, :, j].astype(np.uint32) << np.uint32(j % 32)
    return torch.from_numpy(w.view(np.int32))


def make(seed, B, Hq, Hkv, d, T, lens, cap=None, gain=1.0):
    rng = np.random.default_rng(seed)
    cap = max(max(lens), 1) + 5 if cap is None else cap
    x = dict(B=B, Hq=Hq, Hkv=Hkv, d=d, T=T, lens=np.asarray(lens, np.int32), cap=cap, rng=rng)
    x["qc"] = rng.integers(-127, 128, (B, Hq, T, d)).astype(np.int8)
    x["qs"] = (gain * rng.uniform(0.5, 1.0, (B, Hq)) * 3.0 / (74.0 * 28.0)).astype(np.float32)
    x["kc"] = np.clip(np.rint(rng.normal(size=(B, Hkv, cap, d)) * 28), -127, 127).astype(np.int8)
    x["vc"] = np.clip(np.rint(rng.normal(size=(B, Hkv, cap, d)) * 28), -127, 127).astype(np.int8)
    x["ks"] = rng.uniform(0.02, 0.06, (B, Hkv, d)).astype(np.float32)
    x["vs"] = rng.uniform(0.02, 0.06, (B, Hkv, d)).astype(np.float32)
    x["mean"] = (3.0 * rng.normal(size=(B, Hkv, d))).astype(np.float32)
    x["K"] = bf16(x["mean"][:, :, None] + 1.3 * rng.normal(size=(B, Hkv, T, d)))
    x["V"] = bf16(1.3 * rng.normal(size=(B, Hkv, T, d)))
    return x


def run(x, mode, words=None, out_dtype=qb.DT_F32, q_gran=qb.GRAN_BLOCK, lengths=True, strided=False,
        Nk=None, stream=None, ws_fill=0xFF):
    B, Hq, Hkv, d, T = (x[k] for k in ("B", "Hq", "Hkv", "d", "T"))
    Nk = int(x["lens"].max()) if Nk is None else Nk
    shape = qb.make_shape(B, Hq, Hkv, T, Nk, d)
    params = qb.make_params(causal=mode in ("chain", "cached_causal"), out_dtype=out_dtype, q_gran=q_gran,
                            kv_capacity=x["cap"])
    dt = torch.bfloat16 if out_dtype == qb.DT_BF16 else torch.float32
    O = torch.full((B, Hq, T, d), float("nan"), dtype=dt, device="cuda")
    lse = torch.full((B, Hq, T), float("nan"), device="cuda")
    ws = torch.full((max(qb.tree_workspace_size(shape, params), 256),), ws_fill, dtype=torch.uint8,
                    device="cuda")
    K, V = dev(x["K"], torch.bfloat16), dev(x["V"], torch.bfloat16)
    if strided:  # a packed projection output [B][T][2][Hkv][d]
        pack = torch.stack([K.transpose(1, 2), V.transpose(1, 2)], dim=2).contiguous()
        K, V = pack[:, :, 0].transpose(1, 2), pack[:, :, 1].transpose(1, 2)
        assert not K.is_contiguous() or T == 1 or Hkv == 1
    kw = {}
    if not mode.startswith("cached"):
        kw = dict(K_new=K, V_new=V, k_mean=dev(x["mean"]), tree_mask=None if words is None else words.cuda())
    qb.tree_decode(dev(x["qc"]), dev(x["qs"]), dev(x["kc"]), dev(x["vc"]), dev(x["ks"]), dev(x["vs"]),
                   shape, params, O, lse, ws, lengths=dev(x["lens"]) if lengths else None, stream=stream,
                   **kw)
    torch.cuda.synchronize()
    assert qb.get_error() == 0
    return O, lse


def check(x, mode, O, lse, see=None, sm=None):
    """Against the 64-bit form.  The error allowed per element, with A = sum P |v| / l:
    P's rounding to fp16, half a step each (2^-11 of P, 2^-25 below the normal
    range); e_p = the relative error of one P in fp32, its exponent t - m off by
    two roundings of at most 2 max|t| (2^-24 each, times ln 2) and ex2 by 2^-22,
    counted in the sum and in l; the fp32 additions, one rounding (taken whole,
    2^-23) per 16-key product, per join of shares and per warp; the output's own
    rounding."""
    T, d, G = x["T"], x["d"], x["Hq"] // x["Hkv"]
    sm = 1.0 / np.sqrt(d) if sm is None else sm
    half = torch.finfo(O.dtype).eps / 2
    O, lse = O.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(x["B"]):
        L = int(x["lens"][b])
        for h in range(x["Hkv"]):
            k, v = x["kc"][b, h, :L], x["vc"][b, h, :L]
            if not mode.startswith("cached"):
                dk, dv = R.draft_codes(x["K"][b, h], x["V"][b, h], x["mean"][b, h], x["ks"][b, h], x["vs"][b, h])
                k, v = np.concatenate([k, dk]), np.concatenate([v, dv])
            vis = R.visible(T, L, None if see is None else see[b], mode)
            for hq in range(h * G, (h + 1) * G):
                o, z, A, big = R.attend(x["qc"][b, hq], float(x["qs"].reshape(x["B"], -1)[b, hq]) * sm, k, v,
                                        x["vs"][b, h], vis)
                e_p = np.log(2) * 2 * 2 * big * 2.0 ** -24 + 2.0 ** -22
                adds = (len(k) / 16 + 700) * 2.0 ** -23
                vmax = 127 * float(x["vs"][b, h].max())
                tol = A * (2.0 ** -11 + 2 * e_p + 2 * adds) + len(k) * vmax * 2.0 ** -25 + half * np.abs(o)
                np.testing.assert_array_less(np.abs(O[b, hq] - o), tol + 1e-30, err_msg=f"O b{b} h{hq} {mode}")
                fin = np.isfinite(z)
                assert np.array_equal(np.isfinite(lse[b, hq]), fin) and np.all(lse[b, hq][~fin] == -np.inf)
                ztol = e_p + adds + 2.0 ** -23 * (np.abs(z[fin]) + 2 * big) + 2.0 ** -22
                np.testing.assert_array_less(np.abs(lse[b, hq][fin] - z[fin]), ztol)


SHAPES = [
    # B, Hq, Hkv, d, T, lengths
    (1, 4, 1, 128, 1, [257]),
    (1, 8, 2, 128, 1, [1]),
    (2, 4, 2, 64, 3, [0, 33]),
    (3, 8, 2, 128, 4, [31, 32, 500]),
    (1, 6, 2, 128, 7, [1000]),            # 21 rows: a ragged row block
    (2, 2, 2, 64, 33, [129, 64]),         # two mask words
    (1, 4, 1, 128, 64, [700]),            # 256 rows per KV head
    (1, 2, 1, 64, 128, [200]),            # the most drafts
    (1, 16, 1, 128, 128, [90]),           # 2048 rows of one KV head
    (1, 1, 1, 128, 97, [0]),              # drafts alone
    (5, 4, 2, 128, 2, [4173, 0, 17, 1, 900]),
]


@pytest.mark.parametrize("shape", SHAPES, ids=[f"H{s[1]}-{s[2]}-d{s[3]}-T{s[4]}-L{max(s[5])}" for s in SHAPES])
@pytest.mark.parametrize("mode", ["tree", "chain", "all", "cached", "cached_causal"])
def test_tree_decode_matches_fp64(shape, mode):
    x = make(11, *shape)
    see = words = None
    if mode == "tree":
        see, words = random_mask(x["rng"], x["B"], x["T"])
    O, lse = run(x, mode, words)
    check(x, mode, O, lse, see)


@pytest.mark.parametrize("gain", [0.0, 30.0])
def test_flat_and_sharp_scores(gain):
    """All scores equal (every factor 0), and scores of hundreds: one key takes all."""
    x = make(5, 1, 8, 2, 128, 5, [777], gain=gain)
    see, words = random_mask(x["rng"], 1, 5)
    O, lse = run(x, "tree", words)
    check(x, "tree", O, lse, see)


@pytest.mark.parametrize("d", [64, 128])
def test_rows_that_see_nothing(d):
    """An empty cache and empty mask rows: O = 0, lse = -inf; the other rows count
    only their own drafts.  Bits past the drafts are ignored."""
    x = make(3, 2, 4, 2, d, 6, [0, 40])
    see = np.zeros((2, 6, 6), bool)
    see[:, 2, 2] = see[:, 5, 1] = True
    words = words_of(see)
    words[..., 0] |= 1 << 6  # not a draft
    O, lse = run(x, "tree", words)
    check(x, "tree", O, lse, see)
    assert torch.all(O[0, :, [0, 1, 3, 4]] == 0) and torch.all(lse[0, :, [0, 1, 3, 4]] == -float("inf"))


def test_empty_sequences_without_drafts():
    x = make(4, 3, 4, 2, 64, 2, [0, 0, 9])
    O, lse = run(x, "cached")
    check(x, "cached", O, lse)
    x = make(4, 2, 4, 2, 64, 2, [0, 0], cap=8)
    O, lse = run(x, "cached", Nk=8)
    assert torch.all(O == 0) and torch.all(lse == -float("inf"))
    O, lse = run(x, "cached", Nk=0, lengths=False)
    assert torch.all(O == 0) and torch.all(lse == -float("inf"))


@pytest.mark.parametrize("out_dtype", [qb.DT_F32, qb.DT_BF16])
@pytest.mark.parametrize("strided", [False, True])
def test_output_types_and_strided_drafts(out_dtype, strided):
    x = make(6, 2, 12, 4, 128, 9, [301, 77])
    see, words = random_mask(x["rng"], 2, 9)
    O, lse = run(x, "tree", words, out_dtype=out_dtype, strided=strided)
    check(x, "tree", O, lse, see)


@pytest.mark.parametrize("T", [2, 40])
def test_granules_and_unused_lengths(T):
    """Per-tensor and per-head Q scales; no lengths: Nk rows everywhere."""
    x = make(7, 2, 4, 2, 128, T, [90, 90])
    O, lse = run(x, "chain", q_gran=qb.GRAN_HEAD, lengths=False)
    check(x, "chain", O, lse)
    x["qs"][:] = x["qs"][0, 0]
    O, lse = run(x, "chain", q_gran=qb.GRAN_TENSOR)
    check(x, "chain", O, lse)


@pytest.mark.parametrize("T,d,lens", [(1, 128, [20011]), (48, 128, [20011]), (3, 64, [700, 16111, 0]),
                                      (30, 64, [11, 33333, 0, 20000]),
                                      # many heads, few shares each
                                      (30, 64, [9000, 11, 4000, 0, 700, 8999, 5000]), (48, 128, [9000, 300, 8000, 1]),
                                      (4, 64, [(613 * i * i) % 4101 for i in range(40)])])
def test_tree_decode_long_split(T, d, lens):
    """Long caches in equal shares over every CTA, and their result bit for bit
    whatever the workspace held."""
    x = make(8, len(lens), 8, 2, d, T, lens)
    assert qb.tree_workspace_size(qb.make_shape(len(lens), 8, 2, T, max(lens), d), qb.make_params()) > 0
    see, words = random_mask(x["rng"], len(lens), T)
    O, lse = run(x, "tree", words)
    check(x, "tree", O, lse, see)
    O2, lse2 = run(x, "tree", words, ws_fill=0)
    assert torch.equal(O, O2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("T", [2, 40])
def test_offsets_past_32_bits(T):
    """The last sequence's rows lie 4.9 GB into each cache array."""
    B, Hq, Hkv, d, cap = 8, 16, 8, 128, 600011
    x = make(14, B, Hq, Hkv, d, T, [1] * (B - 1) + [333], cap=400)
    big = []
    for name in ("kc", "vc"):
        t = torch.empty(B, Hkv, cap, d, dtype=torch.int8, device="cuda")
        t[:, :, :400] = dev(x[name])
        big.append(t)
    shape = qb.make_shape(B, Hq, Hkv, T, 333, d)
    params = qb.make_params(causal=True, kv_capacity=cap)
    O = torch.full((B, Hq, T, d), float("nan"), device="cuda")
    lse = torch.full((B, Hq, T), float("nan"), device="cuda")
    ws = torch.empty(max(qb.tree_workspace_size(shape, params), 256), dtype=torch.uint8, device="cuda")
    K, V = dev(x["K"], torch.bfloat16), dev(x["V"], torch.bfloat16)
    qb.tree_decode(dev(x["qc"]), dev(x["qs"]), *big, dev(x["ks"]), dev(x["vs"]), shape, params, O, lse, ws,
                   lengths=dev(x["lens"]), K_new=K, V_new=V, k_mean=dev(x["mean"]))
    torch.cuda.synchronize()
    assert qb.get_error() == 0
    check(x, "chain", O, lse)
    # the same rows through the other operators, last sequence
    w, w_small = torch.zeros(B, Hkv, cap, device="cuda"), torch.zeros(B, Hkv, 400, device="cuda")
    small = qb.make_params(kv_capacity=400)
    wide = qb.make_params(kv_capacity=cap)
    kw = dict(lengths=dev(x["lens"]))
    qb.kv_weights(dev(x["qc"]), dev(x["qs"]), big[0], None, lse, shape, wide, w, **kw)
    qb.kv_weights(dev(x["qc"]), dev(x["qs"]), dev(x["kc"]), None, lse, shape, small, w_small, **kw)
    assert torch.equal(w[:, :, :400], w_small)
    outs = []
    for kc, vc, ww in ((big[0], big[1], w), (dev(x["kc"]), dev(x["vc"]), w_small)):
        o = [torch.zeros(B, Hkv, 50, d, dtype=torch.int8, device="cuda") for _ in range(2)]
        o += [torch.zeros(B, Hkv, 50, device="cuda"), torch.zeros(B, Hkv, 50, dtype=torch.int32, device="cuda"),
              torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, Hkv, d, device="cuda")]
        qb.kv_evict(kc, vc, ww, 50, *o, Nk=333, n_sink=2, n_recent=5, **kw)
        outs.append(o)
    torch.cuda.synchronize()
    assert qb.get_error() == 0 and all(torch.equal(a, b) for a, b in zip(*outs))


def test_cache_and_drafts_agree():
    """Drafts committed to the cache and read from it (causal) give what the chain
    of drafts gave, up to the two calls' own errors; the cache was not touched."""
    x = make(9, 2, 8, 2, 128, 5, [250, 61], cap=300)
    O, lse = run(x, "chain")
    y = dict(x, kc=x["kc"].copy(), vc=x["vc"].copy())
    for b in range(2):
        L = int(x["lens"][b])
        for h in range(2):
            dk, dv = R.draft_codes(x["K"][b, h], x["V"][b, h], x["mean"][b, h], x["ks"][b, h], x["vs"][b, h])
            y["kc"][b, h, L:L + 5], y["vc"][b, h, L:L + 5] = dk, dv
    y["lens"] = x["lens"] + 5
    O2, lse2 = run(y, "cached_causal")
    check(y, "cached_causal", O2, lse2)
    check(x, "chain", O, lse)


@pytest.mark.parametrize("T", [2, 40])
@pytest.mark.parametrize("bad", [41, -1, -2 ** 31, 2 ** 31 - 1])
def test_bad_lengths_are_reported_and_clamped(T, bad):
    x = make(10, 2, 4, 2, 64, T, [40, 30])
    want, _ = run(x, "chain")
    y = dict(x, lens=np.array([bad, 30], np.int32))
    with pytest.raises(AssertionError):
        run(y, "chain", Nk=40)  # run() asserts that the error word is clear
    assert qb.get_error() == 0
    got, _ = run(x, "chain", Nk=40)
    assert torch.equal(want, got)


@pytest.mark.parametrize("T", [4, 40])
def test_two_streams_and_a_captured_graph(T):
    """Two calls at once, each with its own workspace, and a captured call replayed
    with new lengths."""
    x = make(12, 2, 8, 2, 128, T, [600, 450])
    want, _ = run(x, "chain")
    B, Hq, Hkv, d = 2, 8, 2, 128
    shape = qb.make_shape(B, Hq, Hkv, T, 600, d)
    params = qb.make_params(causal=True, kv_capacity=x["cap"])
    arrays = [dev(x[k]) for k in ("qc", "qs", "kc", "vc", "ks", "vs")]
    K, V, mean = dev(x["K"], torch.bfloat16), dev(x["V"], torch.bfloat16), dev(x["mean"])
    lens = dev(x["lens"])
    n = qb.tree_workspace_size(shape, params)
    outs = [(torch.zeros(B, Hq, T, d, device="cuda"), torch.zeros(B, Hq, T, device="cuda"),
             torch.empty(n, dtype=torch.uint8, device="cuda")) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for (O, lse, ws), st in zip(outs, streams):
            qb.tree_decode(*arrays, shape, params, O, lse, ws, lengths=lens, K_new=K, V_new=V, k_mean=mean,
                           stream=st)
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], want) and torch.equal(outs[1][0], want)
    O, lse, ws = outs[0]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qb.tree_decode(*arrays, shape, params, O, lse, ws, lengths=lens, K_new=K, V_new=V, k_mean=mean)
    O.zero_()
    lens.copy_(torch.tensor([17, 600], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    y = dict(x, lens=np.array([17, 600], np.int32))
    check(y, "chain", O, lse)
    assert qb.get_error() == 0


def test_arguments_elsewhere_are_refused():
    """Tensors that are not on the current device, the workspace among them."""
    shape, params = qb.make_shape(1, 8, 1, 4, 20000, 64), qb.make_params(kv_capacity=20000)
    gpu = [torch.zeros(s, dtype=t, device="cuda") for s, t in (
        ((1, 8, 4, 64), torch.int8), ((8,), torch.float32), ((1, 1, 20000, 64), torch.int8),
        ((1, 1, 20000, 64), torch.int8), ((1, 1, 64), torch.float32), ((1, 1, 64), torch.float32))]
    O, lse = torch.zeros(1, 8, 4, 64, device="cuda"), torch.zeros(1, 8, 4, device="cuda")
    ws = torch.zeros(qb.tree_workspace_size(shape, params), dtype=torch.uint8)
    assert ws.numel() > 0
    with pytest.raises((TypeError, ValueError)):
        qb.tree_decode(*gpu, shape, params, O, lse, ws)
    with pytest.raises((TypeError, ValueError)):
        qb.tree_decode(*gpu, shape, params, O, lse, torch.zeros(2 * ws.numel(), dtype=torch.uint8, device="cuda")[::2])
    for i in (0, 1, 2, 4):
        args = [t.cpu() if k == i else t for k, t in enumerate(gpu)]
        if i == 4:  # k_chan_scale is read for drafts only
            args[5] = args[5].cpu()
        with pytest.raises((TypeError, ValueError)):
            qb.tree_decode(*args, shape, params, O, lse, ws.cuda())


# ------------------------------------------------------------------ commit
@pytest.mark.parametrize("B,Hkv,d,T,n", [(1, 1, 64, 1, [1]), (3, 2, 128, 8, [3, 0, 8]), (2, 12, 128, 40, [1, 17]),
                                         (1, 3, 20, 5, [5])])
@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
def test_commit_bit_exact(B, Hkv, d, T, n, strided, in_place):
    if strided and d % 8:
        pytest.skip("rows of 40 bytes do not start on 16-byte boundaries")
    lens = [0, 5, 11][:B]
    x = make(21, B, Hkv, Hkv, d, T, lens, cap=64)
    rng = x["rng"]
    path = np.stack([rng.permutation(T) for _ in range(B)]).astype(np.int32)
    for b in range(B):
        path[b, n[b]:] = 1 << 30  # not read
    seen = np.asarray([3, 5, 400][:B], np.int32)
    amax = np.full((B, Hkv, d), 20, np.float32)
    w = rng.random((B, Hkv, 64)).astype(np.float32)
    kc, vc, rw = x["kc"].copy(), x["vc"].copy(), w.copy()
    ref = [R.commit(x["K"][b], x["V"][b], path[b], n[b], lens[b], int(seen[b]), x["ks"][b], x["vs"][b],
                    x["mean"][b], amax[b], kc[b], vc[b]) for b in range(B)]
    for b in range(B):
        rw[b, :, lens[b]:lens[b] + n[b]] = 0
    K, V = dev(x["K"], torch.bfloat16), dev(x["V"], torch.bfloat16)
    if strided:
        pack = torch.stack([K.transpose(1, 2), V.transpose(1, 2)], dim=2).contiguous()
        K, V = pack[:, :, 0].transpose(1, 2), pack[:, :, 1].transpose(1, 2)
    lengths, s, mean, am = dev(x["lens"]), dev(seen), dev(x["mean"]), dev(amax)
    outs = {} if in_place else dict(lengths_out=torch.zeros_like(lengths), seen_out=torch.zeros_like(s),
                                    k_mean_out=torch.zeros_like(mean), v_code_amax_out=torch.zeros_like(am))
    gk, gv, gw = dev(x["kc"]), dev(x["vc"]), dev(w)
    qb.tree_commit(K, V, dev(path), dev(np.asarray(n, np.int32)), dev(x["ks"]), dev(x["vs"]), lengths, mean, am,
                   gk, gv, seen=s, weights=gw, **outs)
    torch.cuda.synchronize()
    assert qb.get_error() == 0
    got = outs or dict(lengths_out=lengths, seen_out=s, k_mean_out=mean, v_code_amax_out=am)
    assert got["lengths_out"].tolist() == [a + c for a, c in zip(lens, n)]
    assert got["seen_out"].tolist() == [int(a) + c for a, c in zip(seen, n)]
    assert np.array_equal(gk.cpu().numpy(), kc) and np.array_equal(gv.cpu().numpy(), vc)
    assert np.array_equal(gw.cpu().numpy(), rw)
    assert np.array_equal(got["k_mean_out"].cpu().numpy().view(np.uint32),
                          np.stack([r[0] for r in ref]).view(np.uint32))
    assert np.array_equal(got["v_code_amax_out"].cpu().numpy(), np.stack([r[1] for r in ref]))


def test_commit_the_same_draft_twice_and_nothing():
    """A path may name a draft twice; T = 0 appends nothing."""
    x = make(23, 1, 2, 2, 64, 3, [4], cap=9)
    kc, vc = x["kc"].copy(), x["vc"].copy()
    am = np.zeros((1, 2, 64), np.float32)
    m, a = R.commit(x["K"][0], x["V"][0], [2, 2, 0], 3, 4, 4, x["ks"][0], x["vs"][0], x["mean"][0], am[0], kc[0], vc[0])
    gk, gv, lens, mean, gam = dev(x["kc"]), dev(x["vc"]), dev(x["lens"]), dev(x["mean"]), dev(am)
    args = (dev(x["ks"]), dev(x["vs"]), lens, mean, gam, gk, gv)
    K, V = dev(x["K"], torch.bfloat16), dev(x["V"], torch.bfloat16)
    qb.tree_commit(K, V, dev(np.array([[2, 2, 0]], np.int32)), dev(np.array([3], np.int32)), *args)
    none = torch.zeros(1, 0, dtype=torch.int32, device="cuda")
    qb.tree_commit(K[:, :, :0], V[:, :, :0], none, dev(np.array([0], np.int32)), *args)
    torch.cuda.synchronize()
    assert qb.get_error() == 0 and lens.tolist() == [7]
    assert np.array_equal(gk.cpu().numpy(), kc) and np.array_equal(gv.cpu().numpy(), vc)
    assert np.array_equal(mean.cpu().numpy()[0], m) and np.array_equal(gam.cpu().numpy()[0], a)


@pytest.mark.parametrize("n,p,L", [(5, 0, 0), (-1, 0, 0), (2, 4, 0), (2, -1, 0), (2, 0, 7)])
def test_commit_refuses_on_the_device(n, p, L):
    """n_accept, path or room out of range: the sequence is left as it is, its
    neighbour is served, the error word says so."""
    x = make(22, 2, 2, 2, 64, 4, [L, 1], cap=8)
    path = np.array([[p] * 4, [1, 0, 0, 0]], np.int32)
    am = torch.zeros(2, 2, 64, device="cuda")
    gk, gv, lens, mean = dev(x["kc"]), dev(x["vc"]), dev(x["lens"]), dev(x["mean"])
    qb.tree_commit(dev(x["K"], torch.bfloat16), dev(x["V"], torch.bfloat16), dev(path),
                   dev(np.array([n, 1], np.int32)), dev(x["ks"]), dev(x["vs"]), lens, mean, am, gk, gv)
    torch.cuda.synchronize()
    assert qb.get_error() == qb.ERR_INVALID_ARG
    assert lens.tolist() == [L, 2]
    assert torch.equal(gk[0], dev(x["kc"])[0]) and torch.equal(mean[0], dev(x["mean"])[0])
    assert not torch.equal(gk[1, :, 1], dev(x["kc"])[1, :, 1])


def test_commit_refuses_a_token_count_past_32_bits():
    x = make(24, 1, 2, 2, 64, 4, [2], cap=8)
    seen, lens, mean = dev(np.array([2 ** 31 - 2], np.int32)), dev(x["lens"]), dev(x["mean"])
    am, gk, gv = torch.zeros(1, 2, 64, device="cuda"), dev(x["kc"]), dev(x["vc"])
    args = (dev(x["K"], torch.bfloat16), dev(x["V"], torch.bfloat16), dev(np.array([[0, 1, 2, 3]], np.int32)))
    rest = (dev(x["ks"]), dev(x["vs"]), lens, mean, am, gk, gv)
    qb.tree_commit(*args, dev(np.array([2], np.int32)), *rest, seen=seen)
    torch.cuda.synchronize()
    assert qb.get_error() == qb.ERR_INVALID_ARG and lens.tolist() == [2] and seen.tolist() == [2 ** 31 - 2]
    qb.tree_commit(*args, dev(np.array([1], np.int32)), *rest, seen=seen)
    torch.cuda.synchronize()
    assert qb.get_error() == 0 and lens.tolist() == [3] and seen.tolist() == [2 ** 31 - 1]
