"""The serving operators in every division of their work: shares of long caches
and clusters of each size, on two streams, replayed from a graph, without drafts,
and with lengths that are out of range."""
import numpy as np
import pytest
import torch

from quantized_attention_gb300 import binding as qb
from tests.gpu_common import ensure_library
from tests.test_gpu_16_tree import bf16, check, dev, make, random_mask, run
from tests.test_gpu_17_kv_evict import cache, check_evict

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_library()


def need(x, Nk):
    return qb.tree_workspace_size(qb.make_shape(x["B"], x["Hq"], x["Hkv"], x["T"], Nk, x["d"]), qb.make_params())


class Call:
    """A call of the library on fixed tensors, with its own outputs and workspace."""

    def __init__(self, x, Nk, drafts=True):
        B, Hq, T, d = x["B"], x["Hq"], x["T"], x["d"]
        self.shape = qb.make_shape(B, Hq, x["Hkv"], T, Nk, d)
        self.params = qb.make_params(causal=True, kv_capacity=x["cap"], out_dtype=qb.DT_F32)
        self.args = [dev(x[k]) for k in ("qc", "qs", "kc", "vc", "ks", "vs")]
        self.kw = dict(K_new=dev(x["K"], torch.bfloat16), V_new=dev(x["V"], torch.bfloat16),
                       k_mean=dev(x["mean"])) if drafts else {}
        self.lens = dev(x["lens"])
        self.O = torch.full((B, Hq, T, d), float("nan"), device="cuda")
        self.lse = torch.full((B, Hq, T), float("nan"), device="cuda")
        n = qb.tree_workspace_size(self.shape, self.params)
        self.ws = torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device="cuda")

    def __call__(self, stream=None):
        qb.tree_decode(*self.args, self.shape, self.params, self.O, self.lse, self.ws, lengths=self.lens,
                       stream=stream, **self.kw)
        return self.O, self.lse


@pytest.mark.parametrize("T,d", [(3, 64), (30, 64), (2, 128), (40, 128)])
@pytest.mark.parametrize("drafts", [True, False])
def test_shares_on_two_streams_and_replayed_with_other_lengths(T, d, drafts):
    """Long caches, whose shares meet in the workspace: two calls with different
    lengths at once, and a captured call replayed with lengths that move the shares'
    borders, an empty sequence among them."""
    mode = "chain" if drafts else "cached_causal"
    lens = [[12000, 700, 9001], [300, 16111, 5000]]
    if not drafts:
        lens = [[max(n, T) for n in l] for l in lens]
    xs = [make(70 + i, 3, 8, 2, d, T, l, cap=16120) for i, l in enumerate(lens)]
    assert need(xs[0], 16111) > 0
    calls = [Call(x, 16111, drafts) for x in xs]
    want = [[t.clone() for t in c()] for c in calls]
    torch.cuda.synchronize()
    assert qb.get_error() == 0
    for x, (O, lse) in zip(xs, want):
        check(x, mode, O, lse)
    streams = [torch.cuda.Stream() for _ in calls]
    for c in calls:
        c.O.zero_()
        c.lse.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for c, st in zip(calls, streams):
            c(st)
    torch.cuda.synchronize()
    for c, (O, lse) in zip(calls, want):
        assert torch.equal(c.O, O) and torch.equal(c.lse, lse)
    c, g = calls[0], torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c()
    for l in ([0, 16111, 31], [5000, 0, 0], [16111, 16111, 16111], [0, 0, 0]):
        y = dict(xs[0], lens=np.asarray(l, np.int32))
        c.lens.copy_(dev(y["lens"]))
        c.O.fill_(float("nan"))
        c.lse.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        check(y, mode, c.O, c.lse)
    assert qb.get_error() == 0


@pytest.mark.parametrize("mode", ["cached", "cached_causal"])
@pytest.mark.parametrize("T,d,lens", [(1, 128, [20011]), (48, 128, [20011]), (3, 64, [700, 16111, 0]),
                                      (30, 64, [11, 33333, 0, 20000])])
def test_shares_without_drafts(mode, T, d, lens):
    x = make(71, len(lens), 8, 2, d, T, lens)
    assert need(x, max(lens)) > 0
    O, lse = run(x, mode)
    check(x, mode, O, lse)


@pytest.mark.parametrize("B,Hkv,G,T,lens", [
    (3, 20, 2, 3, [130, 0, 77]),       # 60 heads of few rows: clusters of 4
    (4, 25, 2, 3, [300, 1, 0, 257]),   # 100: of 2
    (4, 40, 1, 2, [200, 33, 0, 129]),  # 160: one CTA
    (2, 10, 4, 9, [400, 90]),          # 20 row blocks of 128: clusters of 4
    (5, 10, 4, 9, [400, 90, 0, 1, 129]),   # 50: of 2
    (8, 10, 4, 9, [400, 90, 0, 1, 129, 128, 256, 5]),  # 80: one CTA
    (2, 40, 1, 20, [700, 300]),
])
@pytest.mark.parametrize("mode", ["tree", "cached_causal"])
def test_clusters_of_each_size(B, Hkv, G, T, lens, mode):
    x = make(72, B, Hkv * G, Hkv, 64, T, lens)
    assert need(x, max(lens)) == 0
    see = words = None
    if mode == "tree":
        see, words = random_mask(x["rng"], B, T)
    O, lse = run(x, mode, words)
    check(x, mode, O, lse, see)


@pytest.mark.parametrize("T", [2, 40])
@pytest.mark.parametrize("Nk", [40, 20011])
@pytest.mark.parametrize("bad", [1, -1, -2 ** 31, 2 ** 31 - 1])
def test_lengths_out_of_range_count_as_the_nearest(T, Nk, bad):
    """Reported, and both sequences as with the clamped length: in a head's cluster
    and in shares."""
    bad = Nk + 1 if bad == 1 else bad
    x = make(73, 2, 8, 2, 64, T, [Nk, 30], cap=Nk + 7)
    assert (need(x, Nk) > 0) == (Nk > 40)
    for drafts in (True, False):
        c = Call(dict(x, lens=np.array([0 if bad < 0 else Nk, 30], np.int32)), Nk, drafts)
        want = [t.clone() for t in c()]
        torch.cuda.synchronize()
        assert qb.get_error() == 0
        c.lens.copy_(dev(np.array([bad, 30], np.int32)))
        c.O.fill_(float("nan"))
        c.lse.fill_(float("nan"))
        c()
        torch.cuda.synchronize()
        assert qb.get_error() == qb.ERR_INVALID_ARG and qb.get_error() == 0
        assert torch.equal(c.O, want[0]) and torch.equal(c.lse, want[1])


@pytest.mark.parametrize("T", [2, 40])
def test_many_short_heads_in_shares(T):
    """48 heads of uneven length: shares that hold several heads, borders in their
    drafted steps among them."""
    lens = [(911 * i * i) % 7000 for i in range(24)]
    x = make(74, 24, 8, 2, 64, T, lens)
    assert need(x, max(lens)) > 0
    see, words = random_mask(x["rng"], 24, T)
    O, lse = run(x, "tree", words)
    check(x, "tree", O, lse, see)


# ------------------------------------------------------------------ eviction
@pytest.mark.parametrize("B,H,d,lens,budget,sink,recent", [
    (3, 10, 64, [257, 0, 1000], 100, 2, 30),           # 30 heads: clusters of 4
    (5, 12, 32, [257, 0, 1000, 33, 5], 100, 2, 30),    # 60: of 2
    (13, 10, 128, [257, 0, 300, 33, 5, 1, 101, 100, 99, 64, 200, 31, 129], 100, 2, 30),  # 130: one CTA
    (16, 8, 64, [1801 + 33 * i for i in range(16)], 1999, 4, 128),
])
@pytest.mark.parametrize("kind", ["spread", "ties", "special"])
def test_evict_with_clusters_of_each_size(B, H, d, lens, budget, sink, recent, kind):
    rng = np.random.default_rng(75)
    cap, ocap = max(lens) + 7, budget + 3
    x = cache(rng, B, H, cap, d)
    w = np.exp(2 * rng.normal(size=(B, H, cap))).astype(np.float32)
    if kind == "ties":
        w = rng.choice(np.array([0.0, -0.0, 0.0, 0.25, 1.0], np.float32), size=w.shape)
    if kind == "special":
        w[rng.random(w.shape) < 0.3] = np.nan
        w[rng.random(w.shape) < 0.1] = -np.inf
        w[rng.random(w.shape) < 0.1] = np.finfo(np.float32).min
        w[rng.random(w.shape) < 0.1] = 1e-42
        w[rng.random(w.shape) < 0.02] = np.inf
    check_evict(x, w, budget, sink, recent, lens, max(lens), ocap)


# ------------------------------------------------------------------ commit
@pytest.mark.parametrize("B,H,d,T,pos", [(1, 1, 64, 1, 0), (2, 3, 128, 40, 17), (3, 12, 64, 7, 300), (1, 2, 20, 5, 3)])
def test_commit_of_everything_is_an_append(B, H, d, T, pos):
    """qattn_kv_append and qattn_tree_commit of the same tokens, bit for bit: codes,
    running mean, maxima; values no code holds among them."""
    rng = np.random.default_rng(76)
    cap = pos + T + 2
    mean = (3.0 * rng.normal(size=(B, H, d))).astype(np.float32)
    K = bf16(mean[:, :, None] + 1.3 * rng.normal(size=(B, H, T, d)))
    V = bf16(1.3 * rng.normal(size=(B, H, T, d)))
    K[..., 0], V[..., 0] = 1e30, -1e30
    K[:, :, -1, 1], V[:, :, -1, 1], V[:, :, -1, 2] = np.nan, np.nan, np.inf
    K, V = dev(K, torch.bfloat16), dev(V, torch.bfloat16)
    ks, vs = (dev(rng.uniform(0.02, 0.06, (B, H, d)).astype(np.float32)) for _ in range(2))
    codes = dev(rng.integers(-127, 128, (2, B, H, cap, d)).astype(np.int8))
    out = []
    for append in (True, False):
        kc, vc, mu = codes[0].clone(), codes[1].clone(), dev(mean)
        am = torch.full((B, H, d), 20.0, device="cuda")
        if append:
            qb.kv_append(K, V, pos, ks, vs, mu, am, kc, vc)
        else:
            path = torch.arange(T, dtype=torch.int32, device="cuda").repeat(B, 1)
            lens = torch.full((B,), pos, dtype=torch.int32, device="cuda")
            qb.tree_commit(K, V, path, torch.full_like(lens, T), ks, vs, lens, mu, am, kc, vc)
            assert lens.tolist() == [pos + T] * B
        torch.cuda.synchronize()
        assert qb.get_error() == 0
        out.append((kc, vc, mu.view(torch.int32), am.view(torch.int32)))
    assert all(torch.equal(a, b) for a, b in zip(*out))
