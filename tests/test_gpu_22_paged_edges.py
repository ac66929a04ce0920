"""The paged cache's operators where one kernel hands over to another, and in calls
that share something: a workspace, a pool, a prefix."""
import numpy as np
import pytest
import torch

from quantized_attention_gb300 import binding as qb
from quantized_attention_gb300.pipeline import PagedCache, rope_table
from tests import paged_ref as R
from tests.gpu_common import ensure_library
from tests.test_gpu_21_paged import DT, Pool, check, dev, heads_last, make, run, same_bits, tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_library()


class Call:
    """The call with a bound on the rows (and a page table as wide) far above the lengths,
    as a cache with room has it: work is planned for that bound."""

    def __init__(self, P, Nk, causal=True, ws=None):
        B, Hq, T, d = P.q.shape
        width = -(-Nk // P.page)
        self.pt = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        t = P.table(P.lens)[:, :width]
        self.pt[:, :t.shape[1]] = t
        self.shape = qb.make_shape(B, Hq, P.Hkv, T, Nk, d)
        self.params = qb.make_params(causal=causal, out_dtype=qb.DT_F32)
        self.paging = qb.make_paging(P.n, P.page, width, DT[P.code])
        self.q, self.lens, self.new, self.pool = dev(P.q, torch.bfloat16), dev(P.lens), dev(P.new), P.arrays()
        self.O = torch.full((B, Hq, T, d), 7.0, device="cuda")
        self.lse = torch.full((B, Hq, T), 7.0, device="cuda")
        self.need = qb.paged_workspace_size(self.shape, self.params, self.paging)
        self.ws = torch.full((max(self.need, 256),), 0xFF, dtype=torch.uint8, device="cuda") if ws is None else ws

    def __call__(self):
        qb.paged_fwd(self.q, self.shape, self.params, self.paging, self.pt, self.lens, *self.pool, self.O, self.lse,
                     self.ws, n_new=self.new)
        return self.O, self.lse


def run_bound(P, Nk, causal=True):
    return Call(P, Nk, causal)()


# --------------------------------------------------- few rows, by either kernel
FEW = [
    # B, Hq, Hkv, d, page, code, T, lengths, n_new: 8, 9, 16, 17, 33, 64, 65 rows of a KV head
    (2, 8, 4, 128, 64, "int8", 4, [700, 65], [4, 2]),
    (2, 3, 1, 128, 32, "e4m3", 3, [333, 2], [3, 2]),
    (1, 16, 1, 64, 128, "int8", 1, [1500], None),
    (2, 17, 1, 128, 64, "e4m3", 1, [129, 0], [1, 0]),
    (3, 3, 1, 64, 32, "int8", 11, [640, 11, 100], [11, 11, 5]),
    (1, 8, 1, 128, 128, "e4m3", 8, [1111], None),
    (2, 4, 1, 64, 64, "e4m3", 16, [900, 64], [16, 1]),
    (2, 5, 1, 128, 32, "int8", 13, [257, 500], [13, 12]),
]


@pytest.mark.parametrize("shape", FEW, ids=[f"{s[5]}-{s[1] // s[2] * s[6]}rows-d{s[3]}" for s in FEW])
@pytest.mark.parametrize("bound", [2048, 8192, 1 << 19], ids=["short", "middling", "long"])
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "all"])
def test_few_rows_of_a_short_and_of_a_long_cache(shape, bound, causal):
    P = make(31, *shape)
    O, lse = run_bound(P, bound, causal)
    assert qb.get_error() == 0
    check(P, O, lse, causal)


@pytest.mark.parametrize("T", [1, 8, 20, 70], ids=str)
@pytest.mark.parametrize("bound", [512, 1 << 19], ids=["short", "long"])
@pytest.mark.parametrize("d", [64, 128])
def test_page_scales_of_zero_and_not_numbers(T, bound, d):
    """V scales of 0 beside ordinary ones, a page of NaN scale behind them."""
    P = make(32, 2, 4, 2, d, 32, "e4m3", T, [200, 170], gain=0.3)
    for j in (0, 3, 5):
        P.vs[P.pt[0, j]] = 0
    P.ks[P.pt[0, 2]] = 0
    O, lse = run_bound(P, bound)
    assert qb.get_error() == 0
    check(P, O, lse)
    P.vs[P.pt[1, 5], 1] = np.nan  # rows 160 .. 169 of the second KV head
    O, lse = run_bound(P, bound)
    assert qb.get_error() == 0
    sees = torch.zeros(2, 4, T, dtype=torch.bool)
    sees[1, 2:, max(0, T - 10):] = True
    assert torch.equal(O.isnan().all(-1).cpu(), sees) and torch.equal(lse.isnan().cpu(), sees)
    assert torch.equal(O.isnan().any(-1).cpu(), sees)


@pytest.mark.parametrize("T", [3, 16, 80], ids=str)
@pytest.mark.parametrize("bound", [512, 1 << 19], ids=["short", "long"])
def test_rows_that_see_nothing_and_missing_pages(T, bound):
    """Causal rows before the first cached one, a sequence without rows, one without new
    tokens; a page that does not exist in the middle is reported and hidden."""
    lens = [max(1, T // 2), 0, 300, 300]
    P = make(33, 4, 4, 2, 128, 64, "int8", T, lens, [T, T, 0, T])
    O, lse = run_bound(P, bound)
    assert qb.get_error() == 0
    check(P, O, lse)
    P.pt[3, 1] = P.n + 5
    O, lse = run_bound(P, bound)
    assert qb.get_error() == qb.ERR_INVALID_ARG
    kept = np.r_[0:64, 128:300]
    see = kept[None] <= (300 - T + np.arange(T))[:, None]
    P.pt[3, 1] = P.pt[3, 0]
    for hq in range(4):
        (kc, ks), (vc, vs) = (R.rows(x, s, P.pt[3], hq // 2, 300, 64, "int8") for x, s in ((P.k, P.ks), (P.v, P.vs)))
        o = R.attend(P.q[3, hq], kc[kept], ks[kept], vc[kept], vs[kept], see, 1 / np.sqrt(128))[0]
        # P's half step and the scores' error, well below 2^-9 of the values' size
        assert np.abs(O[3, hq].cpu().numpy() - o).max() < 2.0 ** -9 * np.abs(vc * vs[:, None]).max()
    assert qb.get_error() == 0


def test_a_prefix_in_two_sequences():
    """Pages that several sequences share are read by each: equal queries, equal bits."""
    P = make(34, 3, 8, 2, 128, 32, "int8", 2, [320, 320, 100])
    P.pt[1, :10] = P.pt[0, :10]
    P.q[1] = P.q[0]
    O, lse = run(P)
    assert qb.get_error() == 0 and torch.equal(O[0], O[1]) and torch.equal(lse[0], lse[1])
    check(P, O, lse)


@pytest.mark.parametrize("Nk", [4160, 12288, 12352])
@pytest.mark.parametrize("Hkv,d,code", [(8, 128, "int8"), (3, 64, "e4m3")])
def test_one_long_sequence(Nk, Hkv, d, code):
    """Up to eight KV heads of one sequence around the bound to which they take wide clusters."""
    for L in (Nk, Nk - 63, 33):
        P = make(37, 1, 2 * Hkv, Hkv, d, 64, code, 2, [L])
        O, lse = run_bound(P, Nk)
        assert qb.get_error() == 0
        check(P, O, lse)


@pytest.mark.parametrize("T", [1, 6, 90], ids=str)
@pytest.mark.parametrize("Nk", [3200, 1 << 19], ids=["short", "long"])
def test_two_graphs_share_a_workspace(T, Nk):
    """Two captured calls of other lengths and one workspace, replayed in turn."""
    cases = [make(35, 3, 8, 2, 128, 64, "int8", T, [2900, 91, 700], [T, T, 1]),
             make(36, 3, 8, 2, 128, 64, "int8", T, [95, 3000, 1], [T, 1, 1])]
    first = Call(cases[0], Nk)
    calls, graphs = [first, Call(cases[1], Nk, ws=first.ws)], []
    for call in calls:
        graphs.append(torch.cuda.CUDAGraph())
        torch.cuda.synchronize()
        with torch.cuda.graph(graphs[-1]):
            call()
    for _ in range(5):
        for graph, call in zip(graphs, calls):
            call.O.fill_(7.0)
            call.lse.fill_(7.0)
            graph.replay()
    torch.cuda.synchronize()
    assert qb.get_error() == 0
    for P, call in zip(cases, calls):
        check(P, call.O, call.lse)


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("T", [15, 16, 17, 33], ids=str)
@pytest.mark.parametrize("Hq,Hkv,d,rot", [(9, 3, 64, 24), (20, 2, 128, 128), (1, 1, 128, 40), (7, 7, 64, 48)], ids=str)
@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_append_where_few_tokens_end(T, Hq, Hkv, d, rot, code):
    """Tokens that fill the end of a page and the start of the next, with given positions."""
    B, page = 3, 32
    P = Pool(41, B, Hkv, d, page, code, 200)
    tab = R.table(300, rot)
    before = np.array([0, 25, 63])
    n = np.array([T, T - 1, T], np.int32)
    for b in range(B):
        if before[b]:
            x = tokens(P.rng, Hkv, int(before[b]), d, 0.2)
            P.put(b, 0, x, x)
    K, V, Q = (tokens(P.rng, B * h, T, d).reshape(B, h, T, d) for h in (Hkv, Hkv, Hq))
    pos = P.rng.integers(0, 300, (B, T)).astype(np.int32)
    lens = (before + n).astype(np.int32)
    got = P.arrays()
    q_out = torch.full((B, Hq, T, d), 7.0, dtype=torch.bfloat16, device="cuda")
    k, v, q = (heads_last(dev(x, torch.bfloat16)) for x in (K, V, Q))
    qb.paged_append(k, v, qb.make_shape(B, Hq, Hkv, T, 200, d), P.paging, P.table(lens), dev(lens), *got, n_new=dev(n),
                    positions=dev(pos), rope=qb.make_rope(dev(tab)), Q=q, Q_out=q_out)
    assert qb.get_error() == 0
    want = np.full((B, Hq, T, d), 7.0, np.float32)
    for b in range(B):
        m = int(n[b])
        want[b, :, :m] = R.rotate(Q[b, :, :m], pos[b, :m], tab, False)
        P.put(b, int(before[b]), R.rotate(K[b, :, :m], pos[b, :m], tab, False), V[b, :, :m])
    assert torch.equal(q_out, dev(want, torch.bfloat16))
    assert same_bits(got, P.arrays())


@pytest.mark.parametrize("T", [4, 40], ids=str)
def test_append_positions_outside_the_table(T):
    """A token at a position that the table does not have: neither its Q nor its K is written,
    its V is, and the other tokens' are."""
    P = Pool(42, 1, 2, 64, 32, "int8", 64)
    tab = R.table(50, 64)
    K, V, Q = (tokens(P.rng, h, T, 64) for h in (2, 2, 4))
    pos = np.arange(T, dtype=np.int32)[None].copy()
    pos[0, 2] = 50
    pos[0, 3] = -1
    got = P.arrays()
    q_out = torch.full((1, 4, T, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    qb.paged_append(dev(K[None], torch.bfloat16), dev(V[None], torch.bfloat16), qb.make_shape(1, 4, 2, T, T, 64), P.paging,
                    P.table([T]), torch.tensor([T], dtype=torch.int32, device="cuda"), *got, positions=dev(pos),
                    rope=qb.make_rope(dev(tab)), Q=dev(Q[None], torch.bfloat16), Q_out=q_out)
    assert qb.get_error() == qb.ERR_INVALID_ARG
    safe = np.where((pos[0] < 0) | (pos[0] >= 50), 0, pos[0])
    want, k = R.rotate(Q, safe, tab, False), R.rotate(K, safe, tab, False)
    want[:, 2:4] = 7.0
    held = P.k[P.pt[0, 0], :, 2:4].copy()
    k[:, 2:4] = 0  # they do not count for the page's scale
    P.put(0, 0, k, V)
    P.k[P.pt[0, 0], :, 2:4] = held
    assert torch.equal(q_out[0], dev(want, torch.bfloat16)) and same_bits(got, P.arrays())
    assert qb.get_error() == 0


def test_a_step_on_another_stream_than_the_inputs():
    """Append and attend on a side stream that waits for the inputs' stream."""
    B, Hq, Hkv, d = 2, 8, 2, 128
    rope = qb.make_rope(rope_table(600, d))
    C, E = (PagedCache(40, 32, Hq, Hkv, d, B, 600, rope=rope, out_dtype=qb.DT_F32) for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(5)
    side = torch.cuda.Stream()
    for T in (300, 1, 7, 33):
        x = [torch.randn(B, h, T, d, generator=g, device="cuda").to(torch.bfloat16) for h in (Hq, Hkv, Hkv)]
        want = C.step(*x).clone()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = E.step(*x)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want)
    assert qb.get_error() == 0


def test_a_refused_step_leaves_the_sequences():
    B, Hq, Hkv, d = 2, 4, 2, 64
    C, E = (PagedCache(12, 32, Hq, Hkv, d, B, 128, rope=qb.make_rope(rope_table(128, d)), out_dtype=qb.DT_F32)
            for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(6)

    def new(T):
        return [torch.randn(B, h, T, d, generator=g, device="cuda").to(torch.bfloat16) for h in (Hq, Hkv, Hkv)]

    x = new(40)
    for c in (C, E):
        c.step(*x, n_new=[40, 3])
    Q, K, V = new(30)
    for bad, error in (((Q, K.float(), V), TypeError), ((Q, K, V[:, :1]), ValueError), ((Q, K[:, :, :29], V), ValueError)):
        with pytest.raises(error):
            C.step(*bad)
        assert C.free_pages() == E.free_pages() and C.rows(0) == 40 and C.rows(1) == 3
        assert torch.equal(C.page_table, E.page_table) and torch.equal(C.lengths, E.lengths)
    with pytest.raises(ValueError, match="n_new"):
        C.step(Q, K, V, n_new=[31, 1])
    assert C.rows(0) == 40
    assert torch.equal(C.step(Q, K, V), E.step(Q, K, V)) and torch.equal(C.k_pages, E.k_pages)
    assert qb.get_error() == 0


def test_a_cache_without_rows():
    """Nk = 0: nothing is seen, whatever the pool holds."""
    P = Pool(43, 2, 2, 64, 32, "e4m3", 32)
    for T in (1, 30):
        shape, params = qb.make_shape(2, 8, 2, T, 0, 64), qb.make_params(causal=True, out_dtype=qb.DT_F32)
        paging = qb.make_paging(P.n, 32, 1)
        paging.code_dtype = qb.DT_E4M3
        O, lse = torch.full((2, 8, T, 64), 7.0, device="cuda"), torch.full((2, 8, T), 7.0, device="cuda")
        ws = torch.full((max(qb.paged_workspace_size(shape, params, paging), 256),), 0xFF, dtype=torch.uint8, device="cuda")
        q = torch.randn(2, 8, T, 64, device="cuda").to(torch.bfloat16)
        pt = torch.full((2, 1), -1, dtype=torch.int32, device="cuda")
        lens = torch.zeros(2, dtype=torch.int32, device="cuda")
        qb.paged_fwd(q, shape, params, paging, pt, lens, *P.arrays(), O, lse, ws)
        assert qb.get_error() == 0 and (O == 0).all() and (lse == -float("inf")).all()


@pytest.mark.parametrize("T", [3, 50], ids=str)
def test_append_rotates_q_in_place(T):
    P = Pool(44, 2, 2, 128, 64, "int8", 64)
    tab = R.table(64, 128)
    K, V, Q = (tokens(P.rng, 2 * h, T, 128).reshape(2, h, T, 128) for h in (2, 2, 6))
    q, lens = dev(Q, torch.bfloat16), np.full(2, T, np.int32)
    got = P.arrays()
    qb.paged_append(dev(K, torch.bfloat16), dev(V, torch.bfloat16), qb.make_shape(2, 6, 2, T, 64, 128), P.paging,
                    P.table(lens), dev(lens), *got, rope=qb.make_rope(dev(tab), interleaved=True), Q=q, Q_out=q)
    pos = np.arange(T)
    for b in range(2):
        P.put(b, 0, R.rotate(K[b], pos, tab, True), V[b])
    assert qb.get_error() == 0 and same_bits(got, P.arrays())
    assert torch.equal(q, dev(np.stack([R.rotate(Q[b], pos, tab, True) for b in range(2)]), torch.bfloat16))
