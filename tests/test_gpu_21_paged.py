"""Rotary positions, appending to a paged 8-bit KV cache and attention over it
(qattn_rotate, qattn_paged_append, qattn_paged_fwd) against plain forms."""
import numpy as np
import pytest
import torch

from quantized_attention_gb300 import binding as qb
from quantized_attention_gb300.pipeline import PagedCache, rope_table
from tests import paged_ref as R
from tests.gpu_common import ensure_library

pytestmark = pytest.mark.gpu

DT = {"int8": qb.DT_I8, "e4m3": qb.DT_E4M3}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_library()


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def heads_last(x):
    """[B, H, N, d] laid out as a projection writes it, [B, N, H, d]."""
    return x.transpose(1, 2).contiguous().transpose(1, 2)


# ---------------------------------------------------------------- rotation
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 32, 32), (2, 5, 33, 64, 24), (1, 9, 130, 128, 128), (3, 4, 17, 128, 64),
                                   (2, 1, 300, 64, 8)], ids=str)
@pytest.mark.parametrize("inter", [False, True], ids=["half", "interleaved"])
def test_rotate_bit_exact(shape, inter, dtype):
    B, H, T, d, rot = shape
    rng = np.random.default_rng(3)
    x = R.bf16(rng.normal(size=(B, H, T, d))) if dtype == torch.bfloat16 else rng.normal(size=(B, H, T, d)).astype(np.float32)
    tab = R.table(500, rot)
    pos = rng.integers(0, 500, (B, T)).astype(np.int32)
    for back in (False, True):
        rope = qb.make_rope(dev(tab), interleaved=inter, inverse=back)
        for given in (False, True):
            want = np.stack([R.rotate(x[b], pos[b] if given else np.arange(T), tab, inter, back) for b in range(B)])
            for X in (dev(x, dtype), heads_last(dev(x, dtype))):
                Y = torch.full((B, H, T, d), float("nan"), dtype=dtype, device="cuda")
                qb.rotate(X, Y, rope, positions=dev(pos) if given else None)
                assert qb.get_error() == 0
                assert torch.equal(Y, dev(want).to(dtype))
            X = dev(x, dtype)  # in place
            qb.rotate(X, X, rope, positions=dev(pos) if given else None)
            assert torch.equal(X, dev(want).to(dtype))


@pytest.mark.parametrize("inter", [False, True], ids=["half", "interleaved"])
def test_rotate_gradient(inter):
    """y = R x is linear: <R x, w> = <x, R' w> for every x and w, where R' w is the call
    with an inverse rope; and the difference quotient of <R x, w> along one channel is
    that channel of R' w.  fp32 tensors: each element of either side is off by three
    roundings of products of at most |x| |w|."""
    B, H, T, d, rot = 2, 3, 21, 64, 40
    g = torch.Generator(device="cuda").manual_seed(1)
    x, w = (torch.randn(B, H, T, d, generator=g, device="cuda") for _ in range(2))
    tab = rope_table(64, rot, scaling="ramp", factor=8.0, mscale=1.2)
    f, b = qb.make_rope(tab, interleaved=inter), qb.make_rope(tab, interleaved=inter, inverse=True)
    y, gx = torch.empty_like(x), torch.empty_like(x)
    qb.rotate(x, y, f)
    qb.rotate(w, gx, b)
    lhs, rhs = (y.double() * w.double()).sum(), (x.double() * gx.double()).sum()
    size = (x.abs().double().flatten().norm() * w.abs().double().flatten().norm()) * 1.2 * 2 ** 0.5
    assert abs(float(lhs - rhs)) <= float(size) * 6 * 2.0 ** -24
    for c in (0, 1, 19, 20, 39, 40, 63):
        step = 2.0 ** -3
        xe = x.clone()
        xe[1, 2, 7, c] += step
        ye = torch.empty_like(x)
        qb.rotate(xe, ye, f)
        diff = float(((ye.double() - y.double()) * w.double())[1, 2, 7].sum()) / step
        scale = float(x[1, 2, 7].abs().max() + step) * float(w[1, 2, 7].abs().max()) * 1.2
        assert abs(diff - float(gx[1, 2, 7, c])) <= scale * 16 * 2.0 ** -24 / step


def test_rotate_positions_outside_the_table():
    x = torch.randn(1, 2, 4, 64, device="cuda")
    y = torch.full_like(x, 7.0)
    rope = qb.make_rope(rope_table(10, 64))
    qb.rotate(x, y, rope, positions=torch.tensor([[3, 10, -1, 9]], dtype=torch.int32, device="cuda"))
    assert qb.get_error() == qb.ERR_INVALID_ARG
    assert (y[0, :, 1:3] == 7.0).all() and not (y[0, :, 0] == 7.0).any() and not (y[0, :, 3] == 7.0).any()
    assert qb.get_error() == 0


# ------------------------------------------------------------------ append
class Pool:
    """A pool with shuffled pages, as arrays of the host; rows never written hold
    garbage (e4m3: NaN), pages never used have NaN scales, the page table's unused
    entries point nowhere."""

    def __init__(self, seed, B, Hkv, d, page, code, max_rows, spare=2):
        self.rng = np.random.default_rng(seed)
        self.B, self.Hkv, self.d, self.page, self.code = B, Hkv, d, page, code
        self.width = -(-max(max_rows, 1) // page) + 1
        self.n = B * self.width + spare
        self.pt = self.rng.permutation(self.n)[:B * self.width].reshape(B, self.width).astype(np.int32)
        shape = (self.n, Hkv, page, d)
        junk = np.full(shape, 0x7f, np.uint8) if code == "e4m3" else self.rng.integers(-128, 128, shape).astype(np.int8)
        self.k, self.v = junk.copy(), junk.copy()
        self.ks, self.vs = (np.full((self.n, Hkv), np.nan, np.float32) for _ in range(2))
        self.paging = qb.make_paging(self.n, page, self.width, DT[code])

    def put(self, b, first, k, v):
        R.append(k, first, self.code, self.page, self.pt[b], self.k, self.ks)
        R.append(v, first, self.code, self.page, self.pt[b], self.v, self.vs)

    def table(self, lens):
        """The page table, entries behind the rows in use pointing nowhere."""
        t = self.pt.copy()
        for b, L in enumerate(lens):
            t[b, -(-int(L) // self.page):] = 2 ** 30 if b % 2 else -5
        return dev(t)

    def arrays(self):
        return [dev(x) for x in (self.k, self.v, self.ks, self.vs)]


def same_bits(got, want):
    """Equal bytes; scales equal as numbers or both NaN."""
    return all(torch.equal(a.nan_to_num(nan=-1.0), b.nan_to_num(nan=-1.0)) if a.is_floating_point() else torch.equal(a, b)
               for a, b in zip(got, want))


def tokens(rng, H, n, d, gain=1.0):
    x = rng.normal(size=(H, n, d)) * gain
    x[:, :, 3] *= 8.0
    return R.bf16(x)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("page,d", [(32, 64), (64, 128), (128, 128), (128, 64), (32, 128)])
@pytest.mark.parametrize("inter", [False, True], ids=["half", "interleaved"])
def test_append_bit_exact(page, d, code, inter):
    """Several calls on one pool, some sequences with no new token, magnitudes that
    grow: codes and scales bit for bit, everything else in the pool as it was."""
    B, Hq, Hkv, rot = 3, 6, 2, d - 8 * (page == 64)
    calls = [(page + 9, [page + 9, 0, 1]), (1, [1, 1, 1]), (1, [1, 0, 1]), (2 * page + 5, [7, 2 * page + 5, page]),
             (3, [3, 3, 2]), (1, [1, 1, 1])]
    top = sum(t for t, _ in calls) + 1
    P = Pool(5, B, Hkv, d, page, code, top)
    tab = R.table(top, rot)
    rope = qb.make_rope(dev(tab), interleaved=inter)
    got = P.arrays()
    lens = np.zeros(B, np.int32)
    for step, (T, n) in enumerate(calls):
        K, V, Q = (tokens(P.rng, B * h, T, d, 0.3 * 3.1 ** step).reshape(B, h, T, d) for h in (Hkv, Hkv, Hq))
        lens = lens + np.asarray(n, np.int32)
        shape = qb.make_shape(B, Hq, Hkv, T, int(lens.max()), d)
        q_out = torch.full((B, Hq, T, d), 7.0, dtype=torch.bfloat16, device="cuda")
        q, k, v = (dev(x, torch.bfloat16) for x in (Q, K, V))
        if step % 2:
            q, k, v = heads_last(q), heads_last(k), heads_last(v)
        qb.paged_append(k, v, shape, P.paging, P.table(lens), dev(lens), *got, n_new=dev(np.asarray(n, np.int32)),
                        rope=rope, Q=q, Q_out=q_out)
        assert qb.get_error() == 0
        want_q = np.full((B, Hq, T, d), 7.0, np.float32)
        for b in range(B):
            first, m = int(lens[b]) - n[b], n[b]
            if m:
                pos = np.arange(first, first + m)
                want_q[b, :, :m] = R.rotate(Q[b, :, :m], pos, tab, inter)
                P.put(b, first, R.rotate(K[b, :, :m], pos, tab, inter), V[b, :, :m])
        assert torch.equal(q_out, dev(want_q, torch.bfloat16))
        assert same_bits(got, P.arrays()), f"call {step}"


def test_append_without_rotation_or_counts():
    """No rope, no Q, n_new None (T everywhere), positions given and not used."""
    P = Pool(6, 2, 3, 64, 32, "int8", 50)
    lens = np.array([40, 37], np.int32)
    K, V = (tokens(P.rng, 6, 37, 64).reshape(2, 3, 37, 64) for _ in range(2))
    got = P.arrays()
    for b in range(2):
        seen = tokens(P.rng, 3, 3, 64, 0.1)
        if b == 0:
            P.put(b, 0, seen, seen)
    got = P.arrays()
    qb.paged_append(dev(K, torch.bfloat16), dev(V, torch.bfloat16), qb.make_shape(2, 3, 3, 37, 40, 64), P.paging,
                    P.table(lens), dev(lens), *got)
    for b, L in enumerate(lens):
        P.put(b, L - 37, K[b], V[b])
    assert qb.get_error() == 0 and same_bits(got, P.arrays())


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_append_values_of_all_sizes(code):
    """Zeros, values too small for a scale, NaN and infinity, and what comes behind them
    in the same page; large growth."""
    d, page = 64, 32
    P = Pool(7, 1, 4, d, page, code, 4 * page)
    got = P.arrays()
    rows = [np.zeros((4, 2, d)), np.full((4, 1, d), 2.0 ** -70), np.full((4, 1, d), 1e-3), np.full((4, 1, d), 3e30),
            np.ones((4, 1, d)), np.full((4, 30, d), np.nan), np.ones((4, 2, d)), np.ones((4, 20, d)),
            np.full((4, 1, d), -3.3895e38)]
    rows[5][0, :-1] = rows[5][1, :-1] = 1.0
    rows[5][1, -1] = np.inf
    rows[5][2:, 1:] = -2.0 ** -30
    first = 0
    for x in rows:
        x = R.bf16(x)
        n = x.shape[1]
        lens = np.array([first + n], np.int32)
        t = dev(x[None], torch.bfloat16)
        qb.paged_append(t, t, qb.make_shape(1, 4, 4, n, int(lens[0]), d), P.paging, P.table(lens), dev(lens), *got)
        assert qb.get_error() == 0
        with np.errstate(invalid="ignore"):
            P.put(0, first, x, x)
        assert same_bits(got, P.arrays()), f"row {first}"
        first += n


def test_append_refuses_what_the_device_finds():
    """A length, a count, a page or a position out of range: that part alone is left."""
    d, page = 64, 32
    P = Pool(8, 4, 2, d, page, "int8", 3 * page)
    tab = R.table(60, d)
    T = 40
    K, V = (tokens(P.rng, 8, T, d).reshape(4, 2, T, d) for _ in range(2))
    lens = np.array([T - 1, 97, 50, 45], np.int32)      # fewer rows than new ones; past Nk; page; position
    n = np.array([T, T, T, T], np.int32)
    for b in (2, 3):  # the rows before
        x = tokens(P.rng, 2, int(lens[b]) - T, d, 0.2)
        P.put(b, 0, x, x)
    pt = P.table([96] * 4)
    pt[2, 1] = P.n
    pos = np.tile(np.arange(T, dtype=np.int32), (4, 1))
    pos[3, 35] = 60
    got = P.arrays()
    qb.paged_append(dev(K, torch.bfloat16), dev(V, torch.bfloat16), qb.make_shape(4, 2, 2, T, 96, d), P.paging, pt,
                    dev(lens), *got, n_new=dev(n), positions=dev(pos), rope=qb.make_rope(dev(tab)))
    assert qb.get_error() == qb.ERR_INVALID_ARG
    for b in (2, 3):
        first = int(lens[b]) - T
        k = R.rotate(K[b], np.minimum(pos[b], 59), tab, False)
        if b == 2:  # the rows of the missing page
            m = page - first
            P.put(b, first, k[:, :m], V[b, :, :m])
        else:
            # K of token 35 is not written and does not count for its page's scale
            at = first + 35
            before = P.k[P.pt[b, at // page], :, at % page].copy()
            k0 = k.copy()
            k0[:, 35] = 0
            P.put(b, first, k0, V[b])
            P.k[P.pt[b, at // page], :, at % page] = before
    assert same_bits(got, P.arrays())
    assert qb.get_error() == 0


# ------------------------------------------------------------------ attend
def make(seed, B, Hq, Hkv, d, page, code, T, lens, n=None, gain=1.0, spread=1.0):
    """A filled pool and the queries; codes and scales drawn, not appended."""
    lens = np.asarray(lens, np.int32)
    P = Pool(seed, B, Hkv, d, page, code, int(lens.max()))
    rng = P.rng
    top = 127 if code == "int8" else 448
    for b in range(B):
        for j in range(-(-int(lens[b]) // page)):
            p, m = P.pt[b, j], min(page, int(lens[b]) - j * page)
            z = rng.normal(size=(2, Hkv, m, d)) * top / 4.5
            kv = R.encode(np.clip(z, -top, top).astype(np.float32), code)
            P.k[p, :, :m], P.v[p, :, :m] = kv[0], kv[1]
            P.ks[p] = rng.uniform(0.5, 1.5, Hkv) * 4.5 / top
            P.vs[p] = rng.uniform(0.5, 1.5, Hkv) * 4.5 / top * spread ** rng.uniform(-1, 1, Hkv)
    P.lens, P.T, P.Hq = lens, T, Hq
    P.new = np.full(B, T, np.int32) if n is None else np.asarray(n, np.int32)
    P.q = R.bf16(gain * 1.5 * rng.normal(size=(B, Hq, T, d)))
    return P


def run(P, causal=True, out_dtype=qb.DT_F32, strided=False, counts=True, Nk=None, stream=None, fill=7.0, arrays=None,
        sm_scale=0.0):
    B, Hq, T, d = P.q.shape
    shape = qb.make_shape(B, Hq, P.Hkv, T, int(P.lens.max()) if Nk is None else Nk, d)
    params = qb.make_params(causal=causal, out_dtype=out_dtype, sm_scale=sm_scale)
    O = torch.full((B, Hq, T, d), fill, dtype=torch.bfloat16 if out_dtype == qb.DT_BF16 else torch.float32, device="cuda")
    lse = torch.full((B, Hq, T), fill, device="cuda")
    ws = torch.full((max(qb.paged_workspace_size(shape, params, P.paging), 256),), 0xFF, dtype=torch.uint8, device="cuda")
    q = dev(P.q, torch.bfloat16)
    if strided:
        q = heads_last(q)
    qb.paged_fwd(q, shape, params, P.paging, P.table(P.lens), dev(P.lens), *(P.arrays() if arrays is None else arrays), O,
                 lse, ws, n_new=dev(P.new) if counts else None, stream=stream)
    return O, lse


def check(P, O, lse, causal=True, sm=None, fill=7.0):
    """Against the 64-bit form.  The error allowed per element, with A = sum P |v| / l:
    P's rounding to fp16, half a step (2^-11 of P; below the type's normal range 2^-25,
    which is at most 2^-32 of the row's largest part a key, as the reference lies 7 or
    more below it); S, by d / 16 matrix instructions that may truncate 17 addends each
    at 2^-24 of the largest; the exponent t - m, by eight roundings of at most max |t|
    (2^-24 each), ex2 and the scales by 2^-21; the PV product, by one such instruction
    for 16 keys, and 700 more additions; the output's own rounding."""
    B, Hq, T, d = P.q.shape
    G = Hq // P.Hkv
    sm = 1.0 / np.sqrt(d) if sm is None else sm
    half = torch.finfo(O.dtype).eps / 2
    top = 127 if P.code == "int8" else 448
    O, lse = O.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(B):
        L, n = int(P.lens[b]), int(P.new[b])
        assert (O[b, :, n:] == fill).all() and (lse[b, :, n:] == fill).all()
        see = np.ones((n, L), bool)
        if causal:
            see = np.arange(L)[None] <= (L - n + np.arange(n))[:, None]
        for h in range(P.Hkv):
            kc, ks = R.rows(P.k, P.ks, P.pt[b], h, L, P.page, P.code)
            vc, vs = R.rows(P.v, P.vs, P.pt[b], h, L, P.page, P.code)
            for hq in range(h * G, (h + 1) * G):
                q = P.q[b, hq, :n]
                o, z, A, big, part = R.attend(q, kc, ks, vc, vs, see, sm)
                mass = ((np.abs(q) @ np.abs(kc).T) * ks).max(initial=0.0) * sm / np.log(2.0)
                e_s = d / 16 * 17 * 2.0 ** -24 * mass + d * mass * 2.0 ** -39
                e_p = np.log(2) * (8 * 2.0 ** -24 * big + e_s) + 2.0 ** -21
                adds = L / 16 * 17 * 2.0 ** -24 + 700 * 2.0 ** -23
                tol = A * (2.0 ** -11 + 2 * e_p + 2 * adds) + L * top * part * 2.0 ** -32 + half * np.abs(o)
                np.testing.assert_array_less(np.abs(O[b, hq, :n] - o), tol + 1e-30, err_msg=f"O b{b} h{hq}")
                fin = np.isfinite(z)
                assert np.array_equal(np.isfinite(lse[b, hq, :n]), fin) and np.all(lse[b, hq, :n][~fin] == -np.inf)
                ztol = e_p + adds + 2.0 ** -23 * (np.abs(z[fin]) + 2 * big) + 2.0 ** -21
                np.testing.assert_array_less(np.abs(lse[b, hq, :n][fin] - z[fin]), ztol)


SHAPES = [
    # B, Hq, Hkv, d, page, code, T, lengths, n_new
    (1, 4, 1, 128, 64, "int8", 1, [257], None),
    (1, 8, 2, 128, 32, "e4m3", 1, [1], None),
    (2, 4, 2, 64, 128, "int8", 3, [0, 33], [2, 3]),
    (3, 8, 2, 128, 64, "e4m3", 4, [31, 32, 500], [4, 0, 3]),
    (1, 6, 2, 128, 32, "int8", 7, [1000], None),           # 21 rows: a ragged row block
    (2, 2, 2, 64, 32, "e4m3", 33, [129, 20], [33, 31]),    # rows that see nothing
    (1, 4, 1, 128, 128, "int8", 64, [700], None),          # 256 rows of one KV head
    (1, 16, 1, 64, 64, "e4m3", 128, [200], [117]),         # 2048 rows of one KV head
    (2, 3, 1, 128, 64, "int8", 301, [301, 640], [301, 129]),  # a whole prompt
    (5, 4, 2, 128, 32, "int8", 2, [4173, 0, 17, 1, 900], [1, 2, 2, 0, 2]),
    (40, 2, 1, 64, 32, "e4m3", 1, list(range(0, 1200, 30)), None),  # more sequences than a warp has lanes
    (1, 5, 5, 64, 64, "int8", 1, [9001], None),
    (1, 4, 1, 128, 64, "int8", 200, [5000], None),            # 800 rows over 40 blocks of keys
    (3, 2, 1, 64, 32, "e4m3", 100, [3000, 100, 2049], [100, 65, 30]),  # row blocks of one tile and of two
    (2, 8, 1, 128, 128, "e4m3", 40, [6000, 333], [40, 9]),
    (1, 1, 1, 64, 128, "int8", 700, [2300], None),
    # shares of many steps, blocks of one tile and of two
    (8, 16, 8, 64, 32, "int8", 9, [3000, 2999, 1700, 2100, 40, 3100, 2500, 2000], [9, 9, 8, 9, 9, 9, 1, 9]),
    (3, 12, 12, 64, 64, "e4m3", 515, [1500, 2000, 1030], [515, 260, 300]),
    (2, 32, 8, 128, 64, "int8", 70, [2500, 4000], [70, 20]),
    (7, 4, 4, 128, 32, "int8", 130, [131, 130, 700, 0, 1500, 260, 128], [130, 129, 128, 0, 127, 1, 128]),
]


@pytest.mark.parametrize("shape", SHAPES, ids=[f"{s[5]}-H{s[1]}-{s[2]}-d{s[3]}-T{s[6]}-L{max(s[7])}" for s in SHAPES])
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "all"])
def test_attend_matches_fp64(shape, causal):
    P = make(11, *shape)
    O, lse = run(P, causal)
    assert qb.get_error() == 0
    check(P, O, lse, causal)


@pytest.mark.parametrize("shape", [SHAPES[3], SHAPES[7], SHAPES[8]], ids=["few", "rows", "prompt"])
def test_attend_bf16_strided_sharp(shape):
    """bf16 output, a strided Q, scores that single keys rule, page scales 2^8 apart
    either way, a bound on the rows far above the lengths."""
    P = make(12, *shape, gain=6.0, spread=256.0)
    O, lse = run(P, out_dtype=qb.DT_BF16, strided=True, Nk=P.width * P.page)
    assert qb.get_error() == 0
    check(P, O, lse)


def test_attend_counts_default_and_scale():
    P = make(13, 2, 4, 2, 64, 32, "int8", 5, [70, 6])
    O, lse = run(P, counts=False, sm_scale=0.31)
    assert qb.get_error() == 0
    check(P, O, lse, sm=0.31)


@pytest.mark.parametrize("T", [1, 20], ids=["one", "few"])
@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_attend_page_scales_of_zero(T, code):
    """A V scale of 0 (a page of zeros) takes its share of the weight and gives nothing,
    whatever the other pages' scales and wherever it lies; a K scale of 0 gives scores
    of 0."""
    for big in (2.0 ** -30, 1.0, 2.0 ** 40, 2.0 ** 60):
        P = make(14, 1, 4, 1, 64, 32, code, T, [200], gain=0.3)
        P.vs *= np.float32(big)
        for j in (0, 3, 6):
            P.vs[P.pt[0, j]] = 0
            # codes there need not be zeros
        P.ks[P.pt[0, 2]] = 0
        O, lse = run(P)
        assert qb.get_error() == 0
        if big == 2.0 ** 60:  # V scales above 2^48 are refused as infinite ones are
            assert P.vs[P.pt[0, :7]].max() > 2.0 ** 48 and O.isnan().all() and lse.isnan().all()
        else:
            check(P, O, lse)
    P.vs[P.pt[0, :7]] = 0
    O, lse = run(P)
    assert (O == 0).all()
    check(P, O, lse)


@pytest.mark.parametrize("T", [2, 40], ids=["two", "forty"])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -1.0])
def test_attend_scales_that_are_not_numbers(T, bad):
    """A bad scale gives NaN to the rows that see its page and to no other."""
    for which in ("ks", "vs"):
        P = make(15, 2, 2, 1, 128, 32, "int8", T, [33, 100])
        getattr(P, which)[P.pt[0, 1]] = bad      # holds the last row alone
        O, lse = run(P)
        assert qb.get_error() == 0
        O, lse = O.cpu(), lse.cpu()
        assert O[0, :, T - 1].isnan().all() and lse[0, :, T - 1].isnan().all()
        assert not O[0, :, :T - 1].isnan().any() and not lse[0, :, :T - 1].isnan().any()
        assert not O[1].isnan().any()


@pytest.mark.parametrize("T", [2, 40], ids=["two", "forty"])
def test_attend_queries_that_are_not_numbers(T):
    P = make(16, 2, 2, 1, 64, 64, "int8", T, [0, 100])
    P.q[:, 0, 0, 5] = np.nan
    P.q[:, 1, T - 1, 9] = np.inf
    O, lse = run(P)
    O, lse = O.cpu(), lse.cpu()
    assert (O[0] == 0).all() and (lse[0] == -np.inf).all()  # they see nothing
    want = torch.zeros(2, T, dtype=torch.bool)
    want[0, 0] = want[1, T - 1] = True
    assert torch.equal(lse[1].isnan(), want) and torch.equal(O[1].isnan().all(-1), want)
    assert torch.equal(O[1].isnan().any(-1), want)


@pytest.mark.parametrize("T", [1, 24], ids=["one", "few"])
def test_attend_refuses_what_the_device_finds(T):
    """Lengths and counts out of range are clamped, a page that does not exist is hidden."""
    P = make(17, 3, 2, 1, 64, 32, "int8", T, [96, 96, 96])
    arrays, pt = P.arrays(), P.table([96] * 3)
    pt[2, 1] = P.n
    shape, params = qb.make_shape(3, 2, 1, T, 96, 64), qb.make_params()
    O, lse = torch.zeros(3, 2, T, 64, device="cuda"), torch.zeros(3, 2, T, device="cuda")
    ws = torch.empty(max(qb.paged_workspace_size(shape, params, P.paging), 256), dtype=torch.uint8, device="cuda")
    lens, n = torch.tensor([97, -1, 96], dtype=torch.int32, device="cuda"), torch.tensor([T, T + 1, T], dtype=torch.int32, device="cuda")
    qb.paged_fwd(dev(P.q, torch.bfloat16), shape, params, P.paging, pt, lens, *arrays, O, lse, ws, n_new=n)
    assert qb.get_error() == qb.ERR_INVALID_ARG
    assert (O[1] == 0).all() and (lse[1] == -float("inf")).all()
    P.lens[1] = 0
    keep = np.r_[0:32, 64:96]
    for b, rows in ((0, np.arange(96)), (2, keep)):
        for hq in range(2):
            kc, ks = R.rows(P.k, P.ks, P.pt[b], 0, 96, 32, "int8")
            vc, vs = R.rows(P.v, P.vs, P.pt[b], 0, 96, 32, "int8")
            o = R.attend(P.q[b, hq], kc[rows], ks[rows], vc[rows], vs[rows], np.ones((T, len(rows)), bool), 0.125)[0]
            assert np.abs(O[b, hq].cpu().numpy() - o).max() < 2.0 ** -9 * np.abs(vc * vs[:, None]).max()
    assert qb.get_error() == 0


@pytest.mark.parametrize("T", [1, 5], ids=["one", "few"])
def test_attend_in_a_pool_past_4_GB(T):
    """Pages whose offsets pass 32 bits, with the codes of pages at the start."""
    d, page, Hkv = 128, 128, 8
    n = 2 ** 32 // (Hkv * page * d) + 40
    P = make(18, 1, 8 * 4, Hkv, d, page, "int8", T, [1000])
    k, v = (torch.zeros(n, Hkv, page, d, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((n, Hkv), float("nan"), device="cuda") for _ in range(2))
    far = torch.arange(n - 8, n, device="cuda")
    src = dev(P.pt[0, :8]).long()
    for big, small in zip((k, v, ks, vs), P.arrays()):
        big[far] = small[src]
    shape, params = qb.make_shape(1, 32, Hkv, T, 1000, d), qb.make_params(causal=True)
    paging = qb.make_paging(n, page, 8)
    O, lse = torch.zeros(1, 32, T, d, device="cuda"), torch.zeros(1, 32, T, device="cuda")
    ws = torch.empty(max(qb.paged_workspace_size(shape, params, paging), 256), dtype=torch.uint8, device="cuda")
    qb.paged_fwd(dev(P.q, torch.bfloat16), shape, params, paging, far.int()[None].contiguous(), dev(P.lens), k, v, ks, vs, O, lse, ws)
    assert qb.get_error() == 0
    check(P, O, lse)
    # and appended there
    x = tokens(P.rng, Hkv, 3, d)
    pt = torch.full((1, 8), n - 1, dtype=torch.int32, device="cuda")
    t = dev(x[None], torch.bfloat16)
    qb.paged_append(t, t, qb.make_shape(1, 8, Hkv, 3, 1024, d), paging, pt, torch.tensor([3], dtype=torch.int32, device="cuda"), k, v, ks, vs)
    assert qb.get_error() == 0
    want, ws_ = np.zeros((1, Hkv, page, d), np.int8), np.zeros((1, Hkv), np.float32)
    R.append(x, 0, "int8", page, [0], want, ws_)
    assert np.array_equal(k[n - 1, :, :3].cpu().numpy(), want[0, :, :3]) and np.array_equal(ks[n - 1].cpu().numpy(), ws_[0])


def test_attend_equal_calls_give_equal_bits_on_two_streams():
    """Two calls at once, a workspace each; and the same call again."""
    cases = [make(19, 3, 8, 2, 128, 64, "int8", 1, [30000, 12001, 7]), make(20, 1, 8, 2, 64, 64, "e4m3", 150, [5000])]
    alone = [run(P) for P in cases]
    torch.cuda.synchronize()
    data = [P.arrays() for P in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for P, s, a in zip(cases, streams, data):
            with torch.cuda.stream(s):
                got.append(run(P, arrays=a))
        torch.cuda.synchronize()
        for (O, lse), (O1, lse1) in zip(got, alone):
            assert torch.equal(O, O1) and torch.equal(lse, lse1)
    assert qb.get_error() == 0


# ------------------------------------------------------- a run of them together
@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("inter", [False, True], ids=["half", "interleaved"])
def test_paged_cache_serves(code, inter):
    """Prompts, chunks and single tokens of three sequences, one of them ended and its
    pages used again: codes bit for bit, O against the 64-bit form on those codes."""
    B, Hq, Hkv, d, page, rows = 3, 4, 2, 64, 32, 300
    tab = rope_table(rows, 48, scaling="linear", factor=2.0)
    C = PagedCache(24, page, Hq, Hkv, d, B, rows, code_dtype=DT[code], rope=qb.make_rope(tab, interleaved=inter),
                   out_dtype=qb.DT_F32)
    tab = tab.cpu().numpy()
    rng = np.random.default_rng(9)
    P = Pool(1, B, Hkv, d, page, code, rows)
    P.k, P.v, P.ks, P.vs = (t.cpu().numpy() for t in (C.k_pages, C.v_pages, C.k_scales, C.v_scales))
    lens = np.zeros(B, int)
    steps = [(70, [70, 33, 1]), (1, [1, 1, 1]), (40, [0, 40, 12]), "release", (90, [90, 1, 1]), (1, [1, 1, 1]), (3, [3, 0, 2])]
    for st in steps:
        if st == "release":
            C.release(0)
            lens[0] = 0
            continue
        T, n = st
        K, V, Q = (tokens(rng, B * h, T, d).reshape(B, h, T, d) for h in (Hkv, Hkv, Hq))
        O = C.step(*(heads_last(dev(x, torch.bfloat16)) for x in (Q, K, V)), n_new=n)
        assert qb.get_error() == 0
        lens += n
        P.pt = C.page_table.cpu().numpy()
        P.q = np.zeros((B, Hq, T, d), np.float32)
        for b in range(B):
            pos = np.arange(lens[b] - n[b], lens[b])
            P.q[b, :, :n[b]] = R.bf16(R.rotate(Q[b, :, :n[b]], pos, tab, inter))
            if n[b]:
                P.put(b, int(lens[b]) - n[b], R.rotate(K[b, :, :n[b]], pos, tab, inter), V[b, :, :n[b]])
        assert same_bits([C.k_pages, C.v_pages, C.k_scales, C.v_scales], P.arrays())
        P.lens, P.new = lens.astype(np.int32), np.asarray(n, np.int32)
        live = [O.clone(), C.lse(T).clone()]
        for t in live:  # rows behind a sequence's tokens: checked elsewhere
            for b in range(B):
                t[b, :, n[b]:] = 7.0
        check(P, *live)
        assert C.rows(1) == lens[1]


def test_paged_cache_refuses_and_captures():
    """A pool that runs out changes nothing; append and attend replayed from a graph."""
    B, Hq, Hkv, d, page = 2, 4, 2, 64, 32
    rope = qb.make_rope(rope_table(128, d))
    C = PagedCache(5, page, Hq, Hkv, d, B, 128, rope=rope, out_dtype=qb.DT_F32)
    E = PagedCache(5, page, Hq, Hkv, d, B, 128, rope=rope, out_dtype=qb.DT_F32)
    with pytest.raises(ValueError, match="free pages"):
        C.grow([96, 96])
    with pytest.raises(ValueError, match="max_rows"):
        C.grow([129, 0])
    with pytest.raises(ValueError, match="n_new"):
        C.grow([1])
    assert C.free_pages() == 5 and C.rows(0) == 0
    g = torch.Generator(device="cuda").manual_seed(2)
    new = lambda T: [torch.randn(B, h, T, d, generator=g, device="cuda").to(torch.bfloat16) for h in (Hq, Hkv, Hkv)]  # noqa: E731
    x = new(40)
    for c in (C, E):
        c.step(*x, n_new=[40, 11])
    buf = new(1)
    for c in (C, E):  # the buffers of one-token steps exist before the capture
        c.step(*buf)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        O = C.attend(C.append(*buf))
    for _ in range(30):
        for t, y in zip(buf, new(1)):
            t.copy_(y)
        C.grow([1, 1])
        graph.replay()
        want = E.step(*buf)
        assert torch.equal(O, want) and torch.equal(C.k_pages, E.k_pages) and torch.equal(C.v_scales, E.v_scales)
    assert qb.get_error() == 0
