"""Values at the edges of the serving operators' number formats: scores whose
probabilities are far below the row's largest, and scales that are not finite."""
import numpy as np
import pytest
import torch

from quantized_attention_gb300 import binding as qb
from tests import tree_ref as R
from tests.gpu_common import ensure_library
from tests.test_gpu_16_tree import dev, make, run, words_of

pytestmark = pytest.mark.gpu

# T, lengths: few rows in a head's own cluster and in shares, more than 16 rows in both
FORMS = {"few-cluster": (2, [600, 450]), "few-shares": (1, [20011, 300]),
         "many-cluster": (40, [600, 450]), "many-shares": (48, [20011, 300])}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_library()


def form(name, Hq=8, Hkv=2, d=128):
    """A problem of this form: whether shares are written says the workspace."""
    T, lens = FORMS[name]
    need = qb.tree_workspace_size(qb.make_shape(len(lens), Hq, Hkv, T, max(lens), d), qb.make_params())
    assert (need > 0) == name.endswith("shares")
    return make(17, len(lens), Hq, Hkv, d, T, lens)


@pytest.mark.parametrize("name", FORMS)
@pytest.mark.parametrize("gap", [8.0, 13.0, 14.0, 16.0, 19.0])
@pytest.mark.parametrize("where", ["first", "last"])
def test_one_key_above_all_others(name, gap, where):
    """One key `gap` nats above all others, whose scores are equal and whose V is not
    0 as its own is: every P of the others is e^-gap of the row's largest and their
    roundings do not average out.  P's eleven bits hold down to 2^-29 (20 nats) of the
    largest with at most 16 rows a KV head and to 2^-21 (14.5 nats) with more, so the
    relative error is at most half a step, 2^-11, and the fp32 parts' share as in the
    shapes' test (e_p once in the sum and once in l, the additions)."""
    if gap > 14.5 and name.startswith("many"):
        pytest.skip("P of the others lies below fp16's normal range")
    x = form(name)
    B, Hkv, d, G = x["B"], x["Hkv"], x["d"], x["Hq"] // x["Hkv"]
    x["qc"][:] = 100
    x["kc"][:] = 0
    x["vc"][:] = np.abs(x["vc"]) // 2 + 20
    for b in range(B):
        p = 0 if where == "first" else int(x["lens"][b]) - 1
        x["kc"][b, :, p] = 90
        x["vc"][b, :, p] = 0
    x["qs"][:] = np.float32(gap * np.sqrt(d) / (100 * 90 * d))
    O, lse = run(x, "cached")
    O, lse = O.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(B):
        L = int(x["lens"][b])
        see = R.visible(x["T"], L, mode="cached")
        for h in range(Hkv):
            for hq in range(h * G, (h + 1) * G):
                o, z, _, big = R.attend(x["qc"][b, hq], float(x["qs"][b, hq]) / np.sqrt(d), x["kc"][b, h, :L],
                                        x["vc"][b, h, :L], x["vs"][b, h], see)
                e_p = np.log(2) * 2 * 2 * big * 2.0 ** -24 + 2.0 ** -22
                adds = (L / 16 + 700) * 2.0 ** -23
                assert np.all(o > 0)
                rel = np.abs(O[b, hq] - o) / o
                assert rel.max() <= 2.0 ** -11 + 2 * e_p + 2 * adds, (rel.max(), b, hq)
                assert np.abs(lse[b, hq] - z).max() <= e_p + adds + 2.0 ** -23 * (np.abs(z).max() + 2 * big) + 2.0 ** -22


@pytest.mark.parametrize("name", FORMS)
@pytest.mark.parametrize("big", [2.0 ** 21, 2.0 ** 25])
def test_scores_past_the_lowered_reference(name, big):
    """Scores so large that a reference below the maximum by a few units would round:
    one key takes all, as in 64 bits."""
    x = form(name)
    x["qs"][:] = np.float32(big / (100 * 100 * x["d"]) * np.sqrt(x["d"]))
    x["qc"][:] = 100
    x["kc"] = np.minimum(x["kc"], 90)
    for b in range(x["B"]):
        x["kc"][b, :, int(x["lens"][b]) // 2] = 100
    O, lse = run(x, "cached")
    for b in range(x["B"]):
        p = int(x["lens"][b]) // 2
        for h in range(x["Hkv"]):
            want = torch.from_numpy(x["vc"][b, h, p].astype(np.float32) * x["vs"][b, h]).cuda()
            got = O[b, 4 * h:4 * h + 4]
            # the reference is fl(S c), so P = 2^(S c - fl(S c)) (of size 1 to 2^(ulp / 2), no
            # power of two): rounded to fp16 it is off by 2^-11, while l has it unrounded;
            # ex2, 1 / l and V s: 2^-20
            torch.testing.assert_close(got, want.expand_as(got), rtol=2.0 ** -11 + 2.0 ** -20, atol=0)
        assert torch.isfinite(lse).all()


@pytest.mark.parametrize("name", FORMS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_scale_that_is_not_finite(name, bad):
    """NaN for the query head it belongs to, in O and in lse, whatever the division of
    the work; the other heads keep their bits."""
    x = form(name)
    want_o, want_z = run(x, "chain")
    x["qs"][0, 1] = x["qs"][1, 6] = bad
    O, lse = run(x, "chain")
    hit = torch.zeros(2, 8, dtype=torch.bool, device="cuda")
    hit[0, 1] = hit[1, 6] = True
    assert torch.isnan(O[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(O[~hit], want_o[~hit]) and torch.equal(lse[~hit], want_z[~hit])


@pytest.mark.parametrize("T,lens,cap", [(6, [0, 0], 50), (40, [0, 0], 50), (6, [0, 0], 20011), (40, [0, 0], 20011),
                                        (6, [0, 20011], 20011), (40, [0, 20011], 20011)])
def test_padding_rows_with_scales_that_are_not_finite(T, lens, cap):
    """A row that sees nothing gives O = 0 and lse = -inf whatever its scale."""
    x = make(18, 2, 4, 2, 64, T, lens, cap=cap)
    see = np.zeros((2, T, T), bool)
    see[1] = np.tril(np.ones((T, T), bool))
    x["qs"][0] = [np.nan, np.inf, np.nan, 0.0]
    O, lse = run(x, "tree", words_of(see), Nk=cap)
    assert torch.all(O[0] == 0) and torch.all(lse[0] == -float("inf"))
    assert torch.isfinite(O[1]).all() and torch.isfinite(lse[1]).all()


@pytest.mark.parametrize("T,G", [(3, 2), (40, 4), (70, 1), (300, 2)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_weights_of_masked_queries_with_scales_that_are_not_finite(T, G, bad):
    """A query with lse = -inf gives nothing, whatever its scale: a sequence of
    queries that do not count, and one head's among others that do."""
    rng = np.random.default_rng(19)
    B, Hkv, d, N = 2, 2, 64, 700
    Hq, nb = Hkv * G, (T + 127) // 128
    qc = dev(rng.integers(-127, 128, (B, Hq, T, d)).astype(np.int8))
    kc = dev(rng.integers(-127, 128, (B, Hkv, N, d)).astype(np.int8))
    qs = torch.full((B, Hq, nb), 1e-4, device="cuda")
    lse = torch.full((B, Hq, T), 6.0, device="cuda")
    lse[0] = -float("inf")
    lse[1, 0] = -float("inf")
    base = torch.rand(B, Hkv, N, device="cuda")
    shape, params = qb.make_shape(B, Hq, Hkv, T, N, d), qb.make_params()
    want, got = torch.zeros_like(base), torch.zeros_like(base)
    qb.kv_weights(qc, qs, kc, None, lse, shape, params, want, base=base)
    qs[0] = bad
    qs[1, 0] = bad
    qb.kv_weights(qc, qs, kc, None, lse, shape, params, got, base=base)
    torch.cuda.synchronize()
    assert qb.get_error() == 0
    assert torch.equal(want[0], base[0])
    assert torch.equal(got, want)
