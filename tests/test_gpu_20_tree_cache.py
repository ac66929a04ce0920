"""pipeline.TreeCache: rows that enter by another way than an accepted path, and
what an eviction returns."""
import numpy as np
import pytest
import torch

from quantized_attention_gb300 import binding as qb
from tests import tree_ref as R
from tests.gpu_common import ensure_library
from tests.test_gpu_17_kv_evict import dev, tree_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_library()


def tokens(gen, B, H, T, d):
    return torch.randn(B, H, T, d, device="cuda", generator=gen).to(torch.bfloat16)


def check_weights(C, before, lse):
    """The rows' weights after `weigh`: what they were plus each query's share of the
    rows it sees causally (the last T rows are the queries' own); relative 2^-14 as in
    the serving loop's test."""
    B, Hq, T, d = C.q_codes.shape
    G = Hq // C.k_codes.shape[1]
    qc, qs, lse = C.q_codes.cpu().numpy(), C.q_scales.cpu().numpy().reshape(B, Hq), lse.double().cpu().numpy()
    for b in range(B):
        L = int(C.lengths[b])
        see = np.arange(L)[None, :] <= L - T + np.arange(T)[:, None]
        for h in range(C.k_codes.shape[1]):
            kk = C.k_codes[b, h, :L].cpu().numpy()
            want = before[b, h, :L].astype(np.float64)
            for hq in range(G * h, G * h + G):
                want = want + R.weight(qc[b, hq], np.full(T, qs[b, hq]), kk, np.ones(L), lse[b, hq], see,
                                       1 / np.sqrt(d))[0]
            np.testing.assert_allclose(C.weights[b, h, :L].cpu().numpy().astype(np.float64), want, rtol=2.0 ** -14)


@pytest.mark.parametrize("stream", [False, True])
def test_append_then_verify_without_drafts(stream):
    """Tokens appended and read from the cache, between evictions: the header as after
    one running mean over every token, the new rows' weights from 0."""
    B, Hq, Hkv, d, T, cap = 2, 4, 2, 64, 3, 120
    C = tree_cache(np.random.default_rng(81), B, Hq, Hkv, d, T, cap, [90, 47])
    gen = torch.Generator(device="cuda").manual_seed(82)
    st = torch.cuda.Stream() if stream else None
    torch.cuda.synchronize()
    seen = [90, 47]
    for step in range(4):
        n = T if step < 3 else 11  # as many tokens as queries, or another number
        K, V, Q = tokens(gen, B, Hkv, n, d), tokens(gen, B, Hkv, n, d), tokens(gen, B, Hq, T, d)
        torch.cuda.synchronize()
        old = {k: getattr(C, k).cpu().numpy().copy() for k in ("k_codes", "v_codes", "k_mean", "v_code_amax", "lengths")}
        C.append(K, V, stream=st)
        torch.cuda.synchronize()
        assert qb.get_error() == 0
        for b in range(B):
            L = int(old["lengths"][b])
            kc, vc = old["k_codes"][b].copy(), old["v_codes"][b].copy()
            m, a = R.commit(K[b].float().cpu().numpy(), V[b].float().cpu().numpy(), range(n), n, L, seen[b],
                            C.k_scale[b].cpu().numpy(), C.v_scale[b].cpu().numpy(), old["k_mean"][b],
                            old["v_code_amax"][b], kc, vc)
            assert np.array_equal(C.k_mean[b].cpu().numpy(), m) and np.array_equal(C.v_code_amax[b].cpu().numpy(), a)
            assert np.array_equal(C.k_codes[b].cpu().numpy(), kc) and np.array_equal(C.v_codes[b].cpu().numpy(), vc)
            seen[b] += n
            assert int(C.lengths[b]) == L + n and int(C.seen[b]) == seen[b]
            assert torch.all(C.weights[b, :, L:L + n] == 0)
        before = C.weights.cpu().numpy().copy()
        C.verify(Q, stream=st)
        C.weigh(stream=st)
        torch.cuda.synchronize()
        assert qb.get_error() == 0
        check_weights(C, before, C.lse)
        C.evict(60 - 7 * step, 2, 5, stream=st)
        torch.cuda.synchronize()
        assert qb.get_error() == 0


def test_rows_written_from_outside_start_with_no_weight():
    """After two evictions the arrays of the first set are back: what the rows behind
    the kept ones weighed there is gone."""
    B, Hq, Hkv, d, T, cap = 1, 4, 2, 64, 3, 120
    C = tree_cache(np.random.default_rng(83), B, Hq, Hkv, d, T, cap, [100])
    gen = torch.Generator(device="cuda").manual_seed(84)
    for budget in (80, 50):
        C.verify(tokens(gen, B, Hq, T, d))
        C.weigh()
        C.evict(budget, 2, 5)
    K, V = tokens(gen, B, Hkv, T, d), tokens(gen, B, Hkv, T, d)
    qb.kv_append(K, V, 50, C.k_scale, C.v_scale, C.k_mean, C.v_code_amax, C.k_codes, C.v_codes)
    C.lengths += T
    C.seen += T
    before = C.weights.cpu().numpy().copy()
    before[:, :, 50:] = 0
    C.verify(tokens(gen, B, Hq, T, d))
    C.weigh()
    torch.cuda.synchronize()
    assert qb.get_error() == 0
    check_weights(C, before, C.lse)


def test_evict_marks_the_entries_without_a_row():
    """kept is -1 behind the rows kept, whatever its memory held."""
    C = tree_cache(np.random.default_rng(85), 2, 4, 2, 64, 3, 90, [40, 9])
    torch.full((2, 2, 30), 7, dtype=torch.int32, device="cuda")  # freed: the next of this size lies there
    kept = C.evict(30, 2, 5)
    torch.cuda.synchronize()
    assert qb.get_error() == 0
    assert torch.all(kept[0] >= 0) and torch.all(kept[1, :, :9] >= 0)
    assert torch.all(kept[1, :, 9:] == -1)
