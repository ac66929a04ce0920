"""PagedCache between streams, over many token counts, and after refused steps."""
import pytest
import torch

from quantized_attention_gb300 import binding as qb
from quantized_attention_gb300.pipeline import PagedCache, rope_table
from tests.gpu_common import ensure_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_library()


def caches(n, B, Hq, Hkv, d, rows, page=32, rope=True, **kw):
    turn = qb.make_rope(rope_table(rows, d)) if rope else None
    pages = B * (-(-rows // page)) + 1
    return [PagedCache(pages, page, Hq, Hkv, d, B, rows, rope=turn, **kw) for _ in range(n)]


def tokens(C, g, T, gain=1.0):
    B, Hq, Hkv, d = C._dims
    return [(gain * torch.randn(B, h, T, d, generator=g, device="cuda")).to(torch.bfloat16) for h in (Hq, Hkv, Hkv)]


@pytest.mark.parametrize("rope", [True, False], ids=["rope", "plain"])
def test_steps_on_a_given_stream(rope):
    """step(stream=side) while the current stream is busy: what the first step of a token
    count makes for itself is ready on `side`, and nothing of the current stream's comes
    behind it."""
    C, E = caches(2, 2, 8, 2, 128, 1024, rope=rope, out_dtype=qb.DT_F32)
    g = torch.Generator(device="cuda").manual_seed(1)
    side = torch.cuda.Stream()
    for T in (513, 1, 40, 7):
        x = tokens(C, g, T)
        want, lse = C.step(*x).clone(), C.lse(T).clone()
        spare = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
        del spare  # memory that the allocator has at hand for the current stream
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)  # ~50 ms of the current stream
        got = E.step(*x, stream=side)
        side.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(E.lse(T), lse)
    assert qb.get_error() == 0


@pytest.mark.parametrize("rope", [True, False], ids=["rope", "plain"])
def test_token_counts_share_their_buffers(rope):
    """Steps of many token counts keep what the largest of a power of two needs, and no
    more; each gives what the calls give in buffers of their own."""
    B, Hq, Hkv, d = 2, 8, 2, 64
    C, = caches(1, B, Hq, Hkv, d, 4096, rope=rope, out_dtype=qb.DT_F32)
    g = torch.Generator(device="cuda").manual_seed(2)

    def step(T):
        q, k, v = tokens(C, g, T)
        O, lse = C.step(q, k, v), C.lse(T)
        assert O.shape == (B, Hq, T, d) and O.is_contiguous() and lse.shape == (B, Hq, T) and lse.is_contiguous()
        turned = q
        if rope:
            turned = torch.empty_like(q)
            row = torch.arange(C.rows(0) - T, C.rows(0), dtype=torch.int32, device="cuda")
            qb.rotate(q, turned, C.rope, positions=row.repeat(B, 1))
        shape = qb.make_shape(B, Hq, Hkv, T, C.max_rows, d)
        own, own_lse = torch.empty_like(O), torch.empty_like(lse)
        ws = torch.empty(max(qb.paged_workspace_size(shape, C.params, C.paging), 256), dtype=torch.uint8, device="cuda")
        qb.paged_fwd(turned, shape, C.params, C.paging, C.page_table, C.lengths, C.k_pages, C.v_pages, C.k_scales,
                     C.v_scales, own, own_lse, ws, n_new=C.n_new)
        assert torch.equal(O, own) and torch.equal(lse, own_lse)

    step(33)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for T in (64, 34, 47, 63, 50, 33, 48, 64):
        step(T)
    assert torch.cuda.memory_allocated() == before
    for T in (1, 2, 3, 5, 8, 13, 17, 32, 100):  # seven more sizes: 1, 2, 4, 8, 16, 32, 128
        step(T)
    row = B * Hq * (4 * d + 4 + (2 * d if rope else 0))  # O and lse, and Q if it is rotated
    spaces = sum(max(qb.paged_workspace_size(qb.make_shape(B, Hq, Hkv, T, C.max_rows, d), C.params, C.paging), 256)
                 for T in (1, 2, 4, 8, 16, 32, 128))
    assert torch.cuda.memory_allocated() - before <= row * (1 + 2 + 4 + 8 + 16 + 32 + 128) + 2 * spaces + 28 * 512
    assert qb.get_error() == 0


def test_a_captured_step_keeps_its_buffers():
    """A graph of steps of five tokens, replayed between eager steps of other counts."""
    C, E = caches(2, 2, 4, 2, 64, 2048, out_dtype=qb.DT_F32)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = tokens(C, g, 5)
    for c in (C, E):
        c.step(*x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        O = C.attend(C.append(*x))
    for T in (5, 8, 200, 5, 7, 6, 300, 1, 5):
        if T == 5:
            for t, y in zip(x, tokens(C, g, 5)):
                t.copy_(y)
            C.grow([5, 5])
            graph.replay()
            assert torch.equal(O, E.step(*x))
        else:
            y = tokens(C, g, T)
            assert torch.equal(C.step(*y), E.step(*y))
    assert torch.equal(C.k_pages, E.k_pages) and torch.equal(C.v_scales, E.v_scales)
    assert qb.get_error() == 0


@pytest.mark.parametrize("rope", [True, False], ids=["rope", "plain"])
def test_a_refused_step_leaves_the_pages(rope):
    """A Q that attention refuses, beside K and V that would make the held pages' scales
    grow or end them: nothing of the step has reached the cache."""
    B, Hq, Hkv, d = 2, 4, 2, 64
    C, E = caches(2, B, Hq, Hkv, d, 128, rope=rope, out_dtype=qb.DT_F32)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = tokens(C, g, 40)
    for c in (C, E):
        c.step(*x, n_new=[40, 3])
    Q, K, V = tokens(C, g, 9, 50.0)
    V[1, 0, 2, 5] = float("inf")
    shifted = torch.empty(Q.numel() + 1, dtype=Q.dtype, device="cuda")[1:].view(Q.shape)  # two bytes off
    odd = torch.empty(B, Hq, 9, d + 1, dtype=Q.dtype, device="cuda")[..., :d]             # rows 130 bytes apart
    split = torch.empty(B, Hq, 9, 2 * d, dtype=Q.dtype, device="cuda")[..., ::2]          # channels apart
    for bad, error in ((Q.float(), TypeError), (Q[:, :3], ValueError), (Q[:1], ValueError), (Q[..., :32], ValueError),
                       (Q.cpu(), ValueError), (shifted, qb.QattnError), (odd, qb.QattnError), (split, qb.QattnError)):
        with pytest.raises(error):
            C.step(bad, K, V)
        for a, b in ((C.k_pages, E.k_pages), (C.v_pages, E.v_pages), (C.k_scales, E.k_scales), (C.v_scales, E.v_scales),
                     (C.page_table, E.page_table), (C.lengths, E.lengths), (C.n_new, E.n_new)):
            assert torch.equal(a, b)
        assert C.free_pages() == E.free_pages() and C.rows(0) == 40 and C.rows(1) == 3
    for side in (5, "side"):  # no stream
        with pytest.raises(AttributeError):
            C.step(Q, K, V, stream=side)
        assert C.free_pages() == E.free_pages() and C.rows(0) == 40 and torch.equal(C.n_new, E.n_new)
    V[1, 0, 2, 5] = 1.0
    assert torch.equal(C.step(Q, K, V), E.step(Q, K, V)) and torch.equal(C.k_pages, E.k_pages)
    assert qb.get_error() == 0


@pytest.mark.parametrize("rope", [True, False], ids=["rope", "plain"])
def test_parameters_that_attention_refuses(rope):
    """They are found before the tokens are entered."""
    for kw in (dict(sm_scale=-1.0), dict(sm_scale=float("nan")), dict(out_dtype=qb.DT_I8)):
        C, = caches(1, 1, 4, 2, 64, 64, rope=rope, **kw)
        x = tokens(C, torch.Generator(device="cuda").manual_seed(5), 3)
        with pytest.raises(qb.QattnError):
            C.step(*x)
        assert not C.k_pages.any() and not C.v_scales.any() and C.rows(0) == 0 and C.free_pages() == 3
