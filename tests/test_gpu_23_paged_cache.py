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
