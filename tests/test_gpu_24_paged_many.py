"""qattn_paged_fwd where its list of work is long: more row blocks of a KV head, and more
sequences of several blocks, than a warp has lanes."""
import pytest

from quantized_attention_gb300 import binding as qb
from tests.gpu_common import ensure_library
from tests.test_gpu_21_paged import check, make
from tests.test_gpu_22_paged_edges import run_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_library()


def spread(lo, hi, B):
    """B whole numbers from lo to hi in no order."""
    return [lo + (hi - lo) * ((7 * b) % B) // max(B - 1, 1) for b in range(B)]


MANY = [
    # B, Hq, Hkv, d, page, code, T, lengths, n_new; blocks of 256 rows
    (1, 8, 1, 64, 64, "int8", 1040, [1040], None),                       # 33 blocks: a whole prompt
    (2, 16, 1, 128, 64, "e4m3", 1030, [1030, 1111], [1030, 1027]),       # 65 blocks
    (1, 16, 2, 128, 128, "int8", 1030, [2200], [1025]),                   # 33 blocks of each of two KV heads
    (3, 16, 1, 64, 32, "e4m3", 1100, [1100, 600, 900], [513, 600, 511]), # 33, 38 and 32 blocks
    # more than 32 sequences of several blocks: 2 of 256 rows; 2, 3 and 4 of 16 rows
    (40, 16, 1, 64, 32, "int8", 20, spread(20, 700, 40), spread(0, 20, 40)),
    (70, 8, 1, 128, 64, "e4m3", 40, spread(0, 300, 70), [min(n, L) for n, L in zip(spread(0, 40, 70), spread(0, 300, 70))]),
    (33, 2, 1, 128, 64, "int8", 16, spread(16, 600, 33), None),
    (45, 6, 2, 64, 32, "e4m3", 15, spread(15, 500, 45), spread(0, 15, 45)),
    (65, 4, 1, 64, 128, "int8", 16, spread(0, 400, 65), [min(16, L) for L in spread(0, 400, 65)]),
]


@pytest.mark.parametrize("shape", MANY, ids=[f"{s[5]}-B{s[0]}-H{s[1]}-{s[2]}-d{s[3]}-T{s[6]}" for s in MANY])
@pytest.mark.parametrize("bound", [0, 2048, 1 << 19], ids=["exact", "middling", "long"])
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "all"])
def test_more_blocks_and_sequences_than_lanes(shape, bound, causal):
    P = make(51, *shape)
    O, lse = run_bound(P, max(bound, max(shape[7])), causal)
    assert qb.get_error() == 0
    check(P, O, lse, causal)
