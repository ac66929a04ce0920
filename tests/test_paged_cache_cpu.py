"""Host checks of PagedCache and of what it refuses before anything is launched.  No
GPU needed."""
import os

import pytest
import torch

from quantized_attention_gb300 import binding as qb
from quantized_attention_gb300 import build
from quantized_attention_gb300.pipeline import PagedCache


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not os.path.exists(qb.library_path()):
        build.build()
    qb.lib()


def test_a_grow_that_fails_changes_nothing(monkeypatch):
    """Pages, lengths and counts as they were, on the host too, when the copy to the device
    does not come about."""
    C = PagedCache(12, 32, 4, 2, 64, 2, 128, device="cpu")
    C.grow([40, 3])
    before = C._host.clone()

    def fail(stream):
        raise RuntimeError("no copy")

    with monkeypatch.context() as m:
        m.setattr(C, "_upload", fail)
        with pytest.raises(RuntimeError, match="no copy"):
            C.grow([30, 40])
    assert torch.equal(C._host, before) and C.free_pages() == 9 and C.rows(0) == 40
    C.grow([30, 40])
    assert C.page_table[0].tolist() == [0, 1, 3, -1] and C.page_table[1].tolist() == [2, 4, -1, -1]


def test_inputs_and_parameters_are_refused_before_a_launch(monkeypatch):
    """What attention would refuse, found without it (Q on the device is a device matter)."""
    shape, g = qb.make_shape(2, 8, 2, 4, 200, 128), qb.make_paging(10, 64, 4)
    qb.paged_params(shape, qb.make_params(causal=True), g)
    for p in (qb.make_params(sm_scale=-1.0), qb.make_params(sm_scale=float("nan")), qb.make_params(out_dtype=qb.DT_I8)):
        with pytest.raises(qb.QattnError):
            qb.paged_params(shape, p, g)
    with pytest.raises(qb.QattnError):
        qb.paged_params(shape, qb.make_params(), qb.make_paging(10, 48, 4))
    x = torch.zeros(2, 8, 8, 64, dtype=torch.bfloat16)
    dims = (2, 8, 4, 64)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)  # (what get_device gives of the CPU)
    for good in (x[:, :, :4], x[:, :, ::2], x.transpose(1, 2)[:, :, :4], x[:, :1, :4].expand(2, 8, 4, 64)):
        qb.paged_input("Q", good, dims)
    flat = torch.zeros(2 * 8 * 4 * 64 + 8, dtype=torch.bfloat16)
    for bad in (flat[1:].narrow(0, 0, 4096).view(dims), torch.zeros(2, 8, 4, 65, dtype=torch.bfloat16)[..., :64],
                torch.zeros(2, 8, 4, 128, dtype=torch.bfloat16)[..., ::2]):
        with pytest.raises(qb.QattnError, match="Q"):
            qb.paged_input("Q", bad, dims)
    for bad, error in ((None, ValueError), (x, ValueError), (x[:, :, :4].float(), TypeError)):
        with pytest.raises(error):
            qb.paged_input("Q", bad, dims)
