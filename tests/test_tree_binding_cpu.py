"""Missing tensors are named by the binding of the serving operators.  No GPU needed."""
import pytest
import torch

from quantized_attention_gb300 import binding as qb

T4 = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)


@pytest.mark.parametrize("K_new,k_codes,name", [(None, T4, "K_new"), (T4, None, "k_codes")])
def test_commit_names_what_is_missing(K_new, k_codes, name):
    with pytest.raises(ValueError, match=f"{name} is missing"):
        qb.tree_commit(K_new, T4, *[None] * 7, k_codes, None)


@pytest.mark.parametrize("k_codes,k_out,name", [(None, T4, "k_codes"), (T4, None, "k_out")])
def test_evict_names_what_is_missing(k_codes, k_out, name):
    with pytest.raises(ValueError, match=f"{name} is missing"):
        qb.kv_evict(k_codes, None, None, 1, k_out, *[None] * 5)


def test_scales_and_inputs_name_what_is_missing():
    with pytest.raises(ValueError, match="q_scales is missing"):
        qb._scales_ptr(0, "q_scales", None, qb.GRAN_HEAD, 1, 2, 3)
    with pytest.raises(ValueError, match="V_new is missing"):
        qb._input_ptr(0, "V_new", None, (1, 2, 3, 64))
