"""Forms of qkmla_prefill's queries: both are read by their strides, so that neither may come in another form."""
import pytest
import torch

import qk_normed_latent_gb300 as Q


def zeros(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def call(q, q_rope):
    I32, BF16 = torch.int32, torch.bfloat16
    weights = Q.PrefillWeights(zeros(16, dtype=torch.uint8), 4, 4, 256, 64, 64)
    return Q.prepare_prefill(q, q_rope, zeros(64), zeros(64), zeros(32), weights, zeros(64, 288, dtype=BF16), zeros(64, 4),
                             zeros(3, dtype=I32), zeros(2, dtype=I32), zeros(2, 3, dtype=I32), 16, 3, 60, 0.1, 1e-6,
                             zeros(8, 16, 64, dtype=BF16))


@pytest.mark.parametrize("shape", [(2, 4, 16, 32), (8, 512), (8, 32, 16), (16, 8, 32), (1, 8, 16, 32), (8, 16, 1, 32)])
def test_rope_queries_have_the_queries_form(shape):
    """As many elements as [rows, H, d_r], laid out otherwise (decode takes [B, s_q, H, d_r])."""
    with pytest.raises(ValueError, match="q_rope"):
        call(zeros(8, 16, 64), zeros(*shape))


@pytest.mark.parametrize("shape", [(2, 4, 16, 64), (8, 1024)])
def test_queries_have_three_dimensions(shape):
    with pytest.raises(ValueError, match="q is"):
        call(zeros(*shape), zeros(8, 16, 32))


def test_no_rows_have_no_strides():
    """A tensor without elements may carry any strides (numpy's do): a step without rows is no error."""
    for empty in (torch.empty_strided((0, 16, 64), (0, 0, 0)), torch.empty_strided((0, 16, 64), (1024, 2, 2))):
        with pytest.raises(ValueError, match="CUDA device"):               # what any tensor of the CPU meets
            Q._inner("q", empty)
