"""Rotary positions at their edges: calls that the first tests do not make."""
import pytest
import torch

from tests.test_rope_gpu import _close, _inputs, _turn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def da():
    import differential_attention_v2_b200 as m

    assert torch.cuda.is_available()
    return m


def test_an_output_without_its_input_is_refused(da):
    q, k, pos, inv = (t.cuda() for t in _inputs(4, 2, 1, 64, (16, 16), torch.bfloat16, seed=1))
    out = torch.full_like(k, 3.0)
    with pytest.raises(ValueError):
        da.rope(q, None, pos, inv, (16, 16), k_out=out)
    torch.cuda.synchronize()
    assert out.eq(3.0).all()
    assert da.rope(q, None, pos, inv, (16, 16))[1] is None
