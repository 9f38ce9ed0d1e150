"""What the training binding refuses before it looks for a GPU."""

import pytest

import dense_fp32_gemm_sgemm_gb300 as sg

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("steps", [2.5, 5.0, "5", None])
def test_steps_that_are_not_whole_numbers(steps):
    """2.5 is not two steps."""
    with pytest.raises(TypeError):
        sg.orthogonalize(torch.zeros(4, 8), steps=steps)


def test_a_stack_whose_rows_alternate():
    """The matrices of a transposed stack do not overlap, but lie within one another; the message says what
    is asked for."""
    from dense_fp32_gemm_sgemm_gb300.training import _layout
    t = torch.zeros(6, 3, 8)
    assert _layout(t, "G") == (6, 3, 8, 8, 24)
    with pytest.raises(ValueError, match="begin behind the last element of the one before"):
        _layout(t.transpose(0, 1), "G")
    assert _layout(t[:1].transpose(0, 1)[:1], "G") == (1, 1, 8, 24, 0)  # the pitch of one row counts for nothing
