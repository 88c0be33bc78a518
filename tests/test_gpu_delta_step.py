"""The buffers of DeltaStep: what a call does not write."""
import pytest
import torch

from test_gpu_delta import D, _gen, _i32, _inputs

pytestmark = pytest.mark.gpu


def test_a_prompts_rows_that_are_not_written_are_zeros_or_an_earlier_calls():
    import speculative_decode_verify_append_gb300 as sdva
    from speculative_decode_verify_append_gb300.step import DeltaStep
    hk, hv, T = 1, 2, 60
    torch.use_deterministic_algorithms(True)  # memory that nothing has written holds NaN
    try:
        step = DeltaStep(3, hk, hv, max_tokens=T)
    finally:
        torch.use_deterministic_algorithms(False)
    x = _inputs(_gen(1), (T,), hk, hv)
    cu, seq = _i32([5, 25, 40, 50]), _i32([0, 0, 0])
    out = step.prompt(*x, cu, _i32([0, 9, 2]), seq)
    torch.cuda.synchronize()
    assert int(step.status.item()) == sdva.STATUS_BAD_PAGE
    assert (out[:5] == 0).all() and (out[25:40] == 0).all() and (out[50:] == 0).all()
    first = out.clone()
    assert first[5:25].any() and first[40:50].any()
    step.status.zero_()
    out = step.prompt(*x, _i32([0, 60, 55, 60]), _i32([0, 1, 2]), seq)  # offsets out of order
    torch.cuda.synchronize()
    assert int(step.status.item()) == sdva.STATUS_BAD_COUNT
    assert torch.equal(out, first)


def test_without_lengths_a_prompt_goes_on_from_its_slot():
    from speculative_decode_verify_append_gb300.step import DeltaStep
    hk, hv, n = 1, 2, 20
    step = DeltaStep(1, hk, hv, max_tokens=n)
    x = _inputs(_gen(2), (n,), hk, hv)
    cu, slot = _i32([0, n]), _i32([0])
    fresh = step.prompt(*x, cu, slot, _i32([0])).clone()
    state = step.state.clone()
    assert torch.equal(step.prompt(*x, cu, slot, _i32([0])), fresh) and torch.equal(step.state, state)
    on = step.prompt(*x, cu, slot).clone()
    assert not torch.equal(on, fresh)
    step.state.copy_(state)
    assert torch.equal(step.prompt(*x, cu, slot, _i32([7])), on)
