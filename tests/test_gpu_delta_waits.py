"""The waits of prompt_delta and verify_delta that run out, without a fault: with
a limit of zero cycles a wait for copies that are not there yet gives up.  The
call says so and returns, each CTA's part of a state is what it was or what the
call makes of it, and the next call is right."""
import pytest
import torch

from test_gpu_delta import D, SCALE, _gen, _i32, _inputs, _status, _workspace

pytestmark = pytest.mark.gpu


def _impatient(call):
    import speculative_decode_verify_append_gb300 as sdva
    prev = sdva.sdva_debug_set_wait_limit(0)
    try:
        call()
        torch.cuda.synchronize()
    finally:
        sdva.sdva_debug_set_wait_limit(prev)


def _parts_kept(state, before, after, rows):
    """Every part of `rows` value rows is one or the other; how many are what they were."""
    x, b, a = (y.reshape(-1, rows * D) for y in (state, before, after))
    kept, moved = (x == b).all(1), (x == a).all(1)
    assert (kept | moved).all()
    return int((kept & ~moved).sum())


@pytest.mark.parametrize("lens,hk,hv", [([40], 1, 2), ([700, 1, 0, 64, 333], 2, 4), ([600] * 12, 4, 16)])
def test_a_prompt_that_gives_up_keeps_its_state(lens, hk, hv):
    import speculative_decode_verify_append_gb300 as sdva
    B, T = len(lens), sum(lens)
    g = _gen(1)
    x = _inputs(g, (T,), hk, hv)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    before = torch.randn((B, hv, D, D), generator=g, device="cuda")

    def run(state, out, st):
        sdva.prompt_delta(state, *x, _i32(cu), _i32(range(B)), SCALE, out, _workspace(T, B, hk, hv), status=st)

    good, out, st = before.clone(), torch.empty((T, hv, D), dtype=torch.bfloat16, device="cuda"), _status()
    run(good, out, st)
    assert int(st.item()) == 0
    state, other = before.clone(), torch.empty_like(out)
    _impatient(lambda: run(state, other, st))
    assert int(st.item()) == sdva.STATUS_TIMEOUT
    assert _parts_kept(state, before, good, 32) > 0
    st.zero_()
    state.copy_(before)
    run(state, other, st)
    assert int(st.item()) == 0 and torch.equal(state, good) and torch.equal(other, out)


@pytest.mark.parametrize("W", [4, 16])
@pytest.mark.parametrize("keep", [True, False])
def test_a_window_that_gives_up_keeps_its_state(W, keep):
    import speculative_decode_verify_append_gb300 as sdva
    B, hk, hv = 64, 8, 16
    g = _gen(2)
    x = _inputs(g, (B, W), hk, hv)
    before = torch.randn((B, hv, D, D), generator=g, device="cuda")

    def run(state, out, deltas, st):
        sdva.verify_delta(state, *x, _i32(range(B)), SCALE, out, deltas, status=st)

    def buffers():
        return (before.clone(), torch.empty((B, W, hv, D), dtype=torch.bfloat16, device="cuda"),
                torch.empty((B, W, hv, D), device="cuda") if keep else None)

    good, out, deltas = buffers()
    st = _status()
    run(good, out, deltas, st)
    assert int(st.item()) == 0
    state, o, d = buffers()
    _impatient(lambda: run(state, o, d, st))
    assert int(st.item()) == sdva.STATUS_TIMEOUT
    if keep:
        assert torch.equal(state, before)
    else:
        assert _parts_kept(state, before, good, D) > 0
    st.zero_()
    state.copy_(before)
    run(state, o, d, st)
    assert int(st.item()) == 0 and torch.equal(state, good) and torch.equal(o, out)
    assert d is None or torch.equal(d, deltas)


def test_a_tree_with_a_bad_parent_that_gives_up():
    """The lane is skipped; its copies are waited for all the same."""
    import speculative_decode_verify_append_gb300 as sdva
    B, W, hk, hv = 32, 5, 2, 4
    g = _gen(3)
    x = _inputs(g, (B, W), hk, hv)
    state = torch.randn((B, hv, D, D), generator=g, device="cuda")
    before, st = state.clone(), _status()
    out = torch.full((B, W, hv, D), 7.0, dtype=torch.bfloat16, device="cuda")
    deltas = torch.full((B, W, hv, D), 7.0, device="cuda")
    parent = _i32([[0, 0, 1, 3, 0]] * B)
    _impatient(lambda: sdva.verify_delta(state, *x, _i32(range(B)), SCALE, out, deltas, parent=parent, status=st))
    assert int(st.item()) == sdva.STATUS_BAD_TREE
    assert torch.equal(state, before) and (out == 0).all() and (deltas == 0).all()
