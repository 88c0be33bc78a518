"""Calls whose waits run out late: a warp gives up while the one that copies
has issued its last copy and is done.  No copy may outlive its block, whose
shared memory the next block gets: what runs beside and after is right."""
import numpy as np
import pytest
import torch

import oracle
import synth
from gpu_util import ALL_KV, KV_NAMES, SM_SCALE, assert_close, bf16_dev, fill_both, i32_dev
from test_gpu_prompt import _cu, _gen, _logits, _run_attn, _score, _status

pytestmark = pytest.mark.gpu


def _without_patience(run, beside):
    """run() with a limit of zero cycles, beside() on another stream meanwhile."""
    import speculative_decode_verify_append_gb300 as sdva
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    prev = sdva.sdva_debug_set_wait_limit(0)
    try:
        run()
        with torch.cuda.stream(other):
            got = beside()
        torch.cuda.synchronize()
    finally:
        sdva.sdva_debug_set_wait_limit(prev)
    return got


def _scores_beside():
    """Short rows: small blocks, no waits, in the shared memory that others leave."""
    import speculative_decode_verify_append_gb300 as sdva
    g = _gen(3)
    x = _logits(g, 4000, 5000, torch.float32)
    tokens = torch.randint(5000, (4000,), generator=g, device="cuda", dtype=torch.int32)
    want = _score(x, tokens, 5)
    got = [torch.zeros_like(t) for t in want]

    def beside():
        for _ in range(4):
            sdva.token_logprobs(x, tokens, *got)
        return got
    return want, beside


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sums_that_wait_for_a_long_list(dtype):
    """A NaN and rising values: the list of a row is looked for element by
    element, some hundred microseconds, in which the sums of the rows behind it
    wait for their place and the copies are all issued."""
    g = _gen(1)
    n, V = 1600, 34000
    x = (torch.arange(V, device="cuda") * 1e-3).expand(n, V).to(dtype).contiguous()
    x[:, 100] = float("nan")
    tokens = torch.randint(V, (n,), generator=g, device="cuda", dtype=torch.int32)
    want, beside = _scores_beside()
    st = _status()
    import speculative_decode_verify_append_gb300 as sdva
    out = [torch.empty(n, device="cuda"), torch.empty(n, device="cuda"),
           torch.empty((n, 32), dtype=torch.int32, device="cuda"), torch.empty((n, 32), device="cuda")]
    got = _without_patience(lambda: sdva.token_logprobs(x, tokens, *out, st), beside)
    assert int(st.item()) in (0, sdva.STATUS_TIMEOUT)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # the same call with its usual patience
    st.zero_()
    lp, _, tt, _ = _score(x, tokens, 32, st)
    assert int(st.item()) == 0 and lp.isnan().all()
    xd = x[0].float()
    order = torch.argsort(torch.where(xd.isnan(), float("-inf"), xd), descending=True, stable=True)[:32]
    assert (tt == order.to(torch.int32)).all()


@pytest.mark.parametrize("lens,hq,hkv", [([256] * 400, 1, 1), ([42] * 500, 24, 4), ([128] * 150, 1, 1)])
def test_products_that_wait_for_rows_of_infinities(lens, hq, hkv):
    """Infinities in every row of V: what the guard took out is added again from
    global memory, some hundred microseconds a tile, in which the next tile's
    products wait for their place and the few copies of it are all issued."""
    import speculative_decode_verify_append_gb300 as sdva
    T = sum(lens)
    g = _gen(5)
    q, k, v = (torch.randn((T, h, 128), generator=g, device="cuda").to(torch.bfloat16) for h in (hq, hkv, hkv))
    cu = _cu(lens)
    inf = torch.full_like(v, float("inf"))
    want, beside = _scores_beside()
    good = _run_attn(q, k, v, cu)
    st = _status()
    out = torch.empty_like(q)
    got = _without_patience(lambda: sdva.prompt_attn(q, k, inf, cu, float(SM_SCALE), out, None, st), beside)
    assert int(st.item()) in (0, sdva.STATUS_TIMEOUT)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # the same call with its usual patience, and one with finite values
    st.zero_()
    out, lse = _run_attn(q, k, inf, cu, status=st)
    assert int(st.item()) == 0 and torch.equal(lse, good[1]) and (out == float("inf")).all()
    out, lse = _run_attn(q, k, v, cu, status=st)
    assert int(st.item()) == 0 and torch.equal(out, good[0]) and torch.equal(lse, good[1])


@pytest.mark.parametrize("kind", ALL_KV, ids=[KV_NAMES[k] for k in ALL_KV])
def test_a_window_over_few_pages(kind):
    """verify_attn with no more pages to a CTA than it has stages: the producer
    is done at once, with all its copies in flight, and the others give up."""
    import speculative_decode_verify_append_gb300 as sdva
    lens, W, hq, hkv = [900] * 6, 4, 12, 2
    spec = synth.Spec("late", 72, len(lens), 0, 0, hq, hkv, W, kind, None, 0.7, True)
    step = synth.make_step(spec, seq_lens=np.array(lens, np.int32), with_accept=False)
    gc, oc, _ = fill_both(spec, step)
    q, t, L = bf16_dev(step.q), i32_dev(step.page_table), i32_dev(step.seq_lens)
    ws = torch.empty(sdva.verify_attn_workspace_size(len(lens), W, hq, hkv, max(lens)), dtype=torch.uint8,
                     device="cuda")
    out = torch.zeros((len(lens), W, hq, 128), dtype=torch.bfloat16, device="cuda")
    st = _status()
    want, beside = _scores_beside()

    def run():
        for _ in range(8):
            sdva.verify_attn(gc, q, t, L, max(lens), float(SM_SCALE), out, ws, st)

    got = _without_patience(run, beside)
    assert int(st.item()) == sdva.STATUS_TIMEOUT
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    st.zero_()
    sdva.verify_attn(gc, q, t, L, max(lens), float(SM_SCALE), out, ws, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    ref, _ = oracle.verify_attn(oc, step.q, step.page_table, step.seq_lens, SM_SCALE, threads=16)
    assert_close(out.float().cpu().numpy(), ref, "after the calls that gave up")
