"""The rotated appends and the gated delta rule as a hybrid model's layers use
them together, and at offsets past 32 bits."""
import numpy as np
import pytest
import torch

from test_gpu_delta import D, SCALE, _check_lane, _check_out, _gen, _i32, _inputs, _norm_near, _status, _tol, _walk, _workspace
from test_gpu_rope import _same, _turn

pytestmark = pytest.mark.gpu
HQ, HKV, HK, HV = 6, 2, 2, 4


def _qkv(g, lead):
    x = torch.randn((*lead, HQ + 2 * HKV, D), generator=g, device="cuda").to(torch.bfloat16)
    return x.split([HQ, HKV, HKV], -2)


@pytest.mark.parametrize("fmt", [0, 1, 2, 3])
def test_an_attention_layer_and_a_recurrent_one_through_prompts_and_verify_steps(fmt):
    """Prompts, then verify steps that accept a part of their drafts: the attention
    layer does bit for bit what it does with keys and queries turned before the
    call, and the recurrent one follows the accepted tokens."""
    import speculative_decode_verify_append_gb300 as sdva
    from speculative_decode_verify_append_gb300.step import DeltaStep, PromptStep, VerifyStep, rope_table
    g = _gen(fmt)
    lens, B, W, V = [70, 5, 130], 3, 5, 40
    T = sum(lens)
    cu, seq = _i32(np.concatenate([[0], np.cumsum(lens)])), _i32([0, 0, 0])
    table = _i32(np.arange(12).reshape(3, 4))
    rope = rope_table(300, 64)
    caches = [sdva.KVCache(fmt, 12, HKV) for _ in range(2)]
    prompts = [PromptStep(T, HQ, num_kv_heads=HKV), PromptStep(T, HQ)]
    q, k, v = _qkv(g, (T,))
    pos = torch.cat([torch.arange(n) for n in lens]).cuda()
    out, lse = prompts[0].run(caches[0], q, k, v, cu, table, seq, rope=rope)
    out1, lse1 = prompts[1].run(caches[1], _turn(q, rope, pos, False), _turn(k, rope, pos, False), v, cu, table, seq)
    torch.cuda.synchronize()
    assert torch.equal(out, out1) and torch.equal(lse, lse1)
    with pytest.raises(ValueError, match="num_kv_heads"):
        prompts[1].run(caches[1], q, k, v, cu, table, seq, rope=rope)
    _same(*caches)

    delta = DeltaStep(B, HK, HV, window=W, max_tokens=T)
    x = _inputs(g, (T,), HK, HV, fused=True)
    slots = _i32([1, 2, 0])
    delta.prompt(*x, cu, slots, seq)
    hist = [[[y[int(cu[b]):int(cu[b + 1])] for y in x]] for b in range(B)]
    seq = _i32(lens)
    steps = [VerifyStep(B, W, HQ, HKV, 200, V) for _ in range(2)]
    for step in range(3):
        q, k, v = _qkv(g, (B, W))
        pos = seq.long()[:, None] + torch.arange(W, device="cuda")
        turned = steps[0].append_rope(caches[0], q, k, v, rope, table, seq)
        steps[0].attend(caches[0], turned, table, seq)
        steps[1].append(caches[1], _turn(k, rope, pos, False), v.contiguous(), table, seq)
        steps[1].attend(caches[1], _turn(q, rope, pos, False), table, seq)
        torch.cuda.synchronize()
        assert torch.equal(steps[0].out, steps[1].out)
        _same(*caches)
        x = _inputs(g, (B, W), HK, HV, fused=True)
        out = delta.verify(*x, slots).clone()
        # a target that agrees with some of the drafts
        drafts = torch.randint(V, (B, W - 1), generator=g, device="cuda", dtype=torch.int32)
        logits = torch.randn((B, W, V), generator=g, device="cuda")
        for b in range(B):
            for i in range((step + b) % W):
                logits[b, i, int(drafts[b, i])] += 30.0
        steps[0].accept(logits, drafts, seq)
        delta.commit(x[1], x[3], slots, steps[0].accept_len)
        for b in range(B):
            head = [torch.cat([h[j] for h in hist[b]] + [x[j][b]]) for j in range(5)]
            zero = torch.zeros((HV, D, D), device="cuda")
            wo, _, _, M = _walk(zero, *head)
            _check_out(out[b], wo[-W:], head[0].shape[0], M, ("window", step, b))
            n = int(steps[0].accept_len[b]) + 1
            hist[b].append([y[b, :n] for y in x])
    for b in range(B):
        rows = [torch.cat([h[j] for h in hist[b]]) for j in range(5)]
        _, _, ws, M = _walk(torch.zeros((HV, D, D), device="cuda"), *rows)
        _norm_near(delta.state[int(slots[b])], ws[-1], _tol(rows[0].shape[0], M[0]), "state")
    assert int(steps[0].status.item()) == int(delta.status.item()) == int(prompts[0].status.item()) == 0
    assert int(seq[0]) > lens[0]


def test_a_draft_tree_through_both_layers():
    """Positions by depth in the attention layer, parents in the recurrent one."""
    import speculative_decode_verify_append_gb300 as sdva
    from speculative_decode_verify_append_gb300.step import VerifyStep, rope_table
    g = _gen(9)
    B, W = 2, 6
    parent, depth = [[-1, 0, 0, 1, 1, 4]] * B, [[0, 1, 1, 2, 2, 3]] * B
    lens = [60, 3]
    seq, table, rope = _i32(lens), _i32([[0, 1], [2, 3]]), rope_table(100, 128)
    pos = seq[:, None] + _i32(depth)
    caches = [sdva.KVCache(2, 4, HKV) for _ in range(2)]
    for c in caches:
        k0, v0 = (torch.randn((B, 60, HKV, D), generator=_gen(1), device="cuda").bfloat16() for _ in range(2))
        sdva.kv_append_quant_ragged(c, k0, v0, seq, table, _i32([0, 0]))
    q, k, v = _qkv(g, (B, W))
    step = VerifyStep(B, W, HQ, HKV, 100, None)
    turned = step.append_rope(caches[0], q, k, v, rope, table, seq, positions=pos)
    sdva.kv_append_quant(caches[1], _turn(k, rope, pos, False), v.contiguous(), table, seq)
    torch.cuda.synchronize()
    _same(*caches)
    assert torch.equal(turned, _turn(q, rope, pos, False))
    outs = [torch.empty_like(turned) for _ in range(2)]
    for c, o in zip(caches, outs):
        sdva.verify_attn_tree(c, turned, _i32(parent), table, seq, 100, SCALE, o, step.workspace)
    torch.cuda.synchronize()
    assert torch.equal(*outs)


def test_states_past_32_bit_offsets():
    """A pool of more than 2^31 values: the last slots hold what the first ones would."""
    import speculative_decode_verify_append_gb300 as sdva
    g = _gen(2)
    slots, hk, hv = 2 ** 31 // (16 * D * D) + 3, 8, 16
    state = torch.zeros((slots, hv, D, D), device="cuda")
    assert state.numel() > 2 ** 31
    last = _i32([slots - 1, slots - 2])
    first = torch.randn((2, hv, D, D), generator=g, device="cuda")
    small, idx = first.clone(), _i32([1, 0])
    state[slots - 2:] = first
    x = _inputs(g, (2, 5), hk, hv)
    p = _inputs(g, (60,), hk, hv)
    for keep in (True, False):
        res = []
        for s, i in ((state, last), (small, idx)):
            out, d = torch.empty((2, 5, hv, D), dtype=torch.bfloat16, device="cuda"), torch.empty((2, 5, hv, D), device="cuda")
            sdva.verify_delta(s, *x, i, SCALE, out, d if keep else None)
            if keep:
                sdva.commit_delta(s, x[1], x[3], d, i, _i32([2, 4]))
            po = torch.empty((60, hv, D), dtype=torch.bfloat16, device="cuda")
            sdva.prompt_delta(s, *p, _i32([0, 33, 60]), i, SCALE, po, _workspace(60, 2, hk, hv))
            torch.cuda.synchronize()
            res.append((out, po))
        assert all(torch.equal(a, b) for a, b in zip(*res))
        assert torch.equal(state[slots - 2:], small)
    assert not state[:slots - 2].any()


def _far(g, rows, width, stride):
    """rows of `width` values, `stride` apart, over more than 2^31 values."""
    buf = torch.empty(rows * stride, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((rows, width), (stride, 1))
    x.copy_(torch.randn((rows, width), generator=g, device="cuda"))
    return x


def test_rows_past_32_bit_offsets():
    import speculative_decode_verify_append_gb300 as sdva
    from speculative_decode_verify_append_gb300.step import rope_table
    g = _gen(3)
    B, W, hk, hv = 10, 16, 1, 2
    rows, stride = B * W, 2 ** 31 // (B * W - 1) // 8 * 8 + 4096
    x = _far(g, rows, (2 * hk + hv) * D, stride)
    assert (rows - 1) * stride > 2 ** 31
    q, k, v = x.unflatten(1, (2 * hk + hv, D)).split([hk, hk, hv], 1)
    gd, b = -torch.rand((rows, hv), generator=g, device="cuda"), torch.rand((rows, hv), generator=g, device="cuda")
    cu, slots = _i32(np.arange(0, rows + 1, W)), _i32(range(B))
    start = torch.randn((B, hv, D, D), generator=g, device="cuda")

    def window(t):
        return t.as_strided((B, W, *t.shape[1:]), (W * t.stride(0), *t.stride()))

    def calls(q, k, v):
        s1, s2 = start.clone(), start.clone()
        o1 = torch.empty((rows, hv, D), dtype=torch.bfloat16, device="cuda")
        o2, d = torch.empty((B, W, hv, D), dtype=torch.bfloat16, device="cuda"), torch.empty((B, W, hv, D), device="cuda")
        sdva.prompt_delta(s1, q, k, v, gd, b, cu, slots, SCALE, o1, _workspace(rows, B, hk, hv))
        sdva.verify_delta(s2, *(window(t) for t in (q, k, v)), window(gd), window(b), slots, SCALE, o2, d)
        sdva.commit_delta(s2, window(k), window(gd), d, slots, _i32([W - 1] * B))
        cache = sdva.KVCache(3, B, hk)
        rope, qo, ko = rope_table(W, 128), torch.empty((rows, hv, D), dtype=torch.bfloat16, device="cuda"), torch.empty((rows, hk, D), dtype=torch.bfloat16, device="cuda")
        sdva.kv_append_packed_rope(cache, v, k, q, cu, rope, _i32(range(B)).view(B, 1), _i32([0] * B), qo, ko)
        other = sdva.KVCache(3, B, hk)
        qo2 = torch.empty((B, W, hv, D), dtype=torch.bfloat16, device="cuda")
        sdva.kv_append_rope(other, window(v), window(k), window(q), rope, _i32(range(B)).view(B, 1), _i32([0] * B), qo2)
        torch.cuda.synchronize()
        return [s1, s2, o1, o2, d, qo, ko, qo2, cache.k_codes, cache.v_codes, cache.k_scales, other.k_codes, other.v_codes]

    far = calls(q, k, v)
    near = calls(*(t.contiguous() for t in (q, k, v)))
    for a, c in zip(far, near):
        assert torch.equal(a, c)


def test_pages_past_32_bit_offsets():
    import speculative_decode_verify_append_gb300 as sdva
    from speculative_decode_verify_append_gb300.step import rope_table
    g = _gen(4)
    hkv = 8
    pages = 2 ** 31 // (hkv * 64 * D) + 2
    q, k, v = torch.randn((1, 10, 8 + 2 * hkv, D), generator=g, device="cuda").bfloat16().split([8, hkv, hkv], 2)
    rope = rope_table(80, 64)
    far, near = sdva.KVCache(0, pages, hkv), sdva.KVCache(0, 2, hkv)
    assert far.k_codes.numel() > 2 ** 31
    for c, ids in ((far, [pages - 1, pages - 2]), (near, [1, 0])):
        sdva.kv_append_rope(c, q, k, v, rope, _i32([ids]), _i32([60]), torch.empty((1, 10, 8, D), dtype=torch.bfloat16, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(far.k_codes[-2:], near.k_codes) and torch.equal(far.v_codes[-2:], near.v_codes)
    assert torch.equal(far.k_scales[-2:], near.k_scales) and not far.k_scales[:-2].any()


def test_lanes_that_share_a_state_without_writing_it():
    import speculative_decode_verify_append_gb300 as sdva
    g = _gen(5)
    for W in (2, 9):
        x = _inputs(g, (4, W), 1, 2)
        state = torch.randn((2, 2, D, D), generator=g, device="cuda")
        out, d = torch.empty((4, W, 2, D), dtype=torch.bfloat16, device="cuda"), torch.empty((4, W, 2, D), device="cuda")
        sdva.verify_delta(state, *x, _i32([1, 1, 0, 1]), SCALE, out, d)
        for i, s in enumerate((1, 1, 0, 1)):
            _check_lane(W, state[s], out[i], d[i], None, *(y[i] for y in x))


def test_rows_of_no_lane():
    """Offsets that leave every lane empty, and calls of no rows."""
    import speculative_decode_verify_append_gb300 as sdva
    g = _gen(6)
    q, k, v, gd, b = _inputs(g, (40,), 1, 2)
    state = torch.randn((3, 2, D, D), generator=g, device="cuda")
    before, out, st = state.clone(), torch.full((40, 2, D), 7.0, dtype=torch.bfloat16, device="cuda"), _status()
    for cu in ([0, 0, 0, 0], [40, 40, 40, 40], [13, 13, 13, 13]):
        sdva.prompt_delta(state, q, k, v, gd, b, _i32(cu), _i32([0, 1, 2]), SCALE, out, _workspace(40, 3, 1, 2), status=st)
    empty = [t[:0] for t in (q, k, v, gd, b)]
    sdva.prompt_delta(state, *empty, _i32([0, 0]), _i32([0]), SCALE, out[:0], torch.empty(0, dtype=torch.uint8, device="cuda"), status=st)
    n = torch.zeros(2, dtype=torch.int32, device="cuda")
    w = [t[:8].unflatten(0, (2, 4)) for t in (q, k, v, gd, b)]
    o, d = torch.full((2, 4, 2, D), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((2, 4, 2, D), 7.0, device="cuda")
    sdva.verify_delta(state, *w, _i32([-5, 99]), SCALE, o, d, n, status=st)  # a lane without rows has no slot to check
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and torch.equal(state, before) and (out == 7.0).all() and (o == 0).all() and (d == 0).all()


@pytest.mark.parametrize("hk,hv", [(1, 16), (1, 7), (3, 27)])
def test_many_value_heads_of_a_key_head(hk, hv):
    import speculative_decode_verify_append_gb300 as sdva
    g = _gen(hv)
    x = _inputs(g, (70,), hk, hv, fused=True)
    state = torch.randn((1, hv, D, D), generator=g, device="cuda")
    before, out = state.clone(), torch.empty((70, hv, D), dtype=torch.bfloat16, device="cuda")
    sdva.prompt_delta(state, *x, _i32([0, 70]), _i32([0]), SCALE, out, _workspace(70, 1, hk, hv))
    _check_lane(70, before[0], out, None, state[0], *x)


@pytest.mark.parametrize("lanes", [1, 2, 3, 5, 40, 129])
def test_prompt_shapes_of_grids(lanes):
    """Grids of one, of several and of many rounds of the GPU's SMs (32 heads), with lanes longer and shorter than the
    length at which the shape changes."""
    import speculative_decode_verify_append_gb300 as sdva
    g = _gen(lanes)
    hk, hv = 16, 32
    for long in (True, False):
        lens = [(300 if long else 40) + 7 * (i % 5) for i in range(lanes)] if lanes < 40 else [(270 if long and lanes == 40 else 33)] * lanes
        T = sum(lens)
        x = _inputs(g, (T,), hk, hv)
        state = torch.zeros((lanes, hv, D, D), device="cuda")
        out = torch.empty((T, hv, D), dtype=torch.bfloat16, device="cuda")
        cu = np.concatenate([[0], np.cumsum(lens)])
        sdva.prompt_delta(state, *x, _i32(cu), _i32(range(lanes)), SCALE, out, _workspace(T, lanes, hk, hv))
        for i in sorted({0, lanes // 2, lanes - 1}):
            a, n = int(cu[i]), lens[i]
            h = slice(4, 8)  # of key heads 2 and 3
            _check_lane(n, torch.zeros((4, D, D), device="cuda"), out[a:a + n, h], None, state[i, h],
                        *(y[a:a + n, 2:4] for y in x[:2]), *(y[a:a + n, h] for y in x[2:]))


def test_a_prompt_lane_that_is_skipped_leaves_the_others_right():
    """Of a batch with a bad page in one lane, the status says so and the other lanes' attention is theirs alone."""
    import speculative_decode_verify_append_gb300 as sdva
    from speculative_decode_verify_append_gb300.step import PromptStep, rope_table
    g = torch.Generator(device="cuda").manual_seed(31)
    hq, hkv, lens = 4, 2, [70, 40, 33]
    T = sum(lens)
    q, k, v = (torch.randn((T, h, 128), generator=g, device="cuda").bfloat16() for h in (hq, hkv, hkv))
    cu = torch.tensor([0, 70, 110, 143], dtype=torch.int32, device="cuda")
    zeros = torch.zeros(3, dtype=torch.int32, device="cuda")
    rope = rope_table(128, 128)
    res = []
    for page in (2, 9):  # 9: no page of the cache
        cache = sdva.KVCache(sdva.KV_INT8_G64, 4, hkv)
        table = torch.tensor([[0, 1], [page, -1], [3, -1]], dtype=torch.int32, device="cuda")
        ps = PromptStep(T, hq, num_kv_heads=hkv)
        assert not any(x.any() for x in ps.turned)  # nothing of what the memory held before
        out, lse = ps.run(cache, q, k, v, cu, table, zeros, rope=rope)
        res.append((out.clone(), lse.clone(), int(ps.status)))
    assert res[0][2] == 0 and res[1][2] & sdva.STATUS_BAD_PAGE
    for rows in (slice(0, 70), slice(110, 143)):
        assert torch.equal(res[0][0][rows], res[1][0][rows]) and torch.equal(res[0][1][rows], res[1][1][rows])
