"""prompt_delta, verify_delta and commit_delta on the GPU against the rule
stated token by token in 64 bits.

Tolerances.  A token's map of the state, S -> e^g (I - b kn kn') S + b v kn',
does not expand differences for log decays of at most 0, b in [0, 2] and
|kn| <= 1, so that what each token's roundings add to the state stays as large
as it came in at most.  An operand of a product in two fp16 parts is off by
2^-22 of the largest of its row, and a sum of 128 fp32 products by 2^-24 a
step; a token's update is a chain of a few of these on S and v.  Independent
roundings add in squares:
    |error of S after n tokens| <= 2^-20 sqrt(n + 1) M,  M = max_t (|S_t| + |v_t|)
in the Frobenius norm of a head's state, and as much for every update u (an
update that is recorded is divided by |k|).  Rows that repeat one key repeat its roundings:
there the errors add as they are.  1 / |k| is off by up to 2^-22 (two units in
the last place), |kn|^2 by 2^-21, and 1 - b |kn|^2 at b = 2, which turns the
state's part along the key around, by 2^-20 every time: n + 1 for sqrt(n + 1).
An output is scale qn' S: off by
scale times that, and half a step of bf16 (2^-8 of it).  What goes to the output
alone is taken in one fp16 part, off by 2^-12 of each value of its products:
with R = max_t (|row of S_t| + |its element of v_t|), qn' S by 2^-12 |qn| R, and
the sum over a chunk's updates (at most 32, each an element of u of at most R,
with a weight of at most |qn| |kn|, both operands rounded) by 2^-11 |qn| R each,
in squares: 2^-11 sqrt(33) scale |qn| R together."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

D = 128
SCALE = 1 / math.sqrt(D)
EPS = 1e-6
NAN, INF = float("nan"), float("inf")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _inputs(g, lead, hk, hv, fused=False, similar=0.5, decay=1.0, size=1.0):
    """Keys with a direction in common; decays from hardly any to all within a token."""
    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    q, k, v = normal(*lead, hk, D) * size, normal(*lead, hk, D) + similar * normal(hk, D), normal(*lead, hv, D)
    x = [y.to(torch.bfloat16) for y in (q, k * size, v * size)]
    q, k, v = torch.cat(x, -2).split((hk, hk, hv), -2) if fused else x
    g_ = -decay * torch.exp(2 * normal(*lead, hv) - 3)
    return q, k, v, g_, torch.sigmoid(2 * normal(*lead, hv))


def _norm(x, hv, eps):
    x = x.double()
    if eps >= 0:
        x = x / (x.square().sum(-1, keepdim=True) + eps).sqrt()
    return x.repeat_interleave(hv // x.shape[-2], -2)


def _walk(S, q, k, v, g, b, parent=None, eps=EPS, scale=SCALE):
    """One lane in 64 bits: S [Hv][128][128], rows [n][H][128] -> out, u, the states behind each row, M [Hv] and R
    [Hv][128]."""
    hv = v.shape[-2]
    q, k, v, g, b = _norm(q, hv, eps), _norm(k, hv, eps), v.double(), g.double(), b.double()
    states, out, us = [], [], []
    S = S.double()
    M, R = S.flatten(1).norm(dim=1), S.norm(dim=2)
    for i in range(v.shape[0]):
        p = S if i == 0 else states[i - 1 if parent is None else int(parent[i])]
        x = p * g[i].exp()[:, None, None]
        u = b[i][:, None] * (v[i] - (x @ k[i][..., None]).squeeze(-1))
        x = x + u[:, :, None] * k[i][:, None, :]
        states.append(x)
        us.append(u)
        out.append(scale * (x @ q[i][..., None]).squeeze(-1))
        M = torch.maximum(M, x.flatten(1).norm(dim=1) + v[i].norm(dim=1))
        R = torch.maximum(R, x.norm(dim=2) + v[i].abs())
        if parent is None:
            states[i - 1] = states[i - 1] if i < 1 else None  # a chain needs the last one alone
    return torch.stack(out), torch.stack(us), states, (M, R)


def _near(got, want, tol, what):
    err = (got.double() - want).abs()
    bad = (~(err <= tol)).nonzero()
    assert bad.numel() == 0, (what, len(bad), bad[:4].tolist(), float(err.nan_to_num(1e30).max()))


def _norm_near(got, want, tol, what):
    """Norms over all but the first axis (heads)."""
    err = (got.double() - want).flatten(1).norm(dim=1)
    assert (err <= tol).all(), (what, (err / tol).tolist())


def _tol(n, M, repeated=False):
    return 2.0 ** -20 * (n + 1 if repeated else math.sqrt(n + 1)) * M


def _check_out(got, want, n, M, what, qn=1.0, repeated=False):
    """got, want [n][Hv][128]"""
    M, R = M
    parts = 2.0 ** -11 * math.sqrt(33) * R
    _near(got, want, 2.0 ** -8 * want.abs() + SCALE * qn * (_tol(n, M, repeated)[:, None] + parts), what)


def _check_lane(n, S, out, deltas, state, q, k, v, g, b, parent=None, eps=EPS, repeated=False):
    """One lane's outputs (deltas or the state behind it may be None)."""
    wo, wu, ws, M = _walk(S, q, k, v, g, b, parent, eps)
    qn = 1.0 if eps >= 0 else float(q.double().norm(dim=-1).max())
    _check_out(out, wo, n, M, "out", qn, repeated)
    if deltas is not None:
        r = 1.0 if eps < 0 else (k.double().square().sum(-1) + eps).rsqrt().repeat_interleave(v.shape[1] // k.shape[1], 1)
        err = (deltas.double() - wu * (r[..., None] if eps >= 0 else 1.0)).norm(dim=-1)  # [n][Hv]
        tol = _tol(n, M[0], repeated)[None, :] * r
        assert (err <= tol).all(), ("deltas", float((err / tol).max()))
    if state is not None:
        _norm_near(state, ws[-1], _tol(n, M[0], repeated), "state")


# ---------------------------------------------------------------------------
# verify_delta
# ---------------------------------------------------------------------------
def _tree(rng, W):
    return [-1] + [int(rng.integers(max(0, i - 3), i)) for i in range(1, W)]


def _run_verify(g, lanes, W, hk, hv, counts=None, tree=False, keep=True, fused=False, eps=EPS, slots=None, extra=2, **kw):
    import speculative_decode_verify_append_gb300 as sdva
    rng = np.random.default_rng(lanes * 100 + W)
    q, k, v, gd, b = _inputs(g, (lanes, W), hk, hv, fused, **kw)
    state = torch.randn((lanes + extra, hv, D, D), generator=g, device="cuda") * 0.3
    slots = torch.randperm(lanes + extra, generator=g, device="cuda")[:lanes].int() if slots is None else slots
    parents = [_tree(rng, W) for _ in range(lanes)] if tree else None
    n_lane = None if counts is None else _i32(counts)
    counts = [W] * lanes if counts is None else counts
    for i, n in enumerate(counts):  # rows behind a lane's count are not read
        for x in (q, k, v, gd, b):
            x[i, n:] = NAN
    out = torch.full((lanes, W, hv, D), 7.0, dtype=torch.bfloat16, device="cuda")
    deltas = torch.full((lanes, W, hv, D), 7.0, device="cuda") if keep else None
    before, st = state.clone(), _status()
    sdva.verify_delta(state, q, k, v, gd, b, slots, SCALE, out, deltas, n_lane, _i32(parents) if tree else None, eps, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for i, n in enumerate(counts):
        s = int(slots[i])
        assert (out[i, n:] == 0).all() and (deltas is None or (deltas[i, n:] == 0).all())
        if n:
            row = [x[i, :n] for x in (q, k, v, gd, b)]
            _check_lane(n, before[s], out[i, :n], None if deltas is None else deltas[i, :n],
                        None if keep else state[s], *row, parent=parents[i] if tree else None, eps=eps)
    kept = list(range(lanes + extra)) if keep else sorted(set(range(lanes + extra)) - {int(s) for s, n in zip(slots, counts) if n})
    assert torch.equal(state[kept], before[kept])


@pytest.mark.parametrize("W", list(range(1, 17)))
@pytest.mark.parametrize("keep", [True, False])
def test_verify_windows(W, keep):
    _run_verify(_gen(W), 3, W, 2, 4, keep=keep)


@pytest.mark.parametrize("hk,hv", [(1, 1), (1, 2), (1, 3), (2, 8), (4, 4), (16, 32), (5, 15)])
@pytest.mark.parametrize("W", [1, 5, 16])
def test_verify_heads(hk, hv, W):
    _run_verify(_gen(hk + hv), 2, W, hk, hv, fused=True, keep=W != 5)


@pytest.mark.parametrize("W", [2, 3, 8, 9, 16])
@pytest.mark.parametrize("ragged", [False, True])
def test_verify_trees(W, ragged):
    counts = [W, 0, 1, W // 2, W - 1] if ragged else None
    _run_verify(_gen(W), 5, W, 2, 6, counts=counts, tree=True)


@pytest.mark.parametrize("keep", [True, False])
def test_verify_ragged(keep):
    _run_verify(_gen(5), 20, 16, 2, 2, counts=[16, 0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15, 16, 0, 8], keep=keep)


@pytest.mark.parametrize("keep", [True, False])
def test_verify_many_lanes(keep):
    _run_verify(_gen(6), 70, 4, 4, 8, keep=keep)


@pytest.mark.parametrize("size", [1e-4, 1.0, 300.0, 1e5])
@pytest.mark.parametrize("keep", [True, False])
def test_verify_sizes_of_values(size, keep):
    """Operands far from 1 keep their parts: halves are taken relative to a row's largest."""
    _run_verify(_gen(7), 2, 9, 1, 2, keep=keep, size=size)


def test_verify_without_normalisation():
    import speculative_decode_verify_append_gb300 as sdva
    g = _gen(8)
    q, k, v, gd, b = _inputs(g, (3, 12), 2, 4)
    q, k = ((x.float() / x.float().norm(dim=-1, keepdim=True) * 0.99).to(torch.bfloat16) for x in (q, k))
    state = torch.randn((3, 4, D, D), generator=g, device="cuda")
    out, deltas = torch.empty((3, 12, 4, D), dtype=torch.bfloat16, device="cuda"), torch.empty((3, 12, 4, D), device="cuda")
    sdva.verify_delta(state, q, k, v, gd, b, _i32([0, 1, 2]), SCALE, out, deltas, qk_eps=-1.0)
    for i in range(3):
        _check_lane(12, state[i], out[i], deltas[i], None, q[i], k[i], v[i], gd[i], b[i], eps=-1.0)


@pytest.mark.parametrize("keep", [True, False])
def test_verify_decays_that_forget(keep):
    """Log decays of -inf, of -200 and of 0, and strengths of 0, 1 and 2."""
    import speculative_decode_verify_append_gb300 as sdva
    g = _gen(9)
    q, k, v, gd, b = _inputs(g, (2, 16), 1, 2)
    gd[0, 3], gd[0, 9], gd[1, 0], gd[1, 7] = -INF, -200.0, -INF, 0.0
    gd[:, 12:14] = 0.0
    b[:, 2], b[:, 5], b[:, 12] = 0.0, 2.0, 1.0
    state = torch.randn((2, 2, D, D), generator=g, device="cuda")
    before = state.clone()
    out = torch.empty((2, 16, 2, D), dtype=torch.bfloat16, device="cuda")
    deltas = torch.empty((2, 16, 2, D), device="cuda") if keep else None
    sdva.verify_delta(state, q, k, v, gd, b, _i32([1, 0]), SCALE, out, deltas)
    for i in range(2):
        _check_lane(16, before[1 - i], out[i], deltas[i] if keep else None, None if keep else state[1 - i], q[i], k[i],
                    v[i], gd[i], b[i])


def test_verify_equal_keys():
    """The same key in every row, strengths of 1 and no decay: each update replaces the one before."""
    import speculative_decode_verify_append_gb300 as sdva
    g = _gen(10)
    q, k, v, gd, b = _inputs(g, (1, 16), 1, 1)
    k[:] = k[:, :1]
    gd.zero_()
    b.fill_(1.0)
    state = torch.randn((1, 1, D, D), generator=g, device="cuda")
    out, deltas = torch.empty((1, 16, 1, D), dtype=torch.bfloat16, device="cuda"), torch.empty((1, 16, 1, D), device="cuda")
    sdva.verify_delta(state, q, k, v, gd, b, _i32([0]), SCALE, out, deltas)
    _check_lane(16, state[0], out[0], deltas[0], None, q[0], k[0], v[0], gd[0], b[0])


def test_verify_zero_rows_and_state():
    """Keys and queries of zeros (norm 0), and a state of zeros."""
    import speculative_decode_verify_append_gb300 as sdva
    g = _gen(11)
    q, k, v, gd, b = _inputs(g, (2, 4), 1, 1)
    k[0, 1], q[0, 2], v[0, 3] = 0.0, 0.0, 0.0
    state = torch.zeros((2, 1, D, D), device="cuda")
    out, deltas = torch.empty((2, 4, 1, D), dtype=torch.bfloat16, device="cuda"), torch.empty((2, 4, 1, D), device="cuda")
    sdva.verify_delta(state, q, k, v, gd, b, _i32([0, 1]), SCALE, out, deltas)
    for i in range(2):
        _check_lane(4, state[i], out[i], deltas[i], None, q[i], k[i], v[i], gd[i], b[i])


@pytest.mark.parametrize("what", ["slot_low", "slot_high", "count_low", "count_high", "parent_self", "parent_low"])
def test_verify_skipped_lanes_are_zeros(what):
    import speculative_decode_verify_append_gb300 as sdva
    g = _gen(12)
    q, k, v, gd, b = _inputs(g, (3, 4), 1, 2)
    state = torch.randn((3, 2, D, D), generator=g, device="cuda")
    slots, n_lane, parent, want = [0, 1, 2], None, [[0, 0, 1, 2]] * 3, sdva.STATUS_BAD_TREE
    if what.startswith("slot"):
        slots, want = [0, -1 if what == "slot_low" else 3, 2], sdva.STATUS_BAD_PAGE
    elif what.startswith("count"):
        n_lane, want = _i32([4, -1 if what == "count_low" else 5, 4]), sdva.STATUS_BAD_COUNT
    else:
        parent = [parent[0], [0, 0, 2 if what == "parent_self" else -1, 2], parent[0]]
    st = _status()
    out, deltas = torch.full((3, 4, 2, D), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((3, 4, 2, D), 7.0, device="cuda")
    before = state.clone()
    sdva.verify_delta(state, q, k, v, gd, b, _i32(slots), SCALE, out, deltas, n_lane, _i32(parent), status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == want
    assert (out[1] == 0).all() and (deltas[1] == 0).all() and torch.equal(state, before)
    for i in (0, 2):
        _check_lane(4, state[i], out[i], deltas[i], None, q[i], k[i], v[i], gd[i], b[i], parent=parent[i])
    if what.startswith("parent"):
        return
    # committed: the lane's state stays
    sdva.verify_delta(state, q, k, v, gd, b, _i32(slots), SCALE, out, None, n_lane, status=st)
    torch.cuda.synchronize()
    assert torch.equal(state[1], before[1]) and not torch.equal(state[0], before[0]) and (out[1] == 0).all()


def test_a_bad_parent_behind_a_lanes_count_is_not_read():
    import speculative_decode_verify_append_gb300 as sdva
    g = _gen(13)
    q, k, v, gd, b = _inputs(g, (1, 6), 1, 1)
    state = torch.randn((1, 1, D, D), generator=g, device="cuda")
    out, deltas, st = torch.empty((1, 6, 1, D), dtype=torch.bfloat16, device="cuda"), torch.empty((1, 6, 1, D), device="cuda"), _status()
    sdva.verify_delta(state, q, k, v, gd, b, _i32([0]), SCALE, out, deltas, _i32([3]), _i32([[99, 0, 0, 9, -4, 7]]), status=st)
    assert int(st.item()) == 0
    _check_lane(3, state[0], out[0, :3], deltas[0, :3], None, *(x[0, :3] for x in (q, k, v, gd, b)), parent=[-1, 0, 0])


# ---------------------------------------------------------------------------
# commit_delta
# ---------------------------------------------------------------------------
def _commit_ref(S, k, g, d, order):
    hv = d.shape[1]
    k, g, d = k.double().repeat_interleave(hv // k.shape[1], 1), g.double(), d.double()
    S = S.double()
    mag = S.abs()
    for i in order:
        e = g[i].exp()[:, None, None]
        S = S * e + d[i][:, :, None] * k[i][:, None, :]
        mag = mag * e + (d[i][:, :, None] * k[i][:, None, :]).abs()
    return S, mag


@pytest.mark.parametrize("W", [1, 2, 7, 16])
@pytest.mark.parametrize("hk,hv", [(1, 1), (2, 6), (16, 32)])
@pytest.mark.parametrize("tree", [False, True])
def test_commit(W, hk, hv, tree):
    """fp32 throughout: a product of up to 16 factors and 17 sums, 2^-24 a step, of the magnitudes."""
    import speculative_decode_verify_append_gb300 as sdva
    g = _gen(W + hv)
    rng = np.random.default_rng(W)
    B = 6
    _, k, _, gd, _ = _inputs(g, (B, W), hk, hv, fused=True)
    deltas = torch.randn((B, W, hv, D), generator=g, device="cuda")
    state = torch.randn((B + 1, hv, D, D), generator=g, device="cuda")
    slots = torch.randperm(B + 1, generator=g, device="cuda")[:B].int()
    acc = [W - 1, 0, -1] + [int(x) for x in rng.integers(-1, W, B - 3)]
    path = [sorted(int(x) for x in rng.choice(W, a + 1, replace=False)) + [-1] * (W - a - 1) for a in acc] if tree else None
    orders = [(path[i] if tree else list(range(W)))[:acc[i] + 1] for i in range(B)]
    for i, o in enumerate(orders):  # what is not accepted is not read
        off = [j for j in range(W) if j not in o]
        for x in (k, gd, deltas):
            x[i, off] = NAN
    before, st = state.clone(), _status()
    sdva.commit_delta(state, k, gd, deltas, slots, _i32(acc), _i32(path) if tree else None, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for i, o in enumerate(orders):
        s = int(slots[i])
        want, mag = _commit_ref(before[s], k[i], gd[i], deltas[i], o)
        _near(state[s], want, 40 * 2.0 ** -24 * mag, ("state", i))
        if not o:
            assert torch.equal(state[s], before[s])
    rest = [s for s in range(B + 1) if s not in slots.tolist()]
    assert torch.equal(state[rest], before[rest])


@pytest.mark.parametrize("what", ["low", "high", "slot", "path_low", "path_high"])
def test_commit_skips_bad_lanes(what):
    import speculative_decode_verify_append_gb300 as sdva
    g = _gen(3)
    _, k, _, gd, _ = _inputs(g, (2, 4), 1, 1)
    deltas, state = torch.randn((2, 4, 1, D), generator=g, device="cuda"), torch.randn((2, 1, D, D), generator=g, device="cuda")
    acc, slots, path, want = [1, 2], [0, 1], None, sdva.STATUS_BAD_COUNT
    if what in ("low", "high"):
        acc[0] = -2 if what == "low" else 4
    elif what == "slot":
        slots, want = [2, 1], sdva.STATUS_BAD_PAGE
    else:
        path, want = [[0, -1 if what == "path_low" else 4, -1, -1], [0, 1, 2, -1]], sdva.STATUS_BAD_TREE
    before, st = state.clone(), _status()
    sdva.commit_delta(state, k, gd, deltas, _i32(slots), _i32(acc), None if path is None else _i32(path), st)
    torch.cuda.synchronize()
    assert int(st.item()) == want and torch.equal(state[0], before[0])
    want, mag = _commit_ref(before[1], k[1], gd[1], deltas[1], [0, 1, 2])
    _near(state[1], want, 40 * 2.0 ** -24 * mag, "state")


def test_commit_forgets_at_an_infinite_decay():
    import speculative_decode_verify_append_gb300 as sdva
    g = _gen(4)
    _, k, _, gd, _ = _inputs(g, (1, 5), 1, 1)
    gd[0, 2] = -INF
    deltas, state = torch.randn((1, 5, 1, D), generator=g, device="cuda"), torch.randn((1, 1, D, D), generator=g, device="cuda")
    want, mag = _commit_ref(state[0], k[0], gd[0], deltas[0], range(5))
    sdva.commit_delta(state, k, gd, deltas, _i32([0]), _i32([4]))
    _near(state[0], want, 40 * 2.0 ** -24 * mag, "state")


# ---------------------------------------------------------------------------
# prompt_delta
# ---------------------------------------------------------------------------
def _workspace(T, B, hk, hv):
    import speculative_decode_verify_append_gb300 as sdva
    return torch.full((sdva.prompt_delta_workspace_size(T, B, hk, hv),), 255, dtype=torch.uint8, device="cuda")


def _run_prompt(g, lens, hk, hv, seq=None, start=0, tail=0, fused=False, eps=EPS, change=None, heads=None, repeated=False,
                **kw):
    import speculative_decode_verify_append_gb300 as sdva
    B, T = len(lens), start + sum(lens) + tail
    q, k, v, gd, b = _inputs(g, (T,), hk, hv, fused, **kw)
    if change is not None:
        change(q, k, v, gd, b)
    end = start + sum(lens)
    for x in (q, k, v, gd, b):  # rows outside the lanes hold NaN, which reaches nothing
        x[:start] = NAN
        x[end:] = NAN
    cu = _i32(np.concatenate([[start], start + np.cumsum(lens)]))
    state = torch.randn((B + 2, hv, D, D), generator=g, device="cuda") * 0.3
    slots = torch.randperm(B + 2, generator=g, device="cuda")[:B].int()
    L = [1] * B if seq is None else seq
    for i in range(B):
        if L[i] == 0 and lens[i]:
            state[int(slots[i])] = NAN  # a slot that is started from zeros is not read
    before = state.clone()
    out, st = torch.full((T, hv, D), 7.0, dtype=torch.bfloat16, device="cuda"), _status()
    sdva.prompt_delta(state, q, k, v, gd, b, cu, slots, SCALE, out, _workspace(T, B, hk, hv),
                      None if seq is None else _i32(seq), eps, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert (out[:start] == 7.0).all() and (out[end:] == 7.0).all()
    a = start
    for i, n in enumerate(lens):
        s = int(slots[i])
        if n:
            S = before[s] if L[i] else torch.zeros_like(before[s])
            h = slice(None) if heads is None else heads
            kh = slice(None) if heads is None else slice(heads.start * hk // hv, -(-heads.stop * hk // hv))
            _check_lane(n, S[h], out[a:a + n, h], None, state[s][h], q[a:a + n, kh], k[a:a + n, kh], v[a:a + n, h],
                        gd[a:a + n, h], b[a:a + n, h], eps=eps, repeated=repeated)
        else:
            assert torch.equal(state[s], before[s])
        a += n
    rest = [s for s in range(B + 2) if s not in slots.tolist()]
    assert torch.equal(state[rest], before[rest])
    return out, state


@pytest.mark.parametrize("lens", [[1], [2], [15], [16], [17], [31], [32], [33], [63], [64], [65], [127], [128], [129],
                                  [1, 0, 31, 32, 33, 0, 64, 65, 500], [0, 0, 5, 0], [1] * 40, [300, 1, 700]])
@pytest.mark.parametrize("seq", [False, True])
def test_prompt_lengths(lens, seq):
    L = [i % 2 * 9 for i in range(len(lens))] if seq else None
    _run_prompt(_gen(len(lens)), lens, 2, 4, L)


@pytest.mark.parametrize("hk,hv", [(1, 1), (1, 2), (1, 3), (2, 8), (4, 4), (16, 32), (5, 15), (1, 4)])
def test_prompt_heads(hk, hv):
    _run_prompt(_gen(hv), [100, 3, 70], hk, hv, fused=True, start=5, tail=9)


def test_prompt_long():
    _run_prompt(_gen(1), [3000], 1, 2, [0])
    _run_prompt(_gen(2), [1111, 40, 2000], 2, 2, [0, 3, 3], decay=0.01)


def test_prompt_many_lanes():
    rng = np.random.default_rng(3)
    _run_prompt(_gen(3), [int(x) for x in rng.integers(0, 50, 200)], 1, 2)


@pytest.mark.parametrize("size", [1e-4, 300.0, 1e5])
def test_prompt_sizes_of_values(size):
    _run_prompt(_gen(4), [90, 33], 1, 2, size=size)


def test_prompt_decays_that_forget_and_strengths_at_their_ends():
    def change(q, k, v, gd, b):
        gd[5], gd[40], gd[41], gd[70] = -INF, -200.0, -50.0, -INF
        gd[80:90] = 0.0
        b[10:14], b[20:24], b[50:60] = 0.0, 2.0, 1.0
        gd[100:] = -1e-7
    _run_prompt(_gen(5), [150, 20], 2, 4, change=change)


@pytest.mark.parametrize("beta", [1.0, 0.5, 2.0])
def test_prompt_equal_keys(beta):
    """The same key in every row and no decay: the updates of a chunk depend on one another as much as they can."""
    def change(q, k, v, gd, b):
        k[:] = k[:1]
        gd.zero_()
        b.fill_(beta)
    _run_prompt(_gen(6), [200], 1, 2, [0], change=change, repeated=True)


def test_prompt_zero_rows():
    def change(q, k, v, gd, b):
        k[3:40], q[50:60], v[20:70] = 0.0, 0.0, 0.0
    _run_prompt(_gen(7), [100], 1, 1, [0], change=change)


def test_prompt_without_normalisation():
    def change(q, k, v, gd, b):
        for x in (q, k):
            x.copy_((x.float() / x.float().norm(dim=-1, keepdim=True) * 0.99).to(torch.bfloat16))
    _run_prompt(_gen(8), [130, 7], 2, 2, eps=-1.0, change=change)


@pytest.mark.parametrize("what", ["slot_low", "slot_high", "length"])
def test_prompt_skips_bad_lanes(what):
    import speculative_decode_verify_append_gb300 as sdva
    g = _gen(9)
    lens = [40, 50, 33]
    q, k, v, gd, b = _inputs(g, (123,), 1, 2)
    state = torch.randn((3, 2, D, D), generator=g, device="cuda")
    slots, seq, want = [0, 1, 2], [3, 3, 3], sdva.STATUS_BAD_PAGE
    if what == "length":
        seq, want = [3, -1, 3], sdva.STATUS_OVERFLOW
    else:
        slots[1] = -1 if what == "slot_low" else 3
    before, st = state.clone(), _status()
    out = torch.full((123, 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    sdva.prompt_delta(state, q, k, v, gd, b, _i32([0, 40, 90, 123]), _i32(slots), SCALE, out, _workspace(123, 3, 1, 2),
                      _i32(seq), status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == want
    assert torch.equal(state[1], before[1]) and (out[40:90] == 7.0).all()
    for i, a, n in ((0, 0, 40), (2, 90, 33)):
        _check_lane(n, before[i], out[a:a + n], None, state[i], *(x[a:a + n] for x in (q, k, v, gd, b)))


@pytest.mark.parametrize("cu", [[0, 12, 9, 20], [-1, 5, 9, 20], [0, 5, 9, 21]])
def test_prompt_offsets_out_of_order_write_nothing(cu):
    import speculative_decode_verify_append_gb300 as sdva
    g = _gen(10)
    q, k, v, gd, b = _inputs(g, (20,), 1, 2)
    state = torch.randn((3, 2, D, D), generator=g, device="cuda")
    before, st, out = state.clone(), _status(), torch.full((20, 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    sdva.prompt_delta(state, q, k, v, gd, b, _i32(cu), _i32([0, 1, 2]), SCALE, out, _workspace(20, 3, 1, 2), status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == sdva.STATUS_BAD_COUNT
    assert torch.equal(state, before) and (out == 7.0).all()


def test_prompt_in_two_pieces_is_the_prompt():
    """A prompt that goes on from its state: the same rule, so the same bounds from the 64-bit state."""
    import speculative_decode_verify_append_gb300 as sdva
    g = _gen(11)
    q, k, v, gd, b = _inputs(g, (200,), 1, 2)
    state = torch.zeros((1, 2, D, D), device="cuda")
    out = torch.empty((200, 2, D), dtype=torch.bfloat16, device="cuda")
    done = 0
    for n in (77, 123):
        x = [y[done:done + n] for y in (q, k, v, gd, b)]
        sdva.prompt_delta(state, *x, _i32([0, n]), _i32([0]), SCALE, out[done:done + n], _workspace(n, 1, 1, 2),
                          _i32([done]))
        done += n
    _check_lane(200, torch.zeros((2, D, D), device="cuda"), out, None, state[0], q, k, v, gd, b)


# ---------------------------------------------------------------------------
# all of them
# ---------------------------------------------------------------------------
def test_prompt_verify_commit_together():
    """A prompt, three verify steps of which a part is accepted, and plain steps: the states follow the accepted tokens."""
    import speculative_decode_verify_append_gb300 as sdva
    from speculative_decode_verify_append_gb300.step import DeltaStep
    g = _gen(20)
    hk, hv, B, W = 2, 4, 3, 6
    lens = [50, 7, 33]
    T = sum(lens)
    step = DeltaStep(B, hk, hv, window=W, max_tokens=T)
    q, k, v, gd, b = _inputs(g, (T,), hk, hv, fused=True)
    cu, slots, seq = _i32(np.concatenate([[0], np.cumsum(lens)])), _i32([2, 0, 1]), _i32([0, 0, 0])
    step.state.fill_(NAN)
    step.prompt(q, k, v, gd, b, cu, slots, seq)
    hist = [[[x[int(cu[i]):int(cu[i + 1])] for x in (q, k, v, gd, b)]] for i in range(B)]
    accepted = [_i32([5, 0, 2]), _i32([0, 3, 5]), _i32([1, 1, -1])]
    outs = []
    for acc in accepted:
        x = _inputs(g, (B, W), hk, hv, fused=True)
        outs.append((step.verify(*x, slots).clone(), [[y[i] for y in x] for i in range(B)], acc.tolist()))
        step.commit(x[1], x[3], slots, acc)
        for i in range(B):
            n = int(acc[i]) + 1
            hist[i].append([y[i, :n] for y in x])
    x = _inputs(g, (B, 1), hk, hv)
    last = step.decode(*x, slots)
    for i in range(B):
        hist[i].append([y[i] for y in x])
    assert int(step.status.item()) == 0
    for i in range(B):
        rows = [torch.cat([h[j] for h in hist[i]]) for j in range(5)]
        n = rows[0].shape[0]
        zero = torch.zeros((hv, D, D), device="cuda")
        wo, _, ws, M = _walk(zero, *rows)
        _norm_near(step.state[int(slots[i])], ws[-1], _tol(n, M[0]), "state")
        _check_out(last[i], wo[-1:], n, M, "last")
        # every window's rows, accepted or not, behind what was accepted before
        for w, (out, x, _) in enumerate(outs):
            head = [torch.cat([h[j] for h in hist[i][:w + 1]] + [x[i][j]]) for j in range(5)]
            wo, _, _, M = _walk(zero, *head)
            _check_out(out[i], wo[-W:], head[0].shape[0], M, ("window", w))


def test_tree_accept_and_commit():
    """The acceptance call's path goes to the commit as it is."""
    import speculative_decode_verify_append_gb300 as sdva
    g = _gen(21)
    B, W, hk, hv, V = 4, 8, 1, 2, 50
    rng = np.random.default_rng(5)
    parents = [_tree(rng, W) for _ in range(B)]
    q, k, v, gd, b = _inputs(g, (B, W), hk, hv)
    state = torch.randn((B, hv, D, D), generator=g, device="cuda")
    slots, parent = _i32(range(B)), _i32(parents)
    out, deltas = torch.empty((B, W, hv, D), dtype=torch.bfloat16, device="cuda"), torch.empty((B, W, hv, D), device="cuda")
    before = state.clone()
    sdva.verify_delta(state, q, k, v, gd, b, slots, SCALE, out, deltas, parent=parent)
    tokens = torch.randint(V, (B, W), generator=g, device="cuda", dtype=torch.int32)
    logits = torch.randn((B, W, V), generator=g, device="cuda")
    for i in range(B):  # the target agrees with the first child of every slot but one lane's
        for j in range(W):
            kids = [c for c in range(1, W) if parents[i][c] == j]
            if kids and i:
                logits[i, j, int(tokens[i, kids[0]])] += 20.0
    acc, path, toks = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((B,), (B, W), (B, W)))
    sdva.spec_accept_tree(logits, tokens, parent, acc, path, toks)
    sdva.commit_delta(state, k, gd, deltas, slots, acc, path)
    for i in range(B):
        p = path[i, :int(acc[i]) + 1].long()
        x = [y[i, p] for y in (q, k, v, gd, b)]
        _, _, ws, M = _walk(before[i], *x)
        _norm_near(state[i], ws[-1], _tol(len(p), M[0]), "state")
    assert int(acc.max()) >= 2


@pytest.mark.parametrize("what", ["prompt", "verify", "decode", "commit"])
def test_a_captured_graph_replays(what):
    import speculative_decode_verify_append_gb300 as sdva
    g = _gen(22)
    B, W, hk, hv = 3, 5, 1, 2
    lead = (90,) if what == "prompt" else (B, W)
    x = _inputs(g, lead, hk, hv)
    state = torch.randn((B, hv, D, D), generator=g, device="cuda")
    out, deltas = torch.zeros((*lead, hv, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((*lead, hv, D), device="cuda")
    cu, slots, acc, ws = _i32([0, 40, 41, 90]), _i32([2, 0, 1]), _i32([2, 4, 0]), _workspace(90, B, hk, hv)

    def call(s, o, d, w):
        if what == "prompt":
            sdva.prompt_delta(s, *x, cu, slots, SCALE, o, w)
        elif what == "commit":
            sdva.commit_delta(s, x[1], x[3], deltas, slots, acc)
        else:
            sdva.verify_delta(s, *x, slots, SCALE, o, d if what == "verify" else None)

    call(state.clone(), out, deltas, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(state, out, deltas, ws)
    for seed in (1, 2, 3):
        for y, z in zip(x, _inputs(_gen(seed), lead, hk, hv)):
            y.copy_(z)
        if what == "commit":
            deltas.normal_(generator=g)
        s, o, d = state.clone(), torch.zeros_like(out), torch.zeros_like(deltas)
        call(s, o, d, _workspace(90, B, hk, hv))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(s, state)
        if what != "commit":
            assert torch.equal(o, out)
        if what == "verify":
            assert torch.equal(d, deltas)


def test_calls_at_once_on_several_streams():
    import speculative_decode_verify_append_gb300 as sdva
    g = _gen(23)
    hk, hv, B, W = 4, 8, 6, 16
    lens = [700, 64, 1, 0, 333, 90]
    T = sum(lens)
    p, w = _inputs(g, (T,), hk, hv), _inputs(g, (B, W), hk, hv)
    cu, slots = _i32(np.concatenate([[0], np.cumsum(lens)])), _i32(range(B))
    start = torch.randn((B, hv, D, D), generator=g, device="cuda")

    def calls(streams):
        results = []
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                state = start.clone()
                if i % 2 == 0:
                    out = torch.zeros((T, hv, D), dtype=torch.bfloat16, device="cuda")
                    sdva.prompt_delta(state, *p, cu, slots, SCALE, out, _workspace(T, B, hk, hv))
                    results += [state, out]
                else:
                    out, deltas = torch.zeros((B, W, hv, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((B, W, hv, D), device="cuda")
                    sdva.verify_delta(state, *w, slots, SCALE, out, deltas)
                    sdva.commit_delta(state, w[1], w[3], deltas, slots, _i32([3, 15, 0, 7, 9, 1]))
                    results += [state, out, deltas]
        torch.cuda.synchronize()
        return results

    one = calls([torch.cuda.current_stream()] * 6)
    streams = [torch.cuda.Stream() for _ in range(6)]
    for _ in range(3):
        for a, b in zip(one, calls(streams)):
            assert torch.equal(a, b)


def test_the_binding_refuses():
    import speculative_decode_verify_append_gb300 as sdva
    g = _gen(24)
    q, k, v, gd, b = _inputs(g, (2, 4), 2, 4)
    state, slots = torch.randn((2, 4, D, D), generator=g, device="cuda"), _i32([0, 1])
    out, deltas = torch.empty((2, 4, 4, D), dtype=torch.bfloat16, device="cuda"), torch.empty((2, 4, 4, D), device="cuda")
    good = dict(state=state, q=q, k=k, v=v, log_decay=gd, beta=b, slots=slots, scale=SCALE, out=out, deltas=deltas)
    sdva.verify_delta(**good)
    for change in (dict(state=state[0]), dict(state=state.double()), dict(state=state.transpose(2, 3)), dict(q=q.float()),
                   dict(k=k[:, :, :1]), dict(v=k), dict(log_decay=gd.bfloat16()), dict(beta=b[:, :3]), dict(slots=slots[:1]),
                   dict(out=out.float()), dict(deltas=deltas[:1]), dict(scale=0.0), dict(scale=NAN), dict(scale=INF),
                   dict(qk_eps=NAN), dict(qk_eps=INF), dict(parent=slots), dict(n_lane=_i32([1])),
                   dict(parent=_i32([[0] * 4] * 2), deltas=None), dict(q=q.cpu()), dict(q=q.transpose(0, 1))):
        with pytest.raises((ValueError, sdva.SdvaError)):
            sdva.verify_delta(**{**good, **change})
    with pytest.raises(sdva.SdvaError) as e:
        sdva.prompt_delta(state, q[0], k[0], v[0], gd[0], b[0], _i32([0, 2, 4]), slots, SCALE, out[0],
                          torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert e.value.code == sdva.ERR_WORKSPACE
    acc = _i32([0, 0])
    for change in (dict(k=k[:, :3]), dict(deltas=deltas.half()), dict(accept_len=acc[:1]), dict(path=acc), dict(state=state[:, :3])):
        with pytest.raises((ValueError, sdva.SdvaError)):
            sdva.commit_delta(**{**dict(state=state, k=k, log_decay=gd, deltas=deltas, slots=slots, accept_len=acc), **change})


@pytest.mark.parametrize("W,keep", [(1, True), (2, True), (1, False), (3, False)])
def test_short_chains_give_outputs_of_fp32(W, keep):
    """Chains that fp32 takes owe out nothing but its own rounding: the tolerance of an operand in one fp16 part, which
    the tensor cores' outputs have, is left out here."""
    import speculative_decode_verify_append_gb300 as sdva
    B, hk, hv = 3, 2, 4
    g = _gen(90 + W)
    q, k, v, gd, b = _inputs(g, (B, W), hk, hv)
    state = torch.randn((B, hv, D, D), generator=g, device="cuda") * 0.3
    before, slots = state.clone(), _i32(range(B))
    out = torch.empty((B, W, hv, D), dtype=torch.bfloat16, device="cuda")
    deltas = torch.empty((B, W, hv, D), device="cuda") if keep else None
    sdva.verify_delta(state, q, k, v, gd, b, slots, SCALE, out, deltas)
    for i in range(B):
        want, _, _, (M, _) = _walk(before[i], q[i], k[i], v[i], gd[i], b[i])
        _near(out[i], want, 2.0 ** -8 * want.abs() + SCALE * _tol(W, M)[None, :, None], "out")
