"""The gated delta rule where its values range widely: maps that expand (keys
taken as they are, decays that grow), tokens and value rows of very different
sizes.  Against the rule token by token in 64 bits, with a tolerance per token
and value row that knows nothing of later tokens or of other value rows.

Tolerances.  With g2 = 2^-19 for the relative error of one value of fp32, in
which independent roundings add in squares: a sum of 128 products of operands in
two parts (2^-22 of a value) is off by 2^-23 of the product of the norms a step,
16 steps, 2^-21; a product of up to 32 decays, two units in the last place each,
by sqrt(32) 2^-22, 2^-19.5; a key's factor by 2^-22.  Over tokens errors add as
they are.  In front of a chunk (a window; 32 tokens of a prompt,
of which a plain walk is a special case) a value row of the state has norm S and
is off by E.  With the norms of keys and queries in place of their products,
    x_i = |b_i| (|v_i| + a_i |k_i| (S + E)),  dx_i = g2 x_i + |b_i| a_i |k_i| E
u solves (1 + A) u = x, T = (1 + A)^-1; A is off by g2 L, L_ij = |b_i| D_ij |k_i| |k_j|,
and a product with an inverse that fp32 solved for by g2 |T| (1 + L) |T| x:
    du = |T| (dx + g2 (1 + L) |T| x)
    do_i = scale ((2^-11 + g2) a_i |q_i| (S + E) + a_i |q_i| E
                  + sum_j P_ij (du_j + (2^-10 + g2) |u_j|) + 2^-38 max_j P_ij |u_j|),
P_ij = D_ij |q_i| |k_j|: what goes to the output alone is in one part of 11 bits
(2^-11 of a value), and a score in fp16 is off by 2^-39 of its row's largest at
least.  The output's own rounding is 2^-8 of it.  Behind the chunk
    E <- f E + g2 f S + sum_j D_last,j |k_j| (du_j + g2 |u_j|)."""
import numpy as np
import pytest
import torch

from test_gpu_delta import D, EPS, INF, SCALE, _gen, _i32, _norm, _status, _tree, _workspace

pytestmark = pytest.mark.gpu

G2 = 2.0 ** -19


def _rule(S, q, k, v, g, b, parent=None, eps=EPS):
    """One lane in 64 bits: out, u [n][Hv][128] and the states in front of and behind the tokens (n + 1)."""
    hv = v.shape[-2]
    q, k, v, g, b = _norm(q, hv, eps), _norm(k, hv, eps), v.double(), g.double(), b.double()
    states, out, us = [S.double()], [], []
    for i in range(v.shape[0]):
        x = states[i if parent is None else int(parent[i]) + 1] * g[i].exp()[:, None, None]
        u = b[i][:, None] * (v[i] - torch.einsum("hvk,hk->hv", x, k[i]))
        x = x + u[:, :, None] * k[i][:, None, :]
        states.append(x)
        us.append(u)
        out.append(SCALE * torch.einsum("hvk,hk->hv", x, q[i]))
    return torch.stack(out), torch.stack(us), states


def _bounds(states, us, q, k, v, g, b, parent, eps, chunk):
    """Tolerances of out and u [n][Hv][128], and of the rows of the state behind the last token [Hv][128] (in norm)."""
    n, hv = v.shape[:2]
    q, k, v, eg, b = _norm(q, hv, eps), _norm(k, hv, eps), v.double(), g.double().exp(), b.double()
    E = torch.zeros_like(us[0])
    t_out, t_u = torch.zeros_like(us), torch.zeros_like(us)
    for t0 in range(0, n, chunk):
        c = slice(t0, min(t0 + chunk, n))
        m = c.stop - t0
        Dm, a = torch.zeros((hv, m, m), dtype=torch.float64, device=v.device), torch.zeros((hv, m), dtype=torch.float64, device=v.device)
        for i in range(m):
            p = (i if parent is None else int(parent[i]) + 1) - 1
            a[:, i] = eg[t0 + i] * (a[:, p] if p >= 0 else 1.0)
            if p >= 0:
                Dm[:, i] = eg[t0 + i][:, None] * Dm[:, p]
            Dm[:, i, i] = 1.0
        kk, qq = k[c].norm(dim=-1).T, q[c].norm(dim=-1).T  # [hv][m]
        bb, u = b[c].T.abs(), us[c].abs().transpose(0, 1)
        A = b[c].T[:, :, None] * Dm * torch.einsum("ihd,jhd->hij", k[c], k[c])
        L = bb[:, :, None] * Dm * kk[:, :, None] * kk[:, None, :]
        one = torch.eye(m, dtype=torch.float64, device=v.device)
        A, L = A.tril(-1) + one, L.tril(-1) + one
        T = torch.linalg.solve_triangular(A, one.expand_as(A), upper=False).abs()
        S = states[t0].norm(dim=2)  # [hv][128]
        x = bb[..., None] * (v[c].abs().transpose(0, 1) + (a * kk)[..., None] * (S + E)[:, None])
        dx = G2 * x + (bb * a * kk)[..., None] * E[:, None]
        du = T @ (dx + G2 * (L @ (T @ x)))
        P = Dm * qq[:, :, None] * kk[:, None, :]
        aq = (a * qq)[..., None]
        do = SCALE * ((2.0 ** -11 + G2) * aq * (S + E)[:, None] + aq * E[:, None] + P @ (du + (2.0 ** -10 + G2) * u) +
                      2.0 ** -38 * P.amax(2, keepdim=True) * ((Dm != 0).double() @ u))
        t_out[c], t_u[c] = do.transpose(0, 1), du.transpose(0, 1)
        f, last = a[:, -1, None], (Dm[:, -1] * kk)[..., None]
        E = f * (E + G2 * S) + (last * (du + G2 * u)).sum(1)
    return t_out, t_u, E


def _check(S, out, deltas, state, q, k, v, g, b, parent=None, eps=EPS, chunk=32):
    wo, wu, states = _rule(S, q, k, v, g, b, parent, eps)
    assert float(torch.stack(states).abs().max()) < 1e37 and float(wu.abs().max()) < 1e37  # the case itself is one of fp32
    t_out, t_u, t_S = _bounds(states, wu, q, k, v, g, b, parent, eps, chunk)

    def near(got, want, tol, what):
        err = (got.double() - want).abs()
        bad = (~(err <= tol)).nonzero()
        assert bad.numel() == 0, (what, len(bad), bad[:4].tolist(), float((err / tol).nan_to_num(1e30, 1e30).max()))

    near(out, wo, 2.0 ** -8 * wo.abs() + t_out, "out")
    if deltas is not None:
        r = 1.0
        if eps >= 0:
            r = (k.double().square().sum(-1) + eps).rsqrt().repeat_interleave(v.shape[1] // k.shape[1], 1)[..., None]
        near(deltas, wu * r, t_u * r + 2.0 ** -22 * (wu * r).abs(), "deltas")
    if state is not None:
        err = (state.double() - states[-1]).norm(dim=2)
        assert (err <= t_S).all(), ("state", float((err / t_S).nan_to_num(1e30, 1e30).max()))


def _rows(seed, lead, hk, hv, kind):
    """q, k, v, log_decay, beta, qk_eps of rows whose maps expand."""
    g = _gen(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def unit(x, size):
        return x / x.norm(dim=-1, keepdim=True) * size

    q, k, v = normal(*lead, hk, D), normal(*lead, hk, D), normal(*lead, hv, D)
    gd, b, eps = -0.05 * normal(*lead, hv).abs(), torch.rand((*lead, hv), generator=g, device="cuda"), -1.0
    if kind == "one_key":  # u_i is -2 times the sum in front of it: 3^i
        k = unit(normal(hk, D), 2.0).expand(*lead, hk, D)
        gd, b = torch.zeros_like(gd), torch.ones_like(b)
    elif kind == "long_keys":  # |k|^2 = 128 and more, a direction in common
        k = k + normal(hk, D)
        b = torch.full_like(b, 0.5)
    elif kind == "norms_to_4":
        k = unit(k + 0.5 * normal(hk, D), 2.0) * (1 + torch.rand((*lead, hk, 1), generator=g, device="cuda"))
    elif kind == "growing":  # normalised keys, decays above 0
        gd, eps = 0.4 * torch.rand((*lead, hv), generator=g, device="cuda"), EPS
    elif kind == "small_strengths":  # |k| = 2^10 and b |k|^2 up to 2
        k, b = unit(k + 0.5 * normal(hk, D), 1024.0), 2.0 ** -19 * b
    elif kind == "small_keys":  # |k| = 2^-10, b |k|^2 up to 2
        k, b = unit(k + 0.5 * normal(hk, D), 2.0 ** -10), 2.0 ** 21 * b
    elif kind == "tiny_keys":  # a state of zeros becomes one of their size
        k = unit(k, 2.0 ** -70)
    return q.to(torch.bfloat16), k.to(torch.bfloat16).contiguous(), v.to(torch.bfloat16), gd, b, eps


KINDS = ["one_key", "long_keys", "norms_to_4", "growing", "small_strengths", "small_keys", "tiny_keys"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("W", [1, 2, 3, 4, 9, 16])
@pytest.mark.parametrize("how", ["recorded", "committed", "tree"])
def test_windows_that_expand(kind, W, how):
    import speculative_decode_verify_append_gb300 as sdva
    if how == "tree" and W == 1:
        pytest.skip("a tree of one row is a chain")
    B, hk, hv = 2, 1, 2
    *x, eps = _rows(100 + W, (B, W), hk, hv, kind)
    rng = np.random.default_rng(W)
    parents = [_tree(rng, W) for _ in range(B)] if how == "tree" else None
    state = torch.randn((B, hv, D, D), generator=_gen(W), device="cuda") * (kind != "tiny_keys")
    before, st = state.clone(), _status()
    out = torch.empty((B, W, hv, D), dtype=torch.bfloat16, device="cuda")
    deltas = None if how == "committed" else torch.empty((B, W, hv, D), device="cuda")
    sdva.verify_delta(state, *x, _i32(range(B)), SCALE, out, deltas, parent=_i32(parents) if parents else None, qk_eps=eps, status=st)
    assert int(st.item()) == 0
    for i in range(B):
        _check(before[i], out[i], None if deltas is None else deltas[i], state[i] if deltas is None else None,
               *(y[i] for y in x), parent=parents[i] if parents else None, eps=eps)


@pytest.mark.parametrize("kind,lens", [("one_key", [32, 5, 17]), ("long_keys", [12, 7]), ("norms_to_4", [32, 3]),
                                       ("growing", [64, 33, 20]), ("small_strengths", [64, 40]), ("small_keys", [64, 40]),
                                       ("tiny_keys", [40, 40])])
def test_prompts_that_expand(kind, lens):
    import speculative_decode_verify_append_gb300 as sdva
    hk, hv, B, T = 1, 2, len(lens), sum(lens)
    *x, eps = _rows(200, (T,), hk, hv, kind)
    state = torch.randn((B, hv, D, D), generator=_gen(9), device="cuda") * (kind != "tiny_keys")
    before, st = state.clone(), _status()
    out = torch.empty((T, hv, D), dtype=torch.bfloat16, device="cuda")
    cu = [0, *np.cumsum(lens)]
    sdva.prompt_delta(state, *x, _i32(cu), _i32(range(B)), SCALE, out, _workspace(T, B, hk, hv), qk_eps=eps, status=st)
    assert int(st.item()) == 0
    for i in range(B):
        r = slice(cu[i], cu[i + 1])
        _check(before[i], out[r], None, state[i], *(y[r] for y in x), eps=eps)


@pytest.mark.parametrize("W", [2, 4, 8, 16])
def test_nothing_to_remember_and_growing_decays(W):
    """A state of zeros and updates of zeros stay zeros, whatever the decays are."""
    import speculative_decode_verify_append_gb300 as sdva
    *x, _ = _rows(5, (2, W), 1, 2, "growing")
    x[3].fill_(1.5)
    x[2][0] = 0.0  # one lane by its values, one by its strengths
    x[4][1] = 0.0
    state = torch.zeros((2, 2, D, D), device="cuda")
    out = torch.full((2, W, 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    sdva.verify_delta(state, *x, _i32([0, 1]), SCALE, out)
    assert (state == 0).all() and (out == 0).all()
    n = 40
    *x, _ = _rows(6, (n,), 1, 2, "growing")
    x[3].fill_(1.5)
    x[2].zero_()
    out = torch.full((n, 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    sdva.prompt_delta(state, *x, _i32([0, n]), _i32([0]), SCALE, out, _workspace(n, 1, 1, 2))
    assert (state == 0).all() and (out == 0).all()


def _sized(lead, seed=7):
    """Rows whose values are of size 1; lead[-1] tokens."""
    *x, _ = _rows(seed, lead, 1, 2, "norms_to_4")
    return x


@pytest.mark.parametrize("power", [12, 18, 30])
def test_prompt_tokens_of_different_sizes(power):
    """The last tokens of a chunk are 2^power times the first ones, which do not know of them."""
    import speculative_decode_verify_append_gb300 as sdva
    n = 64
    x = _sized((n,))
    for c in (16, 60):
        x[2][c:c + 4] *= 2.0 ** power
    x[3][32] = -INF  # the second chunk starts small again
    state = torch.randn((1, 2, D, D), generator=_gen(1), device="cuda")
    before = state.clone()
    out = torch.empty((n, 2, D), dtype=torch.bfloat16, device="cuda")
    sdva.prompt_delta(state, *x, _i32([0, n]), _i32([0]), SCALE, out, _workspace(n, 1, 1, 2))
    _check(before[0], out, None, state[0], *x)


@pytest.mark.parametrize("power", [12, 18, 30])
@pytest.mark.parametrize("keep", [True, False])
def test_window_tokens_of_different_sizes(power, keep):
    import speculative_decode_verify_append_gb300 as sdva
    W = 16
    x = _sized((1, W))
    x[2][:, 10:] *= 2.0 ** power
    state = torch.randn((1, 2, D, D), generator=_gen(2), device="cuda")
    before = state.clone()
    out = torch.empty((1, W, 2, D), dtype=torch.bfloat16, device="cuda")
    deltas = torch.empty((1, W, 2, D), device="cuda") if keep else None
    sdva.verify_delta(state, *x, _i32([0]), SCALE, out, deltas)
    _check(before[0], out[0], deltas[0] if keep else None, None if keep else state[0], *(y[0] for y in x))


@pytest.mark.parametrize("power", [12, 18, 30])
@pytest.mark.parametrize("what", ["prompt", "recorded", "committed"])
def test_value_rows_of_different_sizes(power, what):
    """One value row of sixteen is 2^power times the others, in the state and in the values."""
    import speculative_decode_verify_append_gb300 as sdva
    n = 64 if what == "prompt" else 16
    x = _sized((n,) if what == "prompt" else (1, n))
    state = torch.randn((1, 2, D, D), generator=_gen(3), device="cuda")
    state[:, :, 5::16] *= 2.0 ** power
    x[2][..., 5::16] *= 2.0 ** power
    before = state.clone()
    if what == "prompt":
        out, deltas = torch.empty((n, 2, D), dtype=torch.bfloat16, device="cuda"), None
        sdva.prompt_delta(state, *x, _i32([0, n]), _i32([0]), SCALE, out, _workspace(n, 1, 1, 2))
    else:
        out = torch.empty((1, n, 2, D), dtype=torch.bfloat16, device="cuda")
        deltas = torch.empty((1, n, 2, D), device="cuda") if what == "recorded" else None
        sdva.verify_delta(state, *x, _i32([0]), SCALE, out, deltas)
        out, deltas, x = out[0], None if deltas is None else deltas[0], [y[0] for y in x]
    _check(before[0], out, deltas, None if what == "recorded" else state[0], *x)


@pytest.mark.parametrize("power", [-100, 100])
@pytest.mark.parametrize("what", ["prompt", "recorded", "committed"])
def test_values_near_the_ends_of_fp32(power, what):
    import speculative_decode_verify_append_gb300 as sdva
    n = 40 if what == "prompt" else 12
    x = _sized((n,) if what == "prompt" else (1, n))
    x[2] *= 2.0 ** power
    state = torch.randn((1, 2, D, D), generator=_gen(4), device="cuda") * 2.0 ** power
    before, st = state.clone(), _status()
    if what == "prompt":
        out, deltas = torch.empty((n, 2, D), dtype=torch.bfloat16, device="cuda"), None
        sdva.prompt_delta(state, *x, _i32([0, n]), _i32([0]), SCALE, out, _workspace(n, 1, 1, 2), status=st)
    else:
        out = torch.empty((1, n, 2, D), dtype=torch.bfloat16, device="cuda")
        deltas = torch.empty((1, n, 2, D), device="cuda") if what == "recorded" else None
        sdva.verify_delta(state, *x, _i32([0]), SCALE, out, deltas, status=st)
        out, deltas, x = out[0], None if deltas is None else deltas[0], [y[0] for y in x]
    assert int(st.item()) == 0
    _check(before[0], out, deltas, None if what == "recorded" else state[0], *x)


@pytest.mark.parametrize("what", ["prompt", "recorded", "committed"])
def test_a_state_that_is_forgotten_and_one_that_is_replaced(what):
    """Large states that a token forgets (a decay of 0), and small ones behind which all is larger."""
    import speculative_decode_verify_append_gb300 as sdva
    n = 40 if what == "prompt" else 12
    x = _sized((2 * n,) if what == "prompt" else (2, n))
    state = torch.randn((2, 2, D, D), generator=_gen(5), device="cuda")
    state[0] *= 2.0 ** 90
    state[1] *= 2.0 ** -90
    x[2].view(2, n, 2, D)[0, :5] *= 2.0 ** 90
    x[3].view(2, n, 2)[0, 5] = -INF
    before, st = state.clone(), _status()
    out = torch.empty(x[2].shape, dtype=torch.bfloat16, device="cuda")
    if what == "prompt":
        deltas = None
        sdva.prompt_delta(state, *x, _i32([0, n, 2 * n]), _i32([0, 1]), SCALE, out, _workspace(2 * n, 2, 1, 2), status=st)
        out, x = out.view(2, n, 2, D), [y.view(2, n, *y.shape[1:]) for y in x]
    else:
        deltas = torch.empty((2, n, 2, D), device="cuda") if what == "recorded" else None
        sdva.verify_delta(state, *x, _i32([0, 1]), SCALE, out, deltas, status=st)
    assert int(st.item()) == 0
    for i in range(2):
        _check(before[i], out[i], None if deltas is None else deltas[i], None if what == "recorded" else state[i], *(y[i] for y in x))
