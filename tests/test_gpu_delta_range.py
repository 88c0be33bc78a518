"""The gated delta rule where its values range widely."""
import pytest
import torch

from test_gpu_delta import D, EPS, SCALE, _gen, _i32, _workspace

pytestmark = pytest.mark.gpu


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
    return q.to(torch.bfloat16), k.to(torch.bfloat16).contiguous(), v.to(torch.bfloat16), gd, b, eps


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
