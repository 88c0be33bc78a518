"""token_logprobs' long rows, many (a block per row) and few (a cluster per
row), where their fast paths do not hold: forbidden tokens, ties beyond the
candidates' places, rows with fewer finite logits than tokens to list, rows
without a distribution."""
import pytest
import torch

from test_gpu_prompt import DTYPES, INF, NAN, _check_scores, _gen, _logits, _order, _score, _status

pytestmark = pytest.mark.gpu


def _uniform(g, n, V):
    return torch.rand((n, V), generator=g, device="cuda")


def _forbidden(g, x):
    """Nine tokens in ten, then all but a few, at places from the row's start to its end."""
    n, V = x.shape
    r = _uniform(g, n, V)
    x[r < 0.9] = -INF
    x[1::4][r[1::4] < 0.9999] = -INF
    x[2::4] = -INF
    x[2::4, ::V // 7] = 1.0  # eight finite logits
    x[:, V // 2] = 0.5
    return x


def _tied(g, x):
    """A few values only, one value only, and a row's largest value thousands of times."""
    x = (x * 2).round() / 2
    x[1::3] = 0.25
    x[2::3, 5::9] = 20.0
    return x


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,V", [(200, 40000), (200, 40003), (330, 33001), (6, 70001)])
@pytest.mark.parametrize("make", [_forbidden, _tied])
def test_forbidden_and_tied_logits(dtype, n, V, make):
    g = _gen(n + V)
    x = make(g, _logits(g, n, V, torch.float32)).to(dtype)
    tokens = torch.randint(V, (n,), generator=g, device="cuda", dtype=torch.int32)
    tokens[::2] = V // 2
    for top in (0, 5, 32):
        _check_scores(x, tokens, top)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [200, 6])
def test_rows_without_a_distribution_among_others(dtype, n):
    """A NaN (in the first and the last vector, and single), +inf, all -inf:
    NaN in those rows, the list in order, and the others' bits as without them."""
    g = _gen(n)
    V = 40000
    x = _logits(g, n, V, dtype)
    x[3::7, ::2] = -INF
    tokens = torch.randint(V, (n,), generator=g, device="cuda", dtype=torch.int32)
    good = _score(x, tokens, 20)
    bad = torch.zeros(n, dtype=torch.bool, device="cuda")
    for i, (at, value) in enumerate(((0, NAN), (V - 1, NAN), (V // 2, INF), (slice(0, V), -INF), (slice(9, V), NAN))):
        x[i::50, at] = value
        bad[i::50] = True
    st = _status()
    lp, en, tt, tl = _score(x, tokens, 20, st)
    assert int(st.item()) == 0
    assert lp[bad].isnan().all() and en[bad].isnan().all() and tl[bad].isnan().all()
    assert torch.equal(tt, _order(x, 20).to(torch.int32))
    for got, want in zip((lp, en, tt, tl), good):
        assert torch.equal(got[~bad], want[~bad])
