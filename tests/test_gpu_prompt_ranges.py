"""prompt_attn over the range of its values, in both of its kernels: tiles of
one half (few tiles) and of two.  Each test works out which of them its sizes
select."""
import numpy as np
import pytest
import torch

from gpu_util import SM_SCALE
from test_gpu_prompt import INF, NAN, _attn_ref, _check_attn, _cu, _gen, _qkv, _run_attn

pytestmark = pytest.mark.gpu


def _halves(lens, hq, hkv):
    """Halves to a tile: the call's rule on its sizes (csrc/prompt_attn.cu)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    T = 128 // (hq // hkv)
    return 1 if 20 * (sum(lens) + T * len(lens)) * hkv <= 21 * sms * 2 * T else 2


# (lens, q heads, kv heads, halves): groups of 1, 4, 6 and 7
CASES = [([700], 1, 1, 1), ([700], 4, 1, 1), ([413, 287], 6, 1, 1), ([700], 7, 1, 1),
         ([700], 72, 72, 2), ([700], 72, 18, 2), ([413, 287], 72, 12, 2), ([700], 70, 10, 2)]


@pytest.fixture(params=CASES, ids=[f"{hq}x{hkv}_{n}" for _, hq, hkv, n in CASES])
def sizes(request):
    lens, hq, hkv, n = request.param
    assert _halves(lens, hq, hkv) == n
    return lens, hq, hkv


def _scores_about(x, q, k):
    """Adds x (per row of k) to every score: one channel of q and k is theirs alone."""
    q[:, :, 7] = 4.0
    k[:, :, 7] = (torch.as_tensor(x, device="cuda") / (4.0 * float(SM_SCALE))).to(torch.bfloat16).view(-1, 1)


@pytest.mark.parametrize("score", [0.0, 26.0, -26.0])
@pytest.mark.parametrize("size", [1e-33, 1e28, 1e32])
def test_values_far_from_one(sizes, score, size):
    """Scores of one size, far from 0 or not, and values of any size that a sum
    of a row's keys leaves finite: the output is as large as the values."""
    lens, hq, hkv = sizes
    q, k, v = _qkv(_gen(31), sum(lens), hq, hkv)
    _scores_about(np.full(sum(lens), score, np.float32), q, k)
    _check_attn(q, k, (v.float() * size).to(torch.bfloat16), lens)


@pytest.mark.parametrize("ramp", [(-26.0, 26.0), (26.0, -26.0), (-300.0, 300.0), (0.0, 36.0)])
@pytest.mark.parametrize("size", [1.0, 1e32])
def test_scores_that_rise_and_fall_along_the_row(sizes, ramp, size):
    """References that move in many blocks, and sums that follow them."""
    lens, hq, hkv = sizes
    q, k, v = _qkv(_gen(32), sum(lens), hq, hkv)
    _scores_about(np.concatenate([np.linspace(*ramp, n, dtype=np.float32) for n in lens]), q, k)
    _check_attn(q, k, (v.float() * size).to(torch.bfloat16), lens)


def test_the_same_lane_in_both_kernels(sizes):
    """A row's bits do not depend on what its batch makes of the tiles: each
    lane and kv head alone (one half) and in the batch of both kernels."""
    lens, hq, hkv = sizes
    G = hq // hkv
    q, k, v = _qkv(_gen(33), sum(lens), hq, hkv, fused=True)
    k[:, :, ::32] *= 8.0
    out, lse = _run_attn(q, k, v, _cu(lens))
    assert _halves(lens[:1], G, 1) == 1
    a = 0
    for n in lens:
        for h in {0, hkv // 2, hkv - 1}:
            rows, heads = slice(a, a + n), slice(h * G, (h + 1) * G)
            o, z = _run_attn(q[rows, heads], k[rows, h:h + 1], v[rows, h:h + 1], _cu([n]))
            assert torch.equal(o, out[rows, heads]) and torch.equal(z, lse[rows, heads]), (n, h)
        a += n


@pytest.mark.parametrize("gain", [0.0, 1e-3, 30.0])
def test_flat_and_peaked_scores(sizes, gain):
    lens, hq, hkv = sizes
    q, k, v = _qkv(_gen(34), sum(lens), hq, hkv)
    k = (k * torch.linspace(0.1, 1.0, sum(lens), device="cuda")[:, None, None]).to(torch.bfloat16)
    _check_attn((q * gain).to(torch.bfloat16), k, v, lens)


def test_outlier_channels(sizes):
    lens, hq, hkv = sizes
    q, k, v = _qkv(_gen(35), sum(lens), hq, hkv)
    k[:, :, ::32] *= 16.0
    _check_attn(q, k, v, lens)


def _put(x, row, head, channel, value):
    x = x.clone()
    x[row, head, channel] = value
    return x


@pytest.mark.parametrize("value", [INF, -INF, NAN])
@pytest.mark.parametrize("at", [0, 127, 128, 300, 411, 412])
def test_a_value_that_is_not_finite(sizes, at, value):
    """In V: rows from it on in its lane and kv head have it in that channel
    (their weights are far above what fp32 loses: e^-60 at the least, by the
    scores' size), every other element keeps its bits."""
    lens, hq, hkv = sizes
    q, k, v = _qkv(_gen(36), sum(lens), hq, hkv)
    out0, lse0 = _run_attn(q, k, v, _cu(lens))
    scores = q.float().norm(dim=-1).amax() * k.float().norm(dim=-1).amax() * float(SM_SCALE)
    assert 2 * scores < 60
    out, lse = _run_attn(q, k, _put(v, at, hkv - 1, 77, value), _cu(lens))
    assert torch.equal(lse, lse0)
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[at:lens[0], -(hq // hkv):, 77] = True
    assert torch.equal(out[~hit], out0[~hit])
    assert out[hit].isnan().all() if value != value else (out[hit] == value).all()


def test_opposite_infinities_in_one_channel(sizes):
    lens, hq, hkv = sizes
    q, k, v = _qkv(_gen(37), sum(lens), hq, hkv)
    out0, _ = _run_attn(q, k, v, _cu(lens))
    v[140, 0, 3], v[155, 0, 3] = INF, -INF
    out, _ = _run_attn(q, k, v, _cu(lens))
    c = out[:lens[0], :hq // hkv, 3]
    assert torch.equal(c[:140], out0[:140, :hq // hkv, 3])
    assert (c[140:155] == INF).all() and c[155:].isnan().all()


@pytest.mark.parametrize("at", [0, 60, 128, 390])
@pytest.mark.parametrize("value", [INF, -INF])
def test_a_key_that_is_not_finite(sizes, at, value):
    """An infinity in K makes a row's score of that key +inf, where the row is
    NaN, or -inf, where it is as if the key were not there."""
    lens, hq, hkv = sizes
    G = hq // hkv
    q, k, v = _qkv(_gen(38), sum(lens), hq, hkv)
    out0, lse0 = _run_attn(q, k, v, _cu(lens))
    out, lse = _run_attn(q, _put(k, at, hkv - 1, 5, value), v, _cu(lens))
    sign = q[:, :, 5].float() * (1.0 if value > 0 else -1.0)
    seen = torch.zeros_like(sign, dtype=torch.bool)
    seen[at:lens[0], -G:] = True
    assert torch.equal(out[~seen], out0[~seen]) and torch.equal(lse[~seen], lse0[~seen])
    nan = seen & (sign >= 0)  # 0 * inf is a NaN, too
    assert out[nan].isnan().all() and lse[nan].isnan().all()
    alone = seen & (sign < 0)
    if at == 0:  # row 0 sees no other key
        assert out[0][alone[0]].isnan().all() and (lse[0][alone[0]] == -INF).all()
        alone[0] = False
    # the other keys' sum: the key's score far below what any weight holds
    qq, kk, vv = q[:lens[0], -G:], k[:lens[0], -1:].clone(), v[:lens[0], -1:]
    s = torch.einsum("thd,sd->hts", qq.double(), kk[:, 0].double()) * float(SM_SCALE)
    s[:, torch.ones(s.shape[1:], dtype=torch.bool, device="cuda").triu(1)] = -INF
    s[:, :, at] = -INF
    want_l = s.logsumexp(-1).T
    want = torch.einsum("hts,sd->thd", (s - want_l.T[..., None]).exp().nan_to_num(), vv[:, 0].double())
    _, _, to, tl = _attn_ref(qq, kk, vv, [lens[0]], float(SM_SCALE))
    on = alone[:lens[0], -G:]
    # the bounds of _attn_ref, of a sum without one of its keys: as much larger as the others' weights grow
    more = (lse0[:lens[0], -G:].double() - want_l).exp().clamp(min=1.0)[..., None]
    err, near = (out[:lens[0], -G:].double() - want).abs(), 2.0 ** -8 * want.abs() + to * more
    assert (err <= near)[on].all()
    assert ((lse[:lens[0], -G:].double() - want_l).abs() <= tl + 2.0 ** -20 * (1 + want_l.abs()))[on].all()


def test_first_keys_without_weight(sizes):
    """Scores of -inf over more than the first block: the rows behind weigh
    the other keys alone."""
    lens, hq, hkv = sizes
    q, k, v = _qkv(_gen(39), sum(lens), hq, hkv)
    q[:, :, 0] = 1.0
    k[:150, :, 0] = -INF
    out, lse = _run_attn(q, k, v, _cu(lens))
    assert out[:150].isnan().all() and (lse[:150] == -INF).all()
    n = lens[0]
    want, wl, to, tl = _attn_ref(q[150:n], k[150:n], v[150:n], [n - 150], float(SM_SCALE))
    assert ((out[150:n].double() - want).abs() <= to).all()
    assert ((lse[150:n].double() - wl).abs() <= tl).all()
