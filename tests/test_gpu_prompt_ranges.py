"""prompt_attn over the range of its values, in both of its kernels: tiles of
one half (few tiles) and of two.  Each test works out which of them its sizes
select."""
import numpy as np
import pytest
import torch

from gpu_util import SM_SCALE
from test_gpu_prompt import _check_attn, _gen, _qkv

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
