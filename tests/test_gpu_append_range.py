"""Appends at the end of what an int32 position can name."""
import pytest
import torch

from gpu_util import ALL_KV, KV_NAMES

pytestmark = pytest.mark.gpu

LAST = 2 ** 31 - 1
PARTS = ("k_codes", "v_codes", "k_scales", "v_scales")


def _append(call, cache, k, v, table, L, st):
    import speculative_decode_verify_append_gb300 as sdva
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    if call == "packed":
        cu = torch.tensor([0, k.shape[0]], dtype=torch.int32, device="cuda")
        sdva.kv_append_packed(cache, k, v, cu, table, lens, st)
    else:
        sdva.kv_append_quant(cache, k[None], v[None], table, lens, st)
    torch.cuda.synchronize()


@pytest.mark.parametrize("call", ["packed", "quant"])
@pytest.mark.parametrize("kind", ALL_KV, ids=[KV_NAMES[k] for k in ALL_KV])
def test_the_last_positions(kind, call):
    """A lane that ends at position 2^31 - 1 is written as any other; one that
    would go past it is flagged and left, however many pages its row has."""
    import speculative_decode_verify_append_gb300 as sdva
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn((128, 2, 128), generator=g, device="cuda").to(torch.bfloat16) for _ in "kv")
    table = torch.full((1, 2 ** 25 + 2), -1, dtype=torch.int32, device="cuda")
    table[0, -5:] = torch.tensor([3, 1, 4, 2, 0], device="cuda")  # positions 64 (2^25 - 3) and on
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    far, near = sdva.KVCache(kind, 5, 2), sdva.KVCache(kind, 5, 2)
    n = 100
    L = LAST - n
    _append(call, far, k[:n], v[:n], table, L, st)
    _append(call, near, k[:n], v[:n], table[:, L // 64:L // 64 + 2].contiguous(), L % 64, st)
    assert int(st.item()) == 0 and far.k_codes.any()
    for name in PARTS:
        assert torch.equal(getattr(far, name), getattr(near, name)), name
    before = [getattr(far, name).clone() for name in PARTS]
    for L in (LAST - 63, LAST - 127, LAST):
        st.zero_()
        _append(call, far, k, v, table, L, st)
        assert int(st.item()) == sdva.STATUS_OVERFLOW
        assert all(torch.equal(a, getattr(far, name)) for a, name in zip(before, PARTS))
