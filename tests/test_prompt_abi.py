"""Argument checks of prompt_attn, kv_append_packed and token_logprobs (no
GPU): every call below is refused, or found empty, before anything reaches
CUDA, as the header documents."""
import ctypes

import pytest

P, I, L, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
FAKE = 0x1000  # never dereferenced
INVALID, UNSUPPORTED = -1, -2


class _Cache(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("k_codes", P), ("v_codes", P),
                ("k_scales", P), ("v_scales", P)]


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    lib = ctypes.CDLL(__graft_entry__._load_builder().build())
    lib.prompt_attn.argtypes = [P, P, P, L, L, L, I, I, I, P, I, F, P, P, P, P]
    lib.kv_append_packed.argtypes = [P, P, P, L, L, I, P, I, P, I, P, P, P]
    lib.token_logprobs.argtypes = [P, I, L, I, I, P, I, P, P, P, P, P, P]
    return lib


ATTN = dict(q=FAKE, k=FAKE, v=FAKE, qs=512, ks=128, vs=128, hq=4, hkv=1, total=10, cu=FAKE, lanes=1, scale=0.1,
            out=FAKE, lse=None, status=None, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(out=None), INVALID),
    (dict(cu=None), INVALID), (dict(total=-1), INVALID), (dict(lanes=0), INVALID), (dict(hq=0), INVALID),
    (dict(hkv=0), INVALID), (dict(hq=4, hkv=3, ks=384, vs=384), INVALID), (dict(qs=511), INVALID),
    (dict(qs=504), INVALID), (dict(qs=516), INVALID), (dict(ks=120), INVALID), (dict(vs=132), INVALID),
    (dict(q=FAKE + 8), INVALID), (dict(k=FAKE + 2), INVALID), (dict(v=FAKE + 8), INVALID),
    (dict(out=FAKE + 8), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(lanes=1025), UNSUPPORTED),
    (dict(hq=129, qs=129 * 128), UNSUPPORTED), (dict(total=0), 0), (dict(total=0, q=None, cu=None), 0)])
def test_prompt_attn_arguments(lib, change, code):
    assert lib.prompt_attn(*{**ATTN, **change}.values()) == code


def _cache(**change):
    f = dict(dtype=0, num_pages=4, page_size=64, num_kv_heads=1, head_dim=128, k_codes=FAKE, v_codes=FAKE,
             k_scales=FAKE, v_scales=FAKE)
    return _Cache(**{**f, **change})


APPEND = dict(cache=None, k=FAKE, v=FAKE, ks=128, vs=128, total=10, cu=FAKE, lanes=1, table=FAKE, pages=1, lens=FAKE,
              status=None, stream=None)


@pytest.mark.parametrize("cache,change,code", [
    ({}, dict(k=None), INVALID), ({}, dict(v=None), INVALID), ({}, dict(cu=None), INVALID),
    ({}, dict(table=None), INVALID), ({}, dict(lens=None), INVALID), ({}, dict(total=-3), INVALID),
    ({}, dict(lanes=0), INVALID), ({}, dict(pages=0), INVALID), ({}, dict(ks=127), INVALID),
    ({}, dict(ks=120), INVALID), ({}, dict(vs=130), INVALID), ({}, dict(k=FAKE + 8), INVALID),
    ({}, dict(v=FAKE + 2), INVALID), ({}, dict(lanes=65536), UNSUPPORTED), ({}, dict(total=0), 0),
    (dict(head_dim=64), {}, UNSUPPORTED), (dict(page_size=32), {}, UNSUPPORTED), (dict(dtype=4), {}, UNSUPPORTED),
    (dict(k_codes=None), {}, INVALID), (dict(v_scales=FAKE + 4), {}, INVALID), (dict(num_pages=0), {}, INVALID),
    (dict(num_kv_heads=2), {}, INVALID)])
def test_kv_append_packed_arguments(lib, cache, change, code):
    c = _cache(**cache)
    assert lib.kv_append_packed(*{**APPEND, "cache": ctypes.addressof(c), **change}.values()) == code


SCORE = dict(logits=FAKE, dtype=0, stride=100, rows=2, vocab=100, tokens=FAKE, top=5, lp=FAKE, ent=FAKE, tt=FAKE,
             tl=FAKE, status=None, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(logits=None), INVALID), (dict(tokens=None), INVALID), (dict(lp=None), INVALID), (dict(rows=-1), INVALID),
    (dict(vocab=0), INVALID), (dict(stride=99), INVALID), (dict(top=-1), INVALID), (dict(vocab=4), INVALID),
    (dict(tt=None), INVALID), (dict(tl=None), INVALID), (dict(logits=FAKE + 2), INVALID),
    (dict(logits=FAKE + 1, dtype=1), INVALID), (dict(logits=FAKE + 1, dtype=2), INVALID), (dict(top=33), UNSUPPORTED),
    (dict(dtype=3), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED), (dict(rows=0), 0)])
def test_token_logprobs_arguments(lib, change, code):
    assert lib.token_logprobs(*{**SCORE, **change}.values()) == code


def test_constants_match_the_binding(lib):
    import os
    import re

    import speculative_decode_verify_append_gb300 as sdva
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "sdva.h")).read()
    assert int(re.search(r"#define SDVA_MAX_TOP (\d+)", text).group(1)) == sdva.MAX_TOP
    kinds = dict(re.findall(r"SDVA_LOGITS_(\w+) = (\d+)", text))
    assert {k: int(v) for k, v in kinds.items()} == {"F32": 0, "BF16": 1, "F16": 2}
    assert (sdva.LOGITS_F32, sdva.LOGITS_BF16, sdva.LOGITS_F16) == (0, 1, 2)
    assert {"prompt_attn", "kv_append_packed", "token_logprobs"} <= set(sdva.EXPORTED)
