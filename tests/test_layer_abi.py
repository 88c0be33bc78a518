"""Argument checks of the rotated appends and of the gated delta rule's calls (no
GPU): every call below is refused, or found empty, before anything reaches
CUDA, as the header documents; and the binding's checks of devices and rows."""
import ctypes
import types

import pytest
import torch

P, I, L, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
FAKE = 0x1000  # never dereferenced
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
NAN, INF = float("nan"), float("inf")


class _Cache(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("k_codes", P), ("v_codes", P),
                ("k_scales", P), ("v_scales", P)]


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    lib = ctypes.CDLL(__graft_entry__._load_builder().build())
    lib.kv_append_rope.argtypes = [P, P, P, P, L, L, L, I, I, I, P, P, I, I, I, P, P, I, P, P, P, P, P]
    lib.kv_append_packed_rope.argtypes = [P, P, P, P, L, L, L, I, I, P, I, P, I, I, I, P, I, P, P, P, P, P]
    lib.prompt_delta_workspace_size.argtypes, lib.prompt_delta_workspace_size.restype = [I, I, I, I], Z
    lib.prompt_delta.argtypes = [P, I, P, P, P, L, L, L, P, P, I, I, I, P, I, P, P, F, F, P, P, Z, P, P]
    lib.verify_delta.argtypes = [P, I, P, P, P, L, L, L, P, P, I, I, I, I, P, P, P, F, F, P, P, P, P]
    lib.commit_delta.argtypes = [P, I, P, L, P, P, I, I, I, I, P, P, P, P, P]
    return lib


def _cache(**change):
    f = dict(dtype=0, num_pages=4, page_size=64, num_kv_heads=1, head_dim=128, k_codes=FAKE, v_codes=FAKE,
             k_scales=FAKE, v_scales=FAKE)
    return _Cache(**{**f, **change})


ROPE = dict(cache=None, q=FAKE, k=FAKE, v=FAKE, qs=512, ks=128, vs=128, hq=4, lanes=2, n=3, n_lane=None, rope=FAKE,
            far=100, rot=128, pairing=0, positions=None, table=FAKE, pages=1, lens=FAKE, q_out=FAKE, k_out=None,
            status=None, stream=None)
PACKED = dict(cache=None, q=FAKE, k=FAKE, v=FAKE, qs=512, ks=128, vs=128, hq=4, total=10, cu=FAKE, lanes=2, rope=FAKE,
              far=100, rot=128, pairing=0, table=FAKE, pages=1, lens=FAKE, q_out=FAKE, k_out=None, status=None,
              stream=None)
BOTH = [
    ({}, dict(q=None), INVALID), ({}, dict(k=None), INVALID), ({}, dict(v=None), INVALID), ({}, dict(rope=None), INVALID),
    ({}, dict(q_out=None), INVALID), ({}, dict(table=None), INVALID), ({}, dict(lens=None), INVALID),
    ({}, dict(lanes=0), INVALID), ({}, dict(pages=0), INVALID), ({}, dict(far=0), INVALID), ({}, dict(hq=0), INVALID),
    (dict(num_kv_heads=3), dict(ks=384, vs=384), INVALID), ({}, dict(qs=511), INVALID), ({}, dict(qs=504), INVALID),
    ({}, dict(ks=120), INVALID), ({}, dict(vs=132), INVALID), ({}, dict(q=FAKE + 8), INVALID),
    ({}, dict(k=FAKE + 2), INVALID), ({}, dict(v=FAKE + 8), INVALID), ({}, dict(rope=FAKE + 4), INVALID),
    ({}, dict(q_out=FAKE + 8), INVALID), ({}, dict(k_out=FAKE + 8), INVALID), ({}, dict(rot=48), UNSUPPORTED),
    ({}, dict(rot=0), UNSUPPORTED), ({}, dict(rot=256), UNSUPPORTED), ({}, dict(pairing=2), UNSUPPORTED),
    ({}, dict(pairing=-1), UNSUPPORTED), ({}, dict(lanes=65536), UNSUPPORTED),
    (dict(head_dim=64), {}, UNSUPPORTED), (dict(page_size=32), {}, UNSUPPORTED), (dict(dtype=4), {}, UNSUPPORTED),
    (dict(k_codes=None), {}, INVALID), (dict(v_scales=FAKE + 4), {}, INVALID), (dict(num_pages=0), {}, INVALID)]


@pytest.mark.parametrize("cache,change,code", BOTH + [
    ({}, dict(n=0), INVALID), ({}, dict(n=-1), INVALID), ({}, dict(n=2 ** 31 - 1, lanes=65535), UNSUPPORTED)])
def test_kv_append_rope_arguments(lib, cache, change, code):
    c = _cache(**cache)
    assert lib.kv_append_rope(*{**ROPE, "cache": ctypes.addressof(c), **change}.values()) == code
    assert lib.kv_append_rope(*{**ROPE, **change}.values()) == INVALID  # no cache


@pytest.mark.parametrize("cache,change,code", BOTH + [
    ({}, dict(cu=None), INVALID), ({}, dict(total=-1), INVALID), ({}, dict(total=0), 0),
    ({}, dict(total=0, q=None, cu=None), 0)])
def test_kv_append_packed_rope_arguments(lib, cache, change, code):
    c = _cache(**cache)
    assert lib.kv_append_packed_rope(*{**PACKED, "cache": ctypes.addressof(c), **change}.values()) == code


DELTA = [
    (dict(state=None), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(g=None), INVALID), (dict(beta=None), INVALID), (dict(slots=None), INVALID), (dict(out=None), INVALID),
    (dict(num=0), INVALID), (dict(hk=0), INVALID), (dict(hv=0), INVALID), (dict(hk=3, qs=384, ks=384), INVALID),
    (dict(lanes=0), INVALID), (dict(lanes=65536), UNSUPPORTED), (dict(hv=65536, vs=65536 * 128), UNSUPPORTED),
    (dict(qs=255), INVALID), (dict(qs=248), INVALID), (dict(ks=260), INVALID), (dict(vs=504), INVALID),
    (dict(q=FAKE + 8), INVALID), (dict(k=FAKE + 2), INVALID), (dict(v=FAKE + 8), INVALID),
    (dict(state=FAKE + 4), INVALID), (dict(out=FAKE + 8), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID), (dict(eps=NAN), INVALID),
    (dict(eps=INF), INVALID)]
PROMPT = dict(state=FAKE, num=4, q=FAKE, k=FAKE, v=FAKE, qs=256, ks=256, vs=512, g=FAKE, beta=FAKE, hk=2, hv=4,
              total=10, cu=FAKE, lanes=2, slots=FAKE, seq=None, scale=0.1, eps=1e-6, out=FAKE, ws=FAKE, bytes=1 << 40,
              status=None, stream=None)


@pytest.mark.parametrize("change,code", DELTA + [
    (dict(cu=None), INVALID), (dict(total=-1), INVALID), (dict(total=0), 0), (dict(total=0, state=None, q=None), 0),
    (dict(ws=None), WORKSPACE), (dict(ws=FAKE + 128), WORKSPACE), (dict(bytes=0), WORKSPACE)])
def test_prompt_delta_arguments(lib, change, code):
    assert lib.prompt_delta(*{**PROMPT, **change}.values()) == code


def test_prompt_delta_workspace(lib):
    f = lib.prompt_delta_workspace_size
    assert f(10, 2, 2, 4) > 0
    assert f(0, 2, 2, 4) == f(10, 0, 2, 4) == f(10, 2, 0, 4) == f(10, 2, 3, 4) == f(-1, 1, 1, 1) == 0
    assert f(1 << 20, 4, 16, 32) >= f(1 << 10, 4, 16, 32)
    short = {**PROMPT, "bytes": f(10, 2, 2, 4) - 1}
    assert lib.prompt_delta(*short.values()) == WORKSPACE


VERIFY = dict(state=FAKE, num=4, q=FAKE, k=FAKE, v=FAKE, qs=256, ks=256, vs=512, g=FAKE, beta=FAKE, hk=2, hv=4,
              lanes=2, window=3, n_lane=None, parent=None, slots=FAKE, scale=0.1, eps=1e-6, out=FAKE, deltas=FAKE,
              status=None, stream=None)


@pytest.mark.parametrize("change,code", DELTA + [
    (dict(window=0), INVALID), (dict(window=17), UNSUPPORTED), (dict(deltas=FAKE + 8), INVALID),
    (dict(parent=FAKE, deltas=None), INVALID)])
def test_verify_delta_arguments(lib, change, code):
    assert lib.verify_delta(*{**VERIFY, **change}.values()) == code


COMMIT = dict(state=FAKE, num=4, k=FAKE, ks=256, g=FAKE, deltas=FAKE, hk=2, hv=4, lanes=2, window=3, acc=FAKE,
              path=None, slots=FAKE, status=None, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(state=None), INVALID), (dict(k=None), INVALID), (dict(g=None), INVALID), (dict(deltas=None), INVALID),
    (dict(acc=None), INVALID), (dict(slots=None), INVALID), (dict(num=0), INVALID), (dict(hk=0), INVALID),
    (dict(hk=3, ks=384), INVALID), (dict(ks=248), INVALID), (dict(k=FAKE + 8), INVALID), (dict(window=0), INVALID),
    (dict(deltas=FAKE + 8), INVALID), (dict(state=FAKE + 8), INVALID), (dict(window=17), UNSUPPORTED),
    (dict(lanes=65536), UNSUPPORTED), (dict(hv=65536), UNSUPPORTED)])
def test_commit_delta_arguments(lib, change, code):
    assert lib.commit_delta(*{**COMMIT, **change}.values()) == code


def test_constants_match_the_binding(lib):
    import os
    import re

    import speculative_decode_verify_append_gb300 as sdva
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "sdva.h")).read()
    assert dict(re.findall(r"SDVA_ROPE_(\w+) = (\d+)", text)) == {"HALVES": "0", "NEIGHBOURS": "1"}
    assert (sdva.ROPE_HALVES, sdva.ROPE_NEIGHBOURS) == (0, 1)
    assert {"kv_append_rope", "kv_append_packed_rope", "prompt_delta_workspace_size", "prompt_delta", "verify_delta",
            "commit_delta"} <= set(sdva.EXPORTED)


class _OnGpu(torch.Tensor):
    gpu = 0

    def get_device(self):
        return self.gpu

    @property
    def is_cuda(self):
        return True


def _on(t, gpu=0):
    t = t.as_subclass(_OnGpu)
    t.gpu = gpu
    return t


@pytest.fixture
def calls(monkeypatch, lib):
    """name -> (the call, its arguments), on a library that records what reaches it."""
    import speculative_decode_verify_append_gb300 as sdva
    reached = []

    def entry(name):
        return lambda *args: reached.append((name, args)) or 0

    names = ("kv_append_rope", "kv_append_packed_rope", "prompt_delta", "verify_delta", "commit_delta")
    monkeypatch.setattr(sdva, "_lib", types.SimpleNamespace(**{n: entry(n) for n in names}))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(sdva, "_stream", lambda s: 0)

    def bf16(*shape):
        return _on(torch.zeros(shape, dtype=torch.bfloat16))

    def f32(*shape):
        return _on(torch.zeros(shape))

    def i32(*shape):
        return _on(torch.zeros(shape, dtype=torch.int32))

    cache = sdva.KVCache(sdva.KV_FP8_E4M3, 2, 1, tensors=[_on(torch.zeros((2, 1, 64, 128), dtype=torch.uint8)) for _ in range(2)] +
                         [f32(2, 1), f32(2, 1)])
    rope = dict(cache=cache, rope=f32(9, 64), page_table=i32(2, 1), seq_lens=i32(2))
    delta = dict(state=f32(3, 2, 128, 128), slots=i32(2), scale=0.1)
    made = {
        "kv_append_rope": dict(rope, q=bf16(2, 3, 2, 128), k_new=bf16(2, 3, 1, 128), v_new=bf16(2, 3, 1, 128),
                               q_out=bf16(2, 3, 2, 128), k_out=bf16(2, 3, 1, 128), n_lane=i32(2), positions=i32(2, 3)),
        "kv_append_packed_rope": dict(rope, q=bf16(5, 2, 128), k_new=bf16(5, 1, 128), v_new=bf16(5, 1, 128), cu_tokens=i32(3),
                                      q_out=bf16(5, 2, 128), k_out=bf16(5, 1, 128)),
        "prompt_delta": dict(delta, q=bf16(5, 1, 128), k=bf16(5, 1, 128), v=bf16(5, 2, 128), log_decay=f32(5, 2),
                             beta=f32(5, 2), cu_tokens=i32(3), out=bf16(5, 2, 128), seq_lens=i32(2),
                             workspace=_on(torch.zeros(512, dtype=torch.uint8))),
        "verify_delta": dict(delta, q=bf16(2, 3, 1, 128), k=bf16(2, 3, 1, 128), v=bf16(2, 3, 2, 128), log_decay=f32(2, 3, 2),
                             beta=f32(2, 3, 2), out=bf16(2, 3, 2, 128), deltas=f32(2, 3, 2, 128), n_lane=i32(2),
                             parent=i32(2, 3)),
        "commit_delta": dict(state=delta["state"], slots=i32(2), k=bf16(2, 3, 1, 128), log_decay=f32(2, 3, 2),
                             deltas=f32(2, 3, 2, 128), accept_len=i32(2), path=i32(2, 3)),
    }
    return types.SimpleNamespace(args=made, reached=reached,
                                 call=lambda name, **change: getattr(sdva, name)(**{**made[name], **change}))


NAMES = ["kv_append_rope", "kv_append_packed_rope", "prompt_delta", "verify_delta", "commit_delta"]


@pytest.mark.parametrize("name", NAMES)
def test_every_tensor_is_checked_for_its_device_type_and_shape(calls, name):
    status = _on(torch.zeros(1, dtype=torch.int32))
    calls.call(name, status=status)
    assert len(calls.reached) == 1 and calls.reached[0][1][-2] == status.data_ptr()
    for key, t in calls.args[name].items():
        if not isinstance(t, torch.Tensor):
            continue
        bad = [_on(t.as_subclass(torch.Tensor).clone(), 1)]
        if key != "workspace":
            bad.append(_on(t.as_subclass(torch.Tensor).double()))
        if key not in ("workspace", "rope", "state"):  # of these the library refuses an empty one
            bad.append(_on(t.as_subclass(torch.Tensor)[:0]))
        for x in bad:
            with pytest.raises(ValueError):
                calls.call(name, **{key: x})
    for s in (_on(torch.zeros(1, dtype=torch.int32), 1), _on(torch.zeros(0, dtype=torch.int32)), _on(torch.zeros(1))):
        with pytest.raises(ValueError):
            calls.call(name, status=s)
    assert len(calls.reached) == 1


@pytest.mark.parametrize("name,key", [("kv_append_rope", "q"), ("kv_append_rope", "v_new"), ("verify_delta", "k"),
                                      ("verify_delta", "v"), ("commit_delta", "k")])
def test_window_rows_are_one_stride_apart(calls, name, key):
    t = calls.args[name][key].as_subclass(torch.Tensor)
    B, W, H, D = t.shape
    wide = torch.zeros((B, W, H + 3, D), dtype=t.dtype)
    calls.call(name, **{key: _on(wide[:, :, 1:1 + H])})  # slices of a fused projection
    calls.call(name, **{key: _on(torch.zeros((B, W, H, D), dtype=t.dtype))})
    for bad in (torch.zeros((B, W + 1, H, D), dtype=t.dtype)[:, :W], torch.zeros((B, W, H, 2 * D), dtype=t.dtype)[..., ::2],
                torch.zeros((W, B, H, D), dtype=t.dtype).transpose(0, 1)):
        with pytest.raises(ValueError):
            calls.call(name, **{key: _on(bad)})
