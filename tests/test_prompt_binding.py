"""The binding's checks of the prompt calls' devices (no GPU): tensors that say
they are on one, and a library that records what reaches it."""
import types

import pytest
import torch

D = 128


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
def calls(monkeypatch):
    """name -> a call of it with the given status and cache tensors; `calls.reached` lists what got to the library."""
    import __graft_entry__
    __graft_entry__._load_builder().build()
    import speculative_decode_verify_append_gb300 as sdva
    reached = []

    def entry(name):
        def call(*args):
            reached.append((name, args))
            return 0
        return call

    names = ("prompt_attn", "kv_append_packed", "token_logprobs")
    monkeypatch.setattr(sdva, "_lib", types.SimpleNamespace(**{n: entry(n) for n in names}))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(sdva, "_stream", lambda s: 0)

    def bf16(*shape):
        return _on(torch.zeros(shape, dtype=torch.bfloat16))

    def i32(*values):
        return _on(torch.tensor(values, dtype=torch.int32))

    def cache(other=None):
        parts = [_on(torch.zeros((2, 1, 64, D), dtype=torch.uint8), int(other == i)) for i in range(2)]
        parts += [_on(torch.zeros((2, 1)), int(other == i)) for i in (2, 3)]
        return sdva.KVCache(sdva.KV_FP8_E4M3, 2, 1, tensors=parts)

    def prompt_attn(status=None):
        sdva.prompt_attn(bf16(3, 2, D), bf16(3, 1, D), bf16(3, 1, D), i32(0, 3), 0.1, bf16(3, 2, D), None, status)

    def kv_append_packed(status=None, other=None):
        sdva.kv_append_packed(cache(other), bf16(3, 1, D), bf16(3, 1, D), i32(0, 3), _on(i32(0).view(1, 1)), i32(0),
                              status)

    def token_logprobs(status=None):
        sdva.token_logprobs(_on(torch.zeros(2, 9)), i32(1, 2), _on(torch.zeros(2)), status=status)

    return types.SimpleNamespace(prompt_attn=prompt_attn, kv_append_packed=kv_append_packed,
                                 token_logprobs=token_logprobs, reached=reached)


CALLS = ["prompt_attn", "kv_append_packed", "token_logprobs"]


@pytest.mark.parametrize("name", CALLS)
def test_a_status_word_on_the_current_device_reaches_the_call(calls, name):
    status = _on(torch.zeros(1, dtype=torch.int32))
    getattr(calls, name)()
    getattr(calls, name)(status)
    assert [(n, a[-2]) for n, a in calls.reached] == [(name, None), (name, status.data_ptr())]


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("status", [lambda: _on(torch.zeros(1, dtype=torch.int32), 1),
                                    lambda: _on(torch.zeros(0, dtype=torch.int32)),
                                    lambda: _on(torch.zeros(1)),
                                    lambda: torch.zeros(1, dtype=torch.int32)],
                         ids=["other_device", "empty", "float", "cpu"])
def test_any_other_status_word_is_refused(calls, name, status):
    with pytest.raises(ValueError, match="status"):
        getattr(calls, name)(status())
    assert not calls.reached


@pytest.mark.parametrize("part", range(4))
def test_a_cache_with_a_part_on_another_device_is_refused(calls, part):
    calls.kv_append_packed()
    with pytest.raises(ValueError, match="cache"):
        calls.kv_append_packed(other=part)
    assert len(calls.reached) == 1


def test_the_current_stream_with_and_without_its_raw_handle(monkeypatch):
    import __graft_entry__
    __graft_entry__._load_builder().build()
    import speculative_decode_verify_append_gb300 as sdva
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=77))
    monkeypatch.setattr(sdva, "_current_handle", lambda device: 100 + device)
    assert sdva._stream(None) == 103
    monkeypatch.setattr(sdva, "_current_handle", None)
    assert sdva._stream(None) == 77
    assert sdva._stream(5) == 5
