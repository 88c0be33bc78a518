"""Python binding of libsdva, the GB300 verify-step library.

Argument marshalling only: every step of the verify path runs in the CUDA
kernels of ``libsdva.so`` (built in-tree by ``build.py``).  There is no
Python or CPU fallback; importing this package without the built library
raises.  PyTorch supplies device memory and streams.

The calls mirror ``include/sdva.h``:

    kv_append_quant(cache, k_new, v_new, page_table, seq_lens, status=None, stream=None)
    kv_append_quant_ragged(cache, k_new, v_new, n_lane, page_table, seq_lens, status=None, stream=None)
    verify_attn_workspace_size(num_lanes, window, num_q_heads, num_kv_heads, max_context, num_sms=0)
    verify_attn(cache, q, page_table, seq_lens, max_context, sm_scale, out, workspace, status=None, stream=None)
    verify_attn_tree(cache, q, parent, page_table, seq_lens, max_context, sm_scale, out, workspace, status=None,
                     stream=None)
    verify_attn_ragged(cache, q, n_lane, page_table, seq_lens, max_context, sm_scale, out, workspace, status=None,
                       stream=None)
    verify_step(cache, k_new, v_new, q, page_table, seq_lens, max_context, sm_scale, out, workspace, logits, drafts,
                accept_len, out_tokens, commit=True, status=None, stream=None)
    spec_accept(logits, drafts, accept_len, out_tokens, seq_lens_inout=None, status=None, stream=None)
    spec_accept_lazy(logits, drafts, accept_len, out_tokens, num_drafts=None, seq_lens_inout=None, status=None,
                     stream=None)
    spec_accept_tree(logits, tokens, parent, accept_len, path, out_tokens, seq_lens_inout=None, status=None,
                     stream=None)
    spec_accept_sampled_workspace_size(num_lanes, window)
    spec_accept_sampled(logits, draft_probs, drafts, u_accept, u_sample, accept_len, out_tokens, workspace,
                        seq_lens_inout=None, status=None, stream=None)
    kv_append_packed(cache, k_new, v_new, cu_tokens, page_table, seq_lens, status=None, stream=None)
    prompt_attn(q, k, v, cu_tokens, sm_scale, out, lse=None, status=None, stream=None)
    token_logprobs(logits, tokens, logprobs, entropy=None, top_tokens=None, top_logprobs=None, status=None,
                   stream=None)
    kv_append_rope(cache, q, k_new, v_new, rope, page_table, seq_lens, q_out, k_out=None, n_lane=None,
                   positions=None, interleaved=False, status=None, stream=None)
    kv_append_packed_rope(cache, q, k_new, v_new, cu_tokens, rope, page_table, seq_lens, q_out, k_out=None,
                          interleaved=False, status=None, stream=None)
    prompt_delta_workspace_size(total_tokens, num_lanes, num_k_heads, num_v_heads)
    prompt_delta(state, q, k, v, log_decay, beta, cu_tokens, slots, scale, out, workspace, seq_lens=None,
                 qk_eps=1e-6, status=None, stream=None)
    verify_delta(state, q, k, v, log_decay, beta, slots, scale, out, deltas=None, n_lane=None, parent=None,
                 qk_eps=1e-6, status=None, stream=None)
    commit_delta(state, k, log_decay, deltas, slots, accept_len, path=None, status=None, stream=None)
    sdva_status_string(code)
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsdva.so")

KV_FP8_E4M3 = 0
KV_INT4_G32 = 1
KV_INT8_G64 = 2
KV_FP8_ROW = 3
PAGE = 64
HEAD_DIM = 128
MAX_WINDOW = 16

OK = 0
ERR_INVALID = -1
ERR_UNSUPPORTED = -2
ERR_WORKSPACE = -3
ERR_CUDA = -4
STATUS_BAD_PAGE = 1
STATUS_OVERFLOW = 2
STATUS_BAD_DRAFT = 4
STATUS_TIMEOUT = 8
STATUS_BAD_COUNT = 16
STATUS_BAD_TREE = 32
LOGITS_F32 = 0
LOGITS_BF16 = 1
LOGITS_F16 = 2
ROPE_HALVES = 0
ROPE_NEIGHBOURS = 1
MAX_TOP = 32  # SDVA_MAX_TOP: most tokens token_logprobs lists per row
LAZY_WALK_MIN_LANES = 48  # SDVA_LAZY_WALK_MIN_LANES: spec_accept_lazy walks rows from this many lanes on

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()' "
        "or python speculative_decode_verify_append_gb300/build.py)")

_lib = ctypes.CDLL(LIB_PATH)


class _KVCacheStruct(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("k_codes", ctypes.c_void_p),
        ("v_codes", ctypes.c_void_p),
        ("k_scales", ctypes.c_void_p),
        ("v_scales", ctypes.c_void_p),
    ]


_P = ctypes.c_void_p
_I = ctypes.c_int
_lib.kv_append_quant.restype = _I
_lib.kv_append_quant.argtypes = [ctypes.POINTER(_KVCacheStruct), _P, _P, _I, _I, _P, _I, _P, _P, _P]
_lib.kv_append_quant_ragged.restype = _I
_lib.kv_append_quant_ragged.argtypes = [ctypes.POINTER(_KVCacheStruct), _P, _P, _I, _I, _P, _P, _I, _P, _P, _P]
_lib.verify_attn_workspace_size.restype = ctypes.c_size_t
_lib.verify_attn_workspace_size.argtypes = [_I, _I, _I, _I, _I, _I]
_lib.verify_attn.restype = _I
_lib.verify_attn.argtypes = [ctypes.POINTER(_KVCacheStruct), _P, _I, _I, _I, _P, _I, _P, _I, ctypes.c_float, _P,
                             _P, ctypes.c_size_t, _P, _P]
_lib.verify_attn_tree.restype = _I
_lib.verify_attn_tree.argtypes = [ctypes.POINTER(_KVCacheStruct), _P, _I, _I, _I, _P, _P, _I, _P, _I, ctypes.c_float,
                                  _P, _P, ctypes.c_size_t, _P, _P]
_lib.verify_attn_ragged.restype = _I
_lib.verify_attn_ragged.argtypes = [ctypes.POINTER(_KVCacheStruct), _P, _I, _I, _I, _P, _P, _I, _P, _I, ctypes.c_float,
                                    _P, _P, ctypes.c_size_t, _P, _P]
_lib.verify_step.restype = _I
_lib.verify_step.argtypes = [ctypes.POINTER(_KVCacheStruct), _P, _P, _P, _I, _I, _I, _P, _I, _P, _I, ctypes.c_float,
                             _P, _P, ctypes.c_size_t, _P, _I, _P, _P, _P, _I, _P, _P]
_lib.verify_attn_noalloc.restype = _I
_lib.verify_attn_noalloc.argtypes = [ctypes.POINTER(_KVCacheStruct), _P, _I, _I, _I, _P, _I, _P, _I, ctypes.c_float,
                                     _P, _P, _P]
_lib.spec_accept.restype = _I
_lib.spec_accept.argtypes = [_P, _I, _I, _I, _P, _P, _P, _P, _P, _P]
_lib.spec_accept_lazy.restype = _I
_lib.spec_accept_lazy.argtypes = [_P, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P]
_lib.spec_accept_tree.restype = _I
_lib.spec_accept_tree.argtypes = [_P, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P]
_lib.spec_accept_sampled_workspace_size.restype = ctypes.c_size_t
_lib.spec_accept_sampled_workspace_size.argtypes = [_I, _I]
_lib.spec_accept_sampled.restype = _I
_lib.spec_accept_sampled.argtypes = [_P, _P, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P, _P]
_L = ctypes.c_int64
_lib.kv_append_packed.restype = _I
_lib.kv_append_packed.argtypes = [ctypes.POINTER(_KVCacheStruct), _P, _P, _L, _L, _I, _P, _I, _P, _I, _P, _P, _P]
_lib.prompt_attn.restype = _I
_lib.prompt_attn.argtypes = [_P, _P, _P, _L, _L, _L, _I, _I, _I, _P, _I, ctypes.c_float, _P, _P, _P, _P]
_lib.token_logprobs.restype = _I
_lib.token_logprobs.argtypes = [_P, _I, _L, _I, _I, _P, _I, _P, _P, _P, _P, _P, _P]
_F = ctypes.c_float
_lib.kv_append_rope.restype = _I
_lib.kv_append_rope.argtypes = [ctypes.POINTER(_KVCacheStruct), _P, _P, _P, _L, _L, _L, _I, _I, _I, _P, _P, _I, _I, _I,
                                _P, _P, _I, _P, _P, _P, _P, _P]
_lib.kv_append_packed_rope.restype = _I
_lib.kv_append_packed_rope.argtypes = [ctypes.POINTER(_KVCacheStruct), _P, _P, _P, _L, _L, _L, _I, _I, _P, _I, _P, _I,
                                       _I, _I, _P, _I, _P, _P, _P, _P, _P]
_lib.prompt_delta_workspace_size.restype = ctypes.c_size_t
_lib.prompt_delta_workspace_size.argtypes = [_I, _I, _I, _I]
_lib.prompt_delta.restype = _I
_lib.prompt_delta.argtypes = [_P, _I, _P, _P, _P, _L, _L, _L, _P, _P, _I, _I, _I, _P, _I, _P, _P, _F, _F, _P, _P,
                              ctypes.c_size_t, _P, _P]
_lib.verify_delta.restype = _I
_lib.verify_delta.argtypes = [_P, _I, _P, _P, _P, _L, _L, _L, _P, _P, _I, _I, _I, _I, _P, _P, _P, _F, _F, _P, _P, _P, _P]
_lib.commit_delta.restype = _I
_lib.commit_delta.argtypes = [_P, _I, _P, _L, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P]
_lib.sdva_debug_set_wait_limit.restype = ctypes.c_longlong
_lib.sdva_debug_set_wait_limit.argtypes = [ctypes.c_longlong]
_lib.sdva_status_string.restype = ctypes.c_char_p
_lib.sdva_status_string.argtypes = [_I]

EXPORTED = ("kv_append_quant", "kv_append_quant_ragged", "verify_attn_workspace_size", "verify_attn",
            "verify_attn_tree", "verify_attn_ragged", "verify_step", "verify_attn_noalloc", "spec_accept", "spec_accept_lazy", "spec_accept_tree",
            "spec_accept_sampled_workspace_size", "spec_accept_sampled", "kv_append_packed", "prompt_attn",
            "token_logprobs", "kv_append_rope", "kv_append_packed_rope", "prompt_delta_workspace_size", "prompt_delta",
            "verify_delta", "commit_delta", "sdva_debug_set_wait_limit", "sdva_status_string")
NOALLOC_SCRATCH_BYTES = 32 << 20


class SdvaError(RuntimeError):
    def __init__(self, call: str, code: int):
        super().__init__(f"{call}: {sdva_status_string(code)} (code {code})")
        self.code = code


def sdva_debug_set_wait_limit(cycles: int) -> int:
    """Bound every device wait of the tensor-core kernels of verify_attn,
    prompt_attn, prompt_delta and verify_delta and of token_logprobs' kernel for
    long rows at `cycles` clock cycles (negative: the default, about two seconds); returns the
    previous bound.  A wait that runs out raises STATUS_TIMEOUT."""
    return int(_lib.sdva_debug_set_wait_limit(int(cycles)))


def sdva_status_string(code: int) -> str:
    return _lib.sdva_status_string(int(code)).decode()


def _check(call: str, rc: int) -> None:
    if rc != OK:
        raise SdvaError(call, rc)


def _dptr(t: torch.Tensor | None, dtype: torch.dtype | None = None, name: str = "tensor"):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


# The current stream's handle itself, where this build of torch gives it: a
# torch.cuda.Stream object costs a few microseconds.
_current_handle = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int | None:
    if stream is None:
        if _current_handle is None:
            return torch.cuda.current_stream().cuda_stream
        return _current_handle(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


class KVCache:
    """Caller-owned paged KV cache (device tensors in the library's layout).

    FP8:  k_codes/v_codes uint8 [pages][Hkv][64][128]; k_scales/v_scales float32 [pages][Hkv]
    INT4: k_codes/v_codes uint8 [pages][Hkv][64][64];  k_scales/v_scales float16 [pages][Hkv][64][4]
    INT8: k_codes/v_codes uint8 (int8 bits) [pages][Hkv][64][128]; k_scales/v_scales float16 [pages][Hkv][64][2]
    FP8_ROW: k_codes/v_codes uint8 [pages][Hkv][64][128]; k_scales/v_scales float32 [pages][Hkv][64]
    """

    def __init__(self, dtype: int, num_pages: int, num_kv_heads: int, device="cuda", tensors=None):
        self.dtype = int(dtype)
        self.num_pages = int(num_pages)
        self.num_kv_heads = int(num_kv_heads)
        if tensors is not None:
            self.k_codes, self.v_codes, self.k_scales, self.v_scales = tensors
        elif self.dtype == KV_FP8_E4M3:
            shape = (num_pages, num_kv_heads, PAGE, HEAD_DIM)
            self.k_codes = torch.zeros(shape, dtype=torch.uint8, device=device)
            self.v_codes = torch.zeros(shape, dtype=torch.uint8, device=device)
            self.k_scales = torch.zeros((num_pages, num_kv_heads), dtype=torch.float32, device=device)
            self.v_scales = torch.zeros((num_pages, num_kv_heads), dtype=torch.float32, device=device)
        elif self.dtype in (KV_INT4_G32, KV_INT8_G64, KV_FP8_ROW):
            if self.dtype == KV_INT4_G32:
                shape = (num_pages, num_kv_heads, PAGE, HEAD_DIM // 2)
                sshape, sdt = (num_pages, num_kv_heads, PAGE, HEAD_DIM // 32), torch.float16
            elif self.dtype == KV_INT8_G64:
                shape = (num_pages, num_kv_heads, PAGE, HEAD_DIM)
                sshape, sdt = (num_pages, num_kv_heads, PAGE, HEAD_DIM // 64), torch.float16
            else:
                shape = (num_pages, num_kv_heads, PAGE, HEAD_DIM)
                sshape, sdt = (num_pages, num_kv_heads, PAGE), torch.float32
            self.k_codes = torch.zeros(shape, dtype=torch.uint8, device=device)
            self.v_codes = torch.zeros(shape, dtype=torch.uint8, device=device)
            self.k_scales = torch.zeros(sshape, dtype=sdt, device=device)
            self.v_scales = torch.zeros(sshape, dtype=sdt, device=device)
        else:
            raise ValueError(f"unknown kv dtype {dtype}")

    @property
    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.k_codes, self.v_codes, self.k_scales, self.v_scales))

    def struct(self) -> _KVCacheStruct:
        return _KVCacheStruct(self.dtype, self.num_pages, PAGE, self.num_kv_heads, HEAD_DIM,
                              _dptr(self.k_codes, name="k_codes"), _dptr(self.v_codes, name="v_codes"),
                              _dptr(self.k_scales, name="k_scales"), _dptr(self.v_scales, name="v_scales"))


def kv_append_quant(cache: KVCache, k_new: torch.Tensor, v_new: torch.Tensor, page_table: torch.Tensor,
                    seq_lens: torch.Tensor, status: torch.Tensor | None = None, stream=None) -> None:
    """k_new, v_new: bf16 [B][n_new][Hkv][128]; page_table int32 [B][max_pages]; seq_lens int32 [B]."""
    B, n_new = k_new.shape[0], k_new.shape[1]
    s = cache.struct()
    rc = _lib.kv_append_quant(ctypes.byref(s), _dptr(k_new, torch.bfloat16, "k_new"),
                              _dptr(v_new, torch.bfloat16, "v_new"), B, n_new,
                              _dptr(page_table, torch.int32, "page_table"), page_table.shape[1],
                              _dptr(seq_lens, torch.int32, "seq_lens"), _dptr(status, torch.int32, "status"),
                              _stream(stream))
    _check("kv_append_quant", rc)


def kv_append_quant_ragged(cache: KVCache, k_new: torch.Tensor, v_new: torch.Tensor, n_lane: torch.Tensor,
                           page_table: torch.Tensor, seq_lens: torch.Tensor, status: torch.Tensor | None = None,
                           stream=None) -> None:
    """As kv_append_quant; lane b writes only its first n_lane[b] tokens (int32 [B] on the device)."""
    B, n_new = k_new.shape[0], k_new.shape[1]
    if n_lane is None:
        raise ValueError("n_lane is required")
    s = cache.struct()
    rc = _lib.kv_append_quant_ragged(ctypes.byref(s), _dptr(k_new, torch.bfloat16, "k_new"),
                                     _dptr(v_new, torch.bfloat16, "v_new"), B, n_new,
                                     _dptr(n_lane, torch.int32, "n_lane"),
                                     _dptr(page_table, torch.int32, "page_table"), page_table.shape[1],
                                     _dptr(seq_lens, torch.int32, "seq_lens"), _dptr(status, torch.int32, "status"),
                                     _stream(stream))
    _check("kv_append_quant_ragged", rc)


def verify_attn_workspace_size(num_lanes: int, window: int, num_q_heads: int, num_kv_heads: int, max_context: int,
                               num_sms: int = 0) -> int:
    return int(_lib.verify_attn_workspace_size(num_lanes, window, num_q_heads, num_kv_heads, max_context, num_sms))


def verify_attn(cache: KVCache, q: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor,
                max_context: int, sm_scale: float, out: torch.Tensor, workspace: torch.Tensor,
                status: torch.Tensor | None = None, stream=None) -> None:
    """q, out: bf16 [B][W][Hq][128]; workspace: uint8 device tensor of at least
    verify_attn_workspace_size(...) bytes (its contents do not matter)."""
    B, W, Hq = q.shape[0], q.shape[1], q.shape[2]
    s = cache.struct()
    rc = _lib.verify_attn(ctypes.byref(s), _dptr(q, torch.bfloat16, "q"), Hq, B, W,
                          _dptr(page_table, torch.int32, "page_table"), page_table.shape[1],
                          _dptr(seq_lens, torch.int32, "seq_lens"), int(max_context), float(sm_scale),
                          _dptr(out, torch.bfloat16, "out"), _dptr(workspace, None, "workspace"),
                          workspace.numel() * workspace.element_size(), _dptr(status, torch.int32, "status"),
                          _stream(stream))
    _check("verify_attn", rc)


def verify_attn_tree(cache: KVCache, q: torch.Tensor, parent: torch.Tensor | None, page_table: torch.Tensor,
                     seq_lens: torch.Tensor, max_context: int, sm_scale: float, out: torch.Tensor,
                     workspace: torch.Tensor, status: torch.Tensor | None = None, stream=None) -> None:
    """verify_attn over a draft-tree window: parent int32 [B][W] (slot 0 unused);
    row i sees the context and the window keys of its ancestors and itself."""
    B, W, Hq = q.shape[0], q.shape[1], q.shape[2]
    s = cache.struct()
    rc = _lib.verify_attn_tree(ctypes.byref(s), _dptr(q, torch.bfloat16, "q"), Hq, B, W,
                               _dptr(parent, torch.int32, "parent"), _dptr(page_table, torch.int32, "page_table"),
                               page_table.shape[1], _dptr(seq_lens, torch.int32, "seq_lens"), int(max_context),
                               float(sm_scale), _dptr(out, torch.bfloat16, "out"), _dptr(workspace, None, "workspace"),
                               workspace.numel() * workspace.element_size(), _dptr(status, torch.int32, "status"),
                               _stream(stream))
    _check("verify_attn_tree", rc)


def verify_attn_ragged(cache: KVCache, q: torch.Tensor, n_lane: torch.Tensor, page_table: torch.Tensor,
                       seq_lens: torch.Tensor, max_context: int, sm_scale: float, out: torch.Tensor,
                       workspace: torch.Tensor, status: torch.Tensor | None = None, stream=None) -> None:
    """verify_attn with a window row count per lane: n_lane int32 [B]; rows
    past a lane's count are written as zeros."""
    B, W, Hq = q.shape[0], q.shape[1], q.shape[2]
    s = cache.struct()
    rc = _lib.verify_attn_ragged(ctypes.byref(s), _dptr(q, torch.bfloat16, "q"), Hq, B, W,
                                 _dptr(n_lane, torch.int32, "n_lane"), _dptr(page_table, torch.int32, "page_table"),
                                 page_table.shape[1], _dptr(seq_lens, torch.int32, "seq_lens"), int(max_context),
                                 float(sm_scale), _dptr(out, torch.bfloat16, "out"),
                                 _dptr(workspace, None, "workspace"), workspace.numel() * workspace.element_size(),
                                 _dptr(status, torch.int32, "status"), _stream(stream))
    _check("verify_attn_ragged", rc)


def verify_step(cache: KVCache, k_new: torch.Tensor, v_new: torch.Tensor, q: torch.Tensor, page_table: torch.Tensor,
                seq_lens: torch.Tensor, max_context: int, sm_scale: float, out: torch.Tensor, workspace: torch.Tensor,
                logits: torch.Tensor, drafts: torch.Tensor | None, accept_len: torch.Tensor, out_tokens: torch.Tensor,
                commit: bool = True, status: torch.Tensor | None = None, stream=None) -> None:
    """kv_append_quant + verify_attn + spec_accept as one chain of programmatic
    dependent launches (same results as the three calls in order); with commit,
    seq_lens is advanced by 1 + accept_len."""
    B, W, Hq = q.shape[0], q.shape[1], q.shape[2]
    if logits.dim() != 3 or logits.shape[0] != B or logits.shape[1] != W:
        raise ValueError("logits must be [B][W][V]")
    s = cache.struct()
    rc = _lib.verify_step(ctypes.byref(s), _dptr(k_new, torch.bfloat16, "k_new"), _dptr(v_new, torch.bfloat16, "v_new"),
                          _dptr(q, torch.bfloat16, "q"), Hq, B, W, _dptr(page_table, torch.int32, "page_table"),
                          page_table.shape[1], _dptr(seq_lens, torch.int32, "seq_lens"), int(max_context),
                          float(sm_scale), _dptr(out, torch.bfloat16, "out"), _dptr(workspace, None, "workspace"),
                          workspace.numel() * workspace.element_size(), _dptr(logits, torch.float32, "logits"),
                          logits.shape[2], _dptr(drafts, torch.int32, "drafts"),
                          _dptr(accept_len, torch.int32, "accept_len"), _dptr(out_tokens, torch.int32, "out_tokens"),
                          1 if commit else 0, _dptr(status, torch.int32, "status"), _stream(stream))
    _check("verify_step", rc)


def verify_attn_noalloc(cache: KVCache, q: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor,
                        max_context: int, sm_scale: float, out: torch.Tensor, status: torch.Tensor | None = None,
                        stream=None) -> None:
    """verify_attn with the library's fixed device scratch instead of a
    caller workspace (for callers that cannot allocate device memory)."""
    B, W, Hq = q.shape[0], q.shape[1], q.shape[2]
    s = cache.struct()
    rc = _lib.verify_attn_noalloc(ctypes.byref(s), _dptr(q, torch.bfloat16, "q"), Hq, B, W,
                                  _dptr(page_table, torch.int32, "page_table"), page_table.shape[1],
                                  _dptr(seq_lens, torch.int32, "seq_lens"), int(max_context), float(sm_scale),
                                  _dptr(out, torch.bfloat16, "out"), _dptr(status, torch.int32, "status"),
                                  _stream(stream))
    _check("verify_attn_noalloc", rc)


def spec_accept(logits: torch.Tensor, drafts: torch.Tensor | None, accept_len: torch.Tensor,
                out_tokens: torch.Tensor, seq_lens_inout: torch.Tensor | None = None,
                status: torch.Tensor | None = None, stream=None) -> None:
    """logits fp32 [B][W][V]; drafts int32 [B][W-1]; accept_len int32 [B]; out_tokens int32 [B][W]."""
    B, W, V = logits.shape
    rc = _lib.spec_accept(_dptr(logits, torch.float32, "logits"), B, W, V,
                          _dptr(drafts, torch.int32, "drafts") if W > 1 else None,
                          _dptr(accept_len, torch.int32, "accept_len"), _dptr(out_tokens, torch.int32, "out_tokens"),
                          _dptr(seq_lens_inout, torch.int32, "seq_lens_inout"), _dptr(status, torch.int32, "status"),
                          _stream(stream))
    _check("spec_accept", rc)


def spec_accept_lazy(logits: torch.Tensor, drafts: torch.Tensor | None, accept_len: torch.Tensor,
                     out_tokens: torch.Tensor, num_drafts: torch.Tensor | None = None,
                     seq_lens_inout: torch.Tensor | None = None, status: torch.Tensor | None = None,
                     stream=None) -> None:
    """As spec_accept, reading each lane's rows only up to its first disagreement;
    num_drafts int32 [B] (None: W-1 each); out_tokens is -1 after row accept_len."""
    B, W, V = logits.shape
    rc = _lib.spec_accept_lazy(_dptr(logits, torch.float32, "logits"), B, W, V,
                               _dptr(drafts, torch.int32, "drafts") if W > 1 else None,
                               _dptr(num_drafts, torch.int32, "num_drafts"),
                               _dptr(accept_len, torch.int32, "accept_len"),
                               _dptr(out_tokens, torch.int32, "out_tokens"),
                               _dptr(seq_lens_inout, torch.int32, "seq_lens_inout"),
                               _dptr(status, torch.int32, "status"), _stream(stream))
    _check("spec_accept_lazy", rc)


def spec_accept_tree(logits: torch.Tensor, tokens: torch.Tensor | None, parent: torch.Tensor | None,
                     accept_len: torch.Tensor, path: torch.Tensor, out_tokens: torch.Tensor,
                     seq_lens_inout: torch.Tensor | None = None, status: torch.Tensor | None = None,
                     stream=None) -> None:
    """logits fp32 [B][W][V]; tokens, parent int32 [B][W]; accept_len int32 [B];
    path, out_tokens int32 [B][W]."""
    B, W, V = logits.shape
    rc = _lib.spec_accept_tree(_dptr(logits, torch.float32, "logits"), B, W, V,
                               _dptr(tokens, torch.int32, "tokens") if W > 1 else None,
                               _dptr(parent, torch.int32, "parent") if W > 1 else None,
                               _dptr(accept_len, torch.int32, "accept_len"), _dptr(path, torch.int32, "path"),
                               _dptr(out_tokens, torch.int32, "out_tokens"),
                               _dptr(seq_lens_inout, torch.int32, "seq_lens_inout"),
                               _dptr(status, torch.int32, "status"), _stream(stream))
    _check("spec_accept_tree", rc)


def spec_accept_sampled_workspace_size(num_lanes: int, window: int) -> int:
    return int(_lib.spec_accept_sampled_workspace_size(num_lanes, window))


def spec_accept_sampled(logits: torch.Tensor, draft_probs: torch.Tensor | None, drafts: torch.Tensor | None,
                        u_accept: torch.Tensor | None, u_sample: torch.Tensor, accept_len: torch.Tensor,
                        out_tokens: torch.Tensor, workspace: torch.Tensor, seq_lens_inout: torch.Tensor | None = None,
                        status: torch.Tensor | None = None, stream=None) -> None:
    """logits fp32 [B][W][V]; draft_probs fp32 [B][W-1][V]; drafts int32 [B][W-1];
    u_accept fp32 [B][W-1]; u_sample fp32 [B]; workspace: uint8 device tensor of at
    least spec_accept_sampled_workspace_size(B, W) bytes."""
    B, W, V = logits.shape
    rc = _lib.spec_accept_sampled(_dptr(logits, torch.float32, "logits"),
                                  _dptr(draft_probs, torch.float32, "draft_probs") if W > 1 else None, B, W, V,
                                  _dptr(drafts, torch.int32, "drafts") if W > 1 else None,
                                  _dptr(u_accept, torch.float32, "u_accept") if W > 1 else None,
                                  _dptr(u_sample, torch.float32, "u_sample"),
                                  _dptr(accept_len, torch.int32, "accept_len"),
                                  _dptr(out_tokens, torch.int32, "out_tokens"),
                                  _dptr(seq_lens_inout, torch.int32, "seq_lens_inout"),
                                  _dptr(workspace, None, "workspace"), workspace.numel() * workspace.element_size(),
                                  _dptr(status, torch.int32, "status"), _stream(stream))
    _check("spec_accept_sampled", rc)


def _refuse(t, dtype, shape, device: int, name: str) -> None:
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}; the tensors of a call are all on the current device, cuda:{device}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _arg(t: torch.Tensor | None, dtype: torch.dtype, shape: tuple, device: int, name: str):
    """The address of a contiguous tensor of this type and shape on the current device (None: not given)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device or not t.is_contiguous():
        _refuse(t, dtype, shape, device, name)
    return t.data_ptr()


def _status_arg(status: torch.Tensor | None, device: int):
    """The address of a call's status word, on the current device (None: not given)."""
    if status is None:
        return None
    if status.get_device() != device or status.numel() == 0:
        raise ValueError(f"status must be an int32 word on the current device, cuda:{device}; got "
                         f"{status.numel()} on {status.device}")
    return _dptr(status, torch.int32, "status")


def _rows(t: torch.Tensor, shape: tuple, device: int, name: str) -> int:
    """Elements between the token rows of a bf16 [T][H][128] tensor whose rows
    are contiguous inside (a tensor of its own, or a slice of a fused projection)."""
    st = t.stride()
    if (t.dtype is not torch.bfloat16 or t.shape != shape or t.get_device() != device or st[2] != 1 or
            (st[1] != HEAD_DIM and shape[1] > 1)):
        if t.shape == shape and t.dtype is torch.bfloat16 and t.get_device() == device:
            raise ValueError(f"{name} must be contiguous inside a token row")
        _refuse(t, torch.bfloat16, shape, device, name)
    return st[0] if shape[0] > 1 else shape[1] * HEAD_DIM  # of one row the stride means nothing


def kv_append_packed(cache: KVCache, k_new: torch.Tensor, v_new: torch.Tensor, cu_tokens: torch.Tensor,
                     page_table: torch.Tensor, seq_lens: torch.Tensor, status: torch.Tensor | None = None,
                     stream=None) -> None:
    """k_new, v_new: bf16 [T][Hkv][128], token rows of any stride; cu_tokens int32
    [B + 1]: lane b appends rows cu_tokens[b] .. cu_tokens[b + 1] - 1; page_table
    int32 [B][max_pages]; seq_lens int32 [B]."""
    dev = torch.cuda.current_device()
    if k_new.dim() != 3 or v_new.dim() != 3 or page_table.dim() != 2:
        raise ValueError(f"k_new and v_new must be [T][Hkv][{HEAD_DIM}], page_table [B][max_pages]")
    T, B = k_new.shape[0], seq_lens.numel()
    shape = (T, cache.num_kv_heads, HEAD_DIM)
    ks, vs = _rows(k_new, shape, dev, "k_new"), _rows(v_new, shape, dev, "v_new")
    pages = page_table.shape[1]
    s = _cache_on(cache, dev)
    rc = _lib.kv_append_packed(ctypes.byref(s), k_new.data_ptr(), v_new.data_ptr(), ks, vs, T,
                               _arg(cu_tokens, torch.int32, (B + 1,), dev, "cu_tokens"), B,
                               _arg(page_table, torch.int32, (B, pages), dev, "page_table"), pages,
                               _arg(seq_lens, torch.int32, (B,), dev, "seq_lens"),
                               _status_arg(status, dev), _stream(stream))
    _check("kv_append_packed", rc)


def prompt_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_tokens: torch.Tensor, sm_scale: float,
                out: torch.Tensor, lse: torch.Tensor | None = None, status: torch.Tensor | None = None,
                stream=None) -> None:
    """q bf16 [T][Hq][128], k, v bf16 [T][Hkv][128], token rows of any stride;
    cu_tokens int32 [B + 1]; out bf16 [T][Hq][128]; lse fp32 [T][Hq]."""
    dev = torch.cuda.current_device()
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError(f"q, k and v must be [T][H][{HEAD_DIM}]")
    T, Hq, Hkv, B = q.shape[0], q.shape[1], k.shape[1], cu_tokens.numel() - 1
    kv = (T, Hkv, HEAD_DIM)
    qs, ks, vs = _rows(q, (T, Hq, HEAD_DIM), dev, "q"), _rows(k, kv, dev, "k"), _rows(v, kv, dev, "v")
    rc = _lib.prompt_attn(q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, vs, Hq, Hkv, T,
                          _arg(cu_tokens, torch.int32, (B + 1,), dev, "cu_tokens"), B, float(sm_scale),
                          _arg(out, torch.bfloat16, (T, Hq, HEAD_DIM), dev, "out"),
                          _arg(lse, torch.float32, (T, Hq), dev, "lse"),
                          _status_arg(status, dev), _stream(stream))
    _check("prompt_attn", rc)


_LOGITS = {torch.float32: LOGITS_F32, torch.bfloat16: LOGITS_BF16, torch.float16: LOGITS_F16}


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, logprobs: torch.Tensor,
                   entropy: torch.Tensor | None = None, top_tokens: torch.Tensor | None = None,
                   top_logprobs: torch.Tensor | None = None, status: torch.Tensor | None = None, stream=None) -> None:
    """logits fp32, bf16 or fp16 [N][V] (rows of any stride) or contiguous
    [B][W][V]; tokens int32 [N] or [B][W] (-1: row not scored); logprobs,
    entropy fp32 like tokens; top_tokens int32, top_logprobs fp32 with a last
    axis of the number of tokens to list (both or neither)."""
    dev = torch.cuda.current_device()
    kind = _LOGITS.get(logits.dtype)
    if kind is None or logits.get_device() != dev:
        raise ValueError(f"logits must be float32, bfloat16 or float16 on the current device, cuda:{dev}")
    shape = tuple(logits.shape)
    if len(shape) < 2:
        raise ValueError("logits must be [N][V] or contiguous [B][W][V]")
    lead, V = shape[:-1], shape[-1]
    if len(lead) == 1:
        st = logits.stride()
        if st[1] != 1 and V > 1:
            raise ValueError("logits must be contiguous inside a row")
        stride = st[0] if lead[0] > 1 else V
    elif logits.is_contiguous():
        stride = V
    else:
        raise ValueError("logits must be [N][V] or contiguous [B][W][V]")
    if (top_tokens is None) != (top_logprobs is None):
        raise ValueError("top_tokens and top_logprobs go together")
    top = 0 if top_tokens is None else top_tokens.shape[-1]
    rc = _lib.token_logprobs(logits.data_ptr(), kind, stride, math.prod(lead), V,
                             _arg(tokens, torch.int32, lead, dev, "tokens"), top,
                             _arg(logprobs, torch.float32, lead, dev, "logprobs"),
                             _arg(entropy, torch.float32, lead, dev, "entropy"),
                             _arg(top_tokens, torch.int32, lead + (top,), dev, "top_tokens"),
                             _arg(top_logprobs, torch.float32, lead + (top,), dev, "top_logprobs"),
                             _status_arg(status, dev), _stream(stream))
    _check("token_logprobs", rc)


def _window_rows(t: torch.Tensor, shape: tuple, device: int, name: str) -> int:
    """_rows of a bf16 [B][W][H][128] tensor whose B * W token rows are one stride apart."""
    st = t.stride()
    if (t.dtype is not torch.bfloat16 or t.shape != shape or t.get_device() != device or st[3] != 1 or
            (st[2] != HEAD_DIM and shape[2] > 1)):
        if t.shape == shape and t.dtype is torch.bfloat16 and t.get_device() == device:
            raise ValueError(f"{name} must be contiguous inside a token row")
        _refuse(t, torch.bfloat16, shape, device, name)
    if shape[1] == 1:  # of an axis of one the stride means nothing
        return st[0] if shape[0] > 1 else shape[2] * HEAD_DIM
    if shape[0] > 1 and st[0] != shape[1] * st[1]:
        raise ValueError(f"the token rows of {name} must be one stride apart")
    return st[1]


def _cache_on(cache: KVCache, device: int) -> _KVCacheStruct:
    for t in (cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales):
        if t.get_device() != device:
            raise ValueError(f"the cache is on {t.device}, the current device is cuda:{device}")
    return cache.struct()


def kv_append_rope(cache: KVCache, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, rope: torch.Tensor,
                   page_table: torch.Tensor, seq_lens: torch.Tensor, q_out: torch.Tensor,
                   k_out: torch.Tensor | None = None, n_lane: torch.Tensor | None = None,
                   positions: torch.Tensor | None = None, interleaved: bool = False,
                   status: torch.Tensor | None = None, stream=None) -> None:
    """q bf16 [B][W][Hq][128], k_new, v_new bf16 [B][W][Hkv][128], token rows of any
    stride; rope fp32 [positions][rot_dim]: cosines, then sines (step.rope_table);
    page_table int32 [B][max_pages]; seq_lens int32 [B]; q_out, k_out contiguous,
    like q and k_new; n_lane int32 [B]; positions int32 [B][W] (None: seq_lens[b] + i)."""
    dev = torch.cuda.current_device()
    if q.dim() != 4 or k_new.dim() != 4 or v_new.dim() != 4 or page_table.dim() != 2 or rope.dim() != 2:
        raise ValueError(f"q, k_new and v_new must be [B][W][H][{HEAD_DIM}], page_table [B][max_pages], "
                         "rope [positions][rot_dim]")
    B, W, Hq, Hkv, pages = q.shape[0], q.shape[1], q.shape[2], cache.num_kv_heads, page_table.shape[1]
    kv = (B, W, Hkv, HEAD_DIM)
    qs = _window_rows(q, (B, W, Hq, HEAD_DIM), dev, "q")
    ks, vs = _window_rows(k_new, kv, dev, "k_new"), _window_rows(v_new, kv, dev, "v_new")
    s = _cache_on(cache, dev)
    rc = _lib.kv_append_rope(ctypes.byref(s), q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), qs, ks, vs, Hq, B, W,
                             _arg(n_lane, torch.int32, (B,), dev, "n_lane"),
                             _arg(rope, torch.float32, rope.shape, dev, "rope"), rope.shape[0], rope.shape[1],
                             ROPE_NEIGHBOURS if interleaved else ROPE_HALVES,
                             _arg(positions, torch.int32, (B, W), dev, "positions"),
                             _arg(page_table, torch.int32, (B, pages), dev, "page_table"), pages,
                             _arg(seq_lens, torch.int32, (B,), dev, "seq_lens"),
                             _arg(q_out, torch.bfloat16, (B, W, Hq, HEAD_DIM), dev, "q_out"),
                             _arg(k_out, torch.bfloat16, kv, dev, "k_out"), _status_arg(status, dev), _stream(stream))
    _check("kv_append_rope", rc)


def kv_append_packed_rope(cache: KVCache, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                          cu_tokens: torch.Tensor, rope: torch.Tensor, page_table: torch.Tensor,
                          seq_lens: torch.Tensor, q_out: torch.Tensor, k_out: torch.Tensor | None = None,
                          interleaved: bool = False, status: torch.Tensor | None = None, stream=None) -> None:
    """kv_append_packed with the rotation of kv_append_rope: q bf16 [T][Hq][128],
    k_new, v_new bf16 [T][Hkv][128], token rows of any stride; q_out, k_out
    contiguous, like q and k_new."""
    dev = torch.cuda.current_device()
    if q.dim() != 3 or k_new.dim() != 3 or v_new.dim() != 3 or page_table.dim() != 2 or rope.dim() != 2:
        raise ValueError(f"q, k_new and v_new must be [T][H][{HEAD_DIM}], page_table [B][max_pages], "
                         "rope [positions][rot_dim]")
    T, Hq, Hkv, B, pages = q.shape[0], q.shape[1], cache.num_kv_heads, seq_lens.numel(), page_table.shape[1]
    kv = (T, Hkv, HEAD_DIM)
    qs = _rows(q, (T, Hq, HEAD_DIM), dev, "q")
    ks, vs = _rows(k_new, kv, dev, "k_new"), _rows(v_new, kv, dev, "v_new")
    s = _cache_on(cache, dev)
    rc = _lib.kv_append_packed_rope(ctypes.byref(s), q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), qs, ks, vs, Hq, T,
                                    _arg(cu_tokens, torch.int32, (B + 1,), dev, "cu_tokens"), B,
                                    _arg(rope, torch.float32, rope.shape, dev, "rope"), rope.shape[0], rope.shape[1],
                                    ROPE_NEIGHBOURS if interleaved else ROPE_HALVES,
                                    _arg(page_table, torch.int32, (B, pages), dev, "page_table"), pages,
                                    _arg(seq_lens, torch.int32, (B,), dev, "seq_lens"),
                                    _arg(q_out, torch.bfloat16, (T, Hq, HEAD_DIM), dev, "q_out"),
                                    _arg(k_out, torch.bfloat16, kv, dev, "k_out"), _status_arg(status, dev),
                                    _stream(stream))
    _check("kv_append_packed_rope", rc)


def _state(state: torch.Tensor, device: int) -> tuple:
    """The address, slots and heads of a contiguous fp32 [slots][Hv][128][128] pool of states."""
    if state.dim() != 4:
        raise ValueError(f"state must be [slots][Hv][{HEAD_DIM}][{HEAD_DIM}]")
    n, Hv = state.shape[0], state.shape[1]
    return _arg(state, torch.float32, (n, Hv, HEAD_DIM, HEAD_DIM), device, "state"), n, Hv


def prompt_delta_workspace_size(total_tokens: int, num_lanes: int, num_k_heads: int, num_v_heads: int) -> int:
    return int(_lib.prompt_delta_workspace_size(total_tokens, num_lanes, num_k_heads, num_v_heads))


def prompt_delta(state: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                 beta: torch.Tensor, cu_tokens: torch.Tensor, slots: torch.Tensor, scale: float, out: torch.Tensor,
                 workspace: torch.Tensor, seq_lens: torch.Tensor | None = None, qk_eps: float = 1e-6,
                 status: torch.Tensor | None = None, stream=None) -> None:
    """state fp32 [slots][Hv][128][128] (values by keys, in/out); q, k bf16
    [T][Hk][128], v bf16 [T][Hv][128], token rows of any stride; log_decay, beta
    fp32 [T][Hv]; cu_tokens int32 [B + 1]; slots int32 [B]; out bf16 [T][Hv][128];
    workspace: uint8 device tensor of at least prompt_delta_workspace_size(T, B, Hk,
    Hv) bytes; seq_lens int32 [B] (0: the lane starts from zeros)."""
    dev = torch.cuda.current_device()
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError(f"q, k and v must be [T][H][{HEAD_DIM}]")
    p, n, Hv = _state(state, dev)
    T, Hk, B = q.shape[0], q.shape[1], slots.numel()
    qk, vs_ = (T, Hk, HEAD_DIM), (T, Hv, HEAD_DIM)
    qs, ks, vs = _rows(q, qk, dev, "q"), _rows(k, qk, dev, "k"), _rows(v, vs_, dev, "v")
    if workspace.get_device() != dev:
        raise ValueError(f"workspace must be on the current device, cuda:{dev}")
    rc = _lib.prompt_delta(p, n, q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, vs,
                           _arg(log_decay, torch.float32, (T, Hv), dev, "log_decay"),
                           _arg(beta, torch.float32, (T, Hv), dev, "beta"), Hk, Hv, T,
                           _arg(cu_tokens, torch.int32, (B + 1,), dev, "cu_tokens"), B,
                           _arg(slots, torch.int32, (B,), dev, "slots"),
                           _arg(seq_lens, torch.int32, (B,), dev, "seq_lens"), float(scale), float(qk_eps),
                           _arg(out, torch.bfloat16, vs_, dev, "out"), _dptr(workspace, None, "workspace"),
                           workspace.numel() * workspace.element_size(), _status_arg(status, dev), _stream(stream))
    _check("prompt_delta", rc)


def verify_delta(state: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                 beta: torch.Tensor, slots: torch.Tensor, scale: float, out: torch.Tensor,
                 deltas: torch.Tensor | None = None, n_lane: torch.Tensor | None = None,
                 parent: torch.Tensor | None = None, qk_eps: float = 1e-6, status: torch.Tensor | None = None,
                 stream=None) -> None:
    """state fp32 [slots][Hv][128][128] (values by keys); q, k bf16 [B][W][Hk][128],
    v bf16 [B][W][Hv][128], token rows of any stride; log_decay, beta fp32
    [B][W][Hv]; slots int32 [B]; out bf16, deltas fp32 [B][W][Hv][128] (None: the
    window is committed to the state); n_lane int32 [B]; parent int32 [B][W]."""
    dev = torch.cuda.current_device()
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError(f"q, k and v must be [B][W][H][{HEAD_DIM}]")
    p, n, Hv = _state(state, dev)
    B, W, Hk = q.shape[:3]
    qk, vs_, g = (B, W, Hk, HEAD_DIM), (B, W, Hv, HEAD_DIM), (B, W, Hv)
    qs, ks, vs = _window_rows(q, qk, dev, "q"), _window_rows(k, qk, dev, "k"), _window_rows(v, vs_, dev, "v")
    rc = _lib.verify_delta(p, n, q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, vs,
                           _arg(log_decay, torch.float32, g, dev, "log_decay"),
                           _arg(beta, torch.float32, g, dev, "beta"), Hk, Hv, B, W,
                           _arg(n_lane, torch.int32, (B,), dev, "n_lane"),
                           _arg(parent, torch.int32, (B, W), dev, "parent"),
                           _arg(slots, torch.int32, (B,), dev, "slots"), float(scale), float(qk_eps),
                           _arg(out, torch.bfloat16, vs_, dev, "out"), _arg(deltas, torch.float32, vs_, dev, "deltas"),
                           _status_arg(status, dev), _stream(stream))
    _check("verify_delta", rc)


def commit_delta(state: torch.Tensor, k: torch.Tensor, log_decay: torch.Tensor, deltas: torch.Tensor,
                 slots: torch.Tensor, accept_len: torch.Tensor, path: torch.Tensor | None = None,
                 status: torch.Tensor | None = None, stream=None) -> None:
    """state fp32 [slots][Hv][128][128] (in/out); k, log_decay, deltas as verify_delta
    took and wrote them; accept_len int32 [B]; path int32 [B][W] (None: a chain)."""
    dev = torch.cuda.current_device()
    if k.dim() != 4:
        raise ValueError(f"k must be [B][W][Hk][{HEAD_DIM}]")
    p, n, Hv = _state(state, dev)
    B, W, Hk = k.shape[:3]
    ks = _window_rows(k, (B, W, Hk, HEAD_DIM), dev, "k")
    rc = _lib.commit_delta(p, n, k.data_ptr(), ks, _arg(log_decay, torch.float32, (B, W, Hv), dev, "log_decay"),
                           _arg(deltas, torch.float32, (B, W, Hv, HEAD_DIM), dev, "deltas"), Hk, Hv, B, W,
                           _arg(accept_len, torch.int32, (B,), dev, "accept_len"),
                           _arg(path, torch.int32, (B, W), dev, "path"), _arg(slots, torch.int32, (B,), dev, "slots"),
                           _status_arg(status, dev), _stream(stream))
    _check("commit_delta", rc)


def raw_library() -> ctypes.CDLL:
    """The loaded C library (for callers that pass raw pointers themselves)."""
    return _lib
