"""One verify step as a user runs it: append the window, attend, accept.

``VerifyStep`` owns the per-shape device buffers (attention output,
split-K workspace, accept outputs, status word) so that a serving loop, or
a CUDA graph capture, issues exactly the three library calls per step with
no allocation.  With ``num_top`` it also owns the buffers of ``score``, which
reports the log probabilities of the step's tokens.  ``PromptStep`` takes a
packed batch of prompts to where the first verify step can follow: attention
over their own keys and values, and the same K/V into the cache.  ``DeltaStep``
owns the states of a recurrent layer and the buffers of its calls.
``fill_context`` writes one lane's prompt K/V into the cache in page-aligned
chunks (the prefill side of the append call).
"""
from __future__ import annotations

import math

import torch

from . import (KVCache, commit_delta, kv_append_packed, kv_append_packed_rope, kv_append_quant, kv_append_quant_ragged,
               kv_append_rope, prompt_attn, prompt_delta, prompt_delta_workspace_size, spec_accept, spec_accept_lazy,
               token_logprobs, verify_attn, verify_attn_workspace_size, verify_delta, verify_step)


class VerifyStep:
    def __init__(self, num_lanes: int, window: int, num_q_heads: int, num_kv_heads: int, max_context: int,
                 vocab: int | None, device="cuda", sm_scale: float | None = None, num_top: int | None = None):
        self.num_lanes, self.window = num_lanes, window
        self.num_q_heads, self.num_kv_heads = num_q_heads, num_kv_heads
        self.max_context, self.vocab = max_context, vocab
        self.sm_scale = sm_scale if sm_scale is not None else 1.0 / math.sqrt(128.0)
        dev = torch.device(device)
        self.out = torch.empty((num_lanes, window, num_q_heads, 128), dtype=torch.bfloat16, device=dev)
        nbytes = verify_attn_workspace_size(num_lanes, window, num_q_heads, num_kv_heads, max_context)
        self.workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
        self.accept_len = torch.zeros(num_lanes, dtype=torch.int32, device=dev)
        self.out_tokens = torch.zeros((num_lanes, window), dtype=torch.int32, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.q = torch.zeros_like(self.out)  # append_rope's queries
        self.num_top = num_top
        if num_top is not None:
            self.logprobs = torch.zeros((num_lanes, window), device=dev)
            self.entropy = torch.zeros((num_lanes, window), device=dev)
            self.top_tokens = torch.zeros((num_lanes, window, num_top), dtype=torch.int32, device=dev)
            self.top_logprobs = torch.zeros((num_lanes, window, num_top), device=dev)

    def append(self, cache: KVCache, k_win, v_win, page_table, seq_lens, stream=None):
        kv_append_quant(cache, k_win, v_win, page_table, seq_lens, self.status, stream)

    def append_ragged(self, cache: KVCache, k_win, v_win, n_lane, page_table, seq_lens, stream=None):
        """Lane b appends only its first n_lane[b] window tokens (its own 1 + d_b)."""
        kv_append_quant_ragged(cache, k_win, v_win, n_lane, page_table, seq_lens, self.status, stream)

    def append_rope(self, cache: KVCache, q, k_win, v_win, rope, page_table, seq_lens, n_lane=None, positions=None,
                    interleaved=False, stream=None):
        """append of a window whose queries and keys are still to be turned to
        their positions (rope: rope_table); returns the turned queries, which
        attend takes and the next call writes again.  Rows of a lane that the
        append skips (status says so) and rows behind a lane's count are not
        written: they hold zeros or an earlier call's."""
        kv_append_rope(cache, q, k_win, v_win, rope, page_table, seq_lens, self.q, None, n_lane, positions, interleaved,
                       self.status, stream)
        return self.q

    def attend(self, cache: KVCache, q, page_table, seq_lens, stream=None):
        verify_attn(cache, q, page_table, seq_lens, self.max_context, self.sm_scale, self.out, self.workspace,
                    self.status, stream)

    def accept(self, logits, drafts, seq_lens_inout=None, stream=None):
        spec_accept(logits, drafts, self.accept_len, self.out_tokens, seq_lens_inout, self.status, stream)

    def accept_lazy(self, logits, drafts, num_drafts=None, seq_lens_inout=None, stream=None):
        """Acceptance reading each lane's rows only up to its first disagreement."""
        spec_accept_lazy(logits, drafts, self.accept_len, self.out_tokens, num_drafts, seq_lens_inout, self.status,
                         stream)

    def score(self, logits, stream=None):
        """Log probability, entropy and the num_top most probable tokens of every
        position of out_tokens: after accept_lazy the accepted tokens and the
        bonus token (the positions behind them hold -1 and are not read)."""
        if self.num_top is None:
            raise ValueError("score() needs num_top")
        lists = (self.top_tokens, self.top_logprobs) if self.num_top else (None, None)
        token_logprobs(logits, self.out_tokens, self.logprobs, self.entropy, *lists, self.status, stream)

    def step(self, cache: KVCache, q, k_win, v_win, page_table, seq_lens, logits, drafts, commit: bool = True,
             stream=None):
        """The whole step in one library call (verify_step): the same results
        as run(), the three calls chained as programmatic dependent launches."""
        verify_step(cache, k_win, v_win, q, page_table, seq_lens, self.max_context, self.sm_scale, self.out,
                    self.workspace, logits, drafts, self.accept_len, self.out_tokens, commit, self.status, stream)

    def run(self, cache: KVCache, q, k_win, v_win, page_table, seq_lens, logits=None, drafts=None,
            commit: bool = True, stream=None):
        """append -> verify_attn -> spec_accept on one stream; seq_lens is
        advanced by 1 + accept_len when commit is true and logits are given."""
        self.append(cache, k_win, v_win, page_table, seq_lens, stream)
        self.attend(cache, q, page_table, seq_lens, stream)
        if logits is not None:
            self.accept(logits, drafts, seq_lens if commit else None, stream)


class PromptStep:
    """A packed batch of whole prompts of up to max_tokens tokens, cu_tokens int32 [B + 1] (device).
    With num_kv_heads, run can turn queries and keys to their positions."""

    def __init__(self, max_tokens: int, num_q_heads: int, device="cuda", sm_scale: float | None = None,
                 num_kv_heads: int | None = None):
        self.sm_scale = sm_scale if sm_scale is not None else 1.0 / math.sqrt(128.0)
        dev = torch.device(device)
        self.out = torch.empty((max_tokens, num_q_heads, 128), dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty((max_tokens, num_q_heads), device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.turned = None  # run's queries and keys with a rope
        if num_kv_heads is not None:
            self.turned = [torch.zeros((max_tokens, n, 128), dtype=torch.bfloat16, device=dev)
                           for n in (num_q_heads, num_kv_heads)]

    def run(self, cache: KVCache, q, k, v, cu_tokens, page_table, seq_lens, stream=None, rope=None, interleaved=False):
        """The prompts' attention (q [T][Hq][128], k, v [T][Hkv][128], bf16), and
        their K/V into the cache behind the seq_lens tokens that each lane
        holds.  Returns out [T][Hq][128] and lse [T][Hq], which the next run
        writes again.  A lane that goes on from cached tokens attends its new
        ones alone here: whole prompts start at seq_lens 0.  With rope (a
        rope_table) the queries and keys are turned to their positions first;
        of a lane that the append skips (status says so) they are not, and its
        out and lse mean nothing."""
        T = q.shape[0]
        out, lse = self.out[:T], self.lse[:T]
        if rope is not None:
            if self.turned is None:
                raise ValueError("run() with a rope needs num_kv_heads")
            turned = [x[:T] for x in self.turned]
            kv_append_packed_rope(cache, q, k, v, cu_tokens, rope, page_table, seq_lens, *turned, interleaved,
                                  self.status, stream)
            prompt_attn(*turned, v, cu_tokens, self.sm_scale, out, lse, self.status, stream)
            return out, lse
        prompt_attn(q, k, v, cu_tokens, self.sm_scale, out, lse, self.status, stream)
        kv_append_packed(cache, k, v, cu_tokens, page_table, seq_lens, self.status, stream)
        return out, lse


class DeltaStep:
    """The recurrent state of one layer (the gated delta rule) of up to num_slots
    lanes, and the buffers of its calls: prompts of up to max_tokens tokens,
    verify windows of `window` rows, plain decode steps.  Lane b of a call has
    the state slots[b]; log_decay and beta are fp32 [rows][Hv]."""

    def __init__(self, num_slots: int, num_k_heads: int, num_v_heads: int, window: int = 1, max_tokens: int = 0,
                 device="cuda", scale: float | None = None, qk_eps: float = 1e-6):
        self.scale = scale if scale is not None else 1.0 / math.sqrt(128.0)
        self.qk_eps, self.window, self.max_tokens = qk_eps, window, max_tokens
        dev = torch.device(device)
        self.state = torch.zeros((num_slots, num_v_heads, 128, 128), device=dev)
        self.out = torch.empty((num_slots, window, num_v_heads, 128), dtype=torch.bfloat16, device=dev)
        self.deltas = torch.empty((num_slots, window, num_v_heads, 128), device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.prompt_out = torch.zeros((max_tokens, num_v_heads, 128), dtype=torch.bfloat16, device=dev)
        nbytes = prompt_delta_workspace_size(max_tokens, num_slots, num_k_heads, num_v_heads) if max_tokens else 0
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)

    def prompt(self, q, k, v, log_decay, beta, cu_tokens, slots, seq_lens=None, stream=None):
        """Packed prompts (q, k [T][Hk][128], v [T][Hv][128]); lanes with seq_lens 0
        start from zeros, the others, and without seq_lens all, go on from what
        their slots hold: a slot that another request had is started with 0.
        Returns out [T][Hv][128], which the next prompt writes again.  Rows of a
        lane that is skipped (status says so) and rows outside the lanes are not
        written: they hold zeros or an earlier call's."""
        out = self.prompt_out[:q.shape[0]]
        prompt_delta(self.state, q, k, v, log_decay, beta, cu_tokens, slots, self.scale, out, self.workspace, seq_lens,
                     self.qk_eps, self.status, stream)
        return out

    def verify(self, q, k, v, log_decay, beta, slots, n_lane=None, parent=None, stream=None):
        """A verify window ([B][W] rows, a chain or a tree): returns out
        [B][W][Hv][128] and records the updates for commit."""
        B = q.shape[0]
        verify_delta(self.state, q, k, v, log_decay, beta, slots, self.scale, self.out[:B], self.deltas[:B], n_lane,
                     parent, self.qk_eps, self.status, stream)
        return self.out[:B]

    def commit(self, k, log_decay, slots, accept_len, path=None, stream=None):
        """The recorded updates of the accepted tokens of the last verify()."""
        commit_delta(self.state, k, log_decay, self.deltas[:k.shape[0]], slots, accept_len, path, self.status, stream)

    def decode(self, q, k, v, log_decay, beta, slots, n_lane=None, stream=None):
        """verify and commit of all rows in one pass ([B][W] rows, W up to the
        window; a plain decode step has one)."""
        B, W = q.shape[:2]
        out = self.out[:B] if W == self.window else self.out.flatten(0, 1)[:B * W].unflatten(0, (B, W))
        verify_delta(self.state, q, k, v, log_decay, beta, slots, self.scale, out, None, n_lane, None, self.qk_eps,
                     self.status, stream)
        return out


def fill_context(cache: KVCache, k: torch.Tensor, v: torch.Tensor, page_table_row: torch.Tensor, start: int = 0,
                 chunk: int = 4096, status: torch.Tensor | None = None, stream=None) -> None:
    """Append tokens [start, start + len(k)) of one lane.  k, v: bf16
    [n][Hkv][128] on the device; page_table_row: int32 [max_pages] (device)."""
    n = k.shape[0]
    dev = k.device
    row = page_table_row.reshape(1, -1)
    t = 0
    while t < n:
        c = min(chunk - ((start + t) % chunk), n - t)
        lens = torch.tensor([start + t], dtype=torch.int32, device=dev)
        kv_append_quant(cache, k[t:t + c].unsqueeze(0).contiguous(), v[t:t + c].unsqueeze(0).contiguous(), row,
                        lens, status, stream)
        t += c


def rope_table(num_positions: int, rot_dim: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """The cosines and sines of positions 0 .. num_positions - 1 that
    kv_append_rope takes, fp32 [num_positions][rot_dim]: pair i turns by
    position * base^(-2 i / rot_dim).  The angles are taken in 64 bits: at
    position 240,000 an fp32 angle is off by up to 2^-7."""
    rate = base ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    angle = torch.arange(num_positions, dtype=torch.float64, device=device)[:, None] * rate
    return torch.cat([angle.cos(), angle.sin()], 1).float()
