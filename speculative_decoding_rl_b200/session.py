"""Device-resident call objects for the verify-step entry points and the KV commit.

Each object owns the device buffers of one call (inputs copied once with
torch, outputs, workspace) and ``run()`` makes exactly one C-ABI call on the
current torch stream. This is plumbing only: torch allocates memory and
supplies the stream, the library does all the work.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import (PreparedCall, SvAttnDesc, SvKVLayer, SvPagedKV, make_accept_desc, make_cascade_desc, make_kv_layers,
               make_kv_q8, make_kv_q8_layers, make_new_rows, sv_accept, sv_accept_workspace_size,
               sv_cascade_attention_workspace_size, sv_cascade_verify_attention, sv_kv_commit, sv_verify_attention,
               sv_verify_attention_q8_workspace_size, sv_verify_attention_workspace_size)


class AttentionCall:
    def __init__(self, a, device: str = "cuda", out: Optional[torch.Tensor] = None,
                 with_status: bool = True):
        dev = torch.device(device)
        self.inputs = a
        self.desc = SvAttnDesc(a.num_seqs, a.num_q_rows, a.num_q_heads, a.num_kv_heads, a.head_dim,
                               a.block_size, a.max_blocks_per_seq, a.num_blocks)
        self.q = a.q.to(dev)
        self.k_pool = a.k_pool.to(dev)
        self.v_pool = a.v_pool.to(dev)
        self.block_table = a.block_table.to(dev)
        self.ctx_lens = a.ctx_lens.to(dev)
        self.mask = a.draft_mask.to(dev) if a.draft_mask is not None else None
        self.out = out if out is not None else torch.empty_like(self.q)
        self.status = torch.full((a.num_seqs,), -1, dtype=torch.int32, device=dev) if with_status else None
        self.ws_bytes = sv_verify_attention_workspace_size(self.desc)
        self.workspace = torch.empty(max(self.ws_bytes, 256), dtype=torch.uint8, device=dev)
        self.kv = SvPagedKV(self.k_pool.data_ptr(), self.v_pool.data_ptr())

    def run(self, stream=None) -> torch.Tensor:
        sv_verify_attention(self.desc, self.q, self.kv, self.block_table, self.ctx_lens, self.mask,
                            self.out, self.workspace, self.ws_bytes, self.status, stream)
        return self.out

    def kv_bytes(self) -> int:
        return self.inputs.kv_bytes_unique()


class CascadeCall(AttentionCall):
    """sv_cascade_verify_attention over groups of consecutive sequences whose first
    prefix_lens[g] keys sit on the group's first member's pages (default: the
    groups recorded in the inputs)."""

    def __init__(self, a, group_offsets=None, prefix_lens=None, device: str = "cuda",
                 out: Optional[torch.Tensor] = None, with_status: bool = True):
        super().__init__(a, device=device, out=out, with_status=with_status)
        off = a.group_offsets if group_offsets is None else group_offsets
        pre = a.prefix_lens if prefix_lens is None else prefix_lens
        if off is None or pre is None:
            raise ValueError("the inputs carry no groups; pass group_offsets and prefix_lens")
        self.group_offsets, self.prefix_lens = list(off), list(pre)
        self.cdesc = make_cascade_desc(self.group_offsets, self.prefix_lens)
        self.ws_bytes = sv_cascade_attention_workspace_size(self.desc, self.cdesc)
        self.workspace = torch.empty(max(self.ws_bytes, 256), dtype=torch.uint8, device=self.q.device)

    def run(self, stream=None) -> torch.Tensor:
        sv_cascade_verify_attention(self.desc, self.cdesc, self.q, self.kv, self.block_table, self.ctx_lens,
                                    self.mask, self.out, self.workspace, self.ws_bytes, self.status, stream)
        return self.out


class AcceptCall:
    def __init__(self, a, device: str = "cuda", seed: int = 0, with_path: bool = True,
                 with_status: bool = True, temperature: Optional[float] = None):
        dev = torch.device(device)
        self.inputs = a
        self.temperature = a.temperature if temperature is None else float(temperature)
        self.seed = int(seed)
        self.desc = make_accept_desc(a.num_seqs, a.num_rows, a.vocab, a.tree_parents)
        self.logits = a.target_logits.to(dev)
        self.q = a.draft_probs.to(dev)
        self.drafts = a.draft_tokens.to(dev)
        B, N = a.num_seqs, a.num_rows
        self.accept_len = torch.full((B,), -7, dtype=torch.int32, device=dev)
        self.next_token = torch.full((B,), -7, dtype=torch.int32, device=dev)
        self.path = torch.full((B, max(N - 1, 1)), -7, dtype=torch.int32, device=dev) if with_path else None
        self.status = torch.full((B,), -7, dtype=torch.int32, device=dev) if with_status else None
        self.ws_bytes = sv_accept_workspace_size(self.desc)
        self.workspace = torch.empty(max(self.ws_bytes, 256), dtype=torch.uint8, device=dev)

    def run(self, stream=None):
        sv_accept(self.desc, self.logits, self.q if self.q.numel() else None,
                  self.drafts if self.drafts.numel() else None, self.temperature, self.seed,
                  self.accept_len, self.next_token, self.path, self.status, self.workspace, self.ws_bytes,
                  stream)
        return self.accept_len, self.next_token


class CommitCall:
    """KV commit after accept over a fixed set of layers' pools (arguments prepared once)."""

    def __init__(self, desc, layers, block_table, ctx_lens, accept_len, accept_path, device: str = "cuda"):
        dev = torch.device(device)
        B = desc.num_seqs
        self.desc = desc
        self.layers = layers
        self._arr = make_kv_layers(layers)
        self.block_table, self.ctx_lens = block_table, ctx_lens
        self.accept_len, self.accept_path = accept_len, accept_path
        self.new_ctx_lens = torch.empty(B, dtype=torch.int32, device=dev)
        self.status = torch.empty(B, dtype=torch.int32, device=dev)

    def run(self, stream=None):
        sv_kv_commit(self.desc, self._arr, self.block_table, self.ctx_lens, self.accept_len, self.accept_path,
                     self.new_ctx_lens, self.status, stream)
        return self.new_ctx_lens


def _expect(x, name: str, shape, dtype) -> None:
    """The library reads plain contiguous arrays: refuse anything else before its address is taken."""
    if tuple(x.shape) != tuple(shape) or x.dtype != dtype or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}, got {x.dtype} "
                         f"{tuple(x.shape)} with strides {tuple(x.stride())}")


def _expect_cache(desc, kv, q8: bool) -> None:
    pool = (desc.num_blocks, desc.num_kv_heads, desc.block_size, desc.head_dim)
    if len(kv) != (3 if q8 else 2):
        raise ValueError("a layer's cache is (k_pool, v_pool, scales)" if q8 else "a layer's cache is (k_pool, v_pool)")
    for x, name in zip(kv, ("k_pool", "v_pool")):
        _expect(x, name, pool, torch.float8_e4m3fn if q8 else torch.bfloat16)
    if q8:
        _expect(kv[2], "scales", (*pool[:2], 2), torch.float32)


def _expect_lengths(desc, block_table, ctx_lens) -> None:
    _expect(block_table, "block_table", (desc.num_seqs, desc.max_blocks_per_seq), torch.int32)
    _expect(ctx_lens, "ctx_lens", (desc.num_seqs,), torch.int32)


class AppendCall:
    """Rotate the new rows and write them to a layer's bf16 cache (arguments prepared once).

    desc: SvAttnDesc with num_q_rows = N; rope: ``make_rope_desc``; kv: (k_pool, v_pool); q [B][N][Hq][D] or None,
    k and v [B][N][Hkv][D], possibly slices of a fused projection's output, read anew by every run(). q_out is
    allocated unless given. Every tensor is on one device, whose current stream run() uses unless given one."""

    _entry = "sv_kv_append"

    def __init__(self, desc, rope, kv, block_table, ctx_lens, q, k, v, positions=None, new_lens=None,
                 q_out: Optional[torch.Tensor] = None):
        if q is None and q_out is not None:
            raise ValueError("q and q_out go together")
        if tuple(k.shape) != (desc.num_seqs, desc.num_q_rows, desc.num_kv_heads, desc.head_dim) or \
                (q is not None and q.shape[2] != desc.num_q_heads):
            raise ValueError("the new rows' shapes do not match the descriptor")
        _expect_cache(desc, kv, self._entry == "sv_kv_append_q8")
        _expect_lengths(desc, block_table, ctx_lens)
        if q_out is not None:
            _expect(q_out, "q_out", (desc.num_seqs, desc.num_q_rows, desc.num_q_heads, desc.head_dim), torch.bfloat16)
        self.desc, self.rope = desc, rope
        self.rows = make_new_rows(q, k, v, positions, new_lens)
        self.pools, self.kv = kv, self._cache(kv)
        self.block_table, self.ctx_lens = block_table, ctx_lens
        if q is not None and q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        self.q_out = q_out
        self.status = torch.empty(desc.num_seqs, dtype=torch.int32, device=k.device)
        self._call = PreparedCall(self._entry, desc, rope, self.rows, self.kv, block_table, ctx_lens, q_out, self.status,
                                  beside=(q, k, v, positions, new_lens, getattr(rope, "_keep", None), *kv))

    @staticmethod
    def _cache(kv):
        return SvKVLayer(*(x.data_ptr() for x in kv))

    def run(self, stream=None) -> Optional[torch.Tensor]:
        self._call(stream)
        return self.q_out


class AppendQ8Call(AppendCall):
    """AppendCall into a layer's 8-bit cache; kv: (k_pool, v_pool, scales)."""

    _entry = "sv_kv_append_q8"

    @staticmethod
    def _cache(kv):
        return make_kv_q8(*kv)


class AttentionQ8Call:
    """Verify attention over a layer's 8-bit cache; kv: (k_pool, v_pool, scales), q bf16 [B][N][Hq][D]."""

    def __init__(self, desc, kv, block_table, ctx_lens, q, draft_mask=None, out: Optional[torch.Tensor] = None):
        rows = (desc.num_seqs, desc.num_q_rows, desc.num_q_heads, desc.head_dim)
        _expect_cache(desc, kv, True)
        _expect_lengths(desc, block_table, ctx_lens)
        _expect(q, "q", rows, torch.bfloat16)
        if out is not None:
            _expect(out, "out", rows, torch.bfloat16)
        if draft_mask is not None:
            _expect(draft_mask, "draft_mask", rows[:2], torch.int64)
        self.desc = desc
        self.pools, self.kv = kv, make_kv_q8(*kv)
        self.block_table, self.ctx_lens, self.q, self.mask = block_table, ctx_lens, q, draft_mask
        self.out = out if out is not None else torch.empty_like(q)
        self.status = torch.empty(desc.num_seqs, dtype=torch.int32, device=q.device)
        with torch.cuda.device(q.device):
            self.ws_bytes = sv_verify_attention_q8_workspace_size(desc)
        self.workspace = torch.empty(max(self.ws_bytes, 256), dtype=torch.uint8, device=q.device)
        self._call = PreparedCall("sv_verify_attention_q8", desc, q, self.kv, block_table, ctx_lens, draft_mask,
                                  self.out, self.workspace, self.ws_bytes, self.status, beside=kv)

    def run(self, stream=None) -> torch.Tensor:
        self._call(stream)
        return self.out


class CommitQ8Call:
    """KV commit after accept over the 8-bit caches of all layers; layers: (k_pool, v_pool, scales) each, accept_path
    [B][N-1] (one column for N = 1)."""

    def __init__(self, desc, layers, block_table, ctx_lens, accept_len, accept_path):
        for layer in layers:
            _expect_cache(desc, layer, True)
        _expect_lengths(desc, block_table, ctx_lens)
        _expect(accept_len, "accept_len", (desc.num_seqs,), torch.int32)
        _expect(accept_path, "accept_path", (desc.num_seqs, max(desc.num_q_rows - 1, 1)), torch.int32)
        self.desc, self.layers = desc, layers
        self.block_table, self.ctx_lens = block_table, ctx_lens
        self.accept_len, self.accept_path = accept_len, accept_path
        self.new_ctx_lens = torch.empty(desc.num_seqs, dtype=torch.int32, device=ctx_lens.device)
        self.status = torch.empty(desc.num_seqs, dtype=torch.int32, device=ctx_lens.device)
        self._call = PreparedCall("sv_kv_commit_q8", desc, len(layers), make_kv_q8_layers(layers), block_table,
                                  ctx_lens, accept_len, accept_path, self.new_ctx_lens, self.status,
                                  beside=[x for layer in layers for x in layer])

    def run(self, stream=None) -> torch.Tensor:
        self._call(stream)
        return self.new_ctx_lens
