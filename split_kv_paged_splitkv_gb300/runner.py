"""Convenience wrappers: plans, torch-allocated workspaces and outputs.

Marshalling only -- torch allocates device memory and provides the stream;
the computation is in libsplitkv.  ``DecodeSession`` is one decode over given
caches; ``CacheSession`` holds a paged cache through its life: append, decode,
weigh, evict, cross attention.
"""
from __future__ import annotations

import contextlib

import torch

from . import (SPLITKV_BF16, SPLITKV_COMBINE_SEPARATE, SPLITKV_FP8_E4M3, SPLITKV_LAYOUT_HND,
               SPLITKV_LAYOUT_NHD, make_desc, splitkv_combine_workspace, splitkv_decode,
               splitkv_decode_partials,
               splitkv_decode_kv_scales, splitkv_plan, splitkv_plan_fixed,
               splitkv_plan_upload, splitkv_read_stats, splitkv_append,
               splitkv_cross_attend, splitkv_cross_workspace_size, splitkv_evict,
               splitkv_evict_workspace_size, splitkv_key_weights, SPLITKV_EUNSUPPORTED,
               SplitKVError)


class DecodeSession:
    """Holds a plan and its uploaded workspace for one set of KV-cache tensors.

    ``q`` bf16 [B][T][Hq][Dk]; ``k_pages`` bf16 or uint8 (e4m3 codes)
    [N][Hkv][P][Dk] (``kv_layout`` HND) or [N][P][Hkv][Dk] (NHD); ``v_pages``
    likewise or None with ``v_shares_k``;
    ``block_table`` int32 [B][max_pages]; ``seq_lens`` int32 [B] on the device
    and ``seq_lens_host`` the same values on the host.
    """

    def __init__(self, q, k_pages, v_pages, block_table, seq_lens, seq_lens_host, *, scale,
                 kv_scale=1.0, num_splits=0, num_sms=0, v_dim=None, v_shares_k=False,
                 combine_mode=SPLITKV_COMBINE_SEPARATE, stream=None, k_scale=None, v_scale=None,
                 fixed=False, kv_layout=SPLITKV_LAYOUT_HND):
        B, T, Hq, Dk = q.shape
        if kv_layout == SPLITKV_LAYOUT_NHD:
            N, P, Hkv, _ = k_pages.shape
        else:
            N, Hkv, P, _ = k_pages.shape
        if v_dim is None:
            v_dim = Dk if v_pages is None else v_pages.shape[3]
        fp8 = k_pages.dtype == torch.uint8
        self.desc = make_desc(B, T, Hq, Hkv, Dk, v_dim, P, block_table.shape[1], N,
                              SPLITKV_FP8_E4M3 if fp8 else SPLITKV_BF16, int(v_shares_k),
                              combine_mode, kv_layout)
        # fixed: a capacity plan (num_splits items per sequence and head group)
        # whose kernels derive every item from the current device seq_lens,
        # so one captured CUDA graph serves any lengths
        self.fixed = fixed
        self.plan = (splitkv_plan_fixed(self.desc, num_splits) if fixed else
                     splitkv_plan(self.desc, seq_lens_host, num_splits, num_sms))
        self.num_splits = num_splits
        dev = q.device
        self.workspace = torch.empty(max(self.plan.workspace_size, 256), dtype=torch.uint8, device=dev)
        self.stream = stream
        splitkv_plan_upload(self.plan, self.workspace, self.workspace.numel(), stream)
        self.tensors = (q, k_pages, v_pages, block_table, seq_lens)
        self.scale, self.kv_scale = float(scale), float(kv_scale)
        self.k_scale, self.v_scale = k_scale, v_scale  # per-KV-head e4m3 scales, or None
        self.out = torch.empty((B, T, Hq, v_dim), dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty((B, T, Hq), dtype=torch.float32, device=dev)

    def run(self, out=None, lse=None, tensors=None):
        q, k, v, table, lens = tensors if tensors is not None else self.tensors
        o = self.out if out is None else out
        l = self.lse if lse is None else lse
        if self.k_scale is not None:
            splitkv_decode_kv_scales(self.plan, self.workspace, q, k, v, table, lens,
                                     self.num_splits, self.scale, self.k_scale, self.v_scale, o, l,
                                     self.stream)
        else:
            splitkv_decode(self.plan, self.workspace, q, k, v, table, lens, self.num_splits,
                           self.scale, self.kv_scale, o, l, self.stream)
        return self.out if out is None else out, self.lse if lse is None else lse

    def run_partials(self, out=None, lse=None, tensors=None):
        """The split-KV kernel alone (splitkv_decode_partials): rows of sequences
        with one split are final, the others wait for merge()."""
        q, k, v, table, lens = tensors if tensors is not None else self.tensors
        o = self.out if out is None else out
        l = self.lse if lse is None else lse
        splitkv_decode_partials(self.plan, self.workspace, q, k, v, table, lens, self.num_splits,
                                self.scale, self.kv_scale, o, l, self.stream)
        return o, l

    def merge(self, out=None, lse=None):
        """Merges the partials run_partials left in the workspace (splitkv_combine_workspace)."""
        o = self.out if out is None else out
        l = self.lse if lse is None else lse
        splitkv_combine_workspace(self.plan, self.workspace, o, l, self.stream)
        return o, l

    def stats(self):
        """(per-CTA log [n][4], device status word) -- synchronises the stream."""
        return splitkv_read_stats(self.plan, self.workspace, self.stream)


def _on(stream):
    """What is allocated here belongs to ``stream`` (a torch stream, a handle or
    None for the current one), and its memory is reused in that stream's order."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


class CacheSession:
    """A paged cache and the calls that fill, read, weigh and prune it.

    ``desc`` (``make_desc``) describes the cache and the decode step; the pools,
    ``block_table`` and ``seq_lens`` are the caller's tensors, in the layout of
    ``DecodeSession``.  ``seq_lens`` lives on the device: the caller raises it by
    the new tokens before ``append``, ``evict`` lowers it.  Nothing here reads
    a length on the host, so a whole step can be captured into a CUDA graph.

    With ``track`` the session keeps the accumulated weight and the position of
    every cached key, which ``weigh`` and ``evict`` need.  A session's calls
    share its workspaces: one stream (or replayed graph) at a time.  It is made
    outside of captures; the workspaces that it makes then serve every call and
    graph of its life.  Results belong to the stream of the call.
    """

    def __init__(self, desc, k_pages, v_pages, block_table, seq_lens, *, scale, rope=None, kv_scale=1.0,
                 k_scale=None, v_scale=None, num_splits=16, track=False):
        dev = k_pages.device
        self.desc, self.rope = desc, rope
        self.k_pages, self.v_pages = k_pages, v_pages
        self.block_table, self.seq_lens = block_table, seq_lens
        self.scale, self.kv_scale = float(scale), float(kv_scale)
        self.k_scale, self.v_scale = k_scale, v_scale
        self.num_splits = num_splits
        try:
            self.plan = splitkv_plan_fixed(desc, num_splits)
            self.workspace = torch.empty(max(self.plan.workspace_size, 256), dtype=torch.uint8, device=dev)
            splitkv_plan_upload(self.plan, self.workspace, self.workspace.numel())
        except SplitKVError as e:  # (a cache that the decode does not serve may still be filled, and read by cross_attend)
            if e.status != SPLITKV_EUNSUPPORTED:
                raise
            self.plan = None
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        slots = (desc.batch, desc.num_kv_heads, desc.max_pages_per_seq * desc.page_size)
        self.key_weights = torch.zeros(slots, device=dev) if track else None
        self.key_positions = torch.zeros(slots, dtype=torch.int32, device=dev) if track else None
        # (most is needed for a budget of half the slots)
        size = splitkv_evict_workspace_size(desc, max(1, slots[2] // 2)) if track else 0
        self.evict_workspace = torch.empty(size, dtype=torch.uint8, device=dev) if track else None
        torch.cuda.current_stream(dev).synchronize()  # (the calls may come on any stream)

    def append(self, positions, q, k, v, cu_tokens=None, q_out=None, stream=None):
        """Rotates the new tokens' queries (returned) and keys and stores their
        keys and values (``splitkv_append``); ``q`` may be None."""
        if q is not None and q_out is None:
            with _on(stream):
                q_out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
        splitkv_append(self.desc, self.rope, positions, q, k, v, self.block_table, self.seq_lens, q_out,
                       self.k_pages, self.v_pages, cu_tokens=cu_tokens, kv_scale=self.kv_scale,
                       k_scale=self.k_scale, v_scale=self.v_scale, key_weights=self.key_weights,
                       key_positions=self.key_positions, status=self.status, stream=stream)
        return q_out

    def decode(self, q, out=None, lse=None, stream=None):
        """Causal decode attention of ``q`` [B][T][Hq][Dk] through a capacity plan."""
        d = self.desc
        if self.plan is None:
            splitkv_plan_fixed(d, self.num_splits)  # (raises, with the reason)
        with _on(stream):
            if out is None:
                out = torch.empty((d.batch, d.q_tokens, d.num_q_heads, d.v_dim), dtype=torch.bfloat16, device=q.device)
            if lse is None:
                lse = torch.empty((d.batch, d.q_tokens, d.num_q_heads), dtype=torch.float32, device=q.device)
        args = (self.plan, self.workspace, q, self.k_pages, self.v_pages, self.block_table, self.seq_lens,
                self.num_splits, self.scale)
        if self.k_scale is not None:
            splitkv_decode_kv_scales(*args, self.k_scale, self.v_scale, out, lse, stream)
        else:
            splitkv_decode(*args, self.kv_scale, out, lse, stream)
        return out, lse

    def weigh(self, q, lse, decay=1.0, stream=None):
        """Adds the attention every cached key got from ``q`` (``lse`` from ``decode``)."""
        splitkv_key_weights(self.desc, q, self.k_pages, self.block_table, self.seq_lens, lse, self.scale,
                            self.kv_scale, decay, self.key_weights, self.key_weights, k_scale=self.k_scale,
                            status=self.status, stream=stream)

    def evict(self, budget, sink=0, recent=0, stream=None):
        """Cuts every sequence to ``budget`` keys per KV head, in place."""
        splitkv_evict(self.desc, budget, sink, recent, self.k_pages, self.v_pages, self.block_table,
                      self.seq_lens, self.key_weights, self.key_positions, self.key_weights,
                      self.key_positions, self.seq_lens, self.evict_workspace, status=self.status,
                      stream=stream)

    def cross_attend(self, q, cu_tokens=None, stream=None):
        """Attention of ``q`` [n][Hq][128] over all keys of its sequence, without a causal mask."""
        n = q.shape[0]
        size = splitkv_cross_workspace_size(self.desc, n)
        with _on(stream):
            workspace = torch.empty(size, dtype=torch.uint8, device=q.device) if size else None
            out = torch.empty((n, self.desc.num_q_heads, 128), dtype=torch.bfloat16, device=q.device)
            lse = torch.empty((n, self.desc.num_q_heads), dtype=torch.float32, device=q.device)
        splitkv_cross_attend(self.desc, cu_tokens, q, self.k_pages, self.v_pages, self.block_table, self.seq_lens,
                             self.scale, out, lse, workspace, status=self.status, stream=stream)
        return out, lse

    def read_status(self):
        """Device status bits of append, weigh, evict and cross_attend so far (synchronises)."""
        return int(self.status.item())
