"""PackedPlan: where the rows of a packed batch go.

Requests that each bring a number of new tokens of their own (one for a decode, a few
drafts to verify, a chunk of a prompt) are one batch: their rows lie one request after
another in tensors [n_tokens][H][D]. The plan's arrays live on the device and are
filled there from the requests' lengths, so a captured step replays for other lengths:

    plan = PackedPlan(batch, n_tokens)          # once: n_tokens is the most a step takes
    pages.plan(q_lens, plan)                    # a step: pages for the new tokens, the places of its rows
    pages.copy_layer(layer)                     # (where pages may be shared)
    layer.step_packed(q, k_new, v_new, plan)    # every layer of the step

or `layer.plan(q_lens, plan)` over contiguous caches. Layers of one step share the
plan; their `seq_lens` may be one tensor (`cache=dict(seq_lens=pages.seq_lens)`).
"""
from __future__ import annotations

import torch

from . import binding as B


class PackedPlan:
    """q_starts [batch + 1]: the first row of each request (the last entry: rows in use);
    kv_ends [batch]: its length after the step (-1: not served); token_seq, positions
    (int32) and slots (int64) [n_tokens]: each row's request, position and cache slot (-1
    behind the last request, or where there is none)."""

    def __init__(self, batch: int, n_tokens: int, device="cuda"):
        if not torch.cuda.is_available():
            raise RuntimeError("PackedPlan needs a CUDA device; libuaa has no CPU implementation")
        dev = torch.device(device)
        self.device = dev = dev if dev.index is not None else torch.device("cuda", torch.cuda.current_device())
        self._index = dev.index
        self.batch, self.n_tokens = int(batch), int(n_tokens)
        self.filled = 0  # how often plan() has filled it
        new = lambda n, dt=torch.int32: torch.full((n,), -1, dtype=dt, device=dev)
        self.q_starts = torch.zeros(self.batch + 1, dtype=torch.int32, device=dev)
        self.kv_ends = new(self.batch)
        self.token_seq, self.positions, self.slots = new(self.n_tokens), new(self.n_tokens), new(self.n_tokens, torch.int64)
        a = self.args = B.UaaPackedPlan()
        a.batch, a.n_tokens = self.batch, self.n_tokens
        a.q_starts, a.kv_ends = B.ptr(self.q_starts), B.ptr(self.kv_ends)
        a.token_seq, a.positions, a.slots = B.ptr(self.token_seq), B.ptr(self.positions), B.ptr(self.slots)

    def with_lens(self, q_lens, batch: int, index: int):
        """The plan's arguments for the requests' token counts (int32 [batch] on the device), to be
        filled by them."""
        if self.batch != batch or self._index != index:
            raise ValueError(f"the plan is for {self.batch} requests on cuda:{self._index}, not {batch} on cuda:{index}")
        if (q_lens.dtype is not torch.int32 or q_lens.shape != self.kv_ends.shape or q_lens.get_device() != index
                or not q_lens.is_contiguous()):
            raise ValueError("q_lens is not a contiguous int32 tensor [batch] on the device")
        self.args.q_lens = q_lens.data_ptr()
        self.filled += 1
        return self.args


def pair_axes(half_rot: int, sections, order: str) -> list[int]:
    """The axis of each of half_rot rotation pairs. "blocks": the sections one after
    another. "cycle": the axes in turn, where an axis past the first that has had its
    section's pairs leaves its turns to the first axis."""
    sec = [int(x) for x in sections]
    n = len(sec)
    if not 1 <= n <= 4 or min(sec) < 0 or sum(sec) != half_rot:
        raise ValueError(f"rope_sections={sec}: 1 to 4 sections of {half_rot} rotation pairs in all are needed")
    if order == "blocks":
        return [a for a, s in enumerate(sec) for _ in range(s)]
    if order != "cycle":
        raise ValueError(f"rope_axes={order!r} is not \"blocks\" or \"cycle\"")
    axes = [p % n if p < n * sec[p % n] else 0 for p in range(half_rot)]
    if [axes.count(a) for a in range(n)] != sec:
        raise ValueError(f"rope_sections={sec}: {half_rot} pairs in turn do not give each axis its section")
    return axes
