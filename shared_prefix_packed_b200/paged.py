"""PagedCache: a key/value cache of packed groups in pages of 8-bit codes, and the calls that grow, fill and read it.

Allocation (torch) and argument marshalling only; every step runs in libpp's kernels.
"""
from __future__ import annotations

from typing import Sequence

import torch

from . import _lib


class PagedCache:
    """The segments of packed groups (each group's prefix, then its responses) held in pages of a common pool.

    A step of a rollout: ``slots, pos, _ = cache.resize(new_lens, capacity)`` gives the new tokens their slots and
    grouped positions, ``pp_qk_norm_rope`` (or ``pp_rope``) embeds their q and k at ``pos``, ``cache.append(k, v,
    slots)`` rounds them into the pages, and ``cache.decode(q)`` attends. All of it runs on the device and in the order
    of one stream, reads nothing back, and can be captured into a CUDA graph (with ``new_lens`` and the rows in fixed
    buffers, and ``capacity`` the most tokens a step may bring).
    """

    def __init__(self, num_responses: Sequence[int], hq: int, hkv: int, num_pages: int, max_tokens: int,
                 page_size: int = 64, codes: str = "e4m3", d: int = 128, device="cuda"):
        """num_responses[g] = responses of group g; num_pages: the pool; max_tokens: the longest a segment may get;
        codes: "e4m3" or "int8"."""
        if codes not in ("e4m3", "int8"):
            raise ValueError(f"codes must be 'e4m3' or 'int8' (got {codes!r})")
        if page_size not in (16, 32, 64, 128):
            raise ValueError(f"page_size {page_size} not in 16, 32, 64, 128")
        if not len(num_responses) or min(num_responses) < 0 or num_pages < 1 or max_tokens < 1:
            raise ValueError("need a group at least, num_responses >= 0, num_pages >= 1 and max_tokens >= 1")
        self.hq, self.hkv, self.d, self.page_size = hq, hkv, d, page_size
        self.device = torch.device(device)
        start = [0]
        for k in num_responses:
            start.append(start[-1] + 1 + int(k))
        self.num_segments, self.num_groups = start[-1], len(num_responses)
        i32 = dict(dtype=torch.int32, device=self.device)
        self.group_start = torch.tensor(start, **i32)
        self.seg_group = torch.tensor([g for g, k in enumerate(num_responses) for _ in range(1 + int(k))], **i32)
        dt = torch.float8_e4m3fn if codes == "e4m3" else torch.int8
        self.k_pages = torch.zeros(num_pages, hkv, page_size, d, dtype=torch.uint8, device=self.device).view(dt)
        self.v_pages = torch.zeros(num_pages, hkv, d, page_size, dtype=torch.uint8, device=self.device).view(dt)
        self.k_scale = torch.ones(num_pages, hkv, dtype=torch.float32, device=self.device)
        self.v_scale = torch.ones(num_pages, hkv, dtype=torch.float32, device=self.device)
        max_pages = -(-max_tokens // page_size)
        self.page_table = torch.full((self.num_segments, max_pages), -1, **i32)
        self.free_pages = torch.arange(num_pages - 1, -1, -1, **i32)     # taken from its end: page 0 first
        self.n_free = torch.tensor([num_pages], **i32)
        self.lens = torch.zeros(self.num_segments, **i32)
        self.device = self.lens.device                       # "cuda" is the device of now, not of each later call

    def resize(self, new_lens, capacity: int | None = None, stream=None):
        """Bring the segments to new_lens tokens (a sequence, or an int32 tensor on the device): pages are taken for
        those that grow and given back for those that shrink. Returns (slots, pos_ids, counts): one entry of slots and
        pos_ids for each new token in the order of the segments, slot -1 past the last; counts = (new tokens, pages
        taken, pages given back, 1), all 0 if the change did not fit and was not made. ``capacity``: the entries to
        make room for (default, for a sequence: its sum)."""
        if not isinstance(new_lens, torch.Tensor):
            new_lens = [int(n) for n in new_lens]
            capacity = sum(max(n, 0) for n in new_lens) if capacity is None else capacity
            new_lens = torch.tensor(new_lens, dtype=torch.int32)
        if capacity is None:
            raise ValueError("capacity is needed with lengths on the device")
        with _lib.stream_scope(self.device, stream):
            new = new_lens.to(self.device)
            i32 = dict(dtype=torch.int32, device=self.device)
            slots, pos, counts = torch.empty(capacity, **i32), torch.empty(capacity, **i32), torch.empty(4, **i32)
            _lib.pp_pages_resize(self.group_start, self.seg_group, self.lens, new, self.page_size, self.page_table,
                                 self.free_pages, self.n_free, self.n_free, slots, pos, counts)
            # counts[3] is 0 or 1: its first byte is that truth value, so that this is one launch
            torch.where(counts.view(torch.bool)[12], new, self.lens, out=self.lens)
        return slots, pos, counts

    def append(self, k, v, slots, stream=None):
        """Round the rows k, v [n, hkv, d] (bf16 or fp32) to 8 bits and write them at slots [n] (-1 skips a row). Slots
        as ``resize`` gives them; others need the rows of one page to stand together: each within 256 rows of the one
        before, with skipped rows between them and none of another page."""
        _lib.pp_cache_store(k, v, slots, self.k_pages, self.v_pages, self.k_scale, self.v_scale, stream)

    def decode(self, q, softmax_scale: float = 0.0, out=None, lse=None, stream=None):
        """One decoding step: q [n_resp, hq, d] bf16, one query for each response; returns (o [n_resp, hq, d], lse
        [hq, n_resp])."""
        n_resp = self.num_segments - self.num_groups
        with _lib.stream_scope(self.device, stream):
            o = torch.empty_like(q) if out is None else out
            l = torch.empty(self.hq, n_resp, dtype=torch.float32, device=q.device) if lse is None else lse
            ws = torch.empty(_lib.pp_paged_decode_bytes(n_resp, self.hq, self.hkv), dtype=torch.uint8,
                             device=self.device)
            _lib.pp_paged_decode(q, self.k_pages, self.v_pages, self.k_scale, self.v_scale, self.group_start,
                                 self.seg_group, self.lens, self.page_table, o, l, ws, softmax_scale)
        return o, l
