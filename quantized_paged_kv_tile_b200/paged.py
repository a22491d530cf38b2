"""Host-side bookkeeping of a quantized paged KV cache (one attention layer).

``PagedKVCache`` owns the device buffers the C ABI works on (K/V page
pools, fp16 tails, block tables, sequence lengths, decode workspace) and
turns user-level operations into the three library calls:
  prefill(rows)  -> kvq_quantize_tiles for every full tile, then
                    kvq_append_tokens for the unfinished last tile
  append(rows)   -> kvq_append_tokens (quantizes tiles as they fill)
  decode(q)      -> kvq_paged_decode_attention
  prefill_chunk(q, rows) -> kvq_paged_prefill_attention over the cache and
                    the chunk, then kvq_append_tokens of the chunk
  prompt(q, rows) -> kvq_prompt_attention over raw prompts, then prefill(rows)
  evict(keep)    -> kvq_evict_tiles (caches that track masses)
With ``track_mass=True`` prompt() and decode() also add the attention weight
that every tile receives to ``mass`` (kvq_paged_decode_attention_mass).
All arithmetic runs in the library's kernels; this module only sizes and
indexes buffers (PyTorch provides the memory and the stream).
"""

from __future__ import annotations

import math

import contextlib

import numpy as np
import torch

from . import kvq


@contextlib.contextmanager
def _on_stream(stream):
    """Run the enclosed calls on ``stream`` (a torch.cuda.Stream, or None for
    the current stream): temporaries made inside are allocated and copied on
    it, so the caching allocator never hands their memory to other work while
    the stream's kernels still read it."""
    if stream is None:
        yield
    else:
        with torch.cuda.stream(stream):
            yield


def _in_use(buf):
    """Mark a long-lived buffer as used by the current stream (it may have
    been allocated on another), so that freeing it later waits for this use."""
    if buf is not None and buf.is_cuda:
        buf.record_stream(torch.cuda.current_stream(buf.device))


class PagedKVCache:
    def __init__(self, cfg: kvq.Config, num_seqs: int, max_tokens_per_seq: int, device="cuda",
                 block_table: np.ndarray | None = None, num_splits: int = 0, track_mass: bool = False):
        self.cfg = cfg
        self.num_seqs = num_seqs
        self.device = torch.device(device)
        self.layout = kvq.get_layout(cfg)
        self.blocks_per_seq = math.ceil(max_tokens_per_seq / cfg.page_tokens)
        if block_table is None:
            block_table = np.arange(num_seqs * self.blocks_per_seq, dtype=np.int32).reshape(num_seqs, -1)
        if block_table.shape != (num_seqs, self.blocks_per_seq):
            raise ValueError(f"block table shape {block_table.shape} != {(num_seqs, self.blocks_per_seq)}")
        self.num_blocks = int(block_table.max()) + 1
        self.block_tables = torch.from_numpy(np.ascontiguousarray(block_table, dtype=np.int32)).to(self.device)
        h = cfg.num_kv_heads
        self.k_pool = torch.zeros((self.num_blocks, h, self.layout["page_bytes_k"]), dtype=torch.uint8,
                                  device=self.device)
        self.v_pool = torch.zeros((self.num_blocks, h, self.layout["page_bytes_v"]), dtype=torch.uint8,
                                  device=self.device)
        tail_shape = (num_seqs, h, cfg.tile_tokens, cfg.head_dim)
        self.k_tail = torch.zeros(tail_shape, dtype=torch.float16, device=self.device)
        self.v_tail = torch.zeros(tail_shape, dtype=torch.float16, device=self.device)
        self.seq_lens = torch.zeros(num_seqs, dtype=torch.int32, device=self.device)
        self.host_lens = np.zeros(num_seqs, dtype=np.int64)
        self.num_splits = num_splits
        # accumulated attention weight per tile, fp32 [B][max_tiles] (None: not tracked)
        self.max_tiles = -(-self.blocks_per_seq * cfg.page_tokens // cfg.tile_tokens)
        self.mass = torch.zeros((num_seqs, self.max_tiles), dtype=torch.float32,
                                device=self.device) if track_mass else None
        self.workspace = torch.empty(self._decode_bytes(num_splits), dtype=torch.uint8, device=self.device)
        self.prompt_workspace = None  # grown on demand by prompt when it tracks masses
        self.evict_workspace = None
        self.prefill_workspace = None  # grown on demand by prefill_chunk when it splits contexts
        self.dev_status = torch.zeros(1, dtype=torch.int32, device=self.device)

    def _decode_bytes(self, num_splits: int) -> int:
        if self.mass is None:
            return kvq.decode_workspace_bytes(self.cfg, self.num_seqs, num_splits)
        return kvq.decode_mass_workspace_bytes(self.cfg, self.num_seqs, self.blocks_per_seq, num_splits)

    def _run_decode(self, q, out, workspace, num_splits, mass) -> None:
        """The decode call on the current stream, with masses into ``mass`` if given."""
        args = (self.seq_lens, self.block_tables, self.k_pool, self.v_pool, self.k_tail, self.v_tail, workspace)
        kw = dict(num_splits=num_splits, num_blocks=self.num_blocks, dev_status=self.dev_status)
        if mass is None:
            kvq.paged_decode_attention(self.cfg, q, out, *args, **kw)
        else:
            kvq.paged_decode_attention_mass(self.cfg, q, out, mass, *args, **kw)

    # ------------------------------------------------------------------ write
    def prefill_tile_desc(self, lens) -> np.ndarray:
        """{src_row, seq, tile_idx} for every full tile of packed rows with
        per-sequence lengths ``lens`` (rows of seq s start at sum(lens[:s]))."""
        t = self.cfg.tile_tokens
        starts = np.concatenate([[0], np.cumsum(lens)[:-1]]).astype(np.int64)
        desc = [(starts[s] + i * t, s, i) for s in range(len(lens)) for i in range(int(lens[s]) // t)]
        return np.asarray(desc, dtype=np.int32).reshape(-1, 3)

    def prefill(self, rows_k: torch.Tensor, rows_v: torch.Tensor, lens, stream=None) -> None:
        """Load an empty cache with packed rows [sum(lens)][H_kv][d]."""
        lens = np.asarray(lens, dtype=np.int64)
        if np.any(self.host_lens):
            raise RuntimeError("prefill expects an empty cache")
        with _on_stream(stream):
            desc = torch.from_numpy(self.prefill_tile_desc(lens)).to(self.device)
            kvq.quantize_tiles(self.cfg, rows_k, rows_v, desc, self.block_tables, self.k_pool, self.v_pool,
                               num_blocks=self.num_blocks, dev_status=self.dev_status)
            t = self.cfg.tile_tokens
            full = (lens // t) * t
            rest = lens - full
            if rest.any():
                starts = np.concatenate([[0], np.cumsum(lens)[:-1]])
                idx = np.concatenate([np.arange(starts[s] + full[s], starts[s] + lens[s]) for s in range(len(lens))])
                idx_t = torch.from_numpy(idx).to(self.device)
                self._append(rows_k.index_select(0, idx_t), rows_v.index_select(0, idx_t), full, rest)
            self.host_lens = lens.copy()
            self.seq_lens.copy_(torch.from_numpy(lens.astype(np.int32)))

    def _append(self, new_k, new_v, before, counts) -> None:
        # runs on the current stream (callers enter _on_stream first)
        cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        kvq.append_tokens(self.cfg, new_k, new_v, torch.from_numpy(cu).to(self.device),
                          torch.from_numpy(np.asarray(before, dtype=np.int32)).to(self.device),
                          int(np.max(counts)), self.block_tables, self.k_pool, self.v_pool, self.k_tail,
                          self.v_tail, num_blocks=self.num_blocks, dev_status=self.dev_status)

    def append(self, new_k: torch.Tensor, new_v: torch.Tensor, counts=None, stream=None) -> None:
        """Append packed rows (``counts`` per sequence, default one each)."""
        if counts is None:
            counts = np.ones(self.num_seqs, dtype=np.int64)
        counts = np.asarray(counts, dtype=np.int64)
        if np.any(self.host_lens + counts > self.blocks_per_seq * self.cfg.page_tokens):
            raise ValueError("append past the allocated pages")
        with _on_stream(stream):
            self._append(new_k, new_v, self.host_lens, counts)
            self.host_lens = self.host_lens + counts
            self.seq_lens.copy_(torch.from_numpy(self.host_lens.astype(np.int32)))

    # ------------------------------------------------------------------- read
    def decode(self, q: torch.Tensor, out: torch.Tensor | None = None, num_splits: int | None = None,
               stream=None) -> torch.Tensor:
        """One decode step: q fp16 [B][H_q][d] -> out fp16 [B][H_q][d]."""
        splits = self.num_splits if num_splits is None else num_splits
        with _on_stream(stream):
            if out is None:
                out = torch.empty_like(q)
            ws = self.workspace
            need = self._decode_bytes(splits)
            if ws.numel() < need:
                ws = torch.empty(need, dtype=torch.uint8, device=self.device)  # freed after this call's work
            else:
                _in_use(ws)
            _in_use(self.mass)
            self._run_decode(q, out, ws, splits, self.mass)
        return out

    def prompt(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lens, out: torch.Tensor | None = None,
               lse: torch.Tensor | None = None, mass_window: int = 0, stream=None) -> torch.Tensor:
        """Whole prompts into an empty cache: causal attention of the packed rows
        (``lens`` tokens per sequence; q fp16 [N][H_q][d], k / v fp16
        [N][H_kv][d], rows may be strided) over themselves, then ``prefill`` of
        the same rows.  With ``track_mass`` the tiles' masses grow by the weight
        from the last ``mass_window`` tokens of each prompt (0: all).  Returns
        out fp16 [N][H_q][d]; ``lse`` fp32 [N][H_q] is filled if given."""
        lens = np.asarray(lens, dtype=np.int64)
        if lens.shape != (self.num_seqs,) or np.any(lens < 0):
            raise ValueError("lens: one non-negative prompt length per sequence")
        if int(lens.sum()) != q.shape[0]:
            raise ValueError(f"lens sum to {int(lens.sum())}, q has {q.shape[0]} rows")
        if np.any(self.host_lens):
            raise RuntimeError("prompt expects an empty cache")
        if np.any(lens > self.blocks_per_seq * self.cfg.page_tokens):
            raise ValueError("prompt past the allocated pages")
        if mass_window and self.mass is None:
            raise ValueError("mass_window needs a cache with track_mass")
        longest = int(lens.max()) if lens.size else 0
        with _on_stream(stream):
            if out is None:
                out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
            cu = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).to(self.device)
            ws = None
            if self.mass is not None:
                need = kvq.prompt_workspace_bytes(self.cfg, self.num_seqs, q.shape[0], longest, mass_window)
                if self.prompt_workspace is None or self.prompt_workspace.numel() < need:
                    self.prompt_workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=self.device)
                ws = self.prompt_workspace
                _in_use(ws)
                _in_use(self.mass)
            kvq.prompt_attention(self.cfg, q, k, v, out, cu, longest, lse=lse, mass=self.mass,
                                 mass_window=mass_window, workspace=ws, dev_status=self.dev_status)
            if longest > 0:
                self.prefill(k.contiguous(), v.contiguous(), lens)
        return out

    # --------------------------------------------------------------- eviction
    def evict(self, keep_tiles: int, sink_tiles: int = 1, recent_tiles: int = 1, kept: torch.Tensor | None = None,
              stream=None) -> None:
        """Bring every sequence down to ``keep_tiles`` full tiles: those with the
        least mass leave, never the first ``sink_tiles`` or the last
        ``recent_tiles``.  Lengths shrink; rows keep the positions they were
        rotated with.  ``kept`` (int32 [B][max_tiles]) gets the old indices of
        the kept tiles."""
        if self.mass is None:
            raise ValueError("evict needs a cache with track_mass")
        t = self.cfg.tile_tokens
        with _on_stream(stream):
            if self.evict_workspace is None:
                need = kvq.evict_workspace_bytes(self.cfg, self.num_seqs, self.blocks_per_seq)
                self.evict_workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=self.device)
            _in_use(self.evict_workspace)
            _in_use(self.mass)
            kvq.evict_tiles(self.cfg, self.mass, self.seq_lens, self.block_tables, keep_tiles, sink_tiles,
                            recent_tiles, kept=kept, workspace=self.evict_workspace, dev_status=self.dev_status)
        self.host_lens = self.host_lens - np.maximum(0, self.host_lens // t - keep_tiles) * t

    def prefill_chunk(self, q: torch.Tensor, new_k: torch.Tensor, new_v: torch.Tensor, counts,
                      out: torch.Tensor | None = None, append: bool = True, num_splits: int | None = None,
                      stream=None) -> torch.Tensor:
        """Chunked prefill: packed chunk rows (``counts`` tokens per sequence;
        q fp16 [N][H_q][d], new_k / new_v fp16 [N][H_kv][d]) attend to the
        cached context and causally to their own chunk; then (``append``) the
        chunk joins the cache.  ``num_splits`` (default: chosen from the
        context lengths and the SM count) splits long contexts over more
        CTAs.  Returns out fp16 [N][H_q][d].  The chunk's queries do not add to
        the masses of a cache that tracks them."""
        counts = np.asarray(counts, dtype=np.int64)
        if counts.shape != (self.num_seqs,) or np.any(counts < 0):
            raise ValueError("counts: one non-negative chunk length per sequence")
        if append and np.any(self.host_lens + counts > self.blocks_per_seq * self.cfg.page_tokens):
            raise ValueError("append past the allocated pages")
        max_chunk = int(counts.max()) if counts.size else 0
        if num_splits is None:
            num_splits = 1
            if self.device.type == "cuda":  # (anything else is refused by the binding below)
                sms = torch.cuda.get_device_properties(self.device).multi_processor_count
                num_splits = kvq.prefill_splits(self.cfg, self.num_seqs, max_chunk, int(self.host_lens.max()), sms)
        need = kvq.prefill_workspace_bytes(self.cfg, self.num_seqs, max_chunk, num_splits)
        with _on_stream(stream):
            if out is None:
                out = torch.empty_like(q)
            cu = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).to(self.device)
            ws = None
            if need > 0:
                if self.prefill_workspace is None or self.prefill_workspace.numel() < need:
                    # the old buffer (if any) may still be read by earlier work on
                    # another stream: it was marked in use there when it was used
                    self.prefill_workspace = torch.empty(need, dtype=torch.uint8, device=self.device)
                ws = self.prefill_workspace
                _in_use(ws)
            kvq.paged_prefill_attention(self.cfg, q, out, new_k, new_v, cu, self.seq_lens, max_chunk,
                                        self.block_tables, self.k_pool, self.v_pool, self.k_tail, self.v_tail,
                                        num_splits=num_splits, workspace=ws, num_blocks=self.num_blocks,
                                        dev_status=self.dev_status)
            if append and max_chunk > 0:
                self._append(new_k, new_v, self.host_lens, counts)
                self.host_lens = self.host_lens + counts
                self.seq_lens.copy_(torch.from_numpy(self.host_lens.astype(np.int32)))
        return out

    def status(self) -> int:
        """Device status word (0 = no device-detected error); synchronizes."""
        return int(self.dev_status.item())

    def bytes_per_token_head(self) -> float:
        """Stored bytes per (token, KV head) for K+V, pages only."""
        p = self.cfg.page_tokens
        return (self.layout["page_bytes_k"] + self.layout["page_bytes_v"]) / p


class DecodeStepGraph:
    """One serving step of a ``PagedKVCache`` -- append one token per sequence,
    then decode -- captured once in a CUDA graph and replayed.

    Stage the step's rows in ``new_k`` / ``new_v`` ([B][H_kv][d] fp16) and its
    queries in ``q`` ([B][H_q][d] fp16), call ``replay()``, read ``out``.  The
    sequence lengths advance on the device inside the graph (the append reads
    them as the lengths before the step, then they grow by one); the host
    tracks them to refuse a step past the allocated pages.  The first decode
    and append calls happen eagerly before capture.

    ``fused=True``: steps in which no sequence completes a tile replay a graph
    of one launch (kvq_append_decode_step: the token into the tails, the
    decode, the lengths advanced); steps that complete a tile replay the
    append + decode graph (the completed tile has to be quantized first).
    Both use the same split count, so the outputs are those of the unfused
    step bit for bit.  A cache that tracks masses takes the unfused step, whose
    decode adds to them; ``evict`` between replays needs no new capture.
    """

    def __init__(self, cache: PagedKVCache, num_splits: int | None = None, fused: bool = False):
        self.cache = cache
        cfg, b, dev = cache.cfg, cache.num_seqs, cache.device
        if fused and cache.mass is not None:
            raise ValueError("the one-launch step does not track masses: use fused=False")
        self.fused = fused
        if fused and num_splits is None:
            num_splits = kvq.step_splits(cfg, b, torch.cuda.get_device_properties(dev).multi_processor_count)
        self.num_splits = cache.num_splits if num_splits is None else num_splits
        self.new_k = torch.zeros((b, cfg.num_kv_heads, cfg.head_dim), dtype=torch.float16, device=dev)
        self.new_v = torch.zeros_like(self.new_k)
        self.q = torch.zeros((b, cfg.num_q_heads, cfg.head_dim), dtype=torch.float16, device=dev)
        self.out = torch.empty_like(self.q)
        self._cu = torch.arange(b + 1, dtype=torch.int32, device=dev)
        need = cache._decode_bytes(self.num_splits)
        # the graph holds the buffer whose address it records; the cache's stays
        # the cache's, other graphs may have recorded it
        self.workspace = cache.workspace
        if self.workspace.numel() < need:
            self.workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        # the fused step's own workspace: zero-filled once, left zero by every step
        self.step_workspace = torch.zeros(need, dtype=torch.uint8, device=dev) if fused else None
        self.graph = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream(device=dev)
        side.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(side):
            # the decode once eagerly on the current contents (no state change:
            # masses, if tracked, go to a copy)
            self._decode(None if cache.mass is None else cache.mass.clone())
        torch.cuda.current_stream(dev).wait_stream(side)
        torch.cuda.synchronize(dev)
        with torch.cuda.graph(self.graph):
            self._step()
        self.graph_fused = None
        if fused:
            self.graph_fused = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph_fused):
                self._fused_step()

    def _decode(self, mass) -> None:
        self.cache._run_decode(self.q, self.out, self.workspace, self.num_splits, mass)

    def _step(self) -> None:
        c = self.cache
        kvq.append_tokens(c.cfg, self.new_k, self.new_v, self._cu, c.seq_lens, 1, c.block_tables, c.k_pool,
                          c.v_pool, c.k_tail, c.v_tail, num_blocks=c.num_blocks, dev_status=c.dev_status)
        c.seq_lens.add_(1)
        self._decode(c.mass)

    def _fused_step(self) -> None:
        c = self.cache
        kvq.append_decode_step(c.cfg, self.new_k, self.new_v, self.q, self.out, c.seq_lens, c.block_tables,
                               c.k_pool, c.v_pool, c.k_tail, c.v_tail, self.step_workspace, self.num_splits,
                               num_blocks=c.num_blocks, dev_status=c.dev_status)

    def completes_tile(self) -> bool:
        """Whether the next step completes a tile of some sequence."""
        c = self.cache
        return bool(np.any((c.host_lens + 1) % c.cfg.tile_tokens == 0))

    def replay(self) -> torch.Tensor:
        c = self.cache
        if np.any(c.host_lens + 1 > c.blocks_per_seq * c.cfg.page_tokens):
            raise ValueError("append past the allocated pages")
        if self.fused and not self.completes_tile():
            self.graph_fused.replay()
        else:
            self.graph.replay()
        c.host_lens = c.host_lens + 1
        return self.out
