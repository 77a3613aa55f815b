"""Steps over D simulated shards on one GPU: the sparse decode step, a
server's steps with a cache it fills itself, and the projections around them.

Per shard d: filter + convert the global top-k to shard d's slots, then
sparse MLA decode over shard d's pool; finally the LSE-weighted merge of the
D partials (the single-GPU stand-in for the cross-rank LSE all-gather and
output reduce-scatter of "[eldritch] attention: support DCP in SM120
FlashInfer sparse MLA", Why / Scope).

``DcpDecodeStep`` allocates every buffer once in its constructor, so its
``run`` launches 2*D + 1 kernels and allocates nothing.
"""
from __future__ import annotations

from typing import List, Optional

import torch

from . import capi
from .inputs import Workload


class DcpDecodeStep:
    def __init__(self, wl: Workload, device="cuda", stream: Optional[torch.cuda.Stream] = None):
        self.wl = wl
        self.device = torch.device(device)
        self.stream = stream
        T, H, K, D = wl.T, wl.H, wl.K, wl.D
        dev = self.device
        with torch.cuda.stream(stream):  # copied and filled where the step runs
            self.q = wl.q.to(dev).contiguous()
            self.req_id = torch.from_numpy(wl.req_id).to(dev)
            self.topk = torch.from_numpy(wl.topk).to(dev)
            self.pools: List[torch.Tensor] = [s.pool.to(dev) for s in wl.shards]
            self.block_tables = [torch.from_numpy(s.block_table).to(dev) for s in wl.shards]
            self.bt_widths = [s.width for s in wl.shards]
            self.local_slots = [torch.empty((T, K), dtype=torch.int32, device=dev) for _ in range(D)]
            self.valid_count = [torch.empty((T,), dtype=torch.int32, device=dev) for _ in range(D)]
            self.part_out = [torch.empty((T, H, capi.V_DIM), dtype=torch.bfloat16, device=dev)
                             for _ in range(D)]
            self.part_lse = [torch.empty((T, H), dtype=torch.float32, device=dev) for _ in range(D)]
            self.out = torch.empty((T, H, capi.V_DIM), dtype=torch.bfloat16, device=dev)
            self.lse = torch.empty((T, H), dtype=torch.float32, device=dev)
            self.workspace = capi.alloc_decode_workspace(T, H, K, dev, stream)

    @property
    def launches_per_step(self) -> int:
        return 2 * self.wl.D + 1

    def run_shard(self, d: int):
        wl = self.wl
        capi.dcp_filter_convert_index(
            self.req_id, self.block_tables[d], self.topk, wl.D, d, wl.spec.block_size,
            interleave=wl.spec.interleave, bt_width=self.bt_widths[d],
            local_slots=self.local_slots[d],
            valid_count=self.valid_count[d], stream=self.stream)
        capi.sparse_mla_decode(
            self.q, self.pools[d], self.local_slots[d], wl.spec.sm_scale,
            out=self.part_out[d], lse=self.part_lse[d], workspace=self.workspace,
            stream=self.stream)

    def run_fused(self):
        """The same step in one launch (conversion, decode and merge fused)."""
        wl = self.wl
        return capi.dcp_sparse_mla_decode_fused(
            self.q, self.req_id, self.topk, self.pools, self.block_tables,
            wl.spec.block_size, wl.spec.sm_scale, interleave=wl.spec.interleave,
            bt_widths=self.bt_widths,
            out=self.out, lse=self.lse, workspace=self.workspace, stream=self.stream)

    def run_fused_from_host(self, q_host: torch.Tensor, topk_host: torch.Tensor,
                            out_host: torch.Tensor, lse_host: torch.Tensor, chunks: int = 4):
        """The fused step with q and the top-k ids in pinned host memory and
        out/lse returned there: the library copies them in and out through
        this step's device buffers, row groups pipelined."""
        wl = self.wl
        return capi.dcp_sparse_mla_decode_fused_host(
            q_host, topk_host, out_host, lse_host, self.req_id, self.pools, self.block_tables,
            wl.spec.block_size, wl.spec.sm_scale, interleave=wl.spec.interleave,
            bt_widths=self.bt_widths, q_dev=self.q, topk_dev=self.topk, out_dev=self.out,
            lse_dev=self.lse, workspace=self.workspace, chunks=chunks, stream=self.stream)

    def run(self):
        for d in range(self.wl.D):
            self.run_shard(d)
        capi.dcp_lse_merge(self.part_out, self.part_lse, out=self.out, lse=self.lse,
                           stream=self.stream)
        return self.out, self.lse


class DcpServingStep:
    """A server's steps over D simulated shards and a cache it fills itself.

    ``prefill`` writes a chunk of any requests' tokens into the caches;
    ``run`` brings ``tokens_per_req`` new tokens of every request, writes
    them and attends each token's window and sinks over all D pools.  Both
    take device tensors, launch on one stream and read nothing back: the
    block tables grow on the device from each rank's free list.  With a
    ``stream``, everything runs on it, the constructor's fills too; what the
    caller passes in is made ready on it, and results are read behind it, by
    the caller (``stream.wait_stream``).
    ``take_blocks`` then drops the blocks taken since the last call from the
    front of the free lists (it reads their counts, so it synchronises); a
    server that keeps the lengths on the host can do that from them instead.
    A ``prefill`` or ``run`` that raises has taken nothing: called again with
    the same lengths it takes the same blocks.

    With ``max_nodes`` above 0 the server may draft trees of that many tokens
    a request at most: ``verify`` writes their rows into scratch slots that
    each pool has behind its blocks and attends each node's window and sinks
    of its prefix and ancestors, as ``run`` does; ``commit`` takes the
    nodes the model agrees with into the cache.  ``commit`` takes blocks as
    ``run`` does.  Both reuse their results' buffers and allocate nothing; a
    CUDA graph may hold them, with the free lists of its capture.
    """

    def __init__(self, num_reqs: int, tokens_per_req: int, heads: int, dcp: int, block_size: int,
                 blocks_per_rank: int, max_ctx: int, window: int, sinks: int, *, fmt: str = "fp4",
                 gamma: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 cos_sin: Optional[torch.Tensor] = None, rope_pairs: bool = True,
                 sm_scale: float = 192 ** -0.5, interleave: int = 1, max_nodes: int = 0, device="cuda",
                 stream: Optional[torch.cuda.Stream] = None):
        if not 0 <= max_nodes <= capi.MAX_TREE_NODES:
            raise ValueError(f"max_nodes must be 0 .. {capi.MAX_TREE_NODES}, got {max_nodes}")
        dev = torch.device(device)
        self.B, self.S, self.H, self.D = num_reqs, tokens_per_req, heads, dcp
        self.block_size, self.interleave, self.max_ctx = block_size, interleave, max_ctx
        self.window, self.sinks, self.sm_scale = window, sinks, sm_scale
        self.gamma, self.eps, self.cos_sin, self.rope_pairs = gamma, eps, cos_sin, rope_pairs
        self.stream = stream
        row = {"fp8": capi.ROW_BYTES, "fp4": capi.FP4_ROW_BYTES}[fmt]
        width = -(-max_ctx // (interleave * dcp)) * interleave
        width = max(1, -(-width // block_size))
        T = num_reqs * tokens_per_req
        self.max_nodes, drafts = max_nodes, num_reqs * max_nodes
        # Allocated and filled on the stream the steps run on (the current one
        # without a stream), which alone orders the fills before the steps.
        with torch.cuda.stream(stream):
            self.pools = [torch.zeros((blocks_per_rank * block_size + drafts, row), dtype=torch.uint8,
                                      device=dev) for _ in range(dcp)]
            self.block_tables = [torch.full((num_reqs, width), -1, dtype=torch.int32, device=dev)
                                 for _ in range(dcp)]
            self.free_blocks = [torch.arange(blocks_per_rank, dtype=torch.int32, device=dev)
                                for _ in range(dcp)]
            self.q_lens = torch.full((num_reqs,), tokens_per_req, dtype=torch.int32, device=dev)
            self.maps = [capi.alloc_step_maps(num_reqs, T, dev, stream) for _ in range(dcp)]
            self.out = torch.empty((T, heads, capi.V_DIM), dtype=torch.bfloat16, device=dev)
            self.lse = torch.empty((T, heads), dtype=torch.float32, device=dev)
            self.workspace = capi.alloc_window_decode_workspace(T, heads, max_ctx, window, sinks, dcp,
                                                                interleave, -1, dev, stream)
            if drafts:
                # A node's row lies in the same scratch slot of every pool, so
                # that each rank finds the accepted ones it owns.
                self.draft_slots = torch.arange(drafts, dtype=torch.int32, device=dev) + (
                    blocks_per_rank * block_size)
                self.tree = capi.TreeMaps(
                    torch.empty((drafts, -(-max_nodes // 64)), dtype=torch.int64, device=dev),
                    torch.empty((drafts,), dtype=torch.int32, device=dev))
                self.tree_out = torch.empty((drafts, heads, capi.V_DIM), dtype=torch.bfloat16, device=dev)
                self.tree_lse = torch.empty((drafts, heads), dtype=torch.float32, device=dev)
                self.tree_workspace = capi.alloc_tree_decode_workspace(
                    drafts, heads, num_reqs, max_ctx, max_nodes, dcp, interleave, -1, dev, stream)
                self.walk = capi.TreeWalk(*(torch.empty((n,), dtype=torch.int32, device=dev)
                                            for n in (num_reqs, drafts, num_reqs)))
                self.ctx_after = torch.empty((num_reqs,), dtype=torch.int32, device=dev)
                self.tree_maps = [capi.alloc_step_maps(num_reqs, drafts, dev, stream) for _ in range(dcp)]
        self._taken: List[torch.Tensor] = []

    def _append(self, ctx_lens, q_lens, kv, outs):
        if self._taken:
            raise RuntimeError("the last step's blocks are still in the free lists: take_blocks() first")
        taken = []
        for d in range(self.D):
            m = capi.dcp_step_maps(ctx_lens, q_lens, self.free_blocks[d], self.block_tables[d],
                                   kv.shape[0], self.D, d, self.block_size,
                                   interleave=self.interleave, out=outs[d], stream=self.stream)
            taken.append(m.blocks_taken)
            capi.mla_cache_write(kv, m.slots, self.pools[d], gamma=self.gamma, eps=self.eps,
                                 positions=m.positions, cos_sin=self.cos_sin,
                                 rope_pairs=self.rope_pairs, stream=self.stream)
        return taken

    def prefill(self, ctx_lens: torch.Tensor, q_lens: torch.Tensor, kv: torch.Tensor):
        """Write the rows kv [sum(q_lens), 576] of the requests' new tokens."""
        self._taken = self._append(ctx_lens, q_lens, kv, [None] * self.D)

    def run(self, ctx_lens: torch.Tensor, kv: torch.Tensor, q: torch.Tensor):
        """One decode step: rows kv [B*S, 576] go into the caches, q
        [B*S, H, 576] attends.  Returns (out, lse), reused by the next step."""
        taken = self._append(ctx_lens, self.q_lens, kv, self.maps)
        result = capi.dcp_window_mla_decode(
            q, ctx_lens, self.max_ctx, self.S, self.window, self.sinks, self.pools,
            self.block_tables, self.block_size, self.sm_scale, interleave=self.interleave,
            out=self.out, lse=self.lse, workspace=self.workspace, stream=self.stream)
        self._taken = taken
        return result

    def _drafted(self, rows: int) -> int:
        if not 0 <= rows <= self.B * self.max_nodes:
            raise ValueError(f"{rows} drafted rows; this step holds {self.B} trees of {self.max_nodes} nodes")
        return rows

    def verify(self, prefix_lens: torch.Tensor, parents: torch.Tensor, row_start: torch.Tensor,
               kv: torch.Tensor, q: torch.Tensor):
        """Attention of drafted trees over the cached prefixes and themselves,
        each node's window and sinks of them as ``run`` attends a token's.
        Rows kv [T, 576] and q [T, H, 576] are the nodes', request b's at
        row_start[b] .. row_start[b + 1] - 1; their positions (for q's
        rotation) come from ``tree_positions``.  Returns
        (out [T, H, 512], lse [T, H]); rows of no request are left as they
        were."""
        T = self._drafted(parents.shape[0])
        maps = self.tree_positions(prefix_lens, parents, row_start)
        slots = self.draft_slots[:T]
        for pool in self.pools:
            capi.mla_cache_write(kv, slots, pool, gamma=self.gamma, eps=self.eps, positions=maps.positions,
                                 cos_sin=self.cos_sin, rope_pairs=self.rope_pairs, stream=self.stream)
        return capi.dcp_tree_mla_decode(
            q, row_start, prefix_lens, self.max_ctx, maps.masks, self.max_nodes, [slots] * self.D,
            self.pools, self.block_tables, self.block_size, self.sm_scale, interleave=self.interleave,
            window=self.window, sinks=self.sinks, positions=maps.positions, out=self.tree_out[:T], lse=self.tree_lse[:T], workspace=self.tree_workspace,
            stream=self.stream)

    def tree_positions(self, prefix_lens: torch.Tensor, parents: torch.Tensor,
                       row_start: torch.Tensor) -> capi.TreeMaps:
        """The nodes' masks and positions, which verify works with."""
        T = self._drafted(parents.shape[0])
        return capi.tree_maps(parents, row_start, prefix_lens, self.max_nodes,
                              out=capi.TreeMaps(*(t[:T] for t in self.tree)), stream=self.stream)

    def commit(self, prefix_lens: torch.Tensor, parents: torch.Tensor, tokens: torch.Tensor,
               targets: torch.Tensor, row_start: torch.Tensor):
        """Of the trees verified last, the nodes the model agrees with (token
        = its parent's target) move into the cache.  Returns (walk, lengths):
        what tree_accept writes, and the requests' lengths from now on."""
        if self._taken:
            raise RuntimeError("the last step's blocks are still in the free lists: take_blocks() first")
        T = self._drafted(parents.shape[0])
        walk = capi.TreeWalk(self.walk.accepted, self.walk.rows[:T], self.walk.next_tokens)
        capi.tree_accept(parents, tokens, targets, row_start, out=walk, stream=self.stream)
        with torch.cuda.stream(self.stream):
            torch.add(prefix_lens, walk.accepted, out=self.ctx_after)
        taken = []
        for d in range(self.D):
            m = self.tree_maps[d]
            m = capi.dcp_step_maps(self.ctx_after, walk.accepted, self.free_blocks[d], self.block_tables[d],
                                   T, self.D, d, self.block_size, interleave=self.interleave,
                                   out=m._replace(req_id=m.req_id[:T], positions=m.positions[:T],
                                                  slots=m.slots[:T]), stream=self.stream)
            capi.mla_cache_move(self.pools[d], walk.rows, self.draft_slots[:T], m.slots, stream=self.stream)
            taken.append(m.blocks_taken)
        self._taken = taken
        return walk, self.ctx_after

    def take_blocks(self):
        """Drop the blocks the last prefill, run or commit took from the free lists."""
        with torch.cuda.stream(self.stream):
            for d, taken in enumerate(self._taken):
                self.free_blocks[d] = self.free_blocks[d][int(taken.item()):]
        self._taken = []


class Fp8Projections:
    """The matrix products around the attention, in 8 bits, for steps of up to
    ``max_rows`` rows: activations are quantised for each 128 columns, the
    weights come with a scale for each 128 x 128.

      w_q [H * (P + 64), C]   a row's queries from its C activations
      w_k [H, 512, P]         each head's P values without position, absorbed
                              into the latent space
      w_v [H, V, 512]         each head's values from its latent result
      w_o [E, H * V]          the heads' values together

    ``query`` and ``output`` launch on one stream, read nothing back and reuse
    their results' buffers.  ``query`` rotates by torch's own operators, a dozen
    launches with temporaries behind the products; the products and ``output``
    allocate nothing.
    """

    def __init__(self, w_q: capi.Fp8Rows, w_k: capi.Fp8Rows, w_v: capi.Fp8Rows, w_o: capi.Fp8Rows,
                 max_rows: int, *, cos_sin: Optional[torch.Tensor] = None, rope_pairs: bool = True,
                 stream: Optional[torch.cuda.Stream] = None):
        self.w_q, self.w_k, self.w_v, self.w_o = w_q, w_k, w_v, w_o
        self.H, _, self.P = w_k.codes.shape
        self.V, self.E = w_v.codes.shape[1], w_o.codes.shape[0]
        self.rope = capi.QK_DIM - capi.V_DIM
        C = w_q.codes.shape[1]
        if w_q.codes.shape[0] != self.H * (self.P + self.rope):
            raise ValueError("w_q must have P + 64 rows for each of w_k's heads")
        if w_v.codes.shape[0] != self.H or w_o.codes.shape[1] != self.H * self.V:
            raise ValueError("w_v and w_o must be of w_k's heads")
        if w_k.codes.shape[1] != capi.V_DIM or w_v.codes.shape[2] != capi.V_DIM:
            raise ValueError(f"w_k and w_v must be of a latent of {capi.V_DIM}")
        self.max_rows, self.cos_sin, self.rope_pairs, self.stream = max_rows, cos_sin, rope_pairs, stream
        dev, T, H = w_q.codes.device, max_rows, self.H
        new = lambda *shape: capi._new(shape, torch.bfloat16, dev, stream)  # noqa: E731
        self.x8 = capi.alloc_fp8_rows((T, C), dev, stream)
        self.heads = new(T, H, self.P + self.rope)
        self.part8 = capi.alloc_fp8_rows((H, T, self.P), dev, stream)
        self.q = new(T, H, capi.QK_DIM)
        self.latent8 = capi.alloc_fp8_rows((H, T, capi.V_DIM), dev, stream)
        self.values = new(T, H, self.V)
        self.values8 = capi.alloc_fp8_rows((T, H * self.V), dev, stream)
        self.y = new(T, self.E)

    def _product(self, x, x8, w, out):
        a = capi.fp8_quantise(x, out=x8, stream=self.stream)
        return capi.fp8_matmul(a.codes, a.scales, w.codes, w.scales, out=out, stream=self.stream)

    def _rows(self, x8: capi.Fp8Rows, T: int) -> capi.Fp8Rows:
        return capi.Fp8Rows(x8.codes[..., :T, :], x8.scales[..., :T, :])

    def _count(self, rows: int) -> int:
        if rows > self.max_rows:
            raise ValueError(f"{rows} rows; this holds {self.max_rows}")
        return rows

    def query(self, x: torch.Tensor, positions: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Queries [T, H, 576] of rows x [T, C], in the latent space; their
        last 64 values rotated by cos_sin[positions] if this has a table (as
        mla_cache_write rotates a row's; a position outside it takes its
        nearest entry, where that call reports an error)."""
        T, H, P = self._count(x.shape[0]), self.H, self.P
        if self.cos_sin is not None and (positions is None or positions.shape != (T,)):
            raise ValueError(f"a position for each of the {T} rows is needed to rotate them")
        heads, q = self.heads[:T], self.q[:T]
        self._product(x, self._rows(self.x8, T), self.w_q, heads.view(T, H * (P + self.rope)))
        self._product(heads[..., :P].transpose(0, 1), self._rows(self.part8, T), self.w_k,
                      q[..., :capi.V_DIM].transpose(0, 1))
        with torch.cuda.stream(self.stream):
            z, to = heads[..., P:], q[..., capi.V_DIM:]
            if self.cos_sin is None:
                to.copy_(z)
            else:
                at = positions.long().clamp(0, self.cos_sin.shape[0] - 1)
                c, s = self.cos_sin[at][:, None].chunk(2, -1)
                half = self.rope // 2
                a, b = ((z[..., 0::2], z[..., 1::2]) if self.rope_pairs else (z[..., :half], z[..., half:]))
                to_a, to_b = ((to[..., 0::2], to[..., 1::2]) if self.rope_pairs
                              else (to[..., :half], to[..., half:]))
                a, b = a.float(), b.float()
                to_a.copy_(a * c - b * s)
                to_b.copy_(a * s + b * c)
        return q

    def output(self, latent: torch.Tensor) -> torch.Tensor:
        """Rows [T, E] of the attention's results latent [T, H, 512]."""
        T = self._count(latent.shape[0])
        values = self.values[:T]
        self._product(latent.transpose(0, 1), self._rows(self.latent8, T), self.w_v, values.transpose(0, 1))
        return self._product(values.view(T, self.H * self.V), self._rows(self.values8, T), self.w_o, self.y[:T])
