"""One DCP decode step over D simulated shards on one GPU.

Per shard d: filter + convert the global top-k to shard d's slots, then
sparse MLA decode over shard d's pool; finally the LSE-weighted merge of the
D partials (the single-GPU stand-in for the cross-rank LSE all-gather and
output reduce-scatter of "[eldritch] attention: support DCP in SM120
FlashInfer sparse MLA", Why / Scope).

Every buffer is allocated once in the constructor, so ``run`` launches
2*D + 1 kernels and allocates nothing.
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
    """

    def __init__(self, num_reqs: int, tokens_per_req: int, heads: int, dcp: int, block_size: int,
                 blocks_per_rank: int, max_ctx: int, window: int, sinks: int, *, fmt: str = "fp4",
                 gamma: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 cos_sin: Optional[torch.Tensor] = None, rope_pairs: bool = True,
                 sm_scale: float = 192 ** -0.5, interleave: int = 1, device="cuda",
                 stream: Optional[torch.cuda.Stream] = None):
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
        # Allocated and filled on the stream the steps run on (the current one
        # without a stream), which alone orders the fills before the steps.
        with torch.cuda.stream(stream):
            self.pools = [torch.zeros((blocks_per_rank * block_size, row), dtype=torch.uint8, device=dev)
                          for _ in range(dcp)]
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

    def take_blocks(self):
        """Drop the blocks the last prefill or run took from the free lists."""
        with torch.cuda.stream(self.stream):
            for d, taken in enumerate(self._taken):
                self.free_blocks[d] = self.free_blocks[d][int(taken.item()):]
        self._taken = []
