"""Calls of the serving step's operators and of the decodes beside them that
share something with another call or lie at the edge of what the header
allows: one workspace over many shapes, streams, host threads, inputs near
the ends of fp32."""
import ctypes
import threading

import numpy as np
import pytest
import torch

from oracle import step_oracle as so
from sparse_mla_decode_dcp_gb300 import build as smla_build
from sparse_mla_decode_dcp_gb300 import capi
from test_step_operators import (FORMATS, SCALE, _check, _err, _f64, _i32, _np, _paged, _q,
                                 _random_cache)


@pytest.fixture(scope="module")
def lib():
    smla_build.build()
    return capi.load()


# ------------------------------------------------------------- workspaces
def _decode_calls(dev, H):
    """Decodes of many shapes: (workspace bytes, call(out, lse, workspace))."""
    rng = np.random.default_rng(5)
    caches = {f: _random_cache(300, f, 1, dev) for f in FORMATS}
    calls = []

    def add(T, size, run):
        calls.append((T, size, run))

    for T, K in [(38, 2048), (34, 2048), (80, 2048), (77, 2048), (2, 2048), (25, 2000), (9, 700), (90, 2047)]:
        slots = rng.integers(0, 300, (T, K)).astype(np.int32)
        slots[rng.random((T, K)) < 0.1] = -1
        slots[T // 2] = -1
        q, sl = _q(T, H, dev, T), _i32(slots, dev)
        add(T, capi.fp4_decode_workspace_size(T, H, K),
            lambda o, l, w, q=q, sl=sl: capi.sparse_mla_decode_fp4(q, caches["fp4"], sl, SCALE, out=o, lse=l,
                                                                    workspace=w))
        add(T, capi.decode_workspace_size(T, H, K),
            lambda o, l, w, q=q, sl=sl: capi.sparse_mla_decode(q, caches["fp8"], sl, SCALE, out=o, lse=l,
                                                                workspace=w))
    for fmt in FORMATS:
        for ctx in ([2300, 60, 2300], [2200] * 30 + [5] * 8, [2100] * 33):
            pools, tables = _paged(ctx, 2, 16, 1, fmt, len(ctx), dev)
            q, c = _q(len(ctx), H, dev, len(ctx)), _i32(ctx, dev)
            args = (q, c, 2400, 1, 2100, 30, pools, tables, 16, SCALE)
            add(len(ctx), capi.window_decode_workspace_size(len(ctx), H, 2400, 2100, 30, 2),
                lambda o, l, w, a=args: capi.dcp_window_mla_decode(*a, out=o, lse=l, workspace=w))
            if fmt == "fp8":
                add(len(ctx), capi.dense_decode_workspace_size(len(ctx), H, 2400, 2),
                    lambda o, l, w, a=args: capi.dcp_dense_mla_decode(*a[:4], *a[6:], out=o, lse=l, workspace=w))
    return calls


@pytest.mark.gpu
@pytest.mark.parametrize("H", [16, 37])
def test_one_workspace_serves_calls_of_many_shapes(cuda_device, H):
    """Batches of changing size, of all decodes, in turn on one workspace: the
    bits of a call with its own workspace, whatever ran before."""
    dev = cuda_device
    calls = [c for c in _decode_calls(dev, H) if c[1] > 0]
    assert len(calls) >= 12
    shared = torch.zeros(max(n for _, n, _ in calls), dtype=torch.uint8, device=dev)

    def result(call, T, ws):
        out = torch.full((T, H, 512), 7.0, dtype=torch.bfloat16, device=dev)
        lse = torch.full((T, H), 7.0, device=dev)
        call(out, lse, ws)
        return out, lse

    _err()
    want = [result(run, T, torch.zeros(n, dtype=torch.uint8, device=dev)) for T, n, run in calls]
    rng = np.random.default_rng(H)
    for _ in range(3):
        for i in rng.permutation(len(calls)):
            T, n, run = calls[i]
            out, lse = result(run, T, shared)
            assert torch.equal(lse, want[i][1]) and torch.equal(out, want[i][0]), i
            assert not shared[:16384 * 8].any()  # the counters, zero again
    assert _err() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T", [16384, 16385])
def test_splits_merge_on_both_sides_of_the_rows_with_counters(cuda_device, T):
    dev, H, K = cuda_device, 1, 2050
    rng = np.random.default_rng(T)
    cache = _random_cache(300, "fp4", 1, dev)
    slots = np.full((T, K), -1, dtype=np.int32)
    slots[:, ::50] = rng.integers(0, 300, (T, K // 50))
    slots[5] = -1
    q = _q(T, H, dev, 1)
    ws = capi.alloc_fp4_decode_workspace(T, H, K, dev)
    _err()
    for _ in range(2):
        out, lse = capi.sparse_mla_decode_fp4(q, cache, _i32(slots, dev), SCALE, workspace=ws)
    assert _err() == 0
    rows, qf = _np(cache), _f64(q)
    at = [0, 5, 77, T // 2, T - 1]
    _check(out[at], lse[at], [so.attend(qf[t], rows[slots[t][slots[t] >= 0]], SCALE) for t in at])


def test_workspace_sizes_hold_the_counters_of_any_call(lib):
    """Every size that is not 0 begins with the same counters' region, so no
    call's partials reach into it."""
    counters = 16384 * 2 * 4

    def up(n):
        return -(-n // 256) * 256

    for size in (capi.fp4_decode_workspace_size, capi.decode_workspace_size):
        for T, H, K in [(1, 1, 2048), (38, 128, 2048), (34, 16, 2048), (80, 5, 2048), (20000, 3, 2049)]:
            n = size(T, H, K)
            # some count of splits accounts for the whole size
            assert n == 0 or any(n == counters + up(T * s * H * 1024) + up(T * s * H * 16) + 256 for s in range(2, 77))
    assert capi.fp4_decode_workspace_size(38, 128, 2048) > 0


# ---------------------------------------------------------------- streams
def _steps(dev, fmt, stream, ctx, kv, steps):
    """A prefill and decode steps at once behind the constructor: the results
    and everything the steps have written."""
    from sparse_mla_decode_dcp_gb300.pipeline import DcpServingStep
    step = DcpServingStep(num_reqs=3, tokens_per_req=2, heads=16, dcp=3, block_size=8, blocks_per_rank=20000,
                          max_ctx=3100, window=2500, sinks=5, fmt=fmt, sm_scale=SCALE, device=dev, stream=stream)
    step.prefill(ctx, ctx, kv)
    step.take_blocks()
    got = []
    for c, k, q in steps:
        out, lse = step.run(c, k, q)
        with torch.cuda.stream(stream):
            got += [out.clone(), lse.clone()]
        step.take_blocks()
    return got + step.block_tables + step.pools


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_serving_step_on_a_stream_behind_a_busy_one(cuda_device, fmt):
    """Constructed with a stream while the current stream has work queued, and
    used at once: the same results as on the current stream."""
    dev = cuda_device
    ctx = [2400, 1, 33]
    g = torch.Generator(device=dev).manual_seed(3)

    def rows(n):
        return torch.randn((n, 576), generator=g, device=dev).to(torch.bfloat16)

    inputs = (_i32(ctx, dev), rows(sum(ctx)),
              [(_i32([c + 2 * (i + 1) for c in ctx], dev), rows(6), _q(6, 16, dev, i)) for i in range(2)])
    want = _steps(dev, fmt, None, *inputs)
    torch.cuda.synchronize()
    s = torch.cuda.Stream(dev)
    torch.cuda._sleep(400_000_000)  # about 0.2 s on the current stream
    got = _steps(dev, fmt, s, *inputs)
    s.synchronize()
    still_busy = not torch.cuda.current_stream(dev).query()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert still_busy  # nothing of the steps had waited for the current stream


@pytest.mark.gpu
def test_decodes_on_a_stream_with_their_own_workspace(cuda_device):
    """Workspaces that a call allocates for itself are filled, and belong to,
    the stream it launches on, while the current stream is busy."""
    dev = cuda_device
    ctx, H = [2300, 60, 2300], 16
    pools, tables = _paged(ctx, 1, 16, 1, "fp8", 3, dev)
    q, c, req = _q(3, H, dev), _i32(ctx, dev), _i32(range(3), dev)
    ids = _i32(np.stack([np.random.default_rng(b).permutation(2048) % n for b, n in enumerate(ctx)]), dev)
    scores = torch.randn((2, 1 << 18), generator=torch.Generator(device=dev).manual_seed(1), device=dev)
    n_cand = _i32([1 << 18, 200000], dev)
    cache4 = _random_cache(2400, "fp4", 1, dev)
    calls = [
        lambda **k: capi.sparse_mla_decode(q, pools[0], ids, SCALE, **k),
        lambda **k: capi.dcp_sparse_mla_decode_fused(q, req, ids, pools, tables, 16, SCALE, **k),
        lambda **k: capi.dcp_dense_mla_decode(q, c, 2300, 1, pools, tables, 16, SCALE, **k),
        lambda **k: capi.sparse_mla_decode_fp4(q, cache4, ids, SCALE, **k),
    ]
    want = [call() for call in calls]
    top = capi.topk_select(scores, n_cand, 64, workspace=True)
    outs = [(torch.empty_like(o), torch.empty_like(l)) for o, l in want]
    torch.cuda.synchronize()
    s = torch.cuda.Stream(dev)
    torch.cuda._sleep(200_000_000)
    noise = []
    for call, (o, l) in zip(calls, outs):
        call(out=o, lse=l, stream=s)
        noise.append(torch.full((4 << 20,), 255, dtype=torch.uint8, device=dev))  # a reused block would show
    got = capi.topk_select(scores, n_cand, 64, workspace=True, stream=s)
    torch.cuda.synchronize()
    for (o, l), (wo, wl) in zip(outs, want):  # bit by bit: slots nobody holds give NaN
        assert torch.equal(o.view(torch.int16), wo.view(torch.int16))
        assert torch.equal(l.view(torch.int32), wl.view(torch.int32))
    assert torch.equal(got, top)


@pytest.mark.gpu
def test_decode_step_on_a_stream_behind_a_busy_one(cuda_device):
    from sparse_mla_decode_dcp_gb300 import inputs
    from sparse_mla_decode_dcp_gb300.pipeline import DcpDecodeStep
    dev = cuda_device
    wl = inputs.make_workload("tiny", seed=0, device=dev)
    want = [t.clone() for t in DcpDecodeStep(wl, device=dev).run()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream(dev)
    torch.cuda._sleep(200_000_000)
    got = DcpDecodeStep(wl, device=dev, stream=s).run()
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
