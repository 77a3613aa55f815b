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


@pytest.mark.parametrize("ctx", [2 ** 31 - 1, 2 ** 31 - 100, 2 ** 31 - 2048, 2 ** 31 - 2049])
def test_dense_contexts_up_to_31_bits_are_split(lib, ctx):
    """A bound of 2^31 - 1 positions takes as many key ranges as one of a few
    thousand fewer, and the workspace they need, not a single range of 2048."""
    counters = 16384 * 2 * 4 + 256
    for D, I, rank, held in [(4, 1, -1, ctx), (1, 1000, 0, ctx), (1, 2 ** 30, 0, ctx), (2, 16, 1, ctx // 2)]:
        n = capi.dense_decode_workspace_size(1, 1, ctx, D, I, rank)
        assert n >= counters + -(-held // 2048) * (1024 + 16), (D, I)
    arr = lambda typ, x: (typ * 1)(x)  # noqa: E731
    st = lib.smla_dcp_dense_mla_decode(
        0x10000, 1, 1, 1, ctypes.c_float(0.07), 0x10000, ctx, 1, -1, 16, 1, arr(ctypes.c_void_p, 0x10000),
        arr(ctypes.c_int64, 100), arr(ctypes.c_void_p, 0x10000), arr(ctypes.c_int64, 4),
        arr(ctypes.c_int32, 4), 0x10000, 0x10000, None, 0, None)
    assert st == capi.SMLA_ERR_WORKSPACE


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
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


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


@pytest.mark.gpu
def test_serving_step_called_again_after_a_refusal(cuda_device):
    """A prefill and a step that are refused half-way (rows of a wrong width, a
    query of a wrong shape) take no blocks: called again they do what they
    would have done."""
    from sparse_mla_decode_dcp_gb300.pipeline import DcpServingStep
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(4)
    ctx, more = _i32([60, 9], dev), _i32([61, 10], dev)
    kv, kv1 = (torch.randn((n, 576), generator=g, device=dev).to(torch.bfloat16) for n in (69, 2))
    q = _q(2, 4, dev)

    def make():
        return DcpServingStep(num_reqs=2, tokens_per_req=1, heads=4, dcp=2, block_size=4, blocks_per_rank=40,
                              max_ctx=100, window=50, sinks=3, device=dev)

    want = make()
    want.prefill(ctx, ctx, kv)
    want.take_blocks()
    out, lse = (t.clone() for t in want.run(more, kv1, q))
    want.take_blocks()
    step = make()
    with pytest.raises(ValueError):
        step.prefill(ctx, ctx, kv[:, :568].contiguous())
    step.prefill(ctx, ctx, kv)
    step.take_blocks()
    with pytest.raises(ValueError):
        step.run(more, kv1, q[:, :, :512].contiguous())
    with pytest.raises(ValueError):
        step.run(more, kv1.float(), q)
    o, l = step.run(more, kv1, q)
    assert torch.equal(o, out) and torch.equal(l, lse)
    step.take_blocks()
    for a, b in zip(step.free_blocks + step.block_tables + step.pools,
                    want.free_blocks + want.block_tables + want.pools):
        assert torch.equal(a, b)


# ------------------------------------------------------------ ends of fp32
def _fp8_rows(y):
    """Codes and scales of float64 latents y as the header defines them: a
    group whose scale is below 2^-126 is stored as zeros."""
    code, scale = so.quantise_fp8(y)
    low = scale < 2.0 ** -126
    return np.where(np.repeat(low, 128, axis=1), 0, code), np.where(low, np.float32(0), scale)


def _write_latents(x, gamma, fmt, eps=1e-6):
    dev = x.device
    kv = torch.cat([x, torch.zeros((x.shape[0], 64), dtype=x.dtype, device=dev)], 1).contiguous()
    cache = torch.full((x.shape[0], FORMATS[fmt]), 0x5A, dtype=torch.uint8, device=dev)
    capi.mla_cache_write(kv, torch.arange(x.shape[0], dtype=torch.int32, device=dev), cache, gamma=gamma, eps=eps)
    return _np(cache)


@pytest.mark.gpu
@pytest.mark.parametrize("rms", [2.0 ** -40, 2.0 ** -10, 1.0, 2.0 ** 40])
def test_write_tiny_groups(cuda_device, rms):
    """Groups of a normalised row from ordinary size down to below the least
    scale, exact zeros among their values, by small gammas and small latents."""
    dev = cuda_device
    g = torch.Generator().manual_seed(7)
    T = 40
    x = torch.randn((T, 512), generator=g, dtype=torch.float64)
    x[:, 5::37] = 0
    x = (x * rms).to(torch.bfloat16)
    steps = torch.arange(T * 4, dtype=torch.float64).view(T, 4) * -0.85  # 2^0 .. 2^-135 in all
    for t in range(T):
        row = (1 + 0.3 * torch.randn(512, generator=g, dtype=torch.float64))
        gamma = (row * torch.exp2(steps[t]).repeat_interleave(128)).to(torch.bfloat16)
        got = _write_latents(x[t:t + 1].to(dev), gamma.to(dev), "fp8", eps=1e-30)
        y = so.normalise(_f64(x[t:t + 1]), _f64(gamma), 1e-30)
        code, scale = _fp8_rows(y)
        assert np.array_equal(got[:, 512:528].copy().view("<f4"), scale), t
        assert np.array_equal(got[:, :512], code), t


@pytest.mark.gpu
def test_write_tiny_latents(cuda_device):
    """The same from the latents' side: groups of one row far apart, with and
    without a norm."""
    dev = cuda_device
    g = torch.Generator().manual_seed(8)
    T = 160
    x = torch.randn((T, 4, 128), generator=g, dtype=torch.float64)
    x[:, :, 3::29] = 0
    x[:, 1] *= torch.exp2(-torch.arange(T, dtype=torch.float64)[:, None] * 0.85)
    x[:, 2] *= 2.0 ** -100
    x[:, 3] *= 2.0 ** -60
    x = x.view(T, 512).to(torch.bfloat16)
    gamma = torch.full((512,), 1.25, dtype=torch.bfloat16)
    gamma[400:] = 2.0 ** -55
    for gm in (None, gamma):
        got = _write_latents(x.to(dev), None if gm is None else gm.to(dev), "fp8")
        y = so.normalise(_f64(x), None if gm is None else _f64(gm), 1e-6)
        code, scale = _fp8_rows(y)
        assert np.array_equal(got[:, 512:528].copy().view("<f4"), scale)
        assert np.array_equal(got[:, :512], code)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_write_past_fp32(cuda_device, fmt):
    """A normalised value past fp32 makes its group's scale NaN, as an
    infinite one does; the row's other groups are as they are."""
    dev = cuda_device
    g = torch.Generator().manual_seed(9)
    x = torch.randn((8, 512), generator=g, dtype=torch.float64) * 0.01
    x[:, 37] = 0.5  # 50 times the others: 2^127 times its norm does not fit
    x = x.to(torch.bfloat16)
    gamma = torch.ones(512, dtype=torch.bfloat16)
    gamma[:128] = 2.0 ** 127
    gamma[0:16] = 2.0 ** 100
    got = _write_latents(x.to(dev), gamma.to(dev), fmt)
    y = so.normalise(_f64(x), _f64(gamma), 1e-6)
    assert (np.abs(y) > np.finfo(np.float32).max).any(axis=1).all()
    with np.errstate(invalid="ignore"):
        lat = so.parse(got)[0]
    size = 128 if fmt == "fp8" else 16
    past = np.repeat((np.abs(y) > np.finfo(np.float32).max).reshape(8, -1, size).any(axis=2), size, axis=1)
    assert np.array_equal(np.isnan(lat), past)
    if fmt == "fp8":
        code, scale = _fp8_rows(np.where(past, 0, y))
        assert np.array_equal(got[:, :512][~past], code[~past])
        assert np.array_equal(got[:, 512:528].copy().view("<f4")[:, 1:], scale[:, 1:])


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_write_of_values_far_below_their_group(cuda_device, fmt):
    """Quotients too small for fp32, of either sign, beside ones on a rounding
    border (which send the row through the exact quotients)."""
    dev = cuda_device
    x = torch.zeros((8, 512), dtype=torch.float64)
    top = 448.0 * 2.0 ** 52 if fmt == "fp8" else 6.0 * 256
    unit = 2.0 ** 52 if fmt == "fp8" else 256.0
    x[:, ::16] = top
    x[:, 1::16] = 8.5 * unit if fmt == "fp8" else 2.5 * unit  # ties
    x[:, 2::16] = -2.0 ** -110
    x[:, 3::16] = 2.0 ** -110
    x[:, 4::16] = -2.0 ** -133
    x[:, 5::16] = -2.0 ** -130
    x = x.to(torch.bfloat16)
    got = _write_latents(x.to(dev), None, fmt)
    code, scale = so.quantise_fp8(_f64(x)) if fmt == "fp8" else so.quantise_fp4(_f64(x))
    if fmt == "fp8":
        assert np.array_equal(got[:, 512:528].copy().view("<f4"), scale)
        assert np.array_equal(got[:, :512], code)
    else:
        assert np.array_equal(got[:, 256:288], scale)
        assert np.array_equal(got[:, :256], code[:, 0::2] | (code[:, 1::2] << 4))


@pytest.mark.gpu
@pytest.mark.parametrize("D,I", [(16, 1 << 28), (16, (1 << 27) + 1), (9, 1 << 28)])
def test_dense_decode_of_one_rank_with_rounds_past_32_bits(cuda_device, D, I):
    """One rank holds the whole context, the others nothing: runs of I
    positions, D runs a round, more than 32 bits count."""
    dev = cuda_device
    ctx, bs = [150], 16
    pools, tables = _paged(ctx, 1, bs, 1, "fp8", 1, dev)
    q, c = _q(1, 1, dev), _i32(ctx, dev)
    want = so.attend(_f64(q)[0], _np(pools[0])[[int(tables[0][0, t // bs]) * bs + t % bs for t in range(150)]],
                     SCALE, 2.0 ** -11)
    ws = torch.zeros(capi.dense_decode_workspace_size(1, 1, 150, D, I, 0), dtype=torch.uint8, device=dev)
    _err()
    for rank in (0, 1, D - 1):
        use = [pools[0] if d == rank else None for d in range(D)]
        tab = [tables[0] if d == rank else None for d in range(D)]
        out, lse = capi.dcp_dense_mla_decode(q, c, 150, 1, use, tab, bs, SCALE, rank=rank, interleave=I,
                                             workspace=ws)
        if rank == 0:
            _check(out, lse, [want])
        else:
            assert torch.isneginf(lse).all() and not out.any()
    assert _err() == 0


# ------------------------------------------------- overlapping launches
@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_rows_overwritten_and_read_again_without_a_wait(cuda_device, fmt):
    """Step maps, cache write, gather and decodes in one chain of overlapping
    launches, over and over on the same slots with other rows, other tables
    and other lists each time: every reader sees what the writer before it
    wrote, as when the host waits in between."""
    dev = cuda_device
    B, H, bs, n, rounds = 4, 16, 16, 70, 24
    N = B * n
    g = torch.Generator(device=dev).manual_seed(2)
    kv = [torch.randn((N, 576), generator=g, device=dev).to(torch.bfloat16) for _ in range(rounds)]
    free = [torch.randperm(B * 5, generator=g, device=dev).to(torch.int32) for _ in range(rounds)]
    ctx, ql = _i32([n] * B, dev), _i32([n] * B, dev)
    req, topk = _i32(range(B), dev), _i32([list(range(n))] * B, dev)
    cos_sin, q = torch.rand((n, 64), generator=g, device=dev), _q(B, H, dev)
    cache = torch.zeros((B * 5 * bs, FORMATS[fmt]), dtype=torch.uint8, device=dev)
    table = torch.full((B, 5), -1, dtype=torch.int32, device=dev)
    maps = capi.alloc_step_maps(B, N, dev)
    ws = [capi.alloc_window_decode_workspace(B, H, n, n, 0, 1, 1, -1, dev),
          capi.alloc_fp4_decode_workspace(B, H, n, dev)]

    def outs():
        return (torch.empty((N, 576), dtype=torch.bfloat16, device=dev),
                *(torch.empty(s, dtype=t, device=dev) for _ in range(2)
                  for s, t in (((B, H, 512), torch.bfloat16), ((B, H), torch.float32))))

    def chain(i, o, wait):
        capi.dcp_step_maps(ctx, ql, free[i], table, N, 1, 0, bs, out=maps)
        wait()
        capi.mla_cache_write(kv[i], maps.slots, cache, positions=maps.positions, cos_sin=cos_sin)
        wait()
        capi.mla_cache_gather(cache, maps.slots, out=o[0])
        wait()
        capi.dcp_window_mla_decode(q, ctx, n, 1, n, 0, [cache], [table], bs, SCALE, out=o[1], lse=o[2],
                                   workspace=ws[0])
        wait()
        if fmt == "fp4":
            capi.dcp_sparse_mla_decode_fused_fp4(q, req, topk, [cache], [table], bs, SCALE, out=o[3], lse=o[4],
                                                 workspace=ws[1])
        else:
            o[3].zero_()
            o[4].zero_()
        wait()

    got, want = [outs() for _ in range(rounds)], [outs() for _ in range(rounds)]
    _err()
    for i in range(rounds):
        chain(i, want[i], torch.cuda.synchronize)
    for i in range(rounds):
        chain(i, got[i], lambda: None)
    torch.cuda.synchronize()
    assert _err() == 0
    for i in range(rounds):
        for a, b in zip(got[i], want[i]):
            assert torch.equal(a, b), i
    assert not torch.equal(want[0][1], want[1][1])


# ------------------------------------------------------------ host threads
@pytest.mark.gpu
def test_step_maps_from_host_threads_with_large_batches(cuda_device):
    """Batches that need different amounts of shared memory, from several host
    threads and streams: no launch is refused, and every map is right."""
    dev = cuda_device
    failed = []

    def work(B, rounds):
        try:
            s = torch.cuda.Stream(dev)
            with torch.cuda.stream(s):
                ctx, ql = _i32([5] * B, dev), _i32([1] * B, dev)
                free, bt = _i32(range(B), dev), _i32([[7]] * B, dev)
                out = capi.alloc_step_maps(B, B, dev, s)
                want = _i32([7 * 8 + 4] * B, dev)
                for _ in range(rounds):
                    capi.dcp_step_maps(ctx, ql, free, bt, B, 1, 0, 8, out=out, stream=s)
                s.synchronize()
                assert torch.equal(out.slots, want)
        except Exception as e:  # noqa: BLE001
            failed.append((B, e))

    threads = [threading.Thread(target=work, args=(B, 4000)) for B in (8192, 3000, 5000, 100)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    assert _err() == 0


# ---------------------------------------------------------- refused launches
@pytest.mark.gpu
def test_a_refused_launch_is_reported_once(cuda_device):
    """A launch refused on the host (on a stream whose capture has become
    invalid) fails its own call and no later one."""
    dev = cuda_device
    drv = ctypes.CDLL("libcuda.so.1")
    handle = ctypes.c_void_p
    cache = _random_cache(8, "fp4", 1, dev)
    slots, out = _i32(range(8), dev), torch.empty((8, 576), dtype=torch.bfloat16, device=dev)
    ids, table = _i32([[0, 5, 3, -1]], dev), _i32([[1]], dev)
    req = _i32([0], dev)
    ctx, ql, free, maps = _i32([8], dev), _i32([0], dev), _i32([], dev), capi.alloc_step_maps(1, 1, dev)
    q = _q(1, 4, dev)
    o, l = torch.empty((1, 4, 512), dtype=torch.bfloat16, device=dev), torch.empty((1, 4), device=dev)

    def healthy():
        return capi.dcp_filter_convert_index(req, table, ids, 1, 0, 8)[0]

    want = healthy()
    capi.mla_cache_gather(cache, slots, out=out)
    torch.cuda.synchronize()
    s = torch.cuda.Stream(dev)
    for call in (lambda: capi.mla_cache_gather(cache, slots, out=out, stream=s),
                 lambda: capi.dcp_step_maps(ctx, ql, free, table, 1, 1, 0, 8, out=maps, stream=s),
                 lambda: capi.sparse_mla_decode_fp4(q, cache, ids, SCALE, out=o, lse=l, stream=s)):
        st = handle(s.cuda_stream)
        assert drv.cuStreamBeginCapture_v2(st, 2) == 0  # of this stream alone
        assert drv.cuStreamSynchronize(st) != 0  # not allowed in a capture: it is invalid from here on
        with pytest.raises(capi.SmlaError):
            call()
        got = healthy()
        graph = handle()
        assert drv.cuStreamEndCapture(st, ctypes.byref(graph)) != 0
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    capi.mla_cache_gather(cache, slots, out=out, stream=s)  # and the stream works again
    torch.cuda.synchronize()
    assert _err() == 0


# ---------------------------------------------------------------- rounding
def _bf16_once(x):
    """float64 to bf16 (as float64), one rounding, ties to even (normal values)."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 256.0) / 256.0, e)


@pytest.mark.gpu
def test_gather_of_8_bit_rows_rounds_to_bf16_once(cuda_device):
    """Scales whose products with a code lie so close to the middle of two
    bf16 that fp32 would round them onto it."""
    dev = cuda_device
    rng = np.random.default_rng(4)
    # e4m3 codes 1.875, 1.625, 1.125 and their multiples by powers of two
    codes = np.array([0x3F, 0x3D, 0x39, 0xBF, 0x47, 0x35], dtype=np.uint8)
    value = np.array([1.875, 1.625, 1.125, -1.875, 3.75, 0.8125])
    n = 6000
    at = rng.integers(0, len(codes), (n, 4))
    middle = (rng.integers(128, 256, (n, 4)) + 0.5) * 2.0 ** rng.integers(-20, 10, (n, 4))
    scale = (middle / np.abs(value[at])).astype(np.float32)
    rows = np.zeros((n, 656), dtype=np.uint8)
    rows[:, :512] = np.repeat(codes[at], 128, axis=1)
    rows[:, 512:528] = scale.view(np.uint8).reshape(n, 16)
    got = capi.mla_cache_gather(torch.from_numpy(rows).to(dev), _i32(range(n), dev))
    exact = value[at] * scale.astype(np.float64)  # 4 + 24 bits
    twice = _bf16_once(exact.astype(np.float32).astype(np.float64))
    want = _bf16_once(exact)
    assert (want != twice).sum() > 1000  # the inputs tell one rounding from two
    assert np.array_equal(_f64(got)[:, :512], np.repeat(want, 128, axis=1))
    full = capi.mla_cache_gather(torch.from_numpy(rows).to(dev), _i32(range(n), dev), dtype=torch.float32)
    assert np.array_equal(_np(full)[:, :512], np.repeat(exact.astype(np.float32), 128, axis=1))


# ---------------------------------------------------------------- refusals
def test_rows_of_more_entries_than_32_bits_count_are_refused(lib):
    """Not taken as the low 32 bits of their count (of which 64 would run)."""
    q = torch.zeros((0, 4, 576), dtype=torch.bfloat16)
    out, lse = torch.zeros((0, 4, 512), dtype=torch.bfloat16), torch.zeros((0, 4))
    ids = torch.zeros((0, (1 << 32) + 64), dtype=torch.int32)
    cache, table = torch.zeros((8, 416), dtype=torch.uint8), torch.zeros((1, 1), dtype=torch.int32)
    ws = torch.zeros(1, dtype=torch.uint8)
    with pytest.raises(ValueError, match="too many entries"):
        capi.sparse_mla_decode_fp4(q, cache, ids, SCALE, out=out, lse=lse, workspace=ws)
    with pytest.raises(ValueError, match="too many entries"):
        capi.dcp_sparse_mla_decode_fused_fp4(q, torch.zeros(0, dtype=torch.int32), ids, [cache], [table], 8,
                                             SCALE, out=out, lse=lse, workspace=ws)
