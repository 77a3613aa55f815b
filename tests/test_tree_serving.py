"""A server that drafts: projections, tree attention, the walk and the move to
the cache run together through the pipeline, step after step, against the
float64 definitions of oracle/, and against a server that was given the same
tokens at once."""
import math

import numpy as np
import pytest
import torch

from oracle import fp8_oracle as fo
from oracle import step_oracle as so
from oracle import tree_oracle as to
from oracle.smla_oracle import bf16_bits_to_f64
from sparse_mla_decode_dcp_gb300 import capi
from sparse_mla_decode_dcp_gb300.pipeline import DcpServingStep, Fp8Projections

SCALE = 1.0 / math.sqrt(192.0)
KEY_STEP = {"fp8": 2.0 ** -11, "fp4": 0.0}
B, D, BS, H, N, CTX = 3, 3, 8, 16, 12, 200


def _np(t):
    return t.cpu().numpy()


def _i32(a, dev):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).to(dev)


def _f64(t):
    return bf16_bits_to_f64(_np(t.contiguous().view(torch.int16)).astype(np.uint16))


def _err():
    return capi.get_device_error(clear=True)


def _table(n, dev):
    a = torch.arange(n)[:, None] * torch.exp(torch.arange(32) * -0.3)
    return torch.cat([a.cos(), a.sin()], 1).float().to(dev)


def _server(dev, fmt, **kw):
    g = torch.Generator(device=dev).manual_seed(1)
    gamma = (1 + 0.2 * torch.randn(512, generator=g, device=dev)).to(torch.bfloat16)
    a = dict(num_reqs=B, tokens_per_req=1, heads=H, dcp=D, block_size=BS, blocks_per_rank=40, max_ctx=CTX,
             window=60, sinks=5, fmt=fmt, gamma=gamma, cos_sin=_table(CTX + N, dev), sm_scale=SCALE, interleave=2,
             max_nodes=N, device=dev)
    return DcpServingStep(**{**a, **kw})


def _slot(step, tables, b, p):
    """(pool, slot) of a cached position."""
    I = step.interleave
    lp = p // (I * D) * I + p % I
    return p // I % D, int(tables[p // I % D][b][lp // BS]) * BS + lp % BS


def _cached(step, lengths):
    """Every request's cache rows, in order."""
    pools, tables = [_np(p) for p in step.pools], [_np(t) for t in step.block_tables]
    rows = []
    for b, n in enumerate(lengths):
        at = [_slot(step, tables, b, p) for p in range(n)]
        rows.append(np.stack([pools[d][s] for d, s in at]))
    return rows


def _drafts(rng, rows, dev):
    """Trees of 0 .. N nodes for B requests; few tokens, so that walks go on."""
    nodes = rng.integers(1, N + 1, B)
    nodes[rng.integers(B)] = rng.integers(2) * N  # an empty or a full one
    starts = np.concatenate([[0], np.cumsum(nodes)])
    parents = np.concatenate([to.random_tree(rng, n) for n in nodes] + [np.full(rows - starts[-1], -1)])
    tokens, targets = rng.integers(0, 2, rows), rng.integers(0, 2, rows)
    return starts, parents.astype(np.int64), tokens, targets


def _bf16(shape, seed, dev):
    g = torch.Generator(device=dev).manual_seed(seed)
    return torch.randn(shape, generator=g, device=dev).to(torch.bfloat16)


def _weight(shape, seed, dev):
    """Codes and block scales of a weight whose rows keep their input's size."""
    g = torch.Generator(device=dev).manual_seed(seed)
    codes = (torch.randn(shape, generator=g, device=dev) * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
    *batch, R, K = shape
    s = torch.rand((*batch, -(-R // 128), -(-K // 128)), generator=g, device=dev) + 0.5
    rows = capi.alloc_fp8_rows(shape, dev).codes  # 16-byte rows, as the product takes them
    rows.copy_(codes)
    return capi.Fp8Rows(rows, s / (60 * math.sqrt(K)))


def _projections(dev, C=200, P=48, V=40, E=70, **kw):
    return Fp8Projections(_weight((H * (P + 64), C), 1, dev), _weight((H, 512, P), 2, dev),
                          _weight((H, V, 512), 3, dev), _weight((E, H * V), 4, dev), B * N,
                          cos_sin=_table(CTX + N, dev), **kw)


def _check_product(x, w, got):
    """`got` is x (as it is, in bf16) in 8 bits times the weight w."""
    for g in range(x.shape[0]):
        codes, scales = fo.quantise(_f64(x[g]))
        want, tol = fo.matmul(codes, scales, _np(w.codes[g].view(torch.uint8)), _np(w.scales[g]), 2.0 ** -8)
        assert np.all(np.abs(_f64(got[g]) - want) <= tol)


def _check_query(p, x, positions, q):
    heads = p.heads[:len(x)]
    one = lambda w: capi.Fp8Rows(w.codes[None], w.scales[None])  # noqa: E731
    _check_product(x[None], one(p.w_q), heads.reshape(1, len(x), -1))
    _check_product(heads[..., :p.P].transpose(0, 1), p.w_k, q[..., :512].transpose(0, 1))
    z, cs = _f64(heads[..., p.P:]), _f64_table(p.cos_sin)[_np(positions)][:, None]
    want = so.rotate(z.reshape(-1, 64), np.broadcast_to(cs, (*z.shape[:2], 64)).reshape(-1, 64), p.rope_pairs)
    got = _f64(q[..., 512:]).reshape(-1, 64)
    # two products and their sum round in fp32, then the sum to bf16
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 3 * 2.0 ** -24 * 2 * np.abs(z).max())


def _f64_table(t):
    return _np(t).astype(np.float64)


def _check_output(p, latent, y):
    values = p.values[:len(latent)]
    _check_product(latent.transpose(0, 1), p.w_v, values.transpose(0, 1))
    _check_product(values.reshape(1, len(latent), -1), capi.Fp8Rows(p.w_o.codes[None], p.w_o.scales[None]), y[None])


@pytest.mark.gpu
@pytest.mark.parametrize("rope_pairs", [True, False])
@pytest.mark.parametrize("T", [1, 5, 36])
def test_projections_match_their_definition(cuda_device, T, rope_pairs):
    p = _projections(cuda_device, rope_pairs=rope_pairs)
    x, pos = _bf16((T, 200), 7, cuda_device), _i32(np.arange(T) * 5, cuda_device)
    _err()
    q = p.query(x, pos)
    _check_query(p, x, pos, q)
    latent = _bf16((T, H, 512), 8, cuda_device)
    _check_output(p, latent, p.output(latent))
    p.cos_sin = None
    assert torch.equal(p.query(x)[..., 512:], p.heads[:T, :, p.P:])
    assert _err() == 0


@pytest.mark.gpu
def test_projections_of_no_rows_and_of_positions_past_the_table(cuda_device):
    p = _projections(cuda_device)
    n = len(p.cos_sin)
    assert p.query(_bf16((0, 200), 1, cuda_device), _i32([], cuda_device)).shape == (0, H, 576)
    assert p.output(_bf16((0, H, 512), 1, cuda_device)).shape == (0, p.E)
    x = _bf16((4, 200), 2, cuda_device)
    got = p.query(x, _i32([n, -1, 2 ** 31 - 1, 5], cuda_device)).clone()
    assert torch.equal(got, p.query(x, _i32([n - 1, 0, n - 1, 5], cuda_device)))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_no_drafts_change_nothing(cuda_device, fmt):
    """Trees of no nodes, all padding or no rows at all: nothing is accepted,
    the cache and its block tables stay as they were."""
    dev, ctx = cuda_device, [90, 5, 40]
    step = _ready(dev, fmt, ctx)
    keep = _cached(step, ctx)
    pre, rs = _i32(ctx, dev), _i32([0] * (B + 1), dev)
    _err()
    for T in (7, 0):
        par = _i32([-1] * T, dev)
        step.tree_out.fill_(3)
        out, lse = step.verify(pre, par, rs, _bf16((T, 576), 1, dev), _bf16((T, H, 576), 2, dev))
        assert out.shape == (T, H, 512) and out.eq(3).all()
        walk, after = step.commit(pre, par, par, par, rs)
        assert walk.accepted.eq(0).all() and walk.rows.eq(-1).all() and walk.next_tokens.eq(-1).all()
        assert torch.equal(after, pre)
        assert all(int(t) == 0 for t in step._taken)
        step.take_blocks()
    for a, b in zip(_cached(step, ctx), keep):
        assert np.array_equal(a, b)
    assert _err() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_drafting_server(cuda_device, fmt):
    """Prefill, then rounds of trees: each part within its definition's bounds,
    the cache byte by byte that of a server which was given the accepted
    tokens at once, and its next ordinary step the same."""
    dev, rng = cuda_device, np.random.default_rng(5)
    step, proj = _server(dev, fmt), _projections(dev)
    T = B * N - 4
    ctx = np.array([60, 0, 17])
    kv = _bf16((int(ctx.sum()), 576), 2, dev)
    hist = [list(r) for r in torch.split(kv, ctx.tolist())]
    _err()
    step.prefill(_i32(ctx, dev), _i32(ctx, dev), kv)
    step.take_blocks()
    longest = 0
    for i in range(4):
        starts, parents, tokens, targets = _drafts(rng, T, dev)
        while starts[-1] > T:  # T leaves some padding
            starts, parents, tokens, targets = _drafts(rng, T, dev)
        pre, par, rs, tok, tgt = (_i32(v, dev) for v in (ctx, parents, starts, tokens, targets))
        x, kv = _bf16((T, 200), 20 + i, dev), _bf16((T, 576), 30 + i, dev)
        maps = step.tree_positions(pre, par, rs)
        masks, positions = to.tree_maps(parents, starts, ctx, T, N)
        assert np.array_equal(_np(maps.positions), positions)
        q = proj.query(x, maps.positions)
        _check_query(proj, x, maps.positions, q)
        step.tree_out.fill_(0)
        out, lse = step.verify(pre, par, rs, kv, q)
        assert _err() == 0
        pools, tables = [_np(p) for p in step.pools], [_np(t) for t in step.block_tables]
        for b in range(B):
            for j in range(starts[b + 1] - starts[b]):
                t = starts[b] + j
                at = [_slot(step, tables, b, p) for p in range(ctx[b])]
                keys = [pools[d][s] for d, s in at]
                keys += [pools[0][40 * BS + starts[b] + m] for m in range(N) if int(masks[t, 0]) >> m & 1]
                o, l, o_tol, l_tol = so.attend(_f64(q[t]), np.stack(keys), SCALE, KEY_STEP[fmt])
                assert np.all(np.abs(_f64(out[t]) - o) <= o_tol), (i, b, j)
                assert np.all(np.abs(_np(lse[t].double()) - l) <= l_tol), (i, b, j)
        _check_output(proj, out, proj.output(out))
        walk, after = step.commit(pre, par, tok, tgt, rs)
        with pytest.raises(RuntimeError):  # its blocks are still listed as free
            step.commit(pre, par, tok, tgt, rs)
        step.take_blocks()
        acc, line, nexts = to.tree_accept(parents, tokens, targets, starts, T)
        assert np.array_equal(_np(walk.accepted), acc) and np.array_equal(_np(walk.next_tokens), nexts)
        assert np.array_equal(_np(walk.rows), line)
        at = 0
        for b in range(B):
            hist[b] += [kv[r] for r in line[at:at + acc[b]]]
            at += acc[b]
        ctx = ctx + acc
        longest = max(longest, int(acc.max()))
        assert np.array_equal(_np(after), ctx)
    assert longest > 2  # the drafts were worth something
    other = _server(dev, fmt)
    other.prefill(_i32(ctx, dev), _i32(ctx, dev), torch.stack([r for h in hist for r in h]))
    other.take_blocks()
    for a, b in zip(_cached(step, ctx), _cached(other, ctx)):
        assert np.array_equal(a, b)
    kv, q = _bf16((B, 576), 3, dev), _bf16((B, H, 576), 4, dev)
    got, want = (s.run(_i32(ctx + 1, dev), kv, q) for s in (step, other))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert _err() == 0


def _round(step, proj, s):
    """One round on the tensors of s: what it returns, and writes."""
    maps = step.tree_positions(s["pre"], s["par"], s["rs"])
    q = proj.query(s["x"], maps.positions)
    out, lse = step.verify(s["pre"], s["par"], s["rs"], s["kv"], q)
    y = proj.output(out)
    walk, after = step.commit(s["pre"], s["par"], s["tok"], s["tgt"], s["rs"])
    return [out, lse, y, *walk, after, *step.pools, *step.block_tables]


def _inputs(dev, seed, ctx):
    T = B * N
    starts, parents, tokens, targets = _drafts(np.random.default_rng(seed), T, dev)
    s = {k: _i32(v, dev) for k, v in dict(pre=ctx, par=parents, rs=starts, tok=tokens, tgt=targets).items()}
    return {**s, "x": _bf16((T, 200), seed, dev), "kv": _bf16((T, 576), seed + 50, dev)}


def _ready(dev, fmt, ctx, stream=None):
    step = _server(dev, fmt, stream=stream)
    step.prefill(_i32(ctx, dev), _i32(ctx, dev), _bf16((sum(ctx), 576), 2, dev))
    step.take_blocks()
    step.tree_out.fill_(0)
    step.tree_lse.fill_(0)
    return step


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_rounds_in_graphs(cuda_device, fmt):
    """Two servers' rounds captured into a graph each, replayed in turn and at
    once on changed inputs: the results and caches of rounds run eagerly."""
    dev, ctx = cuda_device, [90, 5, 40]
    graphs, owners = [], []  # a graph holds its server's buffers by address
    for k in range(2):
        step, proj, s = _ready(dev, fmt, ctx), _projections(dev), _inputs(dev, 10 + k, ctx)
        keep = [t.clone() for t in step.pools + step.block_tables]
        stream = torch.cuda.Stream(dev)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            _round(step, proj, s)  # whatever is loaded once is loaded
            step._taken = []
        stream.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            res = _round(step, proj, s)
        for t, old in zip(step.pools + step.block_tables, keep):
            t.copy_(old)
        graphs.append((g, s, res, keep, stream))
        owners.append((step, proj))
    for seeds in ((20, 21), (22, 23)):
        for (g, s, res, keep, stream), seed in zip(graphs, seeds):
            for t, old in zip(res[-2 * D:], keep):
                t.copy_(old)
            res[0].zero_(), res[1].zero_()
            for name, t in _inputs(dev, seed, ctx).items():
                s[name].copy_(t)
        torch.cuda.synchronize()
        for g, s, res, keep, stream in graphs:
            with torch.cuda.stream(stream):
                g.replay()
        torch.cuda.synchronize()
        for (g, s, res, keep, stream), seed in zip(graphs, seeds):
            want = _round(_ready(dev, fmt, ctx), _projections(dev), _inputs(dev, seed, ctx))
            for i, (a, b) in enumerate(zip(res, want)):
                assert bool(torch.equal(a, b)), (seed, i)
    assert _err() == 0


@pytest.mark.gpu
def test_rounds_on_a_stream_behind_a_busy_one(cuda_device):
    dev, ctx = cuda_device, [30, 60, 1]
    want = _round(_ready(dev, "fp8", ctx), _projections(dev), _inputs(dev, 3, ctx))
    stream = torch.cuda.Stream(dev)
    s = _inputs(dev, 3, ctx)
    kv, lens = _bf16((sum(ctx), 576), 2, dev), _i32(ctx, dev)
    with torch.cuda.stream(stream):
        proj = _projections(dev, stream=stream)
        table, gamma = _table(CTX + N, dev), _server(dev, "fp8").gamma
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # about 0.1 s on the current stream
    step = _server(dev, "fp8", stream=stream, gamma=gamma, cos_sin=table)
    with torch.cuda.stream(stream):
        step.prefill(lens, lens, kv)
        step.take_blocks()
        step.tree_out.fill_(0), step.tree_lse.fill_(0)
    got = _round(step, proj, s)
    with torch.cuda.stream(stream):
        got = [t.clone() for t in got]
    stream.synchronize()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("max_nodes", [-1, 257])
def test_trees_of_no_size_are_refused(max_nodes):
    with pytest.raises(ValueError):
        _server("cpu", "fp8", max_nodes=max_nodes)


@pytest.mark.gpu
def test_drafts_that_a_server_does_not_hold(cuda_device):
    dev = cuda_device
    plain, step = _server(dev, "fp8", max_nodes=0), _server(dev, "fp8")
    s = _inputs(dev, 1, [0] * B)
    q = _bf16((B * N, H, 576), 1, dev)
    with pytest.raises(ValueError):
        plain.verify(s["pre"], s["par"], s["rs"], s["kv"], q)
    more = torch.cat([s["par"], s["par"][:1]])
    with pytest.raises(ValueError):
        step.verify(s["pre"], more, s["rs"], s["kv"], q)
    with pytest.raises(ValueError):
        step.commit(s["pre"], more, s["tok"], s["tgt"], s["rs"])
    with pytest.raises(ValueError):
        _projections(dev).query(_bf16((B * N + 1, 200), 1, dev), more)
    with pytest.raises(ValueError):
        Fp8Projections(*(_weight(shape, 1, dev) for shape in ((100, 64), (2, 512, 16), (2, 16, 512), (8, 32))), 4)
