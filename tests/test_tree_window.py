"""Drafted trees under a sliding window and sinks: the operator against the
definition, row by row, and the serving step's verification against its own
decode step on the same tokens and cache."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import step_oracle as so
from oracle import tree_oracle as to
from oracle.smla_oracle import bf16_bits_to_f64
from sparse_mla_decode_dcp_gb300 import build as smla_build
from sparse_mla_decode_dcp_gb300 import capi
from sparse_mla_decode_dcp_gb300.pipeline import DcpServingStep
import test_tree_serving as serving
from test_tree_decode import BAD, FAKE, FORMATS, KEY_STEP, OK, SCALE, UNSUP, Case, _err, _i32, _np


@pytest.fixture(scope="module")
def lib():
    smla_build.build()
    return capi.load()


# ---------------------------------------------------------------- refusals
@pytest.mark.parametrize("kw,status", [
    (dict(window=0), BAD), (dict(window=-5), BAD), (dict(sinks=-1), BAD), (dict(pos=None), BAD),
    (dict(pos=FAKE + 2), BAD), (dict(q=None), BAD), (dict(T=-1), BAD), (dict(rank=2), BAD), (dict(fmt=2), BAD),
    (dict(H=129), UNSUP), (dict(n=257), UNSUP), (dict(T=0, q=None, pos=None), OK), (dict(B=0, pos=None), OK),
])
def test_argument_checks(lib, kw, status):
    a = dict(q=FAKE, T=9, H=16, pos=FAKE, B=2, n=8, window=50, sinks=3, rank=-1, fmt=0)
    a.update(kw)
    arr = lambda typ, x: (typ * 2)(x, x)  # noqa: E731
    got = lib.smla_dcp_tree_window_mla_decode(
        a["q"], a["T"], a["H"], ctypes.c_float(0.07), FAKE, FAKE, a["pos"], a["B"], 100, FAKE, a["n"], a["window"],
        a["sinks"], arr(ctypes.c_void_p, FAKE), 2, a["rank"], 16, 1, a["fmt"], arr(ctypes.c_void_p, FAKE),
        arr(ctypes.c_int64, 100), arr(ctypes.c_void_p, FAKE), arr(ctypes.c_int64, 4), arr(ctypes.c_int32, 4),
        FAKE, FAKE, None, 0, None)
    assert got == status


def test_binding_refuses_what_it_cannot_pass(lib):
    z, i32 = torch.zeros, dict(dtype=torch.int32)

    def call(**kw):
        return capi.dcp_tree_mla_decode(
            z(4, 2, 576, dtype=torch.bfloat16), z(2, **i32), z(1, **i32), 5, z(4, 1, dtype=torch.int64), 4,
            [z(4, **i32)], [z(8, 656, dtype=torch.uint8)], [z(1, 3, **i32)], 4, SCALE, **kw)

    with pytest.raises(ValueError):
        call(window=3)
    with pytest.raises(ValueError):
        call(window=3, positions=z(3, **i32))
    with pytest.raises((TypeError, ValueError)):
        call(window=3, positions=z(4, dtype=torch.int64))


# ---------------------------------------------------------------- operator
class Windowed(Case):
    """A Case whose nodes attend t < sinks or t > position - window."""

    def __init__(self, dev, fmt, window, sinks, **kw):
        super().__init__(dev, fmt, **kw)
        self.window, self.sinks = window, sinks
        _, self.positions = to.tree_maps(self.parents, self.starts, self.ctx, self.T, self.max_nodes)

    def run(self, rank=None, **kw):
        return super().run(rank, window=self.window, sinks=self.sinks, positions=_i32(self.positions, self.dev), **kw)

    def seen(self, b, j):
        """Which positions node j of request b sees, as a function."""
        p = self.positions[self.starts[b] + j]
        return lambda t: t < self.sinks or t > p - self.window

    def keys(self, b, j, rank):
        at, seen = self.ctx[b], self.seen(b, j)
        held = [p for p in range(at) if rank < 0 or p // self.I % self.D == rank]
        keys = [k for p, k in zip(held, to.prefix_keys(at, self.D, rank, self.bs, self.I, self.tables, b)) if seen(p)]
        slots = {d: s for d, s in enumerate(self.drafts) if rank < 0 or d == rank}
        t = self.starts[b] + j
        for m in range(self.nodes[b]):
            row = self.starts[b] + m
            if (int(self.masks[t, m // 64]) >> (m % 64)) & 1 and seen(self.positions[row]):
                key = to.draft_key(slots, row)
                if key is not None:
                    keys.append(key)
        return keys


CASES = [
    dict(window=1, sinks=0, nodes=[5, 3], ctx=[70, 0], H=16),                        # itself alone
    dict(window=1, sinks=1, nodes=[4], ctx=[0], H=128),                              # a sink among the drafts
    dict(window=3, sinks=2, nodes=[9, 9, 9], ctx=[100, 1, 3], H=16),                 # less than a tree is deep
    dict(window=60, sinks=5, nodes=[12, 1, 7], ctx=[150, 62, 61], H=16, D=3, bs=8, I=2, pad=3),
    dict(window=64, sinks=64, nodes=[4, 4], ctx=[300, 127], H=37, D=2, bs=48),
    dict(window=100, sinks=400, nodes=[6], ctx=[350], H=16),                         # every position is a sink
    dict(window=90, sinks=0, nodes=[40, 2], ctx=[200, 91], H=64, D=4, bs=16, rank=1),
    dict(window=33, sinks=7, nodes=[8, 8], ctx=[500, 20], H=20, D=3, bs=16, I=4, rank=2),
    dict(window=5, sinks=0, nodes=[6], ctx=[100], H=8, D=8, bs=16, I=16, rank=7),    # a rank without keys
    dict(window=200, sinks=3, nodes=[100, 30], ctx=[333, 190], H=5, max_nodes=128),
    dict(window=1500, sinks=70, nodes=[3, 2], ctx=[4000, 1600], H=16, D=2, bs=64),   # cut into ranges
    dict(window=2 ** 31 - 1, sinks=2 ** 31 - 1, nodes=[3], ctx=[90], H=16),
]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("i", range(len(CASES)))
def test_matches_the_definition(cuda_device, fmt, i):
    c = Windowed(cuda_device, fmt, seed=i, shapes=("chain", "bushy", "star"), **CASES[i]).upload()
    _err()
    out = torch.full((c.T, c.H, 512), 3.0, dtype=torch.bfloat16, device=cuda_device)
    lse = torch.full((c.T, c.H), 5.0, device=cuda_device)
    c.run(out=out, lse=lse)
    c.check(out, lse)
    assert out[c.n:].eq(3).all() and lse[c.n:].eq(5).all()  # rows of nobody
    again = c.run()
    assert torch.equal(out[:c.n], again[0][:c.n]) and torch.equal(lse[:c.n], again[1][:c.n])
    assert _err() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
def test_a_window_past_everything_leaves_nothing_out(cuda_device, fmt):
    c = Windowed(cuda_device, fmt, 150 + 9, 0, nodes=[9, 4], ctx=[150, 80], H=16, D=2, bs=16, seed=3).upload()
    want = Case.run(c)
    got = c.run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c.check(*got)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
def test_many_requests(cuda_device, fmt):
    rng = np.random.default_rng(4)
    B = 700
    nodes, ctx = rng.integers(0, 4, B), rng.integers(0, 90, B)
    ctx[-9], nodes[-9] = 1500, 3
    c = Windowed(cuda_device, fmt, 40, 2, nodes=nodes.tolist(), ctx=ctx.tolist(), H=3, D=2, bs=16, seed=8).upload()
    c.check(*c.run())


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rank", [-1, 0])
def test_blocks_behind_the_window_may_be_given_back(cuda_device, fmt, rank):
    """Their table entries and rows are not read."""
    c = Windowed(cuda_device, fmt, 40, 3, nodes=[7, 2], ctx=[400, 100], H=16, D=2, bs=8, I=2, rank=rank,
                 seed=6).upload()
    want = c.run()
    for b, ctx in enumerate(c.ctx):
        for d in range(c.D):
            kept = {(p // (c.I * c.D) * c.I + p % c.I) // c.bs for p in range(ctx)
                    if p // c.I % c.D == d and (p < 3 or p > ctx - 40)}
            for col in range(c.tables[d].shape[1]):
                if col not in kept:
                    if c.tables[d][b, col] >= 0:
                        rows = c.pools[d][c.tables[d][b, col] * c.bs:][:c.bs]
                        rows[:] = 0xff
                    c.tables[d][b, col] = -1
    c.upload()
    _err()
    got = c.run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert _err() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("at", [31, 32, 34, 36])
def test_a_bad_key_at_the_windows_edge(cuda_device, fmt, at):
    """A cached row that is not finite spoils the nodes that still see it and no
    others: with 100 positions and a window of 70 a node of depth k sees t >= 31
    + k."""
    c = Windowed(cuda_device, fmt, 70, 0, nodes=[6, 2], ctx=[100, 60], H=16, bs=16, seed=9, shapes=("chain",))
    row = c.pools[0][c.tables[0][0][at // 16] * 16 + at % 16]
    if fmt == "fp8":
        row[516:520] = np.array([np.nan], dtype="<f4").view(np.uint8)
    else:
        row[260] = 0x7f
    c.upload()
    out, lse = c.run()
    spoilt = [j for j in range(6) if c.seen(0, j)(at)]
    assert spoilt == list(range(min(at - 30, 6)))
    c.check(out, lse, rows=set(range(c.T)) - set(spoilt))
    assert lse[spoilt].isnan().all()
    _err()


@pytest.mark.gpu
def test_positions_outside_a_tree_count_as_the_nearest(cuda_device):
    c = Windowed(cuda_device, "fp8", 20, 2, nodes=[4], ctx=[90], H=16, bs=16, seed=10, shapes=("chain",)).upload()
    c.positions[:] = [-5, 89, 2 ** 31 - 1, 92]
    got = c.run()
    c.positions[:] = [90, 90, 93, 92]
    want = c.run()
    c.check(*got)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
def test_partials_merge_into_the_whole(cuda_device, fmt):
    c = Windowed(cuda_device, fmt, 50, 4, nodes=[6, 2], ctx=[150, 3], H=16, D=4, bs=16, seed=3).upload()
    parts = [c.run(rank=d) for d in range(c.D)]
    for d, (o, l) in enumerate(parts):
        c.check(o, l, rank=d)
    _, lse = capi.dcp_lse_merge([p[0] for p in parts], [p[1] for p in parts])
    whole = c.run()
    c.check(*whole)
    # each of the logarithms within the checked bounds, a few 10^-3 here
    assert torch.allclose(lse, whole[1], atol=1e-2)


# ------------------------------------------------------------ serving step
B, D, BS, H, CTX = 3, 3, 8, 16, 200


def _bf16(shape, seed, dev):
    g = torch.Generator(device=dev).manual_seed(seed)
    return torch.randn(shape, generator=g, device=dev).to(torch.bfloat16)


def _f64(t):
    return bf16_bits_to_f64(_np(t.contiguous().view(torch.int16)).astype(np.uint16))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window,sinks", [(60, 5), (1, 0), (7, 3), (1000, 0)])
@pytest.mark.parametrize("S,ctx", [(1, [30, 59, 61]), (1, [90, 0, 150]), (4, [90, 5, 150]), (12, [50, 62, 150])])
def test_a_chain_is_verified_as_the_step_decodes_it(cuda_device, fmt, window, sinks, S, ctx):
    """The same S tokens of every request as a drafted chain and as a decode
    step's: both attend the same keys of equal caches."""
    dev = cuda_device
    a = torch.arange(CTX + S)[:, None] * torch.exp(torch.arange(32) * -0.3)
    table = torch.cat([a.cos(), a.sin()], 1).float().to(dev)
    drafts, plain = (DcpServingStep(B, S, H, D, BS, 40, CTX, window, sinks, fmt=fmt, cos_sin=table, sm_scale=SCALE,
                                    interleave=2, max_nodes=S, device=dev) for _ in range(2))
    kv0 = _bf16((sum(ctx), 576), 2, dev)
    for step in (drafts, plain):
        step.prefill(_i32(ctx, dev), _i32(ctx, dev), kv0)
        step.take_blocks()
    kv, q = _bf16((B * S, 576), 3, dev), _bf16((B * S, H, 576), 4, dev)
    _err()
    got = drafts.verify(_i32(ctx, dev), _i32(np.tile(np.arange(S) - 1, B), dev), _i32(np.arange(B + 1) * S, dev), kv, q)
    want = plain.run(_i32(np.array(ctx) + S, dev), kv, q)
    assert _err() == 0
    pools, tables = [_np(p) for p in plain.pools], [_np(t) for t in plain.block_tables]
    for b in range(B):
        for j in range(S):
            t, p = b * S + j, ctx[b] + j
            rows = []
            for k in so.window_positions(p, window, sinks):
                d, lp = k // 2 % D, k // (2 * D) * 2 + k % 2
                rows.append(pools[d][tables[d][b, lp // BS] * BS + lp % BS])
            o, l, o_tol, l_tol = so.attend(_f64(q[t]), np.stack(rows), SCALE, KEY_STEP[fmt])
            for out, lse in (got, want):
                assert np.all(np.abs(_np(lse[t].double()) - l) <= l_tol), (b, j)
                assert np.all(np.abs(_f64(out[t]) - o) <= o_tol), (b, j)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("first", [60, 120])
def test_drafting_server_under_its_window(cuda_device, fmt, first):
    """Rounds of trees by a server with a window of 60 and 5 sinks: queries,
    attention and output within their definitions' bounds, then the accepted
    tokens' cache that of a server which was given them at once, and its next
    ordinary step the same."""
    dev, rng = cuda_device, np.random.default_rng(5)
    step, proj = serving._server(dev, fmt), serving._projections(dev)
    B, D, N, BS = serving.B, serving.D, serving.N, serving.BS
    T = B * N - 4
    ctx = np.array([first, 0, 17])
    kv = _bf16((int(ctx.sum()), 576), 2, dev)
    hist = [list(r) for r in torch.split(kv, ctx.tolist())]
    _err()
    step.prefill(_i32(ctx, dev), _i32(ctx, dev), kv)
    step.take_blocks()
    left_out = 0
    for i in range(4):
        starts, parents, tokens, targets = serving._drafts(rng, T, dev)
        while starts[-1] > T:
            starts, parents, tokens, targets = serving._drafts(rng, T, dev)
        pre, par, rs, tok, tgt = (_i32(v, dev) for v in (ctx, parents, starts, tokens, targets))
        x, kv = _bf16((T, 200), 20 + i, dev), _bf16((T, 576), 30 + i, dev)
        positions = step.tree_positions(pre, par, rs).positions
        q = proj.query(x, positions)
        serving._check_query(proj, x, positions, q)
        step.tree_out.fill_(0)
        out, lse = step.verify(pre, par, rs, kv, q)
        masks, positions = to.tree_maps(parents, starts, ctx, T, N)
        pools, tables = [_np(p) for p in step.pools], [_np(t) for t in step.block_tables]
        for b in range(B):
            for j in range(starts[b + 1] - starts[b]):
                t = starts[b] + j
                seen = lambda at: at < 5 or at > positions[t] - 60  # noqa: E731,B023
                at = [serving._slot(step, tables, b, p) for p in range(ctx[b]) if seen(p)]
                left_out += ctx[b] - len(at)
                keys = [pools[d][s] for d, s in at]
                keys += [pools[0][40 * BS + starts[b] + m] for m in range(N)
                         if int(masks[t, 0]) >> m & 1 and seen(positions[starts[b] + m])]
                o, l, o_tol, l_tol = so.attend(_f64(q[t]), np.stack(keys), SCALE, KEY_STEP[fmt])
                assert np.all(np.abs(_f64(out[t]) - o) <= o_tol), (i, b, j)
                assert np.all(np.abs(_np(lse[t].double()) - l) <= l_tol), (i, b, j)
        serving._check_output(proj, out, proj.output(out))
        walk, after = step.commit(pre, par, tok, tgt, rs)
        step.take_blocks()
        acc, line, nexts = to.tree_accept(parents, tokens, targets, starts, T)
        assert np.array_equal(_np(walk.accepted), acc) and np.array_equal(_np(walk.next_tokens), nexts)
        assert np.array_equal(_np(walk.rows), line)
        at = 0
        for b in range(B):
            hist[b] += [kv[r] for r in line[at:at + acc[b]]]
            at += acc[b]
        ctx = ctx + acc
        assert np.array_equal(_np(after), ctx)
    assert left_out > 0
    other = serving._server(dev, fmt)
    other.prefill(_i32(ctx, dev), _i32(ctx, dev), torch.stack([r for h in hist for r in h]))
    other.take_blocks()
    for a, b in zip(serving._cached(step, ctx), serving._cached(other, ctx)):
        assert np.array_equal(a, b)
    kv, q = _bf16((B, 576), 3, dev), _bf16((B, H, 576), 4, dev)
    got, want = (s.run(_i32(ctx + 1, dev), kv, q) for s in (step, other))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert _err() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("length", [2 ** 30, 2 ** 30 - 37])
@pytest.mark.parametrize("D,rank", [(1, -1), (4, -1), (4, 3)])
def test_the_longest_prefix(cuda_device, fmt, length, D, rank):
    """Only the sinks' and the window's blocks exist, far apart in the table."""
    bs, window, sinks, H, n, I = 2 ** 18, 100, 9, 16, 5, 3
    c = Windowed(cuda_device, fmt, window, sinks, nodes=[n], ctx=[40], H=H, D=D, bs=64, I=I, rank=rank, seed=1,
                 shapes=("chain",))
    rng = np.random.default_rng(2)
    local = lambda p: (p // I % D, p // (I * D) * I + p % I)  # noqa: E731
    cached = {p: c.pools[0][rng.integers(len(c.pools[0]))] for p in (*range(sinks), *range(length - window, length))}
    width = 2 ** 30 // (D * bs) + 2
    pools, tables, drafts = [], [], []
    for d in range(D):
        pool = torch.zeros((3 * bs + n, c.pools[0].shape[1]), dtype=torch.uint8, device=cuda_device)
        table = np.full((1, width), -1, dtype=np.int32)
        cols = sorted({local(p)[1] // bs for p in cached if local(p)[0] == d})
        assert len(cols) <= 3
        table[0, cols] = np.arange(len(cols))
        for p, row in cached.items():
            e, lp = local(p)
            if e == d:
                pool[int(table[0, lp // bs]) * bs + lp % bs] = torch.from_numpy(row.copy()).to(cuda_device)
        own = np.array([3 * bs + j if local(length + j)[0] == d else -1 for j in range(n)])
        for j in np.flatnonzero(own >= 0):
            pool[own[j]] = torch.from_numpy(c.pools[0][j].copy()).to(cuda_device)
        pools.append(pool), tables.append(_i32(table, cuda_device)), drafts.append(_i32(own, cuda_device))
    _err()
    out, lse = capi.dcp_tree_mla_decode(
        c.q.to(cuda_device), _i32([0, n], cuda_device), _i32([length], cuda_device), 2 ** 30,
        torch.from_numpy(c.masks.view(np.int64)).to(cuda_device), c.max_nodes, drafts, pools, tables, bs, SCALE,
        rank=rank, interleave=I, window=window, sinks=sinks, positions=_i32(length + np.arange(n), cuda_device))
    assert _err() == 0
    for j in range(n):
        mine = lambda t: rank < 0 or local(t)[0] == rank  # noqa: E731
        rows = [row for t, row in cached.items() if mine(t) and (t < sinks or t > length + j - window)]
        rows += [c.pools[0][m] for m in range(j + 1) if mine(length + m)]
        o, l, o_tol, l_tol = so.attend(_f64(c.q[j]), np.stack(rows), SCALE, KEY_STEP[fmt])
        assert np.all(np.abs(_f64(out[j]) - o) <= o_tol) and np.all(np.abs(_np(lse[j].double()) - l) <= l_tol), j
