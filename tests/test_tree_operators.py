"""Drafted trees: masks and positions, the greedy walk, the accepted rows'
move.  Refusals run without a GPU; results are compared with
oracle/tree_oracle.py, all of them whole numbers or bytes."""
import numpy as np
import pytest
import torch

from oracle import tree_oracle as to
from sparse_mla_decode_dcp_gb300 import build as smla_build
from sparse_mla_decode_dcp_gb300 import capi

BAD, UNSUP, WS, OK = (capi.SMLA_ERR_INVALID_ARG, capi.SMLA_ERR_UNSUPPORTED,
                      capi.SMLA_ERR_WORKSPACE, capi.SMLA_OK)
FAKE = 0x10000  # aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    smla_build.build()
    return capi.load()


def _np(t):
    return t.cpu().numpy()


def _i32(a, dev):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).to(dev)


def _err():
    return capi.get_device_error(clear=True)


# ------------------------------------------------------------------ oracle
#        0
#      / | \
#     1  2  5
#     |  |\
#     3  4 6        (and 7 on 6)
TREE = [-1, 0, 0, 1, 2, 0, 2, 6]


def test_oracle_on_a_tree_drawn_by_hand():
    masks, pos = to.tree_maps(TREE, [0, 8], [10], 9, 8)
    assert [int(m) for m in masks[:, 0]] == [0b1, 0b11, 0b101, 0b1011, 0b10101, 0b100001, 0b1000101,
                                             0b11000101, 0]
    assert pos.tolist() == [10, 11, 11, 12, 12, 11, 12, 13, 0]
    #         node 0's target is 7: child 2 (node 5 has it too); 2's is 9: child 6; 6's is 4
    tokens, targets = [5, 3, 7, 9, 8, 7, 9, 1], [7, 9, 9, 0, 0, 0, 4, 0]
    acc, rows, nxt = to.tree_accept(TREE, tokens, targets, [0, 8, 8], 9)
    assert acc.tolist() == [3, 0] and nxt.tolist() == [4, -1]
    assert rows.tolist() == [0, 2, 6] + [-1] * 6


# ---------------------------------------------------------------- refusals
@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), BAD), (dict(T=-1), BAD), (dict(n=0), BAD), (dict(n=257), UNSUP),
    (dict(par=None), BAD), (dict(rs=None), BAD), (dict(pre=None), BAD), (dict(masks=None), BAD),
    (dict(par=FAKE + 2), BAD), (dict(rs=FAKE + 1), BAD), (dict(pre=FAKE + 2), BAD),
    (dict(masks=FAKE + 4), BAD), (dict(pos=FAKE + 2), BAD),
    (dict(T=0, par=None, rs=None, pre=None, masks=None), OK),
])
def test_maps_argument_checks(lib, kw, status):
    a = dict(par=FAKE, rs=FAKE, pre=FAKE, B=2, T=9, n=8, masks=FAKE, pos=FAKE)
    a.update(kw)
    assert lib.smla_tree_maps(a["par"], a["rs"], a["pre"], a["B"], a["T"], a["n"], a["masks"], a["pos"],
                              None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), BAD), (dict(T=-1), BAD), (dict(B=capi.MAX_STEP_REQS + 1), UNSUP),
    (dict(par=None), BAD), (dict(tok=None), BAD), (dict(tgt=None), BAD), (dict(rs=None), BAD),
    (dict(acc=None), BAD), (dict(rows=None), BAD), (dict(nxt=None), BAD), (dict(tok=FAKE + 2), BAD),
    (dict(rows=FAKE + 1), BAD), (dict(nxt=FAKE + 3), BAD),
    (dict(B=0, T=0, par=None, tok=None, tgt=None, rs=None, acc=None, rows=None, nxt=None), OK),
])
def test_accept_argument_checks(lib, kw, status):
    a = dict(par=FAKE, tok=FAKE, tgt=FAKE, rs=FAKE, B=2, T=9, acc=FAKE, rows=FAKE, nxt=FAKE)
    a.update(kw)
    assert lib.smla_tree_accept(a["par"], a["tok"], a["tgt"], a["rs"], a["B"], a["T"], a["acc"], a["rows"],
                                a["nxt"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), BAD), (dict(T=-1), BAD), (dict(ns=-1), BAD), (dict(fmt=2), BAD), (dict(kv=None), BAD),
    (dict(rows=None), BAD), (dict(src=None), BAD), (dict(dst=None), BAD), (dict(kv=FAKE + 8), BAD),
    (dict(rows=FAKE + 2), BAD), (dict(src=FAKE + 2), BAD), (dict(dst=FAKE + 2), BAD),
    (dict(N=0, kv=None, rows=None, src=None, dst=None), OK),
])
def test_move_argument_checks(lib, kw, status):
    a = dict(fmt=0, kv=FAKE, ns=9, rows=FAKE, N=4, src=FAKE, T=4, dst=FAKE)
    a.update(kw)
    assert lib.smla_mla_cache_move(a["fmt"], a["kv"], a["ns"], a["rows"], a["N"], a["src"], a["T"],
                                   a["dst"], None) == status


def test_binding_refuses_what_it_cannot_pass(lib):
    i32 = dict(dtype=torch.int32)
    z = torch.zeros
    with pytest.raises(ValueError):  # host tensors never reach the library
        capi.tree_maps(z(4, **i32), z(2, **i32), z(1, **i32), 4)
    with pytest.raises(ValueError):  # row_start is [B + 1]
        capi.tree_maps(z(4, **i32), z(3, **i32), z(1, **i32), 4)
    with pytest.raises(TypeError):
        capi.tree_maps(z(4, dtype=torch.int64), z(2, **i32), z(1, **i32), 4)
    with pytest.raises(ValueError):  # masks of another width
        capi.tree_maps(z(4, **i32), z(2, **i32), z(1, **i32), 65,
                       out=capi.TreeMaps(z(4, 1, dtype=torch.int64), z(4, **i32)))
    with pytest.raises(ValueError):
        capi.tree_accept(z(4, **i32), z(3, **i32), z(4, **i32), z(2, **i32))
    with pytest.raises(ValueError):
        capi.tree_accept(z(4, **i32), z(4, **i32), z(4, **i32), z(2, **i32),
                         out=(z(1, **i32), z(4, **i32)))
    with pytest.raises(ValueError):
        capi.mla_cache_move(z(4, 600, dtype=torch.uint8), z(4, **i32), z(4, **i32), z(4, **i32))
    with pytest.raises(ValueError):  # a destination for each row
        capi.mla_cache_move(z(4, 656, dtype=torch.uint8), z(4, **i32), z(4, **i32), z(3, **i32))


# ------------------------------------------------------------- maps, walk
def _trees(rng, B, lo, hi, shapes=("bushy",)):
    n = rng.integers(lo, hi + 1, B)
    starts = np.concatenate([[0], np.cumsum(n)])
    parents = np.concatenate([to.random_tree(rng, int(k), shapes[b % len(shapes)])
                              for b, k in enumerate(n)] + [np.zeros(0)]).astype(np.int32)
    return starts, parents


SHAPES = ("bushy", "chain", "star", "roots")


@pytest.mark.gpu
@pytest.mark.parametrize("B,lo,hi,max_nodes,pad", [
    (1, 1, 1, 1, 0), (1, 8, 8, 8, 3), (5, 0, 9, 33, 0), (64, 16, 16, 16, 0), (37, 1, 64, 64, 70),
    (9, 30, 65, 65, 1), (11, 100, 200, 200, 0), (4, 256, 256, 256, 5), (3000, 0, 3, 3, 999),
])
def test_maps_match_the_definition(cuda_device, B, lo, hi, max_nodes, pad):
    rng = np.random.default_rng(B + hi)
    starts, parents = _trees(rng, B, lo, hi, SHAPES)
    T = len(parents) + pad
    prefix = rng.integers(0, 2 ** 31 - 300, B)
    parents = np.concatenate([parents, np.full(pad, 12345, dtype=np.int32)])
    want = to.tree_maps(parents, starts, prefix, T, max_nodes)
    _err()
    got = capi.tree_maps(_i32(parents, cuda_device), _i32(starts, cuda_device), _i32(prefix, cuda_device),
                         max_nodes)
    assert np.array_equal(_np(got.masks).view(np.uint64), want[0])
    assert np.array_equal(_np(got.positions), want[1])
    assert _err() == 0


@pytest.mark.gpu
def test_no_request_is_all_padding(cuda_device):
    dev, T = cuda_device, 300
    par, none, start = _i32(np.full(T, -1), dev), _i32([], dev), _i32([0], dev)
    out = capi.TreeMaps(torch.full((T, 2), 5, dtype=torch.int64, device=dev), _i32(np.full(T, 5), dev))
    _err()
    capi.tree_maps(par, start, none, 100, out=out)
    walk = capi.tree_accept(par, par, par, start)
    assert out.masks.eq(0).all() and out.positions.eq(0).all()
    assert walk.rows.eq(-1).all() and len(walk.accepted) == 0 and _err() == 0


@pytest.mark.gpu
def test_maps_report_bad_trees(cuda_device):
    dev = cuda_device

    def run(parents, starts, T=None, max_nodes=4):
        B, T = len(starts) - 1, len(parents)
        out = capi.TreeMaps(torch.full((T, 1), 99, dtype=torch.int64, device=dev),
                            torch.full((T,), 99, dtype=torch.int32, device=dev))
        capi.tree_maps(_i32(parents, dev), _i32(starts, dev), _i32([10] * B, dev), max_nodes, out=out)
        return _np(out.masks)[:, 0].tolist(), _np(out.positions).tolist(), _err()

    _err()
    # its own parent, a later one, one below -1: roots
    masks, pos, err = run([-1, 1, 3, -5], [0, 4])
    assert masks == [1, 2, 4, 8] and pos == [10] * 4 and err == capi.DEVERR_TREE
    # more nodes than the bound; rows behind T; rows that run backwards
    for starts in ([0, 5], [0, 9], [-1, 2], [4, 2]):
        masks, pos, err = run([-1, 0, 0, 0, 0], starts)
        assert err == capi.DEVERR_TREE
        assert pos[:2] == [99, 99] or starts == [-1, 2]
    # the requests around a bad one are served
    masks, pos, err = run([-1, 0, -1, 0, 1, 2, 3, -1, 0], [0, 2, 7, 9])
    assert masks == [1, 3] + [99] * 5 + [1, 3] and err == capi.DEVERR_TREE


@pytest.mark.gpu
@pytest.mark.parametrize("B,lo,hi,pad", [
    (1, 1, 1, 0), (1, 256, 256, 0), (5, 0, 9, 3), (64, 16, 16, 0), (65, 16, 16, 1), (200, 0, 64, 500),
    (1000, 1, 3, 0), (8192, 0, 2, 7), (70, 250, 256, 0), (3, 0, 0, 40),
])
def test_accept_matches_the_definition(cuda_device, B, lo, hi, pad):
    rng = np.random.default_rng(B + hi + 1)
    starts, parents = _trees(rng, B, lo, hi, SHAPES)
    T = len(parents) + pad
    parents = np.concatenate([parents, np.full(pad, -1, dtype=np.int32)])
    tokens, targets = rng.integers(0, 3, T), rng.integers(0, 3, T)  # few: many agree, some twice
    want = to.tree_accept(parents, tokens, targets, starts, T)
    _err()
    got = capi.tree_accept(*(_i32(v, cuda_device) for v in (parents, tokens, targets, starts)))
    for name, g, w in zip(capi.TreeWalk._fields, got, want):
        assert np.array_equal(_np(g), w), name
    assert _err() == 0


@pytest.mark.gpu
def test_a_chain_of_every_node_is_walked_to_its_end(cuda_device):
    n, B = 256, 66
    starts, parents = np.arange(B + 1) * n, np.tile(np.arange(n) - 1, B)
    tokens = np.zeros(n * B)
    got = capi.tree_accept(*(_i32(v, cuda_device) for v in (parents, tokens, tokens, starts)))
    assert _np(got.accepted).tolist() == [n] * B
    assert np.array_equal(_np(got.rows), np.arange(n * B))


@pytest.mark.gpu
@pytest.mark.parametrize("B", [1, 31, 32, 33])
def test_walks_of_wide_and_deep_trees(cuda_device, B):
    """Around the number of requests that one launch takes: many children with
    the same token, the lowest of them far behind others' children; parents
    that are no nodes before them."""
    rng = np.random.default_rng(B)
    starts, parents = _trees(rng, B, 200, 256, ("bushy", "chain", "star"))
    T = len(parents)
    inner = np.arange(T) - np.repeat(starts[:-1], np.diff(starts))  # node numbers
    far = rng.random(T) < 0.3  # children of any node before, not of the nearest
    parents = np.where(far & (inner > 0), rng.integers(0, np.maximum(inner, 1)), parents)
    wrong = (rng.random(T) < 0.1) & (inner > 0)  # themselves, a later node, below -1
    bad = np.where(wrong, np.where(rng.random(T) < 0.5, inner + rng.integers(0, 3, T), -2), parents)
    tokens, targets = rng.integers(0, 2, T), rng.integers(0, 2, T)
    got = capi.tree_accept(*(_i32(v, cuda_device) for v in (bad, tokens, targets, starts)))
    want = to.tree_accept(np.where(wrong, -1, parents), tokens, targets, starts, T)
    for x, y in zip(got, want):
        assert np.array_equal(_np(x), y)
    assert B == 1 or max(want[0]) > 3  # the walks go somewhere
    got = capi.tree_accept(*(_i32(v, cuda_device) for v in (np.arange(T) - 1 - np.repeat(starts[:-1], np.diff(starts)),
                                                            0 * tokens, 0 * tokens, starts)))
    assert np.array_equal(_np(got.accepted), np.diff(starts)) and np.array_equal(_np(got.rows), np.arange(T))


@pytest.mark.gpu
@pytest.mark.parametrize("B", [3, 100])
def test_accept_reports_bad_trees(cuda_device, B):
    """A tree too large or out of the rows counts as empty."""
    dev = cuda_device
    starts = np.arange(B + 1) * 2
    starts[2:] += 300  # request 1 has 302 rows
    T = int(starts[-1]) - 1  # and the last one a row too many
    z = torch.zeros(T, dtype=torch.int32, device=dev)
    par = torch.full((T,), -1, dtype=torch.int32, device=dev)
    _err()
    got = capi.tree_accept(par, z, z, _i32(starts, dev))
    assert _np(got.accepted).tolist() == [1, 0] + [1] * (B - 3) + [0]
    assert _np(got.next_tokens).tolist() == [0, -1] + [0] * (B - 3) + [-1]
    want = [int(s) for b, s in enumerate(starts[:-1]) if b not in (1, B - 1)]
    assert _np(got.rows).tolist() == want + [-1] * (T - len(want))
    assert _err() == capi.DEVERR_TREE


@pytest.mark.gpu
@pytest.mark.parametrize("B", [5, 101])
def test_accepted_rows_of_overlapping_spans_stay_inside(cuda_device, B):
    """Spans that go back over the same rows hold more accepted nodes than there
    are rows: what is behind the last row stays as it was."""
    dev, n = cuda_device, 6
    starts = np.arange(B + 1) % 2 * n  # rows 0 .. 5, then -6 of them, and so on
    par, z = _i32(np.arange(n) - 1, dev), torch.zeros(n, dtype=torch.int32, device=dev)
    rows = torch.full((n + 4000,), 77, dtype=torch.int32, device=dev)
    out = capi.TreeWalk(_i32(np.zeros(B), dev), rows[:n], _i32(np.zeros(B), dev))
    _err()
    capi.tree_accept(par, z, z, _i32(starts, dev), out=out)
    assert _np(out.accepted).tolist() == [n if b % 2 == 0 else 0 for b in range(B)]
    assert _np(out.rows).tolist() == list(range(n))
    assert rows[n:].eq(77).all() and _err() == capi.DEVERR_TREE


# -------------------------------------------------------------------- move
@pytest.mark.gpu
@pytest.mark.parametrize("row", [656, 416])
@pytest.mark.parametrize("N,T", [(1, 1), (7, 9), (64, 64), (1000, 300), (33, 5000)])
def test_move_copies_rows(cuda_device, row, N, T):
    rng = np.random.default_rng(N + T)
    slots = T + N + 5
    pool = torch.from_numpy(rng.integers(0, 256, (slots, row), dtype=np.uint8)).to(cuda_device)
    perm = rng.permutation(slots)
    src, dst = perm[:T].copy(), perm[T:T + N].copy()
    rows = rng.integers(0, T, N)
    rows[rng.random(N) < 0.2] = -1
    dst[rng.random(N) < 0.2] = -1
    want = _np(pool).copy()
    for i in range(N):
        if rows[i] >= 0 and dst[i] >= 0:
            want[dst[i]] = want[src[rows[i]]]
    _err()
    got = capi.mla_cache_move(pool, *(_i32(v, cuda_device) for v in (rows, src, dst)))
    assert got is pool and np.array_equal(_np(pool), want)
    assert _err() == 0


@pytest.mark.gpu
def test_move_past_two_gib_and_its_bad_entries(cuda_device):
    slots = 2 ** 31 // 416 + 1000
    pool = torch.zeros((slots, 416), dtype=torch.uint8, device=cuda_device)
    pool[slots - 1] = 7
    pool[0] = 9
    _err()
    capi.mla_cache_move(pool, _i32([0, 1], cuda_device), _i32([slots - 1, 0], cuda_device),
                        _i32([5, slots - 2], cuda_device))
    assert pool[5].eq(7).all() and pool[slots - 2].eq(9).all() and _err() == 0
    before = pool[:50].clone()
    for rows, src, dst in (([2], [1, 2], [3]), ([-2], [1, 2], [3]), ([0], [-1], [3]), ([0], [slots], [3]),
                           ([0], [1], [slots])):
        capi.mla_cache_move(pool, *(_i32(v, cuda_device) for v in (rows, src, dst)))
        assert _err() == capi.DEVERR_SLOT_RANGE
    assert torch.equal(pool[:50], before)
    capi.mla_cache_move(pool, *(_i32(v, cuda_device) for v in ([0, -1], [-1], [-1, 3])))
    assert torch.equal(pool[:50], before) and _err() == 0  # another rank's


@pytest.mark.gpu
def test_walk_move_and_step_maps_fit_together(cuda_device):
    """The accepted rows of drafts in scratch slots reach the slots that the
    next step's maps give them, and read back in order."""
    dev = cuda_device
    rng = np.random.default_rng(3)
    B, D, bs = 5, 2, 4
    starts, parents = _trees(rng, B, 3, 9)
    T = len(parents)
    tokens, targets = rng.integers(0, 2, T), rng.integers(0, 2, T)
    prefix = rng.integers(0, 20, B)
    walk = capi.tree_accept(*(_i32(v, dev) for v in (parents, tokens, targets, starts)))
    acc, rows, _ = to.tree_accept(parents, tokens, targets, starts, T)
    pools = [torch.from_numpy(rng.integers(0, 256, (400, 656), dtype=np.uint8)).to(dev) for _ in range(D)]
    scratch = _i32(300 + np.arange(T), dev)
    pools[1][300:300 + T] = pools[0][300:300 + T]  # drafts are written on every rank
    drafts = _np(pools[0])[300:300 + T].copy()
    tables = [torch.full((B, 12), -1, dtype=torch.int32, device=dev) for _ in range(D)]
    free = [torch.arange(70, dtype=torch.int32, device=dev) for _ in range(D)]
    for d in range(D):
        m = capi.dcp_step_maps(_i32(prefix, dev), _i32(prefix, dev), free[d], tables[d], int(prefix.sum()),
                               D, d, bs)
        free[d] = free[d][int(m.blocks_taken):]
        m = capi.dcp_step_maps(_i32(prefix, dev) + walk.accepted, walk.accepted, free[d], tables[d], T, D, d, bs)
        capi.mla_cache_move(pools[d], walk.rows, scratch, m.slots)
    i = 0
    for b in range(B):
        for k in range(acc[b]):
            p = int(prefix[b]) + k
            d, lp = p % D, p // D
            slot = int(tables[d][b, lp // bs]) * bs + lp % bs
            assert np.array_equal(_np(pools[d][slot]), drafts[rows[i]])
            i += 1
    assert _err() == 0


@pytest.mark.gpu
def test_calls_follow_their_stream_and_replay_in_a_graph(cuda_device):
    dev = cuda_device
    rng = np.random.default_rng(11)
    starts, parents = _trees(rng, 100, 1, 20)
    T = len(parents)
    tok, tgt = rng.integers(0, 2, T), rng.integers(0, 2, T)
    prefix = rng.integers(0, 50, 100)
    stream = torch.cuda.Stream(dev)
    par, rs, pre, tk, tg = (_i32(v, dev) for v in (parents, starts, prefix, tok, tgt))
    want = to.tree_maps(parents, starts, prefix, T, 20), to.tree_accept(parents, tok, tgt, starts, T)
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        maps = capi.tree_maps(par, rs, pre, 20)
        walk = capi.tree_accept(par, tk, tg, rs)
    stream.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        capi.tree_maps(par, rs, pre, 20, out=maps, stream=stream)
        capi.tree_accept(par, tk, tg, rs, out=walk, stream=stream)
    for t in (*maps, *walk):
        t.fill_(5)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(_np(maps.masks).view(np.uint64), want[0][0])
    assert np.array_equal(_np(maps.positions), want[0][1])
    for a, b in zip(walk, want[1]):
        assert np.array_equal(_np(a), b)
