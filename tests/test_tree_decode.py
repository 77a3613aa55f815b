"""Attention of drafted trees over the paged cache.  Refusals run without a
GPU; results are compared row by row with the float64 definitions of
oracle/tree_oracle.py and oracle/step_oracle.py, tolerances derived there."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import step_oracle as so
from oracle import tree_oracle as to
from oracle.smla_oracle import bf16_bits_to_f64
from sparse_mla_decode_dcp_gb300 import build as smla_build
from sparse_mla_decode_dcp_gb300 import capi

BAD, UNSUP, WS, OK = (capi.SMLA_ERR_INVALID_ARG, capi.SMLA_ERR_UNSUPPORTED,
                      capi.SMLA_ERR_WORKSPACE, capi.SMLA_OK)
FAKE = 0x10000  # aligned, never dereferenced
SCALE = 1.0 / math.sqrt(192.0)
ROW = {"fp8": capi.ROW_BYTES, "fp4": capi.FP4_ROW_BYTES}
# keys round to fp16 from fp8 rows' codes and scales, and are exact from fp4's
KEY_STEP = {"fp8": 2.0 ** -11, "fp4": 0.0}


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


# ---------------------------------------------------------------- refusals
@pytest.mark.parametrize("D,kw,status", [
    (2, dict(T=-1), BAD), (2, dict(H=0), BAD), (2, dict(B=-1), BAD), (2, dict(maxp=-1), BAD),
    (2, dict(n=0), BAD), (0, {}, BAD), (2, dict(rank=2), BAD), (2, dict(rank=-2), BAD), (2, dict(bs=0), BAD),
    (2, dict(I=0), BAD), (2, dict(fmt=2), BAD), (2, dict(scale=0.0), BAD), (2, dict(scale=float("inf")), BAD),
    (2, dict(q=None), BAD), (2, dict(rs=None), BAD), (2, dict(pre=None), BAD), (2, dict(masks=None), BAD),
    (2, dict(out=None), BAD), (2, dict(lse=None), BAD), (2, dict(q=FAKE + 8), BAD), (2, dict(out=FAKE + 8), BAD),
    (2, dict(masks=FAKE + 4), BAD), (2, dict(rs=FAKE + 2), BAD), (2, dict(pools=[FAKE, None]), BAD),
    (2, dict(drafts=[FAKE, None]), BAD), (2, dict(drafts=[FAKE + 2, FAKE]), BAD), (2, dict(widths=[4, 5]), BAD),
    (2, dict(H=129), UNSUP), (17, {}, UNSUP), (2, dict(n=257), UNSUP), (2, dict(maxp=2 ** 30 + 1), UNSUP),
    (2, dict(T=2 ** 25, H=64), UNSUP), (2, dict(T=0, q=None), OK), (2, dict(B=0, rs=None), OK),
])
def test_argument_checks(lib, D, kw, status):
    a = dict(q=FAKE, T=9, H=16, scale=0.07, rs=FAKE, pre=FAKE, B=2, maxp=100, masks=FAKE, n=8, rank=-1, bs=16,
             I=1, fmt=0, out=FAKE, lse=FAKE, pools=None, drafts=None, widths=None)
    a.update(kw)
    n = max(D, 1)
    arr = lambda typ, xs: (typ * n)(*(list(xs) + [0] * n)[:n])  # noqa: E731
    got = lib.smla_dcp_tree_mla_decode(
        a["q"], a["T"], a["H"], ctypes.c_float(a["scale"]), a["rs"], a["pre"], a["B"], a["maxp"], a["masks"],
        a["n"], arr(ctypes.c_void_p, a["drafts"] or [FAKE] * n), D, a["rank"], a["bs"], a["I"], a["fmt"],
        arr(ctypes.c_void_p, a["pools"] or [FAKE] * n), arr(ctypes.c_int64, [100] * n),
        arr(ctypes.c_void_p, [FAKE] * n), arr(ctypes.c_int64, [4] * n), arr(ctypes.c_int32, a["widths"] or [4] * n),
        a["out"], a["lse"], None, 0, None)
    assert got == status


def test_workspace_sizes(lib):
    size = capi.tree_decode_workspace_size
    assert size(-1, 16, 2, 100, 8, 2) == 0 and size(8, 129, 2, 100, 8, 2) == 0
    assert size(8, 16, 2, 100, 257, 2) == 0 and size(8, 16, 2, 100, 8, 2, 1, 2) == 0
    assert size(8, 16, 2, 2 ** 30 + 1, 8, 2) == 0


def test_binding_refuses_what_it_cannot_pass(lib):
    i32 = dict(dtype=torch.int32)
    z = torch.zeros

    def call(**kw):
        a = dict(q=z(4, 2, 576, dtype=torch.bfloat16), rs=z(2, **i32), pre=z(1, **i32), maxp=5,
                 masks=z(4, 1, dtype=torch.int64), n=4, drafts=[z(4, **i32)],
                 kv=[z(8, 656, dtype=torch.uint8)], bt=[z(1, 3, **i32)], rank=-1)
        a.update(kw)
        return capi.dcp_tree_mla_decode(a["q"], a["rs"], a["pre"], a["maxp"], a["masks"], a["n"], a["drafts"],
                                        a["kv"], a["bt"], 4, SCALE, rank=a["rank"])

    with pytest.raises(ValueError):  # host tensors never reach the library
        call()
    with pytest.raises(ValueError):
        call(rs=z(3, **i32))
    with pytest.raises(ValueError):
        call(masks=z(4, 2, dtype=torch.int64))
    with pytest.raises(TypeError):
        call(masks=z(4, 1, **i32))
    with pytest.raises(ValueError):
        call(drafts=[z(3, **i32)])
    with pytest.raises(ValueError):
        call(drafts=[])
    with pytest.raises(ValueError):
        call(bt=[z(0, 3, **i32)])
    with pytest.raises(ValueError):
        call(rank=1)
    with pytest.raises(ValueError):
        call(q=z(4, 576, dtype=torch.bfloat16))


# ----------------------------------------------------------------- results
def _rows(rng, n, fmt):
    lat, rope = rng.standard_normal((n, 512)), rng.standard_normal((n, 64))
    out = np.zeros((n, ROW[fmt]), dtype=np.uint8)
    if fmt == "fp8":
        code, sc = so.quantise_fp8(lat)
        out[:, :512], out[:, 512:528] = code, sc.view(np.uint8).reshape(n, 16)
    else:
        code, sc = so.quantise_fp4(lat)
        out[:, :256], out[:, 256:288] = code[:, 0::2] | (code[:, 1::2] << 4), sc
    bits = torch.from_numpy(rope).to(torch.bfloat16).view(torch.int16).numpy()
    out[:, -128:] = bits.view(np.uint8).reshape(n, 128)
    return out


class Case:
    """Requests' paged prefixes, drafted trees and queries; drafts lie in rows
    behind every block, node i on the pool its linear position belongs to."""

    def __init__(self, dev, fmt, nodes, ctx, H, D=1, bs=16, I=1, rank=-1, seed=0, pad=0, max_nodes=None,
                 shapes=("bushy", "chain", "star")):
        rng = np.random.default_rng(seed)
        self.dev, self.fmt, self.nodes, self.ctx, self.H = dev, fmt, nodes, ctx, H
        self.D, self.bs, self.I, self.rank = D, bs, I, rank
        self.B, self.n = len(nodes), sum(nodes)
        self.T = self.n + pad
        self.starts = np.concatenate([[0], np.cumsum(nodes)])
        self.max_nodes = max_nodes or max(1, max(nodes, default=1))
        self.max_prefix = max(ctx, default=0)
        self.parents = np.concatenate(
            [to.random_tree(rng, k, shapes[b % len(shapes)]) for b, k in enumerate(nodes)]
            + [np.full(pad, -1)]).astype(np.int64)
        self.masks, _ = to.tree_maps(self.parents, self.starts, ctx, self.T, self.max_nodes)
        self.pools, self.tables, self.drafts = [], [], []
        for d in range(D):
            held = [so.rank_rows(c, D, d, I) for c in ctx]
            nb = [-(-h // bs) for h in held]
            total = sum(nb) + 2
            perm = rng.permutation(total)
            table = np.full((max(1, self.B), max(nb, default=0) + 1), -1, dtype=np.int32)
            at = 0
            for b, k in enumerate(nb):
                table[b, :k] = perm[at:at + k]
                at += k
            self.tables.append(table)
            self.pools.append(_rows(rng, total * bs + self.T + 1, fmt))
            slots = np.full(self.T, -1, dtype=np.int32)
            for b in range(self.B):
                for j in range(nodes[b]):
                    if ((ctx[b] + j) // I) % D == d:
                        slots[self.starts[b] + j] = total * bs + self.starts[b] + j
            self.drafts.append(slots)
        self.q = torch.from_numpy(rng.standard_normal((self.T, H, 576))).to(torch.bfloat16)

    def upload(self):
        dev = self.dev
        self.args = (self.q.to(dev), _i32(self.starts, dev), _i32(self.ctx, dev), self.max_prefix,
                     torch.from_numpy(self.masks.view(np.int64)).to(dev), self.max_nodes,
                     [_i32(s, dev) for s in self.drafts], [torch.from_numpy(p).to(dev) for p in self.pools],
                     [_i32(t, dev) for t in self.tables], self.bs, SCALE)
        return self

    def run(self, rank=None, **kw):
        return capi.dcp_tree_mla_decode(*self.args, rank=self.rank if rank is None else rank,
                                        interleave=self.I, **kw)

    def keys(self, b, j, rank):
        """The (pool, slot) rows that node j of request b attends."""
        keys = to.prefix_keys(self.ctx[b], self.D, rank, self.bs, self.I, self.tables, b)
        slots = {d: s for d, s in enumerate(self.drafts) if rank < 0 or d == rank}
        t = self.starts[b] + j
        for m in range(self.nodes[b]):
            if (int(self.masks[t, m // 64]) >> (m % 64)) & 1:
                key = to.draft_key(slots, self.starts[b] + m)
                if key is not None:
                    keys.append(key)
        return keys

    def check(self, out, lse, rank=None, rows=None):
        rank = self.rank if rank is None else rank
        q = bf16_bits_to_f64(self.q.view(torch.int16).numpy().astype(np.uint16))
        out, lse = _np(out.double()), _np(lse.double())
        for b in range(self.B):
            for j in range(self.nodes[b]):
                t = self.starts[b] + j
                if rows is not None and t not in rows:
                    continue
                keys = self.keys(b, j, rank)
                raw = (np.stack([self.pools[d][s] for d, s in keys]) if keys
                       else np.zeros((0, ROW[self.fmt]), dtype=np.uint8))
                o, l, o_tol, l_tol = so.attend(q[t], raw, SCALE, KEY_STEP[self.fmt])
                if not keys:
                    assert np.all(out[t] == 0) and np.all(np.isneginf(lse[t])), (b, j)
                    continue
                assert np.all(np.abs(lse[t] - l) <= l_tol), (b, j, np.abs(lse[t] - l).max(), l_tol.min())
                bad = np.abs(out[t] - o) > o_tol
                assert not bad.any(), (b, j, np.argwhere(bad)[:4].tolist(),
                                       (np.abs(out[t] - o) / o_tol).max())


FORMATS = ["fp8", "fp4"]

CASES = [
    dict(nodes=[1], ctx=[0], H=1),                                   # a token by itself
    dict(nodes=[1], ctx=[1], H=128),
    dict(nodes=[3], ctx=[63], H=16, bs=16),
    dict(nodes=[8], ctx=[64], H=16, bs=1),
    dict(nodes=[9], ctx=[65], H=37, bs=48),                          # rows past two tiles
    dict(nodes=[5, 0, 3, 17], ctx=[127, 50, 0, 300], H=16, bs=16, pad=7),
    dict(nodes=[2, 2], ctx=[200, 129], H=64, D=2, bs=64, I=1),
    dict(nodes=[4, 1, 6], ctx=[90, 311, 5], H=20, D=3, bs=16, I=4),
    dict(nodes=[4, 7], ctx=[33, 190], H=16, D=4, bs=16, rank=2),
    dict(nodes=[2, 3], ctx=[3, 1], H=8, D=8, bs=16, rank=7),         # a rank that holds nothing
    dict(nodes=[3], ctx=[700], H=128, D=2, bs=64, I=64),
    dict(nodes=[70], ctx=[40], H=4, max_nodes=70),                   # two mask words
    dict(nodes=[200, 13], ctx=[10, 100], H=3, max_nodes=256, D=2),
    dict(nodes=[1, 1, 1], ctx=[2000, 1999, 65], H=16, D=1, bs=64),
    dict(nodes=[33], ctx=[500], H=5, shapes=("roots",)),
]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("i", range(len(CASES)))
def test_matches_the_definition(cuda_device, fmt, i):
    c = Case(cuda_device, fmt, seed=i, **CASES[i]).upload()
    _err()
    out = torch.full((c.T, c.H, 512), 3.0, dtype=torch.bfloat16, device=cuda_device)
    lse = torch.full((c.T, c.H), 5.0, device=cuda_device)
    c.run(out=out, lse=lse)
    c.check(out, lse)
    assert out[c.n:].eq(3).all() and lse[c.n:].eq(5).all()  # rows of nobody
    out2, lse2 = c.run()
    assert torch.equal(out[:c.n], out2[:c.n]) and torch.equal(lse[:c.n], lse2[:c.n])  # the same bits again
    assert _err() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rank", [-1, 1])
def test_a_long_prefix_and_few_rows(cuda_device, fmt, rank):
    c = Case(cuda_device, fmt, nodes=[3], ctx=[20011], H=16, D=2, bs=64, rank=rank, seed=5).upload()
    c.check(*c.run())


@pytest.mark.gpu
def test_many_short_requests(cuda_device):
    rng = np.random.default_rng(8)
    c = Case(cuda_device, "fp8", nodes=rng.integers(0, 4, 300).tolist(), ctx=rng.integers(0, 90, 300).tolist(),
             H=16, D=2, bs=16, seed=8).upload()
    c.check(*c.run())


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("B,most", [(640, 40), (1500, 30), (1290, 700)])
def test_more_requests_than_a_block_has_threads(cuda_device, fmt, B, most):
    """Whole and cut row tiles, the longest request among the late ones."""
    rng = np.random.default_rng(B)
    nodes, ctx = rng.integers(0, 3, B), rng.integers(0, 30, B)
    ctx[-7] = most
    nodes[-7] = 2
    c = Case(cuda_device, fmt, nodes=nodes.tolist(), ctx=ctx.tolist(), H=3, D=2, bs=16, seed=8).upload()
    c.check(*c.run())


@pytest.mark.gpu
@pytest.mark.parametrize("ctx", [20, 150])
def test_scales_of_all_sizes(cuda_device, ctx):
    """8-bit rows whose groups' scales reach from 2^-60 to 2^5, next to each other
    and a whole tile of small ones."""
    c = Case(cuda_device, "fp8", nodes=[9], ctx=[ctx], H=16, D=2, bs=16, seed=ctx)
    rng = np.random.default_rng(2)
    for pool in c.pools:
        scale = np.exp2(rng.integers(-60, 6, (len(pool), 4)) * 1.0) * rng.uniform(0.6, 1, (len(pool), 4))
        scale[:len(pool) // 3] = 2.0 ** -12
        pool[:, 512:528] = scale.astype("<f4").view(np.uint8)
    c.upload()
    _err()
    c.check(*c.run())
    assert _err() == capi.DEVERR_RANGE  # the scales below 2^-22, as the header says


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("what", ["scale", "rope", "q"])
def test_what_is_not_finite_stays_in_its_request(cuda_device, fmt, what):
    """A prefix row spoils its request's rows, a query its own row."""
    c = Case(cuda_device, fmt, nodes=[5, 4, 3], ctx=[70, 90, 10], H=16, bs=16, seed=7)
    spoilt = set(range(5, 9))
    slot = c.tables[0][1][4] * 16 + 3
    row = c.pools[0][slot]
    if what == "scale":
        if fmt == "fp8":
            row[520:524] = np.array([np.nan], dtype="<f4").view(np.uint8)
        else:
            row[270] = 0x7f
    elif what == "rope":
        row[-2:] = (0xc0, 0x7f)  # NaN
    else:
        c.q[6, 5, 100] = float("inf")
        spoilt = {6}
    c.upload()
    _err()
    out, lse = c.run()
    # 8-bit rows' rope values go to the tensor cores as they are
    assert _err() == (0 if (fmt, what) == ("fp8", "rope") else capi.DEVERR_RANGE)
    c.check(out, lse, rows=set(range(c.T)) - spoilt)
    if what == "q":
        assert not lse[6, 5].isfinite() and not out[6, 5].isfinite().any()
    else:
        assert lse[5:9].isnan().all() and out[5:9].isnan().all()


@pytest.mark.gpu
def test_a_batch_of_uneven_requests(cuda_device):
    c = Case(cuda_device, "fp8", nodes=[16, 5, 30, 1], ctx=[1500, 9000, 10, 4000], H=128, D=4, bs=64, seed=9).upload()
    out, lse = c.run()
    c.check(out, lse, rows={0, 7, 15, 16, 20, 21, 50, 51})


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
def test_partials_merge_into_the_whole(cuda_device, fmt):
    c = Case(cuda_device, fmt, nodes=[6, 2], ctx=[150, 3], H=16, D=4, bs=16, seed=3).upload()
    parts = [c.run(rank=d) for d in range(c.D)]
    for d, (o, l) in enumerate(parts):
        c.check(o, l, rank=d)
    out, lse = capi.dcp_lse_merge([p[0] for p in parts], [p[1] for p in parts])
    whole, whole_lse = c.run()
    c.check(whole, whole_lse)
    # partials round to bf16 once more each, 2^-8 of their size
    size = sum(p[0].float().abs() for p in parts)
    assert torch.all((out.float() - whole.float()).abs() <= 2.0 ** -6 * size + 1e-3)
    assert torch.allclose(lse, whole_lse, atol=1e-3)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
def test_any_mask(cuda_device, fmt):
    """Masks of no tree: none, all, others' branches, bits of nodes that do
    not exist; drafts that nobody holds, or two pools at once."""
    c = Case(cuda_device, fmt, nodes=[12, 7], ctx=[0, 70], H=16, D=2, bs=16, seed=12)
    rng = np.random.default_rng(1)
    c.masks[:, 0] = rng.integers(0, 2 ** 20, c.T).astype(np.uint64)
    c.masks[0] = 0                       # an empty prefix too: nothing to attend
    c.masks[1] = np.uint64(2 ** 64 - 1)
    c.masks[2] = np.uint64(1) << np.uint64(40)
    c.drafts[0][3] = c.drafts[1][3] = -1
    c.drafts[0][4], c.drafts[1][4] = 2, 3
    c.upload()
    _err()
    out, lse = c.run()
    c.check(out, lse)
    assert lse[0].isneginf().all() and lse[2].isneginf().all() and _err() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("where", ["latent", "rope", "nowhere"])
def test_what_is_masked_does_not_show(cuda_device, fmt, where):
    """A node whose cache row is not finite spoils the rows that see it and no
    others, in its own tile of rows or the next."""
    c = Case(cuda_device, fmt, nodes=[20], ctx=[30], H=16, bs=16, seed=2, shapes=("star",))
    bad = 5
    slot = c.drafts[0][bad]
    row = c.pools[0][slot]
    if where == "latent":
        if fmt == "fp8":
            row[516:520] = np.array([np.nan], dtype=np.float32).view(np.uint8)
        else:
            row[260] = 0x7f
    elif where == "rope":
        row[-128:-126] = (0x80, 0x7f)  # +inf
    else:
        row[:] = 0xff
        c.drafts[0][bad] = -1
    sees = [t for t in range(20) if (int(c.masks[t, 0]) >> bad) & 1]
    assert sees == [bad]
    c.upload()
    _err()
    out, lse = c.run()
    c.check(out, lse, rows=set(range(20)) - ({bad} if where != "nowhere" else set()))
    if where != "nowhere":
        assert not out[bad].isfinite().all()
    _err()


@pytest.mark.gpu
def test_large_scores_and_one_loud_key(cuda_device):
    """Scores far apart: the reference moves late, and early keys vanish."""
    c = Case(cuda_device, "fp4", nodes=[4], ctx=[400], H=16, bs=16, seed=21)
    c.q *= 30
    c.upload()
    c.check(*c.run())


@pytest.mark.gpu
def test_bad_inputs_are_reported(cuda_device):
    dev = cuda_device

    def run(change, max_prefix=None, **kw):
        c = Case(dev, "fp8", nodes=[3, 4, 2], ctx=[40, 50, 33], H=16, bs=16, seed=4)
        change(c)
        c.upload()
        if max_prefix is not None:
            c.args = c.args[:3] + (max_prefix,) + c.args[4:]
        out = torch.full((c.T, c.H, 512), 3.0, dtype=torch.bfloat16, device=dev)
        lse = torch.full((c.T, c.H), 5.0, device=dev)
        _err()
        c.run(out=out, lse=lse)
        return c, out, lse, _err()

    # a prefix past the bound: that request's rows are empty
    c, out, lse, err = run(lambda c: None, max_prefix=45)
    assert err == capi.DEVERR_CONTEXT
    assert out[3:7].eq(0).all() and lse[3:7].isneginf().all()
    c.check(out, lse, rows={0, 1, 2, 7, 8})

    def negative(c):
        c.ctx = [40, -1, 33]
    c, out, lse, err = run(negative)
    assert err == capi.DEVERR_CONTEXT and lse[3:7].isneginf().all()

    # more rows than max_nodes: untouched
    def narrow(c):
        c.max_nodes = 3
    c, out, lse, err = run(narrow)
    assert err == capi.DEVERR_TREE and out[3:7].eq(3).all() and lse[3:7].eq(5).all()
    c.check(out, lse, rows={0, 1, 2, 7, 8})

    # an unallocated block, a block past the pool, a draft past the pool
    def hole(c):
        c.tables[0][1, 2] = -1
        c.keys = lambda b, j, rank: [k for p, k in enumerate(Case.keys(c, b, j, rank)) if b != 1 or not 32 <= p < 48]
    c, out, lse, err = run(hole)
    assert err == capi.DEVERR_BLOCK_TABLE
    c.check(out, lse)

    def past(c):
        c.tables[0][1, 2] = 10 ** 6
        c.keys = lambda b, j, rank: [k for p, k in enumerate(Case.keys(c, b, j, rank)) if b != 1 or not 32 <= p < 48]
    c, out, lse, err = run(past)
    assert err == capi.DEVERR_SLOT_RANGE
    c.check(out, lse)

    def lost(c):
        c.drafts[0][8] = len(c.pools[0])
        c.keys = lambda b, j, rank: [k for k in Case.keys(c, b, j, rank) if k[1] < len(c.pools[0])]
    c, out, lse, err = run(lost)
    assert err == capi.DEVERR_SLOT_RANGE
    c.check(out, lse)

    # a table too narrow
    c = Case(dev, "fp8", nodes=[2], ctx=[40], H=16, bs=16, seed=4).upload()
    c.keys = lambda b, j, rank: [k for p, k in enumerate(Case.keys(c, b, j, rank)) if p < 32 or p >= 40]
    c.check(*c.run(bt_widths=[2]))
    assert _err() == capi.DEVERR_BLOCK_TABLE


@pytest.mark.gpu
def test_slots_and_offsets_past_32_bits(cuda_device):
    """Cache rows past 2^32 bytes, in blocks and as drafts."""
    c = Case(cuda_device, "fp8", nodes=[2], ctx=[20], H=16, bs=16, seed=6)
    far = 2 ** 32 // 656 + 100000
    far -= far % 16
    pool = torch.zeros((far + 64, 656), dtype=torch.uint8, device=cuda_device)
    slots = sorted({s for j in range(2) for _, s in c.keys(0, j, -1)})
    c.upload()
    small = c.args[7][0]
    table = c.tables[0].copy()
    pool[far:far + 16] = small[16 * table[0, 0]:16 * table[0, 0] + 16]
    pool[far + 16:far + 32] = small[16 * table[0, 1]:16 * table[0, 1] + 16]
    drafts = c.drafts[0].copy()
    for i, s in enumerate(drafts):
        pool[far + 32 + i] = small[int(s)]
    assert len(slots) == 22
    table[0, :2] = far // 16, far // 16 + 1
    c.args = (c.args[:6] + ([_i32(far + 32 + np.arange(2), cuda_device)], [pool], [_i32(table, cuda_device)])
              + c.args[9:])
    c.check(*c.run())


@pytest.mark.gpu
def test_workspaces_streams_and_graphs(cuda_device):
    """One workspace serves calls of any shapes in turn and needs no contents;
    two streams run with one each; a captured call replays on new inputs."""
    a = Case(cuda_device, "fp8", nodes=[3, 9], ctx=[2100, 777], H=64, D=2, bs=64, seed=31).upload()
    b = Case(cuda_device, "fp4", nodes=[20], ctx=[3000], H=16, bs=16, seed=32).upload()

    def workspace(c):
        return capi.alloc_tree_decode_workspace(c.T, c.H, c.B, c.max_prefix, c.max_nodes, c.D, c.I, c.rank,
                                                cuda_device)
    sizes = [0 if w is None else w.numel() for w in map(workspace, (a, b))]
    ws = torch.full((max(1, *sizes),), 0xff, dtype=torch.uint8, device=cuda_device)
    ref = [c.run() for c in (a, b)]
    for c, r in ((a, ref[0]), (b, ref[1]), (a, ref[0])):
        got = c.run(workspace=ws)
        assert torch.equal(got[0], r[0]) and torch.equal(got[1], r[1])
    a.check(*ref[0], rows={0, 5})
    b.check(*ref[1], rows={0, 19})
    if max(sizes):
        with pytest.raises(capi.SmlaError):
            a.run(workspace=ws[:256])
    streams = [torch.cuda.Stream(cuda_device) for _ in range(2)]
    both = [torch.full_like(ws, 0xff) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [c.run(workspace=w, stream=s) for c, w, s in zip((a, b), both, streams)]
    torch.cuda.synchronize()
    for g, r in zip(got, ref):
        assert torch.equal(g[0], r[0]) and torch.equal(g[1], r[1])
    out, lse = (torch.zeros_like(t) for t in ref[0])
    q = a.args[0]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=streams[0]):
        a.run(out=out, lse=lse, workspace=both[0], stream=streams[0])
    torch.cuda.synchronize()
    keep = q.clone()
    q.mul_(0.5)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    a.q = q.cpu()
    a.check(out, lse, rows={2, 11})
    q.copy_(keep)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref[0][0]) and _err() == 0
