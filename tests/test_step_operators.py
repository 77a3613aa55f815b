"""The serving step's operators: step maps, cache write and gather, sparse
decode over the 4-bit cache, windowed decode with sinks.  Refusals run
without a GPU; results are compared with the float64 definitions of
oracle/step_oracle.py, tolerances derived there."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import step_oracle as so
from oracle.smla_oracle import bf16_bits_to_f64
from sparse_mla_decode_dcp_gb300 import build as smla_build
from sparse_mla_decode_dcp_gb300 import capi

BAD, UNSUP, WS, OK = (capi.SMLA_ERR_INVALID_ARG, capi.SMLA_ERR_UNSUPPORTED,
                      capi.SMLA_ERR_WORKSPACE, capi.SMLA_OK)
FAKE = 0x10000  # aligned, never dereferenced
SCALE = 1.0 / math.sqrt(192.0)
FORMATS = {"fp8": capi.ROW_BYTES, "fp4": capi.FP4_ROW_BYTES}


@pytest.fixture(scope="module")
def lib():
    smla_build.build()
    return capi.load()


# ---------------------------------------------------------------- refusals
def _maps(lib, **kw):
    a = dict(ctx=FAKE, q=FAKE, B=2, T=4, D=2, rank=0, bs=16, I=1, free=FAKE, nf=4, bt=FAKE,
             stride=8, width=8, rs=None, req=None, pos=None, slots=FAKE, ll=None, taken=None)
    a.update(kw)
    return lib.smla_dcp_step_maps(a["ctx"], a["q"], a["B"], a["T"], a["D"], a["rank"], a["bs"],
                                  a["I"], a["free"], a["nf"], a["bt"], a["stride"], a["width"],
                                  a["rs"], a["req"], a["pos"], a["slots"], a["ll"], a["taken"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), BAD), (dict(T=-1), BAD), (dict(D=0), BAD), (dict(rank=2), BAD),
    (dict(rank=-1), BAD), (dict(bs=0), BAD), (dict(I=0), BAD), (dict(nf=-1), BAD),
    (dict(width=0), BAD), (dict(stride=7), BAD), (dict(ctx=None), BAD), (dict(q=None), BAD),
    (dict(bt=None), BAD), (dict(slots=None), BAD), (dict(free=None), BAD),
    (dict(slots=FAKE + 2), BAD), (dict(pos=FAKE + 1), BAD), (dict(taken=FAKE + 3), BAD),
    (dict(B=capi.MAX_STEP_REQS + 1), UNSUP),
    (dict(B=0, T=0, ctx=None, q=None, bt=None, slots=None), OK),
])
def test_maps_argument_checks(lib, kw, status):
    assert _maps(lib, **kw) == status


def _write(lib, **kw):
    a = dict(kv=FAKE, stride=576, T=2, gamma=FAKE, eps=1e-6, pos=FAKE, cs=FAKE, P=10, pairs=1,
             slots=FAKE, fmt=0, cache=FAKE, ns=10)
    a.update(kw)
    return lib.smla_mla_cache_write(a["kv"], a["stride"], a["T"], a["gamma"],
                                    ctypes.c_float(a["eps"]), a["pos"], a["cs"], a["P"], a["pairs"],
                                    a["slots"], a["fmt"], a["cache"], a["ns"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), BAD), (dict(ns=-1), BAD), (dict(fmt=2), BAD), (dict(fmt=-1), BAD),
    (dict(stride=568), BAD), (dict(stride=580), BAD), (dict(eps=0.0), BAD),
    (dict(eps=float("nan")), BAD), (dict(eps=-1e-6), BAD), (dict(P=0), BAD), (dict(pos=None), BAD),
    (dict(kv=None), BAD), (dict(slots=None), BAD), (dict(cache=None), BAD), (dict(kv=FAKE + 8), BAD),
    (dict(gamma=FAKE + 2), BAD), (dict(cache=FAKE + 8), BAD), (dict(slots=FAKE + 2), BAD),
    (dict(cs=FAKE + 2), BAD), (dict(T=0, kv=None, slots=None, cache=None), OK),
])
def test_write_argument_checks(lib, kw, status):
    assert _write(lib, **kw) == status


def _gather(lib, **kw):
    a = dict(cache=FAKE, ns=10, fmt=1, slots=FAKE, N=3, out=FAKE, stride=576, f32=0)
    a.update(kw)
    return lib.smla_mla_cache_gather(a["cache"], a["ns"], a["fmt"], a["slots"], a["N"], a["out"],
                                     a["stride"], a["f32"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), BAD), (dict(ns=-1), BAD), (dict(fmt=7), BAD), (dict(stride=575), BAD),
    (dict(stride=580), BAD), (dict(stride=578, f32=1), BAD), (dict(cache=None), BAD),
    (dict(slots=None), BAD), (dict(out=None), BAD), (dict(out=FAKE + 8), BAD),
    (dict(N=0, cache=None, slots=None, out=None), OK),
])
def test_gather_argument_checks(lib, kw, status):
    assert _gather(lib, **kw) == status


def _fp4(lib, **kw):
    a = dict(q=FAKE, kv=FAKE, ns=100, slots=FAKE, T=2, H=16, K=64, scale=0.07, out=FAKE, lse=FAKE,
             ws=None, wsb=0)
    a.update(kw)
    return lib.smla_sparse_mla_decode_fp4(a["q"], a["kv"], a["ns"], a["slots"], a["T"], a["H"],
                                          a["K"], ctypes.c_float(a["scale"]), a["out"], a["lse"],
                                          a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), BAD), (dict(K=0), BAD), (dict(H=0), BAD), (dict(H=129), UNSUP), (dict(ns=-1), BAD),
    (dict(scale=0.0), BAD), (dict(scale=float("nan")), BAD), (dict(q=None), BAD),
    (dict(q=FAKE + 8), BAD), (dict(kv=FAKE + 4), BAD), (dict(out=FAKE + 2), BAD),
    (dict(K=4096), WS), (dict(K=2 ** 30 + 1), UNSUP),
    (dict(T=0, q=None, kv=None, slots=None, out=None, lse=None), OK),
])
def test_fp4_decode_argument_checks(lib, kw, status):
    assert _fp4(lib, **kw) == status


def _pools(D, pools=None, widths=None):
    n = max(D, 1)
    arr = lambda typ, xs: (typ * n)(*(list(xs) + [0] * n)[:n])  # noqa: E731
    return (arr(ctypes.c_void_p, pools or [FAKE] * n), arr(ctypes.c_int64, [100] * n),
            arr(ctypes.c_void_p, [FAKE] * n), arr(ctypes.c_int64, [4] * n),
            arr(ctypes.c_int32, widths or [4] * n))


@pytest.mark.parametrize("D,kw,status", [
    (0, {}, BAD), (17, {}, UNSUP), (2, dict(I=0), BAD), (2, dict(bs=0), BAD), (2, dict(H=129), UNSUP),
    (2, dict(pools=[FAKE, None]), BAD), (2, dict(widths=[4, 5]), BAD), (2, dict(req=None), BAD),
    (2, dict(K=4096), WS),
])
def test_fused_fp4_argument_checks(lib, D, kw, status):
    a = dict(T=2, H=16, K=64, req=FAKE, bs=16, I=1, pools=None, widths=None)
    a.update(kw)
    got = lib.smla_dcp_sparse_mla_decode_fused_fp4(
        FAKE, a["T"], a["H"], a["K"], ctypes.c_float(0.07), a["req"], FAKE, 2, D, a["bs"], a["I"],
        *_pools(D, a["pools"], a["widths"]), FAKE, FAKE, None, 0, None)
    assert got == status


@pytest.mark.parametrize("D,kw,status", [
    (2, dict(window=0), BAD), (2, dict(window=-5), BAD), (2, dict(sinks=-1), BAD), (2, dict(fmt=2), BAD),
    (2, dict(rank=2), BAD), (2, dict(rank=-2), BAD), (2, dict(maxc=0), BAD), (2, dict(S=0), BAD),
    (2, dict(B=-1), BAD), (2, dict(H=129), UNSUP), (17, {}, UNSUP), (2, dict(pools=[FAKE, None]), BAD),
    (2, dict(maxc=65536, window=8192), WS), (2, dict(maxc=2 ** 30 + 1), UNSUP),
    (4, dict(I=2 ** 30, rank=0), UNSUP), (2, dict(I=2 ** 30 - 1, maxc=65536, window=8192, rank=0), WS),
    (2, dict(rank=0, maxc=65536, window=2 ** 31 - 1, sinks=2 ** 31 - 1, pools=[FAKE, None]), WS),
    (2, dict(B=0), OK),
])
def test_window_argument_checks(lib, D, kw, status):
    a = dict(B=2, S=1, H=16, maxc=100, window=8, sinks=2, rank=-1, bs=16, I=1, fmt=1, pools=None)
    a.update(kw)
    got = lib.smla_dcp_window_mla_decode(
        FAKE, a["B"], a["S"], a["H"], ctypes.c_float(0.07), FAKE, a["maxc"], a["window"], a["sinks"],
        D, a["rank"], a["bs"], a["I"], a["fmt"], *_pools(D, a["pools"]), FAKE, FAKE, None, 0, None)
    assert got == status


def test_workspace_sizes(lib):
    assert capi.fp4_decode_workspace_size(2, 0, 64) == 0
    assert capi.fp4_decode_workspace_size(-1, 16, 64) == 0
    size = capi.window_decode_workspace_size
    assert size(2, 16, 100, 0, 0, 2) == 0 and size(2, 16, 100, 8, -1, 2) == 0
    assert size(2, 16, 100, 8, 0, 2, 1, 2) == 0
    # the window bounds it, not the context; one rank holds its share
    assert size(8, 128, 65536, 1024, 64, 4) == size(8, 128, 2048, 1024, 64, 4)
    assert size(8, 128, 65536, 2 ** 31 - 1, 2 ** 31 - 1, 4) == size(8, 128, 65536, 65536, 0, 4)
    assert size(8, 128, 65536, 8192, 0, 4, 1, 0) < size(8, 128, 65536, 8192, 0, 4)
    # a rank with long runs holds no more than the window
    assert size(8, 128, 65536, 8192, 0, 2, 2 ** 20, 0) == size(8, 128, 65536, 8192, 0, 1)


def test_binding_refuses_what_it_cannot_pass():
    t = lambda *s, **k: torch.zeros(*s, **k)  # noqa: E731
    i32 = dict(dtype=torch.int32)
    kv = t(4, 576, dtype=torch.bfloat16)
    cache = t(8, 416, dtype=torch.uint8)
    with pytest.raises(ValueError):  # width of neither format
        capi.mla_cache_write(kv, t(4, **i32), t(8, 400, dtype=torch.uint8))
    with pytest.raises(TypeError):
        capi.mla_cache_write(kv, t(4, dtype=torch.int64), cache)
    with pytest.raises(ValueError):  # one slot per row
        capi.mla_cache_write(kv, t(3, **i32), cache)
    with pytest.raises(ValueError):
        capi.mla_cache_write(kv, t(4, **i32), cache, cos_sin=t(9, 64))
    with pytest.raises(ValueError):  # host tensors never reach the library
        capi.mla_cache_write(kv, t(4, **i32), cache)
    with pytest.raises(ValueError):
        capi.mla_cache_gather(cache, t(4, **i32), out=t(4, 576, dtype=torch.float16))
    with pytest.raises(ValueError):
        capi.sparse_mla_decode_fp4(t(2, 4, 576, dtype=torch.bfloat16), t(8, 656, dtype=torch.uint8),
                                   t(2, 5, **i32), 0.07)
    with pytest.raises(ValueError):  # mixed formats
        capi.dcp_window_mla_decode(t(1, 4, 576, dtype=torch.bfloat16), t(1, **i32), 8, 1, 4, 0,
                                   [cache, t(8, 656, dtype=torch.uint8)], [t(1, 2, **i32)] * 2, 4, 0.07)
    with pytest.raises(ValueError):  # fewer table rows than requests
        capi.dcp_window_mla_decode(t(2, 4, 576, dtype=torch.bfloat16), t(2, **i32), 8, 1, 4, 0,
                                   [cache], [t(1, 2, **i32)], 4, 0.07)
    with pytest.raises(ValueError):
        capi.dcp_step_maps(t(2, **i32), t(2, **i32), t(4, **i32), t(1, 4, **i32), 2, 1, 0, 16)


# ------------------------------------------------------------------- maps
def _np(t):
    return t.cpu().numpy()


def _err():
    return capi.get_device_error(clear=True)


def _i32(a, dev):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).to(dev)


def _maps_case(B, q_hi, ctx_hi, D, rank, bs, I, seed):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(1, ctx_hi + 1, B)
    q = np.minimum(ctx, rng.integers(0, q_hi + 1, B))
    W = max(1, max(-(-so.rank_rows(int(c), D, rank, I) // bs) for c in ctx)) + 2
    table = np.full((B, W), -1, dtype=np.int32)
    blocks = rng.permutation(B * W + 5).astype(np.int32)
    at = 0
    for b in range(B):
        n = -(-so.rank_rows(int(ctx[b] - q[b]), D, rank, I) // bs)
        table[b, :n] = blocks[at:at + n]
        at += n
    return ctx, q, blocks[at:], table


@pytest.mark.gpu
@pytest.mark.parametrize("B,q_hi,ctx_hi,D,rank,bs,I,pad", [
    (1, 1, 1, 1, 0, 1, 1, 0), (1, 400, 400, 3, 2, 1, 1, 5), (7, 1, 90, 4, 3, 16, 1, 0),
    (33, 20, 60, 2, 1, 3, 4, 64), (300, 9, 40, 2, 0, 16, 1, 1), (5, 0, 50, 2, 0, 16, 1, 3),
    (700, 3, 30, 8, 7, 64, 64, 0), (64, 500, 900, 5, 2, 48, 7, 11),
])
def test_maps_match_the_definition(cuda_device, B, q_hi, ctx_hi, D, rank, bs, I, pad):
    ctx, q, free, table = _maps_case(B, q_hi, ctx_hi, D, rank, bs, I, seed=B + D)
    T = int(q.sum()) + pad
    wide = torch.full((B, table.shape[1] + 3), 99, dtype=torch.int32, device=cuda_device)
    wide[:, :table.shape[1]] = _i32(table, cuda_device)
    bt = wide[:, :table.shape[1]]  # rows of a wider table
    want = so.step_maps(ctx, q, free, table, T, D, rank, bs, I)
    _err()
    for _ in range(2):  # the same lengths again write the same
        got = capi.dcp_step_maps(_i32(ctx, cuda_device), _i32(q, cuda_device), _i32(free, cuda_device),
                                 bt, T, D, rank, bs, interleave=I)
        for name, g, w in zip(capi.StepMaps._fields, got, want):
            assert np.array_equal(_np(g), w), name
        assert np.array_equal(_np(bt), table)
    assert torch.all(wide[:, table.shape[1]:] == 99)
    assert _err() == 0


@pytest.mark.gpu
def test_maps_of_the_largest_batch_and_of_none(cuda_device):
    B = capi.MAX_STEP_REQS
    ctx, q = np.full(B, 5), np.full(B, 1)
    free = np.arange(B, dtype=np.int32)[::-1].copy()
    table = np.full((B, 1), -1, dtype=np.int32)
    table[1::2, 0] = np.arange(B, B + B // 2)
    q[0::2] = 5  # a whole new request; the others append to their block
    want_table = table.copy()
    T = int(q.sum())
    want = so.step_maps(ctx, q, free, want_table, T, 1, 0, 8, 1)
    bt = _i32(table, cuda_device)
    got = capi.dcp_step_maps(_i32(ctx, cuda_device), _i32(q, cuda_device), _i32(free, cuda_device), bt,
                             T, 1, 0, 8)
    for g, w in zip(got, want):
        assert np.array_equal(_np(g), w)
    assert np.array_equal(_np(bt), want_table)
    got = capi.dcp_step_maps(_i32([], cuda_device), _i32([], cuda_device), _i32([], cuda_device),
                             bt[:0], 3, 1, 0, 8)
    assert _np(got.slots).tolist() == [-1] * 3 and _np(got.row_start).tolist() == [0]
    assert _err() == 0


@pytest.mark.gpu
def test_maps_report_bad_inputs(cuda_device):
    dev = cuda_device

    def run(ctx, q, free, table, T, bs=4, width=None):
        bt = _i32(table, dev)
        got = capi.dcp_step_maps(_i32(ctx, dev), _i32(q, dev), _i32(free, dev), bt, T, 1, 0, bs,
                                 bt_width=width)
        return [_np(g).tolist() for g in got], _np(bt).tolist(), _err()

    _err()
    # more new tokens than positions, a negative length: no new tokens
    (rs, _, pos, slots, _, taken), _, err = run([3, -2, 2], [4, 0, 1], [7, 8], [[-1], [-1], [5]], 2)
    assert rs == [0, 0, 0, 1] and pos == [1, 0] and slots == [21, -1] and taken == [0]
    assert err == capi.DEVERR_CONTEXT
    # more rows than T: those that fit
    (rs, _, _, slots, _, taken), _, err = run([3, 3], [3, 3], [7, 8], [[-1], [-1]], 4)
    assert rs == [0, 3, 6] and slots == [28, 29, 30, 32] and taken == [2]
    assert err == capi.DEVERR_CONTEXT
    # a free list too short
    (_, _, _, slots, _, taken), bt, err = run([3, 3], [3, 3], [7], [[-1], [-1]], 6)
    assert slots == [28, 29, 30, -1, -1, -1] and taken == [2] and bt == [[7], [-1]]
    assert err == capi.DEVERR_FREE_BLOCKS
    # a table too narrow, an unallocated old block
    (_, _, _, slots, _, _), bt, err = run([6], [6], [7, 8], [[-1, 55]], 6, width=1)
    assert slots == [28, 29, 30, 31, -1, -1] and bt == [[7, 55]] and err == capi.DEVERR_BLOCK_TABLE
    (_, _, _, slots, _, _), _, err = run([3], [1], [7], [[-1]], 1)
    assert slots == [-1] and err == capi.DEVERR_BLOCK_TABLE
    # a slot past 2^31 - 1
    (_, _, _, slots, _, _), _, err = run([1], [1], [2 ** 30], [[-1]], 1)
    assert slots == [-1] and err == capi.DEVERR_BLOCK_TABLE


# ------------------------------------------------------------------ write
def _bits(t):
    return _np(t.contiguous().view(torch.int16)).astype(np.uint16)


def _f64(t):
    return _np(t.double())


def _table(n, dev):
    a = torch.arange(n, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)
    return torch.cat([a.cos(), a.sin()], 1).float().to(dev)


def _check_rows(rows, y, rope, rope_size, fmt):
    """Packed rows against float64 latents (bit by bit) and rope values."""
    if fmt == "fp8":
        code, scale = so.quantise_fp8(y)
        assert np.array_equal(rows[:, 512:528].copy().view("<f4"), scale)
        assert np.array_equal(rows[:, :512], code)
        got = bf16_bits_to_f64(rows[:, 528:].copy().view("<u2"))
    else:
        code, scale = so.quantise_fp4(y)
        assert np.array_equal(rows[:, 256:288], scale)
        assert np.array_equal(rows[:, :256], code[:, 0::2] | (code[:, 1::2] << 4))
        got = bf16_bits_to_f64(rows[:, 288:].copy().view("<u2"))
    # bf16's half step, and two fp32 roundings of the products' size
    assert np.all(np.abs(got - rope) <= 2.0 ** -8 * np.abs(rope) + 2 * 2.0 ** -24 * rope_size + 2.0 ** -134)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("T,stride,pairs,norm,rot", [
    (1, 576, True, True, True), (5, 640, False, True, True), (64, 2112, True, True, True),
    (67, 584, False, False, True), (33, 576, True, True, False), (300, 576, True, False, False),
])
def test_write_matches_float64(cuda_device, fmt, T, stride, pairs, norm, rot):
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(T)
    wide = torch.randn((T, stride), generator=g, device=dev) * torch.exp(
        2 * torch.randn((T, 1), generator=g, device=dev))
    kv = wide.to(torch.bfloat16)[:, stride - 576:] if stride % 8 == 0 else None
    kv[0, :128] = 0  # an empty group
    gamma = (1 + 0.3 * torch.randn(512, generator=g, device=dev)).to(torch.bfloat16) if norm else None
    n = 2 * T + 3
    slots = torch.randperm(n, generator=torch.Generator().manual_seed(T))[:T].to(torch.int32)
    if T > 2:
        slots[1] = -1
    pos = torch.randint(0, 5000, (T,), generator=torch.Generator().manual_seed(T)).to(torch.int32)
    table = _table(5000, dev)
    cache = torch.full((n, FORMATS[fmt]), 0x5A, dtype=torch.uint8, device=dev)
    _err()
    capi.mla_cache_write(kv, slots.to(dev), cache, gamma=gamma, eps=1e-6,
                         positions=pos.to(dev) if rot else None, cos_sin=table if rot else None,
                         rope_pairs=pairs)
    assert _err() == 0
    live = slots.numpy() >= 0
    rows = _np(cache)
    untouched = np.setdiff1d(np.arange(n), slots.numpy()[live])
    assert np.all(rows[untouched] == 0x5A)
    x = _f64(kv)[live]
    y = so.normalise(x[:, :512], _f64(gamma) if norm else None, 1e-6)
    cs = _f64(table)[pos.numpy()[live]]
    rope = so.rotate(x[:, 512:], cs, pairs) if rot else x[:, 512:]
    _check_rows(rows[slots.numpy()[live]], y, rope, np.abs(x[:, 512:]).max(axis=1, keepdims=True) * 2, fmt)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_write_rounds_ties_to_even_and_clips(cuda_device, fmt):
    """Latents without a norm that sit on rounding borders of codes and scales."""
    dev = cuda_device
    base = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25, -1.75,
                         -2.5, -3.5, -5.0, 0.0])
    m = torch.cat([base * 2.0 ** e * f for e in range(-12, 12) for f in (1.0, 1.0625, 1.125, 1.25)])
    m = torch.cat([m, torch.zeros(-m.numel() % 512)]).view(-1, 512)
    kv = torch.zeros((m.shape[0], 576))
    kv[:, :512] = m
    kv = kv.to(torch.bfloat16).to(dev)
    cache = torch.zeros((m.shape[0], FORMATS[fmt]), dtype=torch.uint8, device=dev)
    capi.mla_cache_write(kv, torch.arange(m.shape[0], dtype=torch.int32, device=dev), cache)
    _check_rows(_np(cache), _f64(kv)[:, :512], _f64(kv)[:, 512:], 0, fmt)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_write_extreme_rows(cuda_device, fmt):
    dev = cuda_device
    g = torch.Generator().manual_seed(3)
    kv = torch.randn((6, 576), generator=g)
    kv[0] = 0  # 0 / sqrt(eps): an all-zero row
    kv[1, :512] *= 1e-4  # below sqrt(eps)
    kv[2, :512] *= 1e9
    kv[3, 40] = float("inf")
    kv[4, 300] = float("nan")
    kv = kv.to(torch.bfloat16).to(dev)
    gamma = torch.full((512,), 1.5, dtype=torch.bfloat16, device=dev)
    cache = torch.zeros((6, FORMATS[fmt]), dtype=torch.uint8, device=dev)
    slots = torch.arange(6, dtype=torch.int32, device=dev)
    capi.mla_cache_write(kv, slots, cache, gamma=gamma, eps=1e-6)
    rows, x = _np(cache), _f64(kv)
    good = [0, 1, 2, 5]
    _check_rows(rows[good], so.normalise(x[good][:, :512], np.full(512, 1.5), 1e-6), x[good][:, 512:],
                0, fmt)
    lat, _ = so.parse(rows[[3, 4]])
    assert np.all(np.isnan(lat))
    # without a norm only the groups that hold such a value
    capi.mla_cache_write(kv, slots, cache)
    lat, _ = so.parse(_np(cache)[[3, 4]])
    size = 128 if fmt == "fp8" else 16
    for row, at in ((0, 40), (1, 300)):
        bad = np.isnan(lat[row])
        assert np.array_equal(np.nonzero(bad)[0] // size, np.full(size, at // size))


@pytest.mark.gpu
def test_write_reports_and_skips_bad_rows(cuda_device):
    dev = cuda_device
    kv = torch.ones((4, 576), dtype=torch.bfloat16, device=dev)
    cache = torch.zeros((4, 416), dtype=torch.uint8, device=dev)
    _err()
    capi.mla_cache_write(kv, _i32([0, 4, 2, -1], dev), cache)
    assert _err() == capi.DEVERR_SLOT_RANGE
    assert torch.all(cache[[0, 2]].any(1)) and not cache[[1, 3]].any()
    cache.zero_()
    capi.mla_cache_write(kv, _i32([0, 1, 2, -1], dev), cache, positions=_i32([9, 10, -1, 77], dev),
                         cos_sin=_table(10, dev))
    assert _err() == capi.DEVERR_POSITION  # the row without a slot has none to check
    assert cache[0].any() and not cache[1:].any()


# ----------------------------------------------------------------- gather
def _random_cache(n, fmt, seed, dev):
    """Rows of random codes and sensible scales and rope values."""
    rng = np.random.default_rng(seed)
    rows = rng.integers(0, 256, (n, FORMATS[fmt]), dtype=np.uint8)
    rope = torch.from_numpy(rng.standard_normal((n, 64))).to(torch.bfloat16)
    rows[:, -128:] = rope.view(torch.int16).numpy().view(np.uint8)
    if fmt == "fp8":
        codes = rows[:, :512]
        codes[(codes & 0x7F) == 0x7F] = 0x38
        rows[:, 512:528] = (rng.uniform(0.5, 2, (n, 4)) / 100).astype("<f4").view(np.uint8)
    else:
        rows[:, 256:288] = rng.integers(0x18, 0x34, (n, 32))  # 2^-4 .. 0.75
    return torch.from_numpy(rows).to(dev)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N", [1, 3, 4, 31, 257])
def test_gather_matches_float64(cuda_device, fmt, dtype, N):
    cache = _random_cache(100, fmt, N, cuda_device)
    if fmt == "fp4" and N == 257:  # every scale code, subnormal and largest among them
        cache[:, 256:288] = torch.arange(32, dtype=torch.uint8, device=cuda_device) * 4 - 1 & 0x7E
    slots = np.random.default_rng(N).integers(-1, 100, N).astype(np.int32)
    slots[0] = 99
    wide = torch.full((N, 600), 7.0, dtype=dtype, device=cuda_device)
    _err()
    got = capi.mla_cache_gather(cache, _i32(slots, cuda_device), out=wide[:, 8:584])
    assert _err() == 0
    lat, rope = so.parse(_np(cache)[np.maximum(slots, 0)])
    want = np.concatenate([lat, rope], 1) * (slots >= 0)[:, None]
    # one rounding (bf16 values of fp8 rows: after one to fp32)
    half = torch.finfo(dtype).eps / 2 * (1 + 2.0 ** -15)
    assert np.all(np.abs(_f64(got) - want) <= half * np.abs(want))
    assert torch.all(wide[:, :8] == 7) and torch.all(wide[:, 584:] == 7)
    assert torch.equal(capi.mla_cache_gather(cache, _i32(slots, cuda_device), dtype=dtype), got)


@pytest.mark.gpu
def test_gather_reports_bad_slots(cuda_device):
    cache = _random_cache(5, "fp4", 0, cuda_device)
    _err()
    got = capi.mla_cache_gather(cache, _i32([4, 5, 2 ** 31 - 1, -7], cuda_device))
    assert _err() == capi.DEVERR_SLOT_RANGE
    assert got[0].any() and not got[1:].any()


# ----------------------------------------------------------------- decode
def _check(out, lse, refs, where=""):
    """refs: per row (out, lse, out_tol, lse_tol)."""
    o, l = _f64(out), _f64(lse)
    for t, (ro, rl, to, tl) in enumerate(refs):
        empty = np.isneginf(rl)
        assert np.array_equal(np.isneginf(l[t]), empty), f"{where} row {t}"
        if empty.all():
            assert not out[t].any(), f"{where} row {t}: not zero"
            continue
        assert np.all(np.abs(l[t] - rl) <= tl), f"{where} row {t}: lse {np.abs(l[t] - rl).max()}"
        assert np.all(np.abs(o[t] - ro) <= to), f"{where} row {t}: out {np.abs(o[t] - ro).max()}"


def _q(T, H, dev, seed=0):
    g = torch.Generator(device=dev).manual_seed(seed)
    return torch.randn((T, H, 576), generator=g, device=dev).to(torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,K", [
    (1, 1, 1), (3, 16, 63), (2, 128, 64), (5, 37, 65), (4, 128, 129), (1, 64, 700), (3, 8, 2049),
    (80, 16, 128),
])
def test_fp4_sparse_decode_matches_float64(cuda_device, T, H, K):
    dev = cuda_device
    rng = np.random.default_rng(K)
    n = 500
    cache = _random_cache(n, "fp4", K, dev)
    slots = rng.integers(0, n, (T, K)).astype(np.int32)  # repeats among them
    slots[rng.random((T, K)) < 0.2] = -1
    if T > 1:
        slots[T - 1] = -1  # an empty row
    if T > 2:
        slots[1] = -1
        slots[1, K // 2] = n - 1  # a single key
    q = _q(T, H, dev, K)
    _err()
    out, lse = capi.sparse_mla_decode_fp4(q, cache, _i32(slots, dev), SCALE)
    assert _err() == 0
    rows, qf = _np(cache), _f64(q)
    _check(out, lse, [so.attend(qf[t], rows[slots[t][slots[t] >= 0]], SCALE) for t in range(T)])


def _paged(ctx, D, bs, I, fmt, seed, dev):
    """Random pools and tables of D shards; numpy views for the oracle."""
    rng = np.random.default_rng(seed)
    pools, tables = [], []
    for d in range(D):
        nb = [-(-so.rank_rows(int(c), D, d, I) // bs) for c in ctx]
        perm = rng.permutation(sum(nb) + 2).astype(np.int32)
        table = np.full((len(ctx), max(1, max(nb)) + 1), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(nb):
            table[b, :n] = perm[at:at + n]
            at += n
        tables.append(_i32(table, dev))
        pool = _random_cache((sum(nb) + 2) * bs, fmt, seed + d, dev)
        held = np.zeros(pool.shape[0], dtype=bool)
        for b, c in enumerate(ctx):
            lp = np.arange(so.rank_rows(int(c), D, d, I))
            held[table[b, lp // bs] * bs + lp % bs] = True
        pool[torch.from_numpy(~held).to(dev)] = 0xFF  # NaN scales, codes and rope nobody may read
        pools.append(pool)
    return pools, tables


def _rows_at(pools, tables, b, ids, D, bs, I, rank=-1):
    """Cache rows of request b's positions ids (rank's only, where given)."""
    rows = []
    for t in ids:
        d = (t // I) % D
        if rank >= 0 and d != rank:
            continue
        lp = (t // (I * D)) * I + t % I
        rows.append(pools[d][int(tables[d][b, lp // bs]) * bs + lp % bs])
    width = pools[max(rank, 0)].shape[1]
    return np.stack(rows) if rows else np.zeros((0, width), dtype=np.uint8)


@pytest.mark.gpu
@pytest.mark.parametrize("D,I,bs,H,K", [(2, 1, 16, 16, 64), (3, 4, 1, 37, 100), (8, 1, 64, 128, 300)])
def test_fp4_fused_step_matches_float64_and_the_three_calls(cuda_device, D, I, bs, H, K):
    dev = cuda_device
    ctx = [700, 3, 250, 64]
    pools, tables = _paged(ctx, D, bs, I, "fp4", 11 * D, dev)
    rng = np.random.default_rng(D)
    topk = np.full((4, K), -1, dtype=np.int32)
    for b, c in enumerate(ctx):
        n = min(K, c)
        topk[b, rng.permutation(K)[:n]] = rng.choice(c, n, replace=False)
    topk[3] = -1
    q = _q(4, H, dev, D)
    req = _i32(range(4), dev)
    _err()
    out, lse = capi.dcp_sparse_mla_decode_fused_fp4(q, req, _i32(topk, dev), pools, tables, bs, SCALE,
                                                    interleave=I)
    npools, ntables, qf = [_np(p) for p in pools], [_np(t) for t in tables], _f64(q)
    refs = [so.attend(qf[b], _rows_at(npools, ntables, b, topk[b][topk[b] >= 0], D, bs, I), SCALE)
            for b in range(4)]
    _check(out, lse, refs, "fused")
    outs, lses = [], []
    for r in range(D):
        sl, _ = capi.dcp_filter_convert_index(req, tables[r], _i32(topk, dev), D, r, bs, interleave=I)
        o, l = capi.sparse_mla_decode_fp4(q, pools[r], sl, SCALE)
        outs.append(o)
        lses.append(l)
    # the shards' partials add a bf16 rounding of each
    m_out, m_lse = capi.dcp_lse_merge(outs, lses)
    _check(m_out, m_lse, [(o, l, to + 2.0 ** -8 * np.abs(o).max(), 2 * tl) for o, l, to, tl in refs],
           "three calls")
    assert _err() == 0


WINDOWS = [(1, 0), (1, 1), (7, 0), (64, 4), (65, 63), (200, 300), (2 ** 31 - 1, 0), (3, 2 ** 31 - 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("D,I,bs,S,rank", [(1, 1, 16, 1, -1), (3, 1, 8, 2, -1), (2, 4, 3, 3, 1),
                                           (2, 100, 16, 1, 0)])
def test_window_matches_float64(cuda_device, fmt, window, sinks, D, I, bs, S, rank):
    dev = cuda_device
    ctx = [S, 5 + S, 64, 131, 430]
    B, H = len(ctx), 16
    pools, tables = _paged(ctx, D, bs, I, fmt, 5, dev)
    q = _q(B * S, H, dev, window % 97)
    use = [r if rank < 0 or d == rank else None for d, r in enumerate(pools)]
    tab = [r if rank < 0 or d == rank else None for d, r in enumerate(tables)]
    _err()
    out, lse = capi.dcp_window_mla_decode(q, _i32(ctx, dev), 430, S, window, sinks, use, tab, bs, SCALE,
                                          rank=rank, interleave=I)
    assert _err() == 0
    npools, ntables, qf = [_np(p) for p in pools], [_np(t) for t in tables], _f64(q)
    refs = []
    for t in range(B * S):
        b, s = divmod(t, S)
        ids = so.window_positions(ctx[b] - S + s, window, sinks)
        refs.append(so.attend(qf[t], _rows_at(npools, ntables, b, ids, D, bs, I, rank), SCALE,
                              2.0 ** -11 if fmt == "fp8" else 0.0))
    _check(out, lse, refs)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_window_over_splits_long_contexts_and_freed_blocks(cuda_device, fmt):
    """Many key ranges a row; the blocks between sinks and window are gone."""
    dev = cuda_device
    ctx, bs, window, sinks = [9000, 40, 5000], 16, 4500, 40
    pools, tables = _paged(ctx, 1, bs, 1, fmt, 2, dev)
    for b, c in enumerate(ctx):
        lo, hi = -(-sinks // bs), max(c - window, 0) // bs
        if hi > lo:
            tables[0][b, lo:hi] = -1
    q = _q(3, 128, dev, 4)
    _err()
    ws = capi.alloc_window_decode_workspace(3, 128, 9000, window, sinks, 1, 1, -1, dev)
    assert ws is not None
    npools, ntables, qf = [_np(p) for p in pools], [_np(t) for t in tables], _f64(q)
    refs = [so.attend(qf[b], _rows_at(npools, ntables, b, so.window_positions(c - 1, window, sinks), 1, bs, 1),
                      SCALE, 2.0 ** -11 if fmt == "fp8" else 0.0) for b, c in enumerate(ctx)]
    for _ in range(2):  # the workspace is left as it has to be found
        out, lse = capi.dcp_window_mla_decode(q, _i32(ctx, dev), 9000, 1, window, sinks, pools, tables, bs,
                                              SCALE, workspace=ws)
        _check(out, lse, refs)
    assert _err() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_window_rows_longer_than_a_pairs_list(cuda_device, fmt):
    """Up to 4100 keys a row, over several key ranges.  Then the same with
    blocks missing."""
    dev = cuda_device
    B, S, H, D, bs, window, sinks = 4, 19, 3, 2, 16, 4090, 10
    ctx = [4150, 2049, 2100, 3000]
    pools, tables = _paged(ctx, D, bs, 1, fmt, 6, dev)
    q = _q(B * S, H, dev, 9)
    npools, qf = [_np(p) for p in pools], _f64(q)
    step = 2.0 ** -11 if fmt == "fp8" else 0.0

    def refs():
        nt, out = [_np(t) for t in tables], []
        for t in range(0, B * S, 7):  # every seventh token
            b, i = divmod(t, S)
            ids = [x for x in so.window_positions(ctx[b] - S + i, window, sinks)
                   if nt[x % D][b, (x // D) // bs] >= 0]
            out.append(so.attend(qf[t], _rows_at(npools, nt, b, ids, D, bs, 1), SCALE, step))
        return out

    _err()
    out, lse = capi.dcp_window_mla_decode(q, _i32(ctx, dev), 4150, S, window, sinks, pools, tables, bs, SCALE)
    assert _err() == 0
    _check(out[::7], lse[::7], refs(), "whole")
    tables[0][0, 3] = tables[1][0, 90] = tables[0][0, 129] = -1
    tables[0][3], tables[1][3] = -1, -1  # a request without any
    tables[1][2, 64] = -1  # the last block of a row just longer than the list
    out, lse = capi.dcp_window_mla_decode(q, _i32(ctx, dev), 4150, S, window, sinks, pools, tables, bs, SCALE)
    assert _err() == capi.DEVERR_BLOCK_TABLE
    _check(out[::7], lse[::7], refs(), "holes")
    assert torch.isneginf(lse[3 * S:]).all() and not out[3 * S:].any()


@pytest.mark.gpu
@pytest.mark.parametrize("T,K", [(77, 2048), (90, 2047), (100, 1985), (153, 2048)])
def test_fp4_sparse_decode_past_one_wave_of_pairs(cuda_device, T, K):
    """Rows cut into a large and a small key range; a workspace serves call
    after call, with the same bits."""
    dev, H = cuda_device, 5
    rng = np.random.default_rng(T)
    cache = _random_cache(700, "fp4", 3, dev)
    slots = rng.integers(0, 700, (T, K)).astype(np.int32)
    slots[rng.random((T, K)) < 0.1] = -1
    slots[7] = -1
    slots[16, :1900] = -1  # its keys are all in the last range
    slots[25, 64:] = -1
    q = _q(T, H, dev, T)
    ws = capi.alloc_fp4_decode_workspace(T, H, K, dev)
    _err()
    out, lse = capi.sparse_mla_decode_fp4(q, cache, _i32(slots, dev), SCALE, workspace=ws)
    for _ in range(3):
        out2, lse2 = capi.sparse_mla_decode_fp4(q, cache, _i32(slots, dev), SCALE, workspace=ws)
        assert torch.equal(out, out2) and torch.equal(lse, lse2)
    assert _err() == 0
    rows, qf = _np(cache), _f64(q)
    at = list(range(7, T, 9))
    _check(out[at], lse[at], [so.attend(qf[t], rows[slots[t][slots[t] >= 0]], SCALE) for t in at])


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_long_windows_past_one_wave_of_pairs(cuda_device, fmt):
    """64 rows of up to 4112 keys, short contexts among them (ranges without
    a key)."""
    dev = cuda_device
    B, S, H, D, bs, window, sinks = 32, 2, 4, 2, 64, 4096, 16
    ctx = [4300 if b % 3 == 0 else 2 + 130 * b for b in range(B)]
    pools, tables = _paged(ctx, D, bs, 1, fmt, 8, dev)
    q = _q(B * S, H, dev, 3)
    ws = capi.alloc_window_decode_workspace(B * S, H, 4300, window, sinks, D, 1, -1, dev)
    _err()
    for _ in range(2):
        out, lse = capi.dcp_window_mla_decode(q, _i32(ctx, dev), 4300, S, window, sinks, pools, tables, bs,
                                              SCALE, workspace=ws)
    assert _err() == 0
    npools, ntables, qf = [_np(p) for p in pools], [_np(t) for t in tables], _f64(q)
    at = list(range(0, B * S, 5))
    refs = [so.attend(qf[t], _rows_at(npools, ntables, t // S, so.window_positions(
        ctx[t // S] - S + t % S, window, sinks), D, bs, 1), SCALE, 2.0 ** -11 if fmt == "fp8" else 0.0)
            for t in at]
    _check(out[at], lse[at], refs)


@pytest.mark.gpu
def test_window_wide_enough_is_the_dense_decode(cuda_device):
    """Two kernels, one definition: both within its bounds."""
    dev = cuda_device
    ctx = [300, 77]
    pools, tables = _paged(ctx, 2, 16, 1, "fp8", 8, dev)
    q = _q(4, 32, dev)
    npools, ntables, qf = [_np(p) for p in pools], [_np(t) for t in tables], _f64(q)
    refs = [so.attend(qf[t], _rows_at(npools, ntables, t // 2, range(ctx[t // 2] - 1 + t % 2), 2, 16, 1), SCALE,
                      2.0 ** -11) for t in range(4)]
    _check(*capi.dcp_dense_mla_decode(q, _i32(ctx, dev), 300, 2, pools, tables, 16, SCALE), refs, "dense")
    _check(*capi.dcp_window_mla_decode(q, _i32(ctx, dev), 300, 2, 300, 0, pools, tables, 16, SCALE), refs,
           "window")


@pytest.mark.gpu
def test_window_reports_bad_contexts_and_tables(cuda_device):
    dev = cuda_device
    pools, tables = _paged([50, 50, 50], 1, 16, 1, "fp4", 1, dev)
    q = _q(3, 4, dev)
    _err()
    out, lse = capi.dcp_window_mla_decode(q, _i32([0, 51, 50], dev), 50, 1, 8, 2, pools, tables, 16, SCALE)
    assert _err() == capi.DEVERR_CONTEXT
    assert torch.isneginf(lse[:2]).all() and not out[:2].any() and torch.isfinite(lse[2]).all()
    tables[0][2, 3] = -1
    out, lse = capi.dcp_window_mla_decode(q, _i32([50, 50, 50], dev), 50, 1, 8, 2, pools, tables, 16, SCALE)
    assert _err() == capi.DEVERR_BLOCK_TABLE and torch.isfinite(lse).all()


@pytest.mark.gpu
def test_nan_scale_sets_the_range_bit(cuda_device):
    dev = cuda_device
    cache = _random_cache(70, "fp4", 0, dev)
    cache[69, 256 + 5] = 0x7F
    q = _q(1, 4, dev)
    _err()
    capi.sparse_mla_decode_fp4(q, cache, _i32([list(range(69))], dev), SCALE)
    assert _err() == 0
    capi.sparse_mla_decode_fp4(q, cache, _i32([list(range(70))], dev), SCALE)
    assert _err() & capi.DEVERR_RANGE


@pytest.mark.gpu
def test_row_offsets_past_32_bits(cuda_device):
    """A 4-bit cache of more than 4 GiB: write, gather and decode at its end."""
    dev = cuda_device
    n = (1 << 32) // 416 + 1000
    cache = torch.empty((n, 416), dtype=torch.uint8, device=dev)
    kv = torch.randn((64, 576), device=dev).to(torch.bfloat16)
    slots = _i32(range(n - 64, n), dev)
    capi.mla_cache_write(kv, slots, cache)
    small = torch.zeros((64, 416), dtype=torch.uint8, device=dev)
    capi.mla_cache_write(kv, _i32(range(64), dev), small)
    assert torch.equal(cache[-64:], small)
    assert torch.equal(capi.mla_cache_gather(cache, slots), capi.mla_cache_gather(small, _i32(range(64), dev)))
    q = _q(1, 16, dev)
    a = capi.sparse_mla_decode_fp4(q, cache, slots[None], SCALE)
    b = capi.sparse_mla_decode_fp4(q, small, _i32([list(range(64))], dev), SCALE)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# --------------------------------------------------------------- together
@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_serving_step_runs_together(cuda_device, fmt):
    """Prefill, then decode steps through the pipeline: maps, write, windowed
    decode over three pools, against attention over the rows as defined."""
    from sparse_mla_decode_dcp_gb300.pipeline import DcpServingStep
    dev = cuda_device
    D, bs, S, H, window, sinks = 3, 8, 2, 16, 60, 5
    g = torch.Generator(device=dev).manual_seed(1)
    gamma = (1 + 0.2 * torch.randn(512, generator=g, device=dev)).to(torch.bfloat16)
    table = _table(300, dev)
    step = DcpServingStep(num_reqs=3, tokens_per_req=S, heads=H, dcp=D, block_size=bs, blocks_per_rank=40,
                          max_ctx=200, window=window, sinks=sinks, fmt=fmt, gamma=gamma, cos_sin=table,
                          sm_scale=SCALE, device=dev)
    ctx = np.array([90, 1, 33])
    hist = [[] for _ in ctx]  # every request's latent rows, in order

    def bring(q):
        kv = torch.randn((int(q.sum()), 576), generator=g, device=dev).to(torch.bfloat16)
        at = 0
        for b, n in enumerate(q):
            hist[b].extend(_f64(kv)[at:at + n])
            at += n
        return kv

    _err()
    step.prefill(_i32(ctx, dev), _i32(ctx, dev), bring(ctx))
    with pytest.raises(RuntimeError):  # the blocks it took are still listed as free
        step.run(_i32(ctx, dev), torch.zeros((3 * S, 576), dtype=torch.bfloat16, device=dev), _q(3 * S, H, dev))
    step.take_blocks()
    for i in range(3):
        ctx = ctx + S
        q = _q(3 * S, H, dev, i)
        out, lse = step.run(_i32(ctx, dev), bring(np.full(3, S)), q)
        torch.cuda.synchronize()
        step.take_blocks()
        refs = []
        for t in range(3 * S):
            b, s = divmod(t, S)
            ids = so.window_positions(int(ctx[b]) - S + s, window, sinks)
            x = np.stack([hist[b][p] for p in ids])
            y = so.normalise(x[:, :512], _f64(gamma), 1e-6)
            rope = so.rotate(x[:, 512:], _f64(table)[ids], True)
            row = np.zeros((len(ids), FORMATS[fmt]), dtype=np.uint8)
            if fmt == "fp8":
                row[:, :512], sc = so.quantise_fp8(y)
                row[:, 512:528] = sc.view(np.uint8)
            else:
                code, row[:, 256:288] = so.quantise_fp4(y)
                row[:, :256] = code[:, 0::2] | (code[:, 1::2] << 4)
            row[:, -128:] = torch.from_numpy(rope).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint8)
            # a rope value next to a bf16 border may be one step (2^-7) off
            refs.append(so.attend(_f64(q)[t], row, SCALE, 2.0 ** -11 if fmt == "fp8" else 2.0 ** -14))
        _check(out, lse, refs, f"step {i}")
    assert _err() == 0


@pytest.mark.gpu
def test_captured_steps_replay_and_share_nothing(cuda_device):
    """Maps, write and decode captured into two graphs with their own
    workspaces, replayed in turn on changed lengths and rows."""
    dev = cuda_device
    ctx_h = [400, 80]
    T, H, bs = 2, 16, 16
    graphs = []
    for k in range(2):
        pools, tables = _paged(ctx_h, 1, bs, 1, "fp4", k, dev)
        st = dict(pool=pools[0], table=tables[0], ctx=_i32(ctx_h, dev), ql=_i32([1, 1], dev),
                  free=_i32([], dev), kv=torch.randn((T, 576), device=dev).to(torch.bfloat16), q=_q(T, H, dev, k))
        st["maps"] = capi.alloc_step_maps(2, T, dev)
        st["out"] = torch.empty((T, H, 512), dtype=torch.bfloat16, device=dev)
        st["lse"] = torch.empty((T, H), dtype=torch.float32, device=dev)
        st["ws"] = capi.alloc_window_decode_workspace(T, H, 512, 300, 4, 1, 1, -1, dev)

        def run(st=st):
            m = capi.dcp_step_maps(st["ctx"], st["ql"], st["free"], st["table"], T, 1, 0, bs, out=st["maps"])
            capi.mla_cache_write(st["kv"], m.slots, st["pool"])
            capi.dcp_window_mla_decode(st["q"], st["ctx"], 512, 1, 300, 4, [st["pool"]], [st["table"]], bs,
                                       SCALE, out=st["out"], lse=st["lse"], workspace=st["ws"])

        run()  # kernels' attributes are set outside the capture
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        graphs.append((graph, st, run))
    _err()
    for i in range(3):
        for k, (graph, st, run) in enumerate(graphs):
            st["ctx"].copy_(_i32([400 - 3 * i, 80 - i], dev))
            st["kv"].copy_(torch.randn((T, 576), device=dev).to(torch.bfloat16))
            graph.replay()
        torch.cuda.synchronize()
        for graph, st, run in graphs:
            out, lse = st["out"].clone(), st["lse"].clone()
            run()
            torch.cuda.synchronize()
            assert torch.equal(out, st["out"]) and torch.equal(lse, st["lse"])
    assert _err() == 0


@pytest.mark.gpu
def test_another_stream_with_nothing_passed(cuda_device):
    """Outputs and workspaces allocated by the call belong to its stream."""
    dev = cuda_device
    pools, tables = _paged([3000], 1, 16, 1, "fp4", 3, dev)
    q, ctx = _q(1, 64, dev), _i32([3000], dev)
    ref = capi.dcp_window_mla_decode(q, ctx, 3000, 1, 2500, 9, pools, tables, 16, SCALE)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        got = capi.dcp_window_mla_decode(q, ctx, 3000, 1, 2500, 9, pools, tables, 16, SCALE, stream=s)
        noise = torch.full((1 << 20,), 255, dtype=torch.uint8, device=dev)  # a reused block would show
        s.synchronize()
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
        del noise
