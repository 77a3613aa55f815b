"""Tree attention at the edges of what its queries, calls and buffers may be."""
import itertools

import numpy as np
import pytest
import torch

from oracle import step_oracle as so
from oracle.smla_oracle import bf16_bits_to_f64
from sparse_mla_decode_dcp_gb300 import build as smla_build
from sparse_mla_decode_dcp_gb300 import capi
from sparse_mla_decode_dcp_gb300.pipeline import DcpServingStep
from test_tree_decode import FORMATS, SCALE, Case, _err


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("at", [0, 511, 512, 575])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
def test_a_query_that_is_not_finite_is_reported(cuda_device, fmt, at, value):
    """Wherever in the row it is; the other rows are as they were."""
    c = Case(cuda_device, fmt, nodes=[5, 2], ctx=[70, 9], H=16, bs=16, seed=7).upload()
    clean = c.run()
    assert _err() == 0
    c.q[2, 5, at] = value
    c.upload()
    out, lse = c.run()
    assert _err() == capi.DEVERR_RANGE
    assert not lse[2, 5].isfinite() and not out[2, 5].isfinite().any()
    keep = torch.ones(c.T, c.H, dtype=torch.bool)
    keep[2, 5] = False
    assert torch.equal(out[keep], clean[0][keep]) and torch.equal(lse[keep], clean[1][keep])


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("low", [-60, -100, -113, -120, -126])
def test_tiny_latents_beside_an_ordinary_rope_part(cuda_device, fmt, low):
    """Finite scores whatever the sizes of the two parts are."""
    c = Case(cuda_device, fmt, nodes=[5], ctx=[70], H=16, bs=16, seed=7)
    c.q[:, ::2, :512] *= 2.0 ** low
    c.q[:, ::3, 512:] *= 300
    c.upload()
    out, lse = c.run()
    assert _err() == 0
    c.check(out, lse)


@pytest.mark.gpu
def test_latents_of_all_sizes(cuda_device):
    """8-bit rows: nodes whose latents are from 2^-126 to 2^16 of ordinary ones."""
    c = Case(cuda_device, "fp8", nodes=[72], ctx=[70], H=16, bs=16, seed=8, max_nodes=72)
    by = torch.exp2(torch.arange(-126, 18, 2).double())[:, None, None]
    c.q[..., :512] = (c.q[..., :512].double() * by).bfloat16()
    c.upload()
    out, lse = c.run()
    assert _err() == 0
    assert out.isfinite().all() and lse.isfinite().all()
    c.check(out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("ctx", [70, 900])
@pytest.mark.parametrize("fmt,low,high", [("fp8", 12, 100), ("fp4", 4, 12)])
def test_scores_past_the_exponentials_range(cuda_device, fmt, low, high, ctx):
    """Scores from some 2^13 to 2^100: the largest key alone counts, in whole
    tiles and in merged ranges."""
    c = Case(cuda_device, fmt, nodes=[8], ctx=[ctx], H=16, bs=16, seed=9)
    by = torch.exp2(torch.linspace(low, high, 8).floor().double())[:, None, None]
    c.q = (c.q.double() * by).bfloat16()
    if fmt == "fp4":  # groups' scales as large as they may be
        for pool in c.pools:
            pool[:, 256:288] = 0x70
    c.upload()
    out, lse = c.run()
    assert _err() == 0
    assert out.isfinite().all() and lse.isfinite().all()
    q = bf16_bits_to_f64(c.q.view(torch.int16).numpy().astype(np.uint16))
    checked = 0
    for j in range(8):
        lat, rope = so.parse(np.stack([c.pools[d][s] for d, s in c.keys(0, j, -1)]))
        s = SCALE * q[j] @ np.concatenate([lat, rope], axis=1).T
        size = SCALE * (np.abs(q[j]) @ np.abs(np.concatenate([lat, rope], axis=1)).T).max(axis=1)
        first, second = np.argmax(s, axis=1), np.sort(s, axis=1)[:, -2]
        tol = size * 2.0 ** -17  # 42 steps of 2^-23 of the products' sum, as so.attend has it, and the keys' rope in fp16
        assert np.all(np.abs(lse[j].cpu().double().numpy() - s.max(axis=1)) <= tol + np.log(ctx + 8))
        for h in range(16):
            if s[h].max() - second[h] > 2 * tol[h] + 20:  # another key's weight is below e^-20
                want = lat[first[h]]
                assert np.all(np.abs(out[j, h].cpu().double().numpy() - want) <= 2.0 ** -7 * np.abs(want) + 2.0 ** -12)
                checked += 1
    assert checked > 60


# --------------------------------------------------------------- workspaces
@pytest.mark.parametrize("H", [1, 16, 128])
@pytest.mark.parametrize("B", [1, 5, 32, 200])
@pytest.mark.parametrize("rank", [-1, 1])
def test_a_workspace_serves_every_smaller_call(H, B, rank):
    smla_build.build()
    size = capi.tree_decode_workspace_size
    rows, prefixes = [1, 2, 3, 8, 16, 17, 32, 64, 100, 256, 512, 3000], [0, 60, 130, 300, 400, 496, 600, 5000]
    got = {(T, p): size(T, H, B, p, 16, 4, 1, rank) for T, p in itertools.product(rows, prefixes)}
    for (T, p), n in got.items():
        for (T2, p2), m in got.items():
            assert T2 > T or p2 > p or m <= n, (T, p, T2, p2)
    assert all(size(64, H, b, 300, 16, 4, 1, rank) <= size(64, H, B, 300, 16, 4, 1, rank) for b in range(1, B + 1))
    assert all(size(64, h, B, 300, 16, 4, 1, rank) <= size(64, H, B, 300, 16, 4, 1, rank) for h in range(1, H + 1))
    assert all(size(64, H, B, 300, n, 4, 1, rank) <= size(64, H, B, 300, 16, 4, 1, rank) for n in range(1, 17))


@pytest.mark.gpu
@pytest.mark.parametrize("window", [150, 1000])
def test_steps_of_any_rows_allocate_nothing(cuda_device, window):
    """A server whose full steps are not cut into key ranges and whose small
    ones are."""
    dev, B, N, H = cuda_device, 32, 16, 128
    step = DcpServingStep(B, 1, H, 2, 16, 700, 300, window, 4, fmt="fp8", max_nodes=N, device=dev)
    ctx = torch.full((B,), 260, dtype=torch.int32, device=dev)
    g = torch.Generator(device=dev).manual_seed(1)
    step.prefill(ctx, ctx, torch.randn((260 * B, 576), generator=g, device=dev).bfloat16())
    step.take_blocks()
    for T in (512, 300, 64, 40, 32, 16, 3, 1):
        par = torch.full((T,), -1, dtype=torch.int32, device=dev)
        starts = torch.arange(B + 1, device=dev) * T // B
        rs, tok = starts.to(torch.int32), torch.zeros_like(par)
        kv = torch.randn((T, 576), generator=g, device=dev).bfloat16()
        q = torch.randn((T, H, 576), generator=g, device=dev).bfloat16()
        torch.cuda.synchronize()
        before = torch.cuda.memory_stats(dev)["allocation.all.allocated"]
        out, lse = step.verify(ctx, par, rs, kv, q)
        step.commit(ctx, par, tok, tok, rs)
        torch.cuda.synchronize()
        assert torch.cuda.memory_stats(dev)["allocation.all.allocated"] == before, T
        assert lse.isfinite().all() and _err() == 0
        step._taken = []  # the same lengths again


# -------------------------------------------------- the log-sums of 8-bit rows
def _bounds(q, raw):
    """One node's log-sums and their tolerance, as the header promises them over
    8-bit rows: exact products in fp32 sums (so.attend without a rounding of the
    keys), but latents of q below 2^-10 of the row's largest to within 2^-17 of
    it."""
    _, lse, _, tol = so.attend(q, raw, SCALE, 0.0)
    lat = np.abs(so.parse(raw)[0])
    top = np.abs(q[:, :512]).max(axis=1, keepdims=True)
    small = np.where(np.abs(q[:, :512]) < 2.0 ** -10 * top, 2.0 ** -17 * top, 0)
    return lse, tol + SCALE * (small @ lat.T).max(axis=1)


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [
    dict(nodes=[9, 3], ctx=[65, 700], H=16, D=2), dict(nodes=[16], ctx=[130], H=128), dict(nodes=[5], ctx=[0], H=37),
])
@pytest.mark.parametrize("what", ["plain", "sizes of rows", "small latents", "scales"])
def test_log_sums_are_as_good_as_fp32_sums(cuda_device, kw, what):
    c = Case(cuda_device, "fp8", bs=16, seed=len(what), **kw)
    g = torch.Generator().manual_seed(3)
    if what == "sizes of rows":
        c.q *= torch.exp2(torch.randint(-40, 7, (c.T, c.H, 1), generator=g)).bfloat16()
    elif what == "small latents":  # down to 2^-20 of the row's largest
        c.q[..., :512] *= torch.exp2(torch.randint(-20, 1, (c.T, c.H, 512), generator=g)).bfloat16()
    elif what == "scales":
        rng = np.random.default_rng(4)
        for pool in c.pools:
            by = np.exp2(rng.integers(-8, 4, (len(pool), 4))).astype("<f4")
            pool[:, 512:528] = (pool[:, 512:528].copy().view("<f4") * by).view(np.uint8)
    c.upload()
    _, got = c.run()
    assert _err() == 0
    q = bf16_bits_to_f64(c.q.view(torch.int16).numpy().astype(np.uint16))
    for b in range(c.B):
        for j in range(c.nodes[b]):
            t = c.starts[b] + j
            want, tol = _bounds(q[t], np.stack([c.pools[d][s] for d, s in c.keys(b, j, -1)]))
            err = np.abs(got[t].cpu().double().numpy() - want)
            assert np.all(err <= tol), (b, j, (err / tol).max())


def test_the_bounds_tell_rounded_keys_apart():
    """Keys rounded to fp16 would be outside them where a node sees few keys (over
    many their errors cancel, and the bounds' worst case does not)."""
    c = Case("cpu", "fp8", nodes=[5], ctx=[0], H=37, bs=16, seed=5)  # as one of the cases above
    q = bf16_bits_to_f64(c.q.view(torch.int16).numpy().astype(np.uint16))
    worst = 0
    for j in range(5):
        raw = np.stack([c.pools[d][s] for d, s in c.keys(0, j, -1)])
        want, tol = _bounds(q[j], raw)
        lat, rope = so.parse(raw)
        s = SCALE * q[j] @ np.concatenate([lat.astype(np.float16), rope], axis=1).astype(np.float64).T
        off = np.log(np.exp(s - s.max(axis=1, keepdims=True)).sum(axis=1)) + s.max(axis=1) - want
        worst = max(worst, (np.abs(off) / tol).max())
    assert worst > 2
