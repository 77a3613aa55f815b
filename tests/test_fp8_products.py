"""The projections in 8 bits: rows to e4m3 and the block-scaled product.
Refusals run without a GPU; codes and scales are compared bit by bit with
oracle/fp8_oracle.py, products within the tolerance derived there."""
import numpy as np
import pytest
import torch

from oracle import fp8_oracle as fo
from oracle.smla_oracle import E4M3_TABLE
from sparse_mla_decode_dcp_gb300 import build as smla_build
from sparse_mla_decode_dcp_gb300 import capi

BAD, UNSUP, WS, OK = (capi.SMLA_ERR_INVALID_ARG, capi.SMLA_ERR_UNSUPPORTED,
                      capi.SMLA_ERR_WORKSPACE, capi.SMLA_OK)
FAKE = 0x10000  # aligned, never dereferenced
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    smla_build.build()
    return capi.load()


def _np(t):
    return t.cpu().numpy()


def _codes(t):
    return _np(t.contiguous().view(torch.uint8))


def _err():
    return capi.get_device_error(clear=True)


# ------------------------------------------------------------------ oracle
def test_oracle_quantises_a_group_by_hand():
    x = np.zeros((1, 130))
    x[0, :6] = [448.0, -224.0, 17.0, 18.0, 19.0, 2.0 ** -10]  # 17 and 19 are halfway
    x[0, 129] = -896.0
    codes, scales = fo.quantise(x)
    assert scales.tolist() == [[1.0, 2.0]]
    assert E4M3_TABLE[codes[0, :6]].tolist() == [448.0, -224.0, 16.0, 18.0, 20.0, 0.0]
    assert E4M3_TABLE[codes[0, 129]] == -448.0


def test_oracle_rounds_as_the_cast_does():
    x = np.random.default_rng(0).standard_normal((4, 128))
    codes, scales = fo.quantise(x)
    q = torch.from_numpy((x / scales).astype(np.float32)).to(E4M3)
    assert np.array_equal(codes, q.view(torch.uint8).numpy())


# ---------------------------------------------------------------- refusals
@pytest.mark.parametrize("kw,status", [
    (dict(G=-1), BAD), (dict(M=-1), BAD), (dict(K=0), BAD), (dict(xr=-1), BAD), (dict(cr=-1), BAD),
    (dict(sc=-1), BAD), (dict(x=None), BAD), (dict(c=None), BAD), (dict(s=None), BAD),
    (dict(x=FAKE + 1), BAD), (dict(s=FAKE + 2), BAD), (dict(M=0, x=None, c=None, s=None), OK),
    (dict(G=0, x=None, c=None, s=None), OK),
])
def test_quantise_argument_checks(lib, kw, status):
    a = dict(x=FAKE, xb=0, xr=128, G=1, M=2, K=128, c=FAKE, cb=0, cr=128, s=FAKE, sb=0, sr=1, sc=2)
    a.update(kw)
    assert lib.smla_fp8_quantise(a["x"], a["xb"], a["xr"], a["G"], a["M"], a["K"], a["c"], a["cb"], a["cr"],
                                 a["s"], a["sb"], a["sr"], a["sc"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(G=-1), BAD), (dict(M=-1), BAD), (dict(N=-1), BAD), (dict(K=0), BAD), (dict(a=None), BAD),
    (dict(b=None), BAD), (dict(sa=None), BAD), (dict(sb=None), BAD), (dict(o=None), BAD),
    (dict(a=FAKE + 8), BAD), (dict(b=FAKE + 4), BAD), (dict(sa=FAKE + 2), BAD), (dict(o=FAKE + 1), BAD),
    (dict(o=FAKE + 2, f32=1), BAD), (dict(ar=120), BAD), (dict(br=136), BAD), (dict(ar=0), BAD),
    (dict(G=2, ab=8), BAD), (dict(G=2, bb=0), BAD), (dict(G=2, ob=0), BAD), (dict(our=0), BAD),
    (dict(sac=-1), BAD), (dict(ar=1 << 40), UNSUP), (dict(M=2 ** 31 - 1, N=2 ** 31 - 1), UNSUP),
    (dict(M=0, a=None), OK), (dict(N=0, b=None), OK), (dict(G=0, o=None), OK),
])
def test_matmul_argument_checks(lib, kw, status):
    d = dict(a=FAKE, ab=256, ar=128, sa=FAKE, sac=2, b=FAKE, bb=256, br=128, sb=FAKE, G=1, M=2, N=2, K=128,
             o=FAKE, ob=4, our=2, f32=0)
    d.update(kw)
    assert lib.smla_fp8_matmul(d["a"], d["ab"], d["ar"], d["sa"], 2, 1, d["sac"], d["b"], d["bb"], d["br"],
                               d["sb"], 1, 1, 1, d["G"], d["M"], d["N"], d["K"], d["o"], d["ob"], d["our"],
                               d["f32"], None) == status


def test_binding_refuses_what_it_cannot_pass(lib):
    z = torch.zeros
    x, c, s = z(2, 130, dtype=torch.bfloat16), z(2, 130).to(E4M3), z(2, 2)
    with pytest.raises(ValueError):  # host tensors never reach the library
        capi.fp8_quantise(x)
    with pytest.raises(ValueError):
        capi.fp8_quantise(z(4, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        capi.fp8_quantise(z(2, 130))
    with pytest.raises(ValueError):  # a scale for each 128 columns
        capi.fp8_quantise(x, out=(c, z(2, 1)))
    with pytest.raises(ValueError):
        capi.fp8_quantise(x.t(), out=(c, s))
    with pytest.raises(TypeError):
        capi.fp8_matmul(z(2, 128, dtype=torch.uint8), z(2, 1), z(4, 128).to(E4M3), z(1, 1))
    with pytest.raises(ValueError):  # other columns
        capi.fp8_matmul(z(2, 128).to(E4M3), z(2, 1), z(4, 256).to(E4M3), z(1, 2))
    with pytest.raises(ValueError):
        capi.fp8_matmul(z(2, 128).to(E4M3), z(2, 1), z(130, 128).to(E4M3), z(1, 1))
    with pytest.raises(ValueError):
        capi.fp8_matmul(z(2, 128).to(E4M3), z(2, 1), z(1, 4, 128).to(E4M3), z(1, 1))
    with pytest.raises(TypeError):
        capi.fp8_matmul(z(2, 128).to(E4M3), z(2, 1), z(4, 128).to(E4M3), z(1, 1),
                        out=z(2, 4, dtype=torch.float16))


# ---------------------------------------------------------------- quantise
def _check_quantised(x, got):
    codes, scales = fo.quantise(_np(x.double()))
    assert np.array_equal(_np(got.scales).view(np.uint32)[~np.isnan(scales)],
                          scales.view(np.uint32)[~np.isnan(scales)])
    assert np.array_equal(np.isnan(_np(got.scales)), np.isnan(scales))
    assert np.array_equal(_codes(got.codes), codes)


@pytest.mark.gpu
@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (2, 127), (5, 128), (4, 129), (33, 576), (1, 16384), (300, 200)])
def test_quantise_matches_the_definition(cuda_device, M, K):
    g = torch.Generator().manual_seed(M + K)
    x = (torch.randn((M, K), generator=g) * torch.exp(4 * torch.randn((M, 1), generator=g))).bfloat16()
    _check_quantised(x, capi.fp8_quantise(x.to(cuda_device)))


@pytest.mark.gpu
def test_quantise_next_to_the_halves(cuda_device):
    """Every bf16 mantissa against maxima of every mantissa: quotients on, just
    above and just below the halfway points, at scales from tiny to huge."""
    top = (1 + torch.arange(128) / 128)[:, None]
    x = torch.cat([top.expand(128, 1), torch.arange(1, 128).expand(128, 127) * top.new_tensor(1 / 128)], 1)
    low = x.clone()
    low[:, 1:] *= 2.0 ** -9  # e4m3's small numbers
    rows = torch.cat([x, -x, low])
    for e in (-126, -117, -100, -60, 0, 3, 100, 126):
        v = (rows.double() * 2.0 ** e).bfloat16()
        _check_quantised(v, capi.fp8_quantise(v.to(cuda_device)))


@pytest.mark.gpu
def test_quantise_odd_groups(cuda_device):
    x = torch.randn((9, 256), generator=torch.Generator().manual_seed(1)).bfloat16()
    x[0] = 0
    x[1] = -0.0
    x[2, 3] = float("inf")
    x[3, 200] = float("nan")
    x[4] = 2.0 ** -133       # bf16's smallest: a scale below 2^-126
    x[5, :128] = 2.0 ** -120
    x[6] = 3.38e38
    x[7, 130] = -float("inf")
    x[8, 7] = 1e30           # the rest of its group is nothing beside it
    got = capi.fp8_quantise(x.to(cuda_device))
    _check_quantised(x, got)
    assert _np(got.scales)[0].tolist() == [0, 0]


@pytest.mark.gpu
@pytest.mark.parametrize("offset", [0, 1, 4, 8])
def test_quantise_strided_batches(cuda_device, offset):
    """A head's part of wider rows, at any alignment, into any layout; what
    lies around it stays."""
    G, M, K = 3, 5, 200
    g = torch.Generator().manual_seed(offset)
    wide = torch.randn((M, G, 300), generator=g).bfloat16().to(cuda_device)
    x = wide[:, :, offset:offset + K].transpose(0, 1)
    buf = torch.full((M, G, 256), 3.0, device=cuda_device).to(E4M3)
    codes = buf[:, :, offset:offset + K].transpose(0, 1)
    scales = torch.full((G, M, 4), 5.0, device=cuda_device)
    got = capi.fp8_quantise(x, out=capi.Fp8Rows(codes, scales[:, :, :2]))
    for i in range(G):
        _check_quantised(x[i], capi.Fp8Rows(got.codes[i], got.scales[i]))
    rest = torch.ones_like(buf.view(torch.uint8), dtype=torch.bool)
    rest[:, :, offset:offset + K] = False
    assert torch.all(buf.float()[rest] == 3.0) and torch.all(scales[:, :, 2:] == 5.0)


# ----------------------------------------------------------------- product
def _operand(shape, seed, block_rows, dev):
    """Codes of all sizes and scales over three decades."""
    g = torch.Generator().manual_seed(seed)
    *batch, R, K = shape
    codes = (torch.randn((*batch, R, K), generator=g) * 60).clamp(-448, 448).to(E4M3)
    s = torch.exp(torch.empty((*batch, -(-R // block_rows), -(-K // 128))).uniform_(-4, 3, generator=g))
    buf = torch.zeros((*batch, R, -(-K // 16) * 16)).to(E4M3).to(dev)
    buf[..., :K] = codes.to(dev)
    return buf[..., :K], s.to(dev)


def _check_product(got, a, sa, b, sb):
    dims = a.dim()
    for g in range(a.shape[0] if dims == 3 else 1):
        pick = (lambda t: t[g]) if dims == 3 else (lambda t: t)  # noqa: E731
        want, tol = fo.matmul(_codes(pick(a)), _np(pick(sa)), _codes(pick(b)), _np(pick(sb)), HALF[got.dtype])
        err = np.abs(_np(pick(got).double()) - want)
        assert np.all(err <= tol), (float((err / tol).max()), np.argwhere(err > tol)[:5].tolist())


SIZES = [(1, 1, 1), (1, 1, 16), (1, 576, 2048), (2, 5, 127), (3, 200, 130), (16, 129, 128), (17, 128, 1000),
         (33, 300, 272), (64, 257, 640), (65, 128, 384), (128, 130, 129), (130, 64, 16), (200, 300, 2176),
         (257, 513, 1152), (5, 40, 16384), (64, 128, 8192), (100, 128, 4112),
         (20, 45000, 130), (50, 40001, 300),                             # columns' tiles in turn
         (300, 4990, 400), (1100, 2049, 144), (259, 9000, 1300), (2000, 3000, 48)]  # pairs' tiles


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product_matches_the_definition(cuda_device, M, N, K):
    a, sa = _operand((M, K), M + K, 1, cuda_device)
    b, sb = _operand((N, K), N + K, 128, cuda_device)
    _err()
    got = capi.fp8_matmul(a, sa, b, sb)
    _check_product(got, a, sa, b, sb)
    assert torch.equal(got, capi.fp8_matmul(a, sa, b, sb))  # the same bits again
    _check_product(capi.fp8_matmul(a, sa, b, sb, dtype=torch.float32), a, sa, b, sb)
    assert _err() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("G,M,N,K", [(3, 1, 512, 128), (5, 64, 128, 512), (128, 2, 16, 128), (2, 100, 300, 400),
                                     (7, 129, 33, 48), (2, 20, 60, 4096),
                                     (40, 130, 33, 176), (20, 300, 260, 272)])
def test_batches_in_and_out_of_interleaved_rows(cuda_device, G, M, N, K):
    """A product for each head, from and into the heads' parts of wider rows."""
    a0, sa = _operand((M, G, K), G + M, 1, cuda_device)
    pad = -(-K // 16) * 16
    a = a0.transpose(0, 1)
    sa = sa.transpose(0, 1)
    b, sb = _operand((G, N, K), G + N, 128, cuda_device)
    assert a.stride(0) == pad
    for dtype in (torch.bfloat16, torch.float32):
        wide = torch.full((M, G, N + 9), 7.0, dtype=dtype, device=cuda_device)
        out = wide[:, :, 4:4 + N].transpose(0, 1)
        got = capi.fp8_matmul(a, sa, b, sb, out=out)
        assert got is out
        _check_product(got, a, sa, b, sb)
        assert torch.all(wide[:, :, :4] == 7) and torch.all(wide[:, :, 4 + N:] == 7)


@pytest.mark.gpu
@pytest.mark.parametrize("G,M,N,K", [(1, 1500, 3300, 400), (1, 300, 7168, 272), (1, 257, 8400, 300),
                                     (9, 513, 500, 144), (5, 300, 1000, 1040)])
def test_each_width_of_the_pairs_tiles(cuda_device, G, M, N, K):
    """Tiles of 160, 192, 224 and 256 columns, whose weight scales change at
    other columns than they end; rows and columns past the end untouched."""
    shape = lambda *s: s if G > 1 else s[1:]  # noqa: E731
    a, sa = _operand(shape(G, M, K), M + K, 1, cuda_device)
    b, sb = _operand(shape(G, N, K), N + K, 128, cuda_device)
    wide = torch.full(shape(G, M + 1, N + 16), 7.0, dtype=torch.bfloat16, device=cuda_device)
    got = capi.fp8_matmul(a, sa, b, sb, out=wide[..., :M, :N])
    _check_product(got, a, sa, b, sb)
    assert torch.all(wide[..., M:, :] == 7) and torch.all(wide[..., N:] == 7)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [3, 40, 150])
def test_whole_numbers_come_out_exactly(cuda_device, M):
    """Sums of whole numbers below 2^24 are exact in fp32, so any lost bit of
    an accumulation or a misplaced element shows."""
    N, K = 200, 1024
    g = torch.Generator().manual_seed(M)
    a = torch.randint(-15, 16, (M, K), generator=g).float().to(E4M3)
    b = torch.randint(-15, 16, (N, K), generator=g).float().to(E4M3)
    sa, sb = torch.full((M, 8), 2.0), torch.full((2, 8), 0.5)
    want = a.double() @ b.double().T
    got = capi.fp8_matmul(*(t.to(cuda_device) for t in (a, sa, b, sb)), dtype=torch.float32)
    assert torch.equal(got.cpu().double(), want)


@pytest.mark.gpu
def test_shared_scales_and_row_major_ones(cuda_device):
    M, N, K = 70, 140, 300
    a, sa = _operand((M, K), 1, 1, cuda_device)
    b, sb = _operand((N, K), 2, 128, cuda_device)
    one = torch.full((1, 1), 0.25, device=cuda_device)
    _check_product(capi.fp8_matmul(a, one.expand(M, 3), b, one.expand(2, 3)), a, one.expand(M, 3), b,
                   one.expand(2, 3))
    cols = sa.t().contiguous().t()
    assert torch.equal(capi.fp8_matmul(a, sa, b, sb), capi.fp8_matmul(a, cols, b, sb))


@pytest.mark.gpu
@pytest.mark.parametrize("M", [4, 100])
def test_a_bad_row_stays_by_itself(cuda_device, M):
    N, K = 150, 400
    a, sa = _operand((M, K), 3, 1, cuda_device)
    b, sb = _operand((N, K), 4, 128, cuda_device)
    clean = capi.fp8_matmul(a, sa, b, sb)
    a.view(torch.uint8)[2, 5] = 0x7f  # e4m3's NaN
    sa[3, 1] = float("nan")
    got = capi.fp8_matmul(a, sa, b, sb)
    assert got[2:4].isnan().all()
    keep = [i for i in range(M) if i not in (2, 3)]
    assert torch.equal(got[keep], clean[keep])


@pytest.mark.gpu
@pytest.mark.parametrize("M", [2, 129])
def test_weights_past_two_gib(cuda_device, M):
    N, K = 280000, 8192
    a, sa = _operand((M, K), 5, 1, cuda_device)
    b = torch.zeros((N, K), dtype=torch.uint8, device=cuda_device)
    b[::4096] = 0x38  # 1.0
    b[N - 1] = 0x40   # 2.0
    sb = torch.ones((-(-N // 128), K // 128), device=cuda_device)
    got = capi.fp8_matmul(a, sa, b.view(E4M3), sb)
    rows = torch.tensor([0, 4096, 4097, 266240, 270336, N - 2, N - 1])
    small = torch.zeros((len(rows), K), dtype=torch.uint8)
    small[:] = b[rows.to(cuda_device)].cpu()
    want, tol = fo.matmul(_codes(a), _np(sa), small.numpy(), np.ones((1, K // 128)), HALF[torch.bfloat16])
    assert np.all(np.abs(_np(got[:, rows.to(cuda_device)].double()) - want) <= tol)
    assert got[:, 1:4096].eq(0).all()


@pytest.mark.gpu
def test_empty_calls(cuda_device):
    e = lambda *s: torch.zeros(s, device=cuda_device)  # noqa: E731
    assert capi.fp8_quantise(e(0, 128).bfloat16()).codes.shape == (0, 128)
    assert capi.fp8_matmul(e(0, 128).to(E4M3), e(0, 1), e(3, 128).to(E4M3), e(1, 1)).shape == (0, 3)
    assert capi.fp8_matmul(e(3, 128).to(E4M3), e(3, 1), e(0, 128).to(E4M3), e(0, 1)).shape == (3, 0)


@pytest.mark.gpu
def test_quantise_and_product_on_a_stream_and_in_a_graph(cuda_device):
    """A projection as a step runs it: quantise, multiply, quantise again,
    multiply; on a stream of its own, replayed on new inputs."""
    M, N, K = 24, 512, 384
    w1, s1 = _operand((N, K), 6, 128, cuda_device)
    w2, s2 = _operand((200, N), 7, 128, cuda_device)
    xs = [(torch.randn((M, K), generator=torch.Generator().manual_seed(i))).bfloat16().to(cuda_device)
          for i in range(2)]
    x = xs[0].clone()
    stream = torch.cuda.Stream(cuda_device)
    torch.cuda.synchronize()

    def step():
        r = capi.fp8_quantise(x, stream=stream)
        h = capi.fp8_matmul(r.codes, r.scales, w1, s1, stream=stream)
        r2 = capi.fp8_quantise(h, stream=stream)
        return r, h, r2, capi.fp8_matmul(r2.codes, r2.scales, w2, s2, stream=stream)

    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        r, h, r2, y = step()
    for v in xs:
        x.copy_(v)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        _check_quantised(v.cpu(), r)
        _check_product(h, r.codes, r.scales, w1, s1)
        _check_quantised(h.cpu(), r2)
        _check_product(y, r2.codes, r2.scales, w2, s2)
    assert _err() == 0
