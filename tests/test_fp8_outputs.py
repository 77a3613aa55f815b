"""The 8-bit calls' outputs lie apart: layouts in which two entries would share
a place are refused before anything runs."""
import pytest
import torch

from sparse_mla_decode_dcp_gb300 import build as smla_build
from sparse_mla_decode_dcp_gb300 import capi

BAD, UNSUP, OK = capi.SMLA_ERR_INVALID_ARG, capi.SMLA_ERR_UNSUPPORTED, capi.SMLA_OK
FAKE = 0x10000  # aligned, never dereferenced
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    smla_build.build()
    return capi.load()


@pytest.mark.parametrize("kw", [
    dict(cr=0), dict(cr=299), dict(G=2, cb=0), dict(G=2, cb=300), dict(G=2, cb=299, cr=1000),
    dict(G=3, cb=400, cr=1000), dict(sr=0), dict(sc=0), dict(sr=2, sc=1), dict(sr=1, sc=4), dict(G=2, sb=0),
    dict(G=2, sb=14), dict(G=2, sb=1, sr=3, sc=2), dict(G=2 ** 31 - 1, M=2 ** 31 - 1, cb=2 ** 62, cr=2 ** 62),
])
def test_quantise_refuses_shared_places(lib, kw):
    """Five rows of 300 columns, three scales each."""
    a = dict(G=1, M=5, cb=10 ** 6, cr=300, sb=10 ** 6, sr=1, sc=5)
    a.update(kw)
    assert lib.smla_fp8_quantise(FAKE, 0, 300, a["G"], a["M"], 300, FAKE, a["cb"], a["cr"], FAKE, a["sb"], a["sr"],
                                 a["sc"], None) == BAD


@pytest.mark.parametrize("kw,status", [
    (dict(our=199), BAD), (dict(our=1), BAD), (dict(G=2, ob=1199), BAD), (dict(G=2, ob=199, our=1000), BAD),
    (dict(G=6, ob=200, our=1000), BAD), (dict(M=2 ** 31 - 1, N=2 ** 31 - 1), UNSUP),
])
def test_product_refuses_shared_places(lib, kw, status):
    """Six rows of 200 results."""
    d = dict(G=1, M=6, N=200, ob=0, our=200)
    d.update(kw)
    assert lib.smla_fp8_matmul(FAKE, 1024, 128, FAKE, 6, 1, 6, FAKE, 1024, 128, FAKE, 1, 1, 1, d["G"], d["M"], d["N"],
                               128, FAKE, d["ob"], d["our"], 0, None) == status


@pytest.mark.gpu
def test_expanded_outputs_are_refused(cuda_device):
    x = torch.randn((4, 256), device=cuda_device).bfloat16()
    codes, scales = torch.zeros((4, 256), device=cuda_device).to(E4M3), torch.zeros((4, 2), device=cuda_device)
    for out in ((codes[:1].expand(4, 256), scales), (codes, scales[:1].expand(4, 2)),
                (codes, scales[:, :1].expand(4, 2)), (codes.view(-1).as_strided((4, 256), (128, 1)), scales)):
        with pytest.raises(capi.SmlaError):
            capi.fp8_quantise(x, out=out)
    a = capi.fp8_quantise(x)
    with pytest.raises(capi.SmlaError):
        capi.fp8_matmul(a.codes, a.scales, codes, torch.ones((1, 2), device=cuda_device),
                        out=torch.zeros(16, device=cuda_device).as_strided((4, 4), (2, 1)))


@pytest.mark.gpu
@pytest.mark.parametrize("G,M", [(1, 1), (1, 5), (4, 1), (3, 5)])
def test_every_order_of_dimensions_is_taken(cuda_device, G, M):
    """Outputs whose dimensions lie in any order, one-entry ones with any stride."""
    x = torch.randn((G, M, 300), device=cuda_device).bfloat16()
    want = capi.fp8_quantise(x)
    for order in ((0, 1, 2), (0, 2, 1), (1, 0, 2), (1, 2, 0), (2, 0, 1), (2, 1, 0)):
        shape = [(G, M, 3)[i] for i in order]
        back = [order.index(i) for i in range(3)]
        scales = torch.zeros(shape, device=cuda_device).permute(back)
        wide = torch.zeros((G, M, 320) if order[0] != 1 else (M, G, 320), device=cuda_device).to(E4M3)
        codes = (wide if order[0] != 1 else wide.transpose(0, 1))[..., :300]
        got = capi.fp8_quantise(x, out=capi.Fp8Rows(codes, scales))
        assert torch.equal(got.codes.float(), want.codes.float()) and torch.equal(got.scales, want.scales)
