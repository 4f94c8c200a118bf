"""int8 rows without columns."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def ox():
    import conv_implicit_gemm_amd as ox
    return ox


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N", [(3, 5), (40, 300), (700, 600)])
@pytest.mark.parametrize("scale", [float("nan"), float("inf"), 1.0])
def test_without_k_no_scale_is_read(ox, scale, M, N, out):
    A, B = torch.empty((M, 0), dtype=torch.int8, device="cuda"), torch.empty((N, 0), dtype=torch.int8, device="cuda")
    b = (torch.arange(N, device="cuda") % 9 - 4).to(out)
    sa, sb = torch.full((M,), scale, device="cuda"), torch.full((N,), scale, device="cuda")
    for bias, want in ((b, b.clamp(min=0)), (None, torch.zeros_like(b))):
        Y = ox.ox_gemm_i8(A, sa, B, sb, bias=bias, act="relu" if bias is not None else "none", out_dtype=out)
        assert torch.equal(Y, want.expand(M, N))
