"""The e4m3 and expert-grouped products at the ends of their ranges: offsets of
any content, infinite weights and scales, sizes next to 2^31 elements, exact
halfway points, and the precision that each result type keeps."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

F8 = torch.float8_e4m3fn


def say(*a):
    print("[case]", *a, flush=True)


@pytest.fixture(scope="module")
def ox():
    import conv_implicit_gemm_amd as ox
    return ox


def test_offsets_whose_tiles_leave_32_bits(ox):
    # 32768 experts' offsets that swing over all rows: 2^26 row tiles of 32 rows
    # times 32 column tiles.  Y is undefined, its neighbours are not written.
    E, T, N, K = 32768, 131072, 2048, 16
    say("wild offsets", E, T, N, K)
    A = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    B = torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, T] * (E // 2) + [0], dtype=torch.int32, device="cuda")
    whole = torch.full((T * N + 4096,), 77, dtype=torch.bfloat16, device="cuda")
    ox.ox_gemm_grouped(A, B, off, Y=whole[2048:2048 + T * N].view(T, N))
    torch.cuda.synchronize()
    assert (whole[:2048] == 77).all().item() and (whole[-2048:] == 77).all().item()
