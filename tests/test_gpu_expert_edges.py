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


@pytest.mark.parametrize("K", [2 ** 31 - 1, 2 ** 31 - 16, 2 ** 31 - 500])
def test_quantize_a_row_next_to_the_limit(ox, K):
    # 128-wide blocks whose last one ends on, or a little before, 2^31 elements
    say("quantise one row of", K)
    tail = 640 + K % 128
    X = torch.zeros(1, K, dtype=torch.bfloat16, device="cuda")
    X[0, -tail:].normal_()
    whole = torch.full((K + 4096,), 77, dtype=torch.uint8, device="cuda")
    Q, S = ox.ox_quantize_fp8(X, Q=whole[2048:2048 + K].view(1, K))
    q, s = ox.ox_quantize_fp8(X[:, -tail:].contiguous())
    torch.cuda.synchronize()
    assert (whole[:2048] == 77).all().item() and (whole[-2048:] == 77).all().item()
    assert torch.equal(Q[:, -tail:], q.view(torch.uint8)) and torch.equal(S[-s.shape[0]:], s)
    assert not Q[:, :-tail].any().item()
