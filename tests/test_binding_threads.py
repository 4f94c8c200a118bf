"""The binding's tables of torch's types: threads that make their first calls
together, and a torch without the raw stream lookup (no GPU needed)."""
import importlib.util
import threading

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def fresh():
    """A copy of the binding that no call has been made of."""
    import conv_implicit_gemm_amd as ox
    spec = importlib.util.spec_from_file_location("conv_implicit_gemm_amd_fresh", ox.__file__)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("table", ["_types", "_dtype_code"])
def test_first_calls_of_threads(fresh, table):
    t = torch.zeros(1)
    call = fresh._types if table == "_types" else lambda: fresh._dtype_code(t)
    together = threading.Barrier(4, timeout=10)
    real = fresh._torch

    def torch_when_all_are_here():      # every thread is between its look at the table and making it
        together.wait()
        return real()
    fresh._torch = torch_when_all_are_here
    got = []
    threads = [threading.Thread(target=lambda: got.append(call())) for _ in range(4)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    fresh._torch = real
    assert len(got) == 4
    if table == "_types":
        for types in got + [call()]:
            f8, u8, f32, i32, raw = types
            assert (f8, u8, f32, i32) == (torch.float8_e4m3fn, torch.uint8, torch.float32, torch.int32)
    else:
        assert got == [fresh.OX_F32] * 4 and call() == fresh.OX_F32


def test_without_the_raw_stream_lookup(fresh, monkeypatch):
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    fresh._stream = lambda stream: 7 if stream is None else stream
    assert fresh._types()[4](0) == 7
