"""Whose memory the binding hands to a launch on a stream that is not torch's
current one (no GPU needed: torch's allocator and the library are stand-ins).

torch's allocator keeps memory by the stream it was asked for under: what is
given back serves the next tensor of that stream, whose work comes behind, and
may still be in use by kernels of any other stream.  So what a call makes for a
launch has to be of the launch's stream."""
import contextlib
import ctypes
import importlib.util
import itertools
import types

import pytest

torch = pytest.importorskip("torch")

CURRENT = 5          # the current stream's handle


class Tensor:
    """A dense tensor on GPU 0 that remembers the stream it was made under."""
    places = itertools.count(1 << 20, 1 << 20)

    def __init__(self, shape, dtype, stream=CURRENT):
        self.shape, self.dtype, self.stream = torch.Size(shape), dtype, stream
        self.device, self.place, self.recorded = torch.device("cuda", 0), next(self.places), []

    def data_ptr(self):
        return self.place

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()

    def record_stream(self, stream):
        self.recorded.append(stream.cuda_stream)


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Torch:
    """torch with an allocator of stand-ins and a current stream of its own."""

    def __init__(self):
        self.now, self.made = [CURRENT], []

        def external(handle, device=None):
            assert handle != 0, "torch takes a stream of its pool for handle 0"
            return Stream(handle)

        @contextlib.contextmanager
        def under(stream):
            self.now.append(stream.cuda_stream)
            yield
            self.now.pop()

        self.cuda = types.SimpleNamespace(Stream=Stream, ExternalStream=external, stream=under,
                                          default_stream=lambda device=None: Stream(0),
                                          current_stream=lambda device=None: Stream(self.now[-1]))

    def empty(self, *shape, dtype=None, device=None):
        shape = shape[0] if len(shape) == 1 and not isinstance(shape[0], int) else shape
        self.made.append(Tensor(shape, dtype or torch.float32, self.now[-1]))
        return self.made[-1]

    def __getattr__(self, name):
        return getattr(torch, name)


@pytest.fixture
def ox():
    """A copy of the binding over a library that only takes down its arguments."""
    import conv_implicit_gemm_amd as real
    spec = importlib.util.spec_from_file_location("conv_implicit_gemm_amd_streams", real.__file__)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    fake = Torch()
    mod._types()
    mod._F8 = mod._F8[:4] + (lambda device: fake.now[-1],)
    mod._current_device = lambda: 0
    mod._torch = lambda: fake
    mod.fake, mod.calls, library = fake, [], mod.lib

    class Library:
        def __getattr__(self, name):
            if name.endswith("_bytes"):
                return getattr(library, name)

            def call(*args):
                mod.calls.append((name, args))
                return 0
            return call
    mod.lib = Library()
    return mod


def made_of(ox, place):
    """The stand-in at an address that the library was given."""
    found = [t for t in ox.fake.made if t.place == place]
    assert len(found) == 1
    return found[0]


STREAMS = [(None, CURRENT), (7, 7), (Stream(7), 7), (0, 0), (Stream(0), 0), (CURRENT, CURRENT), (Stream(CURRENT), CURRENT),
           (ctypes.c_void_p(7), 7), (ctypes.c_void_p(0), 0), (ctypes.c_void_p(CURRENT), CURRENT)]
IDS = ["none", "handle", "object", "default-handle", "default-object", "current-handle", "current-object", "pointer",
       "default-pointer", "current-pointer"]


def handle_of(at):
    """The handle that the library was given, as a number."""
    return (at.value or 0) if isinstance(at, ctypes.c_void_p) else at


@pytest.mark.parametrize("stream,launched", STREAMS, ids=IDS)
def test_scratch_of_the_routed_layer(ox, stream, launched):
    T, D, H, E, top = 4, 64, 96, 8, 2
    bf = torch.bfloat16
    ox.ox_moe_few(Tensor((T, D), bf), Tensor((T, E), torch.float32), Tensor((E, 2 * H, D), bf), Tensor((E, D, H), bf), top,
                  Y=Tensor((T, D), bf), stream=stream)
    (name, args), = ox.calls
    assert name == "ox_moe_few" and handle_of(args[-1]) == launched
    scratch = made_of(ox, args[-3])
    assert scratch.numel() == args[-2] == ox.ox_moe_few_workspace_bytes(T, D, H, E, top)
    assert scratch.stream == launched


@pytest.mark.parametrize("stream,launched", STREAMS, ids=IDS)
def test_scratch_of_the_dynamic_quantisation(ox, stream, launched):
    u8, f32 = torch.uint8, torch.float32
    ox.ox_dynamic_quantize_linear(Tensor((9, 100), f32), Tensor((9, 100), u8), Tensor((1,), f32), Tensor((1,), u8), stream=stream)
    (name, args), = ox.calls
    assert name == "ox_dynamic_quantize_linear" and handle_of(args[-1]) == launched
    scratch = made_of(ox, args[-3])
    assert scratch.numel() == args[-2] == ox.lib.ox_dynamic_quantize_workspace_bytes()
    assert scratch.stream == launched


def calls(ox, stream):
    """One call of every entry point that makes its results."""
    f32, bf, i8, u8, i32, f8 = torch.float32, torch.bfloat16, torch.int8, torch.uint8, torch.int32, torch.float8_e4m3fn
    T, kw = Tensor, dict(stream=stream)
    X4, W4 = T((2, 8, 6, 6), bf), T((16, 8, 3, 3), bf)
    c = [T((8,), f32) for _ in range(4)]
    A8, B8, kb = T((4, 256), f8), T((64, 256), f8), T((2, 4), f32)
    Ai, Bi, si, sb = T((4, 256), i8), T((64, 256), i8), T((4,), f32), T((64,), f32)
    return {
        "matmul_batched": lambda: ox.ox_matmul_batched(T((2, 4, 8), f32), T((8, 6), f32), **kw),
        "gemm_fused": lambda: ox.ox_gemm_fused(T((4, 8), f32), T((8, 6), f32), **kw),
        "gemm_fused_i8": lambda: ox.ox_gemm_fused(T((4, 8), i8), T((6, 8), i8), transB=True, **kw),
        "gemm_fused_ws": lambda: ox.ox_gemm_fused_ws(T((4, 8), f32), T((8, 6), f32), None, **kw),
        "conv2d_fused": lambda: ox.ox_conv2d_fused(X4, W4, **kw),
        "conv2d_fused_res": lambda: ox.ox_conv2d_fused_res(X4, W4, T((2, 16, 4, 4), bf), **kw),
        "conv2d_fused_packed": lambda: ox.ox_conv2d_fused_packed(X4, T((16 * 8 * 9,), bf), **kw),
        "conv2d_int8": lambda: ox.ox_conv2d_int8(T((2, 8, 6, 6), i8), T((16, 8, 3, 3), i8), T((64,), u8), **kw),
        "matmul_nbits": lambda: ox.ox_matmul_nbits(T((4, 64), bf), T((6, 2, 16), u8), T((6, 2), f32), 64, **kw),
        "dynamic_quantize_linear": lambda: ox.ox_dynamic_quantize_linear(T((9, 10), f32), workspace=T((8192,), u8), **kw),
        "batchnorm_act": lambda: ox.ox_batchnorm_act(X4, *c, **kw),
        "maxpool2d": lambda: ox.ox_maxpool2d(X4, (2, 2), **kw),
        "global_avgpool": lambda: ox.ox_global_avgpool(X4, **kw),
        "quantize_fp8": lambda: ox.ox_quantize_fp8(T((4, 256), bf), **kw),
        "gemm_fp8": lambda: ox.ox_gemm_fp8(A8, kb, B8, T((1, 2), f32), **kw),
        "gemm_grouped": lambda: ox.ox_gemm_grouped(T((4, 8), bf), T((3, 6, 8), bf), T((4,), i32), **kw),
        "gemm_grouped_fp8": lambda: ox.ox_gemm_grouped_fp8(A8, kb, T((3, 64, 256), f8), T((3, 1, 2), f32), T((4,), i32), **kw),
        "quantize_i8": lambda: ox.ox_quantize_i8(T((4, 256), bf), **kw),
        "gemm_i8": lambda: ox.ox_gemm_i8(Ai, si, Bi, sb, **kw),
        "rmsnorm": lambda: ox.ox_rmsnorm(T((4, 256), bf), residual=T((4, 256), bf), out="fp8", **kw),
        "moe_few": lambda: ox.ox_moe_few(T((4, 64), bf), T((4, 8), f32), T((8, 192, 64), bf), T((8, 64, 96), bf), 2,
                                         workspace=T((1 << 22,), u8), **kw),
    }


@pytest.mark.parametrize("stream,launched", STREAMS, ids=IDS)
def test_results(ox, stream, launched):
    """A result is of the launch's stream, so that nothing else still uses its
    memory, and known to be used by the caller's stream too, so that nothing
    gets it while that one still reads."""
    makes = {"dynamic_quantize_linear": 3, "quantize_fp8": 2, "quantize_i8": 2, "rmsnorm": 3}
    for name, call in calls(ox, stream).items():
        ox.calls.clear()
        ox.fake.made.clear()
        call()
        (entry, args), = ox.calls
        assert entry.startswith("ox_" + name.replace("_i8", "")) and handle_of(args[-1]) == launched, name
        assert len(ox.fake.made) == makes.get(name, 1), name
        for t in ox.fake.made:
            assert t.place in args and t.stream == launched, name
            assert t.recorded == ([] if launched == CURRENT else [CURRENT]), name


FLAT = ["quantize_fp8", "gemm_fp8", "gemm_grouped", "gemm_grouped_fp8", "quantize_i8", "gemm_i8", "rmsnorm", "moe_few"]


@pytest.mark.parametrize("current", [0, 1])
@pytest.mark.parametrize("stream", [None, 9, 0])
@pytest.mark.parametrize("name", FLAT)
def test_tensors_on_another_gpu_than_the_current_one(ox, name, stream, current, monkeypatch):
    """The calls that take tensors of any GPU launch with that GPU as the current
    one: the default stream's handle, 0, names the current GPU's."""
    at, of = [current], 1 - current

    @contextlib.contextmanager
    def device(index):
        at.append(getattr(index, "index", index))
        yield
        at.pop()
    monkeypatch.setattr(Tensor, "get_device", lambda t: of)
    ox.fake.cuda.device = device
    ox._current_device = lambda: at[-1]
    seen = []

    class Library:
        def __getattr__(self, entry):
            def call(*args):
                seen.append((entry, at[-1]))
                return 0
            return call if not entry.endswith("_bytes") else lambda *args: 64
    ox.lib = Library()
    calls(ox, stream)[name]()
    assert seen == [("ox_" + name, of)] and at == [current]


def test_host_tensors_are_refused_whatever_the_stream():
    import conv_implicit_gemm_amd as real
    X, s, W1, W2 = torch.zeros(4, 64), torch.zeros(4, 8), torch.zeros(8, 192, 64), torch.zeros(8, 64, 96)
    for stream in (None, 0, 7):
        for call in (lambda: real.ox_moe_few(X, s, W1, W2, 2, stream=stream), lambda: real.ox_rmsnorm(X, out="i8", stream=stream),
                     lambda: real.ox_quantize_i8(X, stream=stream)):
            with pytest.raises(ValueError, match="GPU"):
                call()
