"""Calls on streams that are not torch's current one, with memory that the
binding makes: nothing is handed on while the launch still uses it."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

WAIT = 5_000_000          # clock ticks of the kernel that holds a stream back: milliseconds


@pytest.fixture(scope="module")
def ox():
    import conv_implicit_gemm_amd as ox
    return ox


def layer(T, E, D, H, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")
    return (normal(T, D).bfloat16(), normal(T, E), (normal(E, 2 * H, D) * D ** -0.5).bfloat16(),
            (normal(E, D, H) * H ** -0.5).bfloat16(), 2)


@pytest.mark.parametrize("handle", [False, True])
def test_routed_layers_on_two_streams_make_a_workspace_each(ox, handle):
    cases = [layer(48, 8, 512, 256, 1), layer(7, 16, 512, 256, 2)]
    want = [ox.ox_moe_few(*c) for c in cases]
    Y = [[torch.zeros_like(w) for _ in range(10)] for w in want]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for s in streams:
        with torch.cuda.stream(s):
            torch.cuda._sleep(WAIT)
    for i in range(10):
        for c, y, s in zip(cases, Y, streams):
            ox.ox_moe_few(*c, Y=y[i], stream=s.cuda_stream if handle else s)
    # the current stream's next tensors, over anything that was given back
    over = [torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(40)]
    torch.cuda.synchronize()
    for ys, w in zip(Y, want):
        assert all(torch.equal(y, w) for y in ys)
    assert all((o == 255).all().item() for o in over)


def test_the_default_stream_by_its_handle(ox):
    c = layer(5, 8, 256, 128, 3)
    want = ox.ox_moe_few(*c)
    side = torch.cuda.Stream()
    Y = torch.zeros_like(want)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        ox.ox_moe_few(*c, Y=Y, stream=torch.cuda.default_stream())
        ox.ox_moe_few(*c, Y=Y, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(Y, want)


def test_dynamic_quantisation_on_two_streams(ox):
    g = torch.Generator(device="cuda").manual_seed(4)
    X = [torch.randn((1 << 20,), generator=g, device="cuda") * k for k in (1.0, 30.0)]
    want = [ox.ox_dynamic_quantize_linear(x) for x in X]
    out = [[[torch.zeros_like(w) for w in ws] for _ in range(10)] for ws in want]
    streams = [torch.cuda.Stream() for _ in X]
    torch.cuda.synchronize()
    for s in streams:
        with torch.cuda.stream(s):
            torch.cuda._sleep(WAIT)
    for i in range(10):
        for x, o, s in zip(X, out, streams):
            ox.ox_dynamic_quantize_linear(x, *o[i], stream=s)
    over = [torch.full((1 << 14,), 255, dtype=torch.uint8, device="cuda") for _ in range(40)]
    torch.cuda.synchronize()
    for os_, ws in zip(out, want):
        for o in os_:
            assert all(torch.equal(a, b) for a, b in zip(o, ws))
    assert all((o == 255).all().item() for o in over)


def test_results_on_another_stream_are_of_memory_that_nothing_uses(ox):
    """Memory that the current stream gave back and still reads is not the next
    result's on another stream, and a result that is dropped at once is not the
    current stream's next tensor while the launch still writes it."""
    rows, K = 512, 2048
    g = torch.Generator(device="cuda").manual_seed(5)
    X, R = (torch.randn((rows, K), generator=g, device="cuda").bfloat16() for _ in range(2))
    want = ox.ox_rmsnorm(X, residual=R, out="i8")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(WAIT)
    given_back = [torch.full((rows, K), 3.0, device="cuda").bfloat16() for _ in range(8)]
    doubled = [2 * t for t in given_back]
    del given_back
    early = [ox.ox_rmsnorm(X, residual=R, out="i8", stream=side) for _ in range(4)]
    torch.cuda.synchronize()
    assert all((d == 6.0).all().item() for d in doubled)
    assert all(torch.equal(a, b) for e in early for a, b in zip(e, want))
    with torch.cuda.stream(side):
        torch.cuda._sleep(WAIT)
    for handle in (side, side.cuda_stream):
        ox.ox_rmsnorm(X, residual=R, out="i8", stream=handle)
    over = [torch.full((rows, K), 7.0, device="cuda").bfloat16() for _ in range(12)]
    torch.cuda.synchronize()
    assert all((o == 7.0).all().item() for o in over)
