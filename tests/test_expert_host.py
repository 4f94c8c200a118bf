"""Refusals of the e4m3 and expert-grouped products (no GPU needed): every bad
argument is named before anything reaches the HIP runtime, and empty problems
are accepted."""
import pytest

torch = pytest.importorskip("torch")

F32, BF16, I8 = 0, 1, 2
INVALID, SHAPE, UNSUPPORTED = 1, 2, 3
P = 1 << 20          # a pointer no call may follow


@pytest.fixture(scope="module")
def ox():
    import conv_implicit_gemm_amd as ox
    return ox


def quant(ox, **kw):
    a = dict(t=BF16, rows=4, K=256, X=P, R=4, index=None, br=1, Q=P, s=P)
    a.update(kw)
    return ox.lib.ox_quantize_fp8(a["t"], a["rows"], a["K"], a["X"], a["R"], a["index"], a["br"], a["Q"], a["s"], None)


def fp8(ox, **kw):
    a = dict(t=BF16, M=4, N=64, K=256, A=P, sa=P, B=P, sb=P, bias=None, act=0, Y=P)
    a.update(kw)
    return ox.lib.ox_gemm_fp8(a["t"], a["M"], a["N"], a["K"], a["A"], a["sa"], a["B"], a["sb"], a["bias"], a["act"],
                              a["Y"], None)


def grp(ox, **kw):
    a = dict(t=BF16, T=4, N=64, K=256, E=2, tB=1, A=P, B=P, off=P, bias=None, act=0, Y=P)
    a.update(kw)
    return ox.lib.ox_gemm_grouped(a["t"], a["T"], a["N"], a["K"], a["E"], a["tB"], a["A"], a["B"], a["off"],
                                  a["bias"], a["act"], a["Y"], None)


def grp8(ox, **kw):
    a = dict(t=BF16, T=4, N=64, K=256, E=2, A=P, sa=P, B=P, sb=P, off=P, bias=None, act=0, Y=P)
    a.update(kw)
    return ox.lib.ox_gemm_grouped_fp8(a["t"], a["T"], a["N"], a["K"], a["E"], a["A"], a["sa"], a["B"], a["sb"],
                                      a["off"], a["bias"], a["act"], a["Y"], None)


REFUSED = [
    (quant, dict(t=I8), UNSUPPORTED, "dtype"), (quant, dict(rows=-1, R=-1), SHAPE, "negative"),
    (quant, dict(K=-1), SHAPE, "negative"), (quant, dict(br=64), UNSUPPORTED, "block_rows"),
    (quant, dict(br=128, index=P), UNSUPPORTED, "index"), (quant, dict(R=5), SHAPE, "R=5"),
    (quant, dict(rows=1 << 16, R=1 << 16, K=1 << 15), UNSUPPORTED, "2^31"),
    (quant, dict(X=None), INVALID, "NULL"), (quant, dict(Q=None), INVALID, "NULL"),
    (quant, dict(s=None), INVALID, "NULL"), (quant, dict(X=P + 1), INVALID, "aligned"),
    (quant, dict(s=P + 2), INVALID, "aligned"), (quant, dict(index=P + 2), INVALID, "aligned"),
    (fp8, dict(t=I8), UNSUPPORTED, "dtype"), (fp8, dict(act=9), INVALID, "act"), (fp8, dict(M=-1), SHAPE, "negative"),
    (fp8, dict(N=-2), SHAPE, "negative"), (fp8, dict(K=-3), SHAPE, "negative"),
    (fp8, dict(M=1 << 16, K=1 << 15), UNSUPPORTED, "2^31"), (fp8, dict(A=None), INVALID, "NULL"),
    (fp8, dict(B=None), INVALID, "NULL"), (fp8, dict(sa=None), INVALID, "scales"), (fp8, dict(sb=None), INVALID, "scales"),
    (fp8, dict(Y=None), INVALID, "Y"), (fp8, dict(Y=P + 1), INVALID, "aligned"), (fp8, dict(sa=P + 1), INVALID, "aligned"),
    (fp8, dict(bias=P + 1), INVALID, "aligned"),
    (grp, dict(t=I8), UNSUPPORTED, "dtype"), (grp, dict(off=None), INVALID, "offsets"),
    (grp, dict(off=P + 2), INVALID, "aligned"), (grp, dict(E=0), SHAPE, "experts"), (grp, dict(E=-1), SHAPE, "negative"),
    (grp, dict(E=1 << 12, N=1 << 10, K=1 << 10), UNSUPPORTED, "2^31"), (grp, dict(A=P + 1), INVALID, "aligned"),
    (grp, dict(act=-1), INVALID, "act"), (grp, dict(Y=None), INVALID, "Y"),
    (grp8, dict(off=None), INVALID, "offsets"), (grp8, dict(sb=None), INVALID, "scales"),
    (grp8, dict(t=I8), UNSUPPORTED, "dtype"), (grp8, dict(T=-1), SHAPE, "negative"),
]


@pytest.mark.parametrize("case", REFUSED, ids=["%s-%s" % (c[0].__name__, "-".join(c[1])) for c in REFUSED])
def test_refusals_name_the_argument(ox, case):
    call, kw, status, word = case
    assert call(ox, **kw) == status
    assert word in ox.ox_last_error(), ox.ox_last_error()


@pytest.mark.parametrize("call,kw", [(quant, dict(rows=0, R=0, X=None)), (quant, dict(K=0, X=None, Q=None)),
                                     (fp8, dict(M=0, A=None, Y=None)), (fp8, dict(N=0, B=None, Y=None)),
                                     (grp, dict(T=0, E=0, off=None)), (grp8, dict(N=0, off=None))])
def test_empty_problems_enqueue_nothing(ox, call, kw):
    assert call(ox, **kw) == 0


def test_binding_checks_shapes_and_types(ox):
    f8 = torch.float8_e4m3fn
    A, B = torch.zeros(4, 256).to(f8), torch.zeros(64, 256).to(f8)
    sa, sb = torch.ones(2, 4), torch.ones(1, 2)
    with pytest.raises(ValueError):
        ox.ox_gemm_fp8(A, sa.t().contiguous(), B, sb)          # scales row first
    with pytest.raises(ValueError):
        ox.ox_gemm_fp8(A, sa, torch.zeros(64, 128).to(f8), sb)
    with pytest.raises(ValueError):
        ox.ox_gemm_fp8(A, sa, B, torch.ones(2, 2))
    with pytest.raises(TypeError):
        ox.ox_gemm_fp8(A.float(), sa, B, sb)
    with pytest.raises(TypeError):
        ox.ox_gemm_fp8(A, sa.double(), B, sb)
    with pytest.raises(TypeError):
        ox.ox_gemm_fp8(A, sa, B, sb, bias=torch.zeros(64))     # bias float32, Y bfloat16
    with pytest.raises(ValueError):
        ox.ox_gemm_fp8(A, sa, B, sb, Y=torch.zeros(4, 63, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        ox.ox_gemm_fp8(A.t().contiguous().t(), sa, B, sb)      # not dense
    X, W, off = torch.zeros(4, 32), torch.zeros(2, 8, 32), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        ox.ox_gemm_grouped(X, W, off[:2])
    with pytest.raises(TypeError):
        ox.ox_gemm_grouped(X, W, off.long())
    with pytest.raises(ValueError):
        ox.ox_gemm_grouped(X, W, off, transB=False)
    with pytest.raises(TypeError):
        ox.ox_gemm_grouped(X, W.bfloat16(), off)
    with pytest.raises(ValueError):
        ox.ox_gemm_grouped(X, W, off, bias=torch.zeros(8))
    with pytest.raises(TypeError):
        ox.ox_quantize_fp8(X, index=off.long())
    with pytest.raises(ValueError):
        ox.ox_quantize_fp8(X, scales=torch.zeros(4, 1))
    with pytest.raises(ValueError):
        ox.ox_quantize_fp8(X, block_rows=32)
    with pytest.raises(ValueError):
        ox.ox_quantize_fp8(X, index=off, block_rows=128)
    with pytest.raises(ValueError):
        ox.ox_quantize_fp8(X)                                  # host memory
    with pytest.raises(ValueError):
        ox.ox_gemm_grouped(X, W, off)
