"""Refusals of the RMS norm, the int8 quantisation of rows and the int8 product
(no GPU needed): every bad argument is named before anything reaches the HIP
runtime, and empty problems are accepted."""
import pytest

torch = pytest.importorskip("torch")

F32, BF16, I8, I32, F8 = 0, 1, 2, 3, 4
INVALID, SHAPE, UNSUPPORTED = 1, 2, 3
P = 1 << 20          # a pointer no call may follow


@pytest.fixture(scope="module")
def ox():
    import conv_implicit_gemm_amd as ox
    return ox


def quant(ox, **kw):
    a = dict(t=BF16, rows=4, K=256, X=P, Q=P, s=P)
    a.update(kw)
    return ox.lib.ox_quantize_i8(a["t"], a["rows"], a["K"], a["X"], a["Q"], a["s"], None)


def gemm(ox, **kw):
    a = dict(t=BF16, M=4, N=64, K=256, A=P, sa=P, B=P, sb=P, bias=None, act=0, Y=P)
    a.update(kw)
    return ox.lib.ox_gemm_i8(a["t"], a["M"], a["N"], a["K"], a["A"], a["sa"], a["B"], a["sb"], a["bias"], a["act"],
                             a["Y"], None)


def norm(ox, **kw):
    a = dict(t=BF16, rows=4, K=256, X=P, R=2 * P, g=P, eps=1e-6, S=3 * P, yt=F8, Y=4 * P, s=P)
    a.update(kw)
    return ox.lib.ox_rmsnorm(a["t"], a["rows"], a["K"], a["X"], a["R"], a["g"], a["eps"], a["S"], a["yt"], a["Y"],
                             a["s"], None)


REFUSED = [
    (quant, dict(t=I8), UNSUPPORTED, "dtype"), (quant, dict(rows=-1), SHAPE, "negative"), (quant, dict(K=-1), SHAPE, "negative"),
    (quant, dict(K=65537), UNSUPPORTED, "65536"), (quant, dict(rows=1 << 16, K=1 << 15), UNSUPPORTED, "2^31"),
    (quant, dict(X=None), INVALID, "NULL"), (quant, dict(Q=None), INVALID, "NULL"), (quant, dict(s=None), INVALID, "NULL"),
    (quant, dict(X=P + 1), INVALID, "aligned"), (quant, dict(s=P + 2), INVALID, "aligned"),
    (quant, dict(rows=(1 << 31) - 1, K=1), UNSUPPORTED, "launch"),
    (gemm, dict(t=I8), UNSUPPORTED, "dtype"), (gemm, dict(act=4), INVALID, "act"), (gemm, dict(M=-1), SHAPE, "negative"),
    (gemm, dict(N=-1), SHAPE, "negative"), (gemm, dict(K=-1), SHAPE, "negative"), (gemm, dict(K=1 << 17), UNSUPPORTED, "131071"),
    (gemm, dict(M=1 << 16, N=1 << 15), UNSUPPORTED, "2^31"), (gemm, dict(A=None), INVALID, "NULL"),
    (gemm, dict(B=None), INVALID, "NULL"), (gemm, dict(sa=None), INVALID, "scales"), (gemm, dict(sb=None), INVALID, "scales"),
    (gemm, dict(sa=None, K=0), INVALID, "scales"), (gemm, dict(Y=None), INVALID, "Y"), (gemm, dict(Y=P + 1), INVALID, "aligned"),
    (gemm, dict(sb=P + 1), INVALID, "aligned"), (gemm, dict(bias=P + 1), INVALID, "aligned"),
    (norm, dict(t=I8), UNSUPPORTED, "dtype"), (norm, dict(yt=I32), UNSUPPORTED, "y_type"), (norm, dict(yt=F32), UNSUPPORTED, "y_type"),
    (norm, dict(eps=0.0), INVALID, "eps"), (norm, dict(eps=float("nan")), INVALID, "eps"), (norm, dict(eps=float("inf")), INVALID, "eps"),
    (norm, dict(rows=-1), SHAPE, "negative"), (norm, dict(K=65537), UNSUPPORTED, "65536"),
    (norm, dict(rows=1 << 16, K=1 << 15), UNSUPPORTED, "2^31"), (norm, dict(X=None), INVALID, "NULL"),
    (norm, dict(Y=None), INVALID, "NULL"), (norm, dict(s=None), INVALID, "NULL"), (norm, dict(R=None), INVALID, "residual"),
    (norm, dict(S=4 * P), INVALID, "sum_out"), (norm, dict(X=P + 1), INVALID, "aligned"), (norm, dict(R=P + 1), INVALID, "aligned"),
    (norm, dict(g=P + 1), INVALID, "aligned"), (norm, dict(S=P + 1), INVALID, "aligned"), (norm, dict(s=P + 2), INVALID, "aligned"),
    (norm, dict(yt=BF16, Y=P + 1), INVALID, "aligned"),
]


@pytest.mark.parametrize("case", REFUSED, ids=["%s-%s" % (c[0].__name__, "-".join(c[1])) for c in REFUSED])
def test_refusals_name_the_argument(ox, case):
    call, kw, status, word = case
    assert call(ox, **kw) == status
    assert word in ox.ox_last_error(), ox.ox_last_error()


@pytest.mark.parametrize("call,kw", [(quant, dict(rows=0, X=None)), (quant, dict(K=0, Q=None)), (gemm, dict(M=0, A=None, Y=None)),
                                     (gemm, dict(N=0, B=None)), (norm, dict(rows=0, X=None)), (norm, dict(K=0, Y=None)),
                                     (quant, dict(rows=0, K=70000)), (norm, dict(rows=0, K=70000))])
def test_empty_problems_enqueue_nothing(ox, call, kw):
    assert call(ox, **kw) == 0


def test_binding_checks_shapes_and_types(ox):
    i8 = torch.int8
    A, B, sa, sb = torch.zeros(4, 256, dtype=i8), torch.zeros(64, 256, dtype=i8), torch.ones(4), torch.ones(64)
    X, g = torch.zeros(4, 256), torch.ones(256)
    bad = [
        (ValueError, lambda: ox.ox_gemm_i8(A, sb, B, sb)), (ValueError, lambda: ox.ox_gemm_i8(A, sa, B, sa)),
        (ValueError, lambda: ox.ox_gemm_i8(A, sa[:, None], B, sb)), (ValueError, lambda: ox.ox_gemm_i8(A, sa, B[:, :128], sb)),
        (TypeError, lambda: ox.ox_gemm_i8(A.float(), sa, B, sb)), (TypeError, lambda: ox.ox_gemm_i8(A, sa, B.view(torch.uint8), sb)),
        (TypeError, lambda: ox.ox_gemm_i8(A, sa.double(), B, sb)), (TypeError, lambda: ox.ox_gemm_i8(A, sa, B, sb, bias=torch.zeros(64))),
        (ValueError, lambda: ox.ox_gemm_i8(A, sa, B, sb, Y=torch.zeros(4, 63, dtype=torch.bfloat16))),
        (ValueError, lambda: ox.ox_gemm_i8(A, sa, B, sb)),                        # host memory
        (ValueError, lambda: ox.ox_quantize_i8(X, scales=torch.zeros(1, 4))), (TypeError, lambda: ox.ox_quantize_i8(X, Q=X)),
        (TypeError, lambda: ox.ox_quantize_i8(X, scales=torch.zeros(4).double())), (TypeError, lambda: ox.ox_quantize_i8(X.double())),
        (ValueError, lambda: ox.ox_quantize_i8(X, Q=A[:3])), (ValueError, lambda: ox.ox_quantize_i8(X)),
        (ValueError, lambda: ox.ox_rmsnorm(X, g, out="e4m3")), (ValueError, lambda: ox.ox_rmsnorm(X, g[:9])),
        (TypeError, lambda: ox.ox_rmsnorm(X, g.bfloat16())), (ValueError, lambda: ox.ox_rmsnorm(X, g, S=X)),
        (ValueError, lambda: ox.ox_rmsnorm(X, g, residual=X[:3])), (TypeError, lambda: ox.ox_rmsnorm(X, g, residual=X.bfloat16())),
        (TypeError, lambda: ox.ox_rmsnorm(X, g, residual=X, S=X.bfloat16())), (ValueError, lambda: ox.ox_rmsnorm(X, g, scales=sa)),
        (ValueError, lambda: ox.ox_rmsnorm(X, g, out="fp8", scales=torch.zeros(4, 2))), (TypeError, lambda: ox.ox_rmsnorm(X, g, out="i8", Y=X)),
        (ValueError, lambda: ox.ox_rmsnorm(X, g)),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()
