"""Refusals of the routed layer of a few tokens (no GPU needed): every bad
argument is named before anything reaches the HIP runtime, and empty problems
are accepted."""
import pytest

torch = pytest.importorskip("torch")

F32, BF16, I8, I32, F8 = 0, 1, 2, 3, 4
INVALID, SHAPE, UNSUPPORTED = 1, 2, 3
P = 1 << 20          # a pointer no call may follow


@pytest.fixture(scope="module")
def ox():
    import conv_implicit_gemm_amd as ox
    return ox


def moe(ox, **kw):
    a = dict(t=BF16, wt=BF16, T=4, D=64, H=96, E=8, top=2, X=P, st=F32, s=P, re=1, W1=P, s1=None, b1=None, act=4, gated=1,
             W2=P, s2=None, b2=None, ids=None, w=None, Y=P, ws=P, nb=1 << 40)
    a.update(kw)
    return ox.lib.ox_moe_few(a["t"], a["wt"], a["T"], a["D"], a["H"], a["E"], a["top"], a["X"], a["st"], a["s"], a["re"], a["W1"],
                             a["s1"], a["b1"], a["act"], a["gated"], a["W2"], a["s2"], a["b2"], a["ids"], a["w"], a["Y"], a["ws"],
                             a["nb"], None)


REFUSED = [
    (dict(t=I8), UNSUPPORTED, "dtype"), (dict(wt=F32), UNSUPPORTED, "w_type"), (dict(t=F32, wt=F8), UNSUPPORTED, "w_type"),
    (dict(wt=I8), UNSUPPORTED, "w_type"), (dict(st=I32), UNSUPPORTED, "scores_type"), (dict(act=5), INVALID, "act"),
    (dict(act=-1), INVALID, "act"), (dict(T=-1), SHAPE, "negative"), (dict(D=-1), SHAPE, "negative"), (dict(H=-1), SHAPE, "negative"),
    (dict(E=-1), SHAPE, "negative"), (dict(T=65), UNSUPPORTED, "64 tokens"), (dict(E=513), UNSUPPORTED, "512"),
    (dict(E=0), SHAPE, "top"), (dict(top=0), SHAPE, "top"), (dict(top=9), SHAPE, "top"), (dict(E=64, top=17), UNSUPPORTED, "16"),
    (dict(D=(1 << 22) + 1), UNSUPPORTED, "D="), (dict(H=(1 << 22) + 1), UNSUPPORTED, "H="),
    (dict(X=None), INVALID, "NULL"), (dict(s=None), INVALID, "NULL"),
    (dict(Y=None), INVALID, "NULL"), (dict(W1=None), INVALID, "W1"), (dict(W2=None), INVALID, "W2"),
    (dict(wt=F8, s1=P), INVALID, "scales"), (dict(wt=F8, s2=P), INVALID, "scales"), (dict(X=P + 1), INVALID, "aligned"),
    (dict(Y=P + 1), INVALID, "aligned"), (dict(W1=P + 1), INVALID, "aligned"), (dict(W2=P + 1), INVALID, "aligned"),
    (dict(b1=P + 1), INVALID, "aligned"), (dict(b2=P + 1), INVALID, "aligned"), (dict(s=P + 2), INVALID, "aligned"),
    (dict(ids=P + 2), INVALID, "aligned"), (dict(w=P + 2), INVALID, "aligned"), (dict(wt=F8, s1=P, s2=P + 2), INVALID, "aligned"),
    (dict(ws=None), INVALID, "workspace"), (dict(ws=P + 8), INVALID, "workspace"), (dict(nb=64), INVALID, "workspace"),
]


@pytest.mark.parametrize("case", REFUSED, ids=["-".join("%s=%s" % i for i in c[0].items()) for c in REFUSED])
def test_refusals_name_the_argument(ox, case):
    kw, status, word = case
    assert moe(ox, **kw) == status
    assert word in ox.ox_last_error(), ox.ox_last_error()


@pytest.mark.parametrize("kw", [dict(T=0, X=None, Y=None, ws=None), dict(D=0, X=None, W1=None, ws=None), dict(T=0, E=0)])
def test_empty_problems_enqueue_nothing(ox, kw):
    assert moe(ox, **kw) == 0


def test_silu_is_for_this_call_alone(ox):
    assert ox.lib.ox_gemm_fp8(BF16, 4, 64, 256, P, P, P, P, None, 4, P, None) == INVALID
    assert ox.lib.ox_gemm_grouped(BF16, 4, 64, 256, 2, 1, P, P, P, None, 4, P, None) == INVALID
    assert "activation" in ox.ox_last_error()


def test_workspace_bytes(ox):
    f = ox.ox_moe_few_workspace_bytes
    for bad in [(0, 64, 96, 8, 2), (65, 64, 96, 8, 2), (4, 0, 96, 8, 2), (4, 64, -1, 8, 2), (4, 64, 96, 513, 2), (4, 64, 96, 8, 9),
                (4, 64, 96, 8, 0), (4, 64, 96, 64, 17), (4, (1 << 22) + 1, 96, 8, 2)]:
        assert f(*bad) == 0
    for T, D, H, E, top in [(1, 1, 0, 1, 1), (1, 1024, 4096, 8, 2), (64, 2048, 1024, 64, 8), (64, 1 << 22, 1, 1, 1), (1, 1, 1 << 22, 1, 1),
                            (64, 1 << 13, 1 << 11, 512, 16), (64, 1 << 22, 1 << 22, 512, 16)]:
        # at least the hidden rows and one set of sums
        assert f(T, D, H, E, top) >= 4 * T * top * H + 4 * T * D
        need = f(T, D, H, E, top)
        assert moe(ox, T=T, D=D, H=H, E=E, top=top, nb=need - 1, gated=0) == INVALID and "workspace" in ox.ox_last_error()


def test_binding_checks_shapes_and_types(ox):
    f8 = torch.float8_e4m3fn
    X, s = torch.zeros(4, 64), torch.zeros(4, 8)
    W1, W2 = torch.zeros(8, 192, 64), torch.zeros(8, 64, 96)
    Xb, Q1, Q2 = X.bfloat16(), W1.to(f8), W2.to(f8)
    s1, s2 = torch.ones(8, 2, 1), torch.ones(8, 1, 1)
    bad = [
        (ValueError, lambda: ox.ox_moe_few(X, s, W1, W2[:, :, :95], 2)), (ValueError, lambda: ox.ox_moe_few(X, s, W1, W2[:7], 2)),
        (ValueError, lambda: ox.ox_moe_few(X, s, W1, W2, 2, gated=False)), (ValueError, lambda: ox.ox_moe_few(X, s, W1[:, :191], W2, 2)),
        (ValueError, lambda: ox.ox_moe_few(X[:, :63], s, W1, W2, 2)), (ValueError, lambda: ox.ox_moe_few(X, s[:, :7], W1, W2, 2)),
        (TypeError, lambda: ox.ox_moe_few(X, s.double(), W1, W2, 2)), (TypeError, lambda: ox.ox_moe_few(X, s, W1.bfloat16(), W2, 2)),
        (TypeError, lambda: ox.ox_moe_few(Xb, s, W1, W2, 2)), (TypeError, lambda: ox.ox_moe_few(X, s, Q1, Q2, 2)),
        (ValueError, lambda: ox.ox_moe_few(X, s, W1, W2, 2, w1_scales=s1)), (ValueError, lambda: ox.ox_moe_few(Xb, s, Q1, Q2, 2)),
        (ValueError, lambda: ox.ox_moe_few(Xb, s, Q1, Q2, 2, w1_scales=s2, w2_scales=s2)),
        (TypeError, lambda: ox.ox_moe_few(Xb, s, Q1, Q2, 2, w1_scales=s1, w2_scales=s2.double())),
        (ValueError, lambda: ox.ox_moe_few(X, s, W1, W2, 2, b1=torch.zeros(8, 96))),
        (TypeError, lambda: ox.ox_moe_few(X, s, W1, W2, 2, b2=torch.zeros(8, 64).bfloat16())),
        (ValueError, lambda: ox.ox_moe_few(X, s, W1, W2, 2, Y=X[:3])), (TypeError, lambda: ox.ox_moe_few(X, s, W1, W2, 2, Y=Xb)),
        (ValueError, lambda: ox.ox_moe_few(X, s, W1, W2, 2, experts=torch.zeros(4, 2))),
        (ValueError, lambda: ox.ox_moe_few(X, s, W1, W2, 2, weights=torch.zeros(4, 3))),
        (ValueError, lambda: ox.ox_moe_few(X, s, W1, W2, 2)),                                 # host memory
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()
