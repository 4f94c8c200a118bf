"""The routed layer of a few tokens where its weights are not finite, against
the formula in 64 bits (an e4m3 block's scale multiplies the block's sum)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_moe_few import BF, F32, Layer, chosen_plain, say      # noqa: E402

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def ox():
    import conv_implicit_gemm_amd as ox
    return ox


def bf16_hidden(layer, e):
    """Expert e's hidden values are tokens' elements: exact in bf16."""
    W = torch.zeros(layer.W[0][e].shape, dtype=layer.t)
    for j in range(layer.H):
        W[j, j % layer.D] = 1.0
    layer.W[0][e] = W.cuda()
    layer.w64[0][e] = W.double().numpy()


def same_kind(got, ref):
    """Infinities with their signs, and NaN, where the formula has them."""
    for kind in (np.isposinf, np.isneginf, np.isnan):
        np.testing.assert_array_equal(kind(got), kind(ref), err_msg=kind.__name__)


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("T,D", [(3, 72), (12, 72), (40, 72), (40, 8200)])
def test_infinities_among_the_second_weights(ox, t, T, D):
    E, top, H = 4, 2, 200
    say("infinite W2", t, T, D)
    layer = Layer([40, T, D], t, E, D, H, False, False)
    bf16_hidden(layer, 0)
    inf, nan = float("inf"), float("nan")
    for e, row, k, v in [(0, 5, 3, inf), (0, 6, 4, -inf), (1, 7, 11, inf), (1, 8, 12, inf), (1, 8, 13, -inf), (2, 9, 190, nan),
                         (2, 10, 70, -inf), (3, 11, H - 1, inf), (3, D - 1, 0, -inf)]:
        layer.W[1][e, row, k] = v
        layer.w64[1][e][row, k] = v
    X = torch.from_numpy(layer.rng.standard_normal((T, D))).to(layer.t)
    scores = torch.from_numpy(layer.rng.standard_normal((T, E))).float()
    s = scores.double().numpy()
    ids, w = chosen_plain(s, top, True)
    with np.errstate(invalid="ignore"):
        ref, tol = layer.plain(X.double().numpy(), ids, w, s, "none")
    got = ox.ox_moe_few(X.cuda(), scores.cuda(), layer.W[0], layer.W[1], top, act="none", gated=False).double().cpu().numpy()
    assert np.isinf(ref).sum() > 3 * T / 2 and np.isnan(ref).any()
    same_kind(got, ref)
    ok = np.isfinite(ref)
    half = torch.finfo(layer.t).eps / 2
    got, ref, tol = got[ok], ref[ok], tol[ok]
    assert (np.abs(got - ref) <= 1.02 * tol + half * (np.abs(ref) + tol) * 1.01 + 2.0 ** -126).all()


@pytest.mark.parametrize("T", [3, 12, 40])
def test_infinite_scales_of_the_second_weights(ox, T):
    E, D, H = 2, 200, 300
    say("infinite scales of W2", T)
    layer = Layer([41, T], "fp8", E, D, H, False, False)
    ones = torch.ones((E, H, D), dtype=F32)
    ones[:, :, 1:] = 0                       # every hidden value is the token's first element
    W1 = ones.to(torch.float8_e4m3fn).cuda()
    s1 = torch.ones_like(layer.scales[0])
    W2, s2 = layer.W[1].float(), layer.scales[1]
    W2[W2 == 0] = 1.0
    s2[0, 0, 1] = float("inf")               # rows 0 .. 127, k 128 .. 255 of the first expert
    s2[1, 1, 2] = float("-inf")              # rows 128 .. 199, k 256 .. 299 of the second
    X = torch.from_numpy(layer.rng.standard_normal((T, D))).to(BF)
    X[0, 0] = 3.0
    scores = torch.full((T, E), float("-inf"))
    scores[torch.arange(T), torch.arange(T) % 2] = 0.0
    got = ox.ox_moe_few(X.cuda(), scores.cuda(), W1, W2.to(torch.float8_e4m3fn), 1, w1_scales=s1, w2_scales=s2, act="none",
                        gated=False).double().cpu().numpy()
    q, h = W2.double().cpu().numpy(), X[:, 0].double().numpy()
    sign = np.zeros((T, D))
    for i in range(T):
        if i % 2 == 0:
            sign[i, :128] = np.sign(h[i] * q[0, :128, 128:256].sum(axis=1))
        else:
            sign[i, 128:] = -np.sign(h[i] * q[1, 128:, 256:].sum(axis=1))
    assert (sign > 0).any() and (sign < 0).any()
    with np.errstate(invalid="ignore"):
        far = sign != 0
        np.testing.assert_array_equal(got[far], (sign * np.inf)[far])
    # (a block's sum of exactly zero has no infinity to give)
    blocks = np.zeros((T, D), bool)
    blocks[::2, :128] = blocks[1::2, 128:] = True
    assert np.isfinite(got[~blocks]).all() and np.isnan(got[blocks & ~far]).all()
