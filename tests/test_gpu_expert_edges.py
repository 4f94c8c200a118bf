"""The e4m3 and expert-grouped products at the ends of their ranges: offsets of
any content, infinite weights and scales, sizes next to 2^31 elements, exact
halfway points, and the precision that each result type keeps."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

from test_gpu_expert import VARIANTS, check, check_codes, grouped_plain, quantize_plain, wide  # noqa: E402

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


def products64(A, B, off):
    """A [T, K], B [E, N, K] float64; (Y, sum of magnitudes), infinities and all"""
    Y, S = np.zeros((A.shape[0], B.shape[1])), np.zeros((A.shape[0], B.shape[1]))
    with np.errstate(invalid="ignore"):
        for e in range(B.shape[0]):
            rows = slice(off[e], off[e + 1])
            # term by term: a library's product may pad, and 0 * inf is NaN
            Y[rows] = (A[rows][:, None, :] * B[e][None]).sum(axis=2)
            S[rows] = np.abs(A[rows][:, None, :] * B[e][None]).sum(axis=2)
    return Y, S


def check_infinities(got, Y, S, K, dtype):
    """The same infinities and NaN; the finite results within the rounding of K
    additions in fp32 (2^-23 of the sum of magnitudes each) and of the result."""
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(Y))
    inf = np.isinf(Y)
    assert np.array_equal(np.isinf(got), inf) and np.array_equal(got[inf], Y[inf])
    fin = np.isfinite(Y)
    eps = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    assert (np.abs(got[fin] - Y[fin]) <= 1.2 * (K + 8) * 2.0 ** -23 * S[fin] + eps * np.abs(Y[fin])).all()


@pytest.mark.parametrize("variant", ["", "stream", "32x64", "64x64x2", "regs"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
# blocks of 128 bytes of K that do not divide into slices of four, and rows that
# end inside a block
@pytest.mark.parametrize("blocks,tail", [(24, 0), (9, 0), (17, 16), (33, 112), (3, 48)])
def test_infinite_operands(ox, monkeypatch, variant, dtype, blocks, tail):
    say("infinities", variant, dtype, blocks, tail)
    if variant:
        monkeypatch.setenv("OX_FORCE_KERNEL", variant)
    size = 2 if dtype == torch.bfloat16 else 4
    K, N, off = (blocks * 128 + tail) // size, 48, [0, 1, 1, 4]
    rng = np.random.default_rng([11, blocks, tail])
    A = torch.from_numpy(rng.standard_normal((4, K))).to(dtype)
    B = torch.from_numpy(rng.standard_normal((3, N, K))).to(dtype)
    for i, k in enumerate([0, 1, K // 2, K - 1, K - 2, K - 16 // size, K - 128 // size, K - 256 // size, K - 512 // size]):
        B[:, 2 * i, k] = np.inf * (-1) ** i
    A[2, K - 1] = np.inf
    Y, S = products64(A.double().numpy(), B.double().numpy(), off)
    assert np.isinf(Y).sum() > 30
    dev = [A.cuda(), B.cuda(), torch.tensor(off, dtype=torch.int32, device="cuda")]
    check_infinities(ox.ox_gemm_grouped(*dev), Y, S, K, dtype)
    if variant != "stream":                                    # weights stored [K, N] are not streamed
        Bt = dev[1].transpose(1, 2).contiguous()
        check_infinities(ox.ox_gemm_grouped(dev[0], Bt, dev[2], transB=False), Y, S, K, dtype)
    got = ox.ox_gemm_grouped(*dev, act="relu").double().cpu().numpy()
    assert (got[Y == np.inf] == np.inf).all() and (got[Y == -np.inf] == 0).all()


@pytest.mark.parametrize("variant", ["", "stream", "32x32x4", "64x64x2", "128x128x2", "64x64", "regs"])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", [1152, 1024, 2064, 4224, 368])
def test_infinite_scales(ox, monkeypatch, variant, out, K):
    say("infinite scales", variant, out, K)
    if variant:
        monkeypatch.setenv("OX_FORCE_KERNEL", variant)
    M, N, kb = 3, 256, -(-K // 128)
    rng = np.random.default_rng([12, K])
    # positive codes: every block's sum is above zero
    qa, qb = (torch.from_numpy(rng.uniform(0.5, 2.0, (n, K))).float().to(F8) for n in (M, N))
    sa, sb = rng.uniform(0.5, 2.0, (M, kb)).astype(np.float32), rng.uniform(0.5, 2.0, (2, kb)).astype(np.float32)
    sa[1, kb - 1] = np.inf
    sb[1, kb - 1] = -np.inf
    Y = ox.ox_gemm_fp8(qa.cuda(), torch.from_numpy(sa.T.copy()).cuda(), qb.cuda(), torch.from_numpy(sb).cuda(), out_dtype=out)
    want = np.zeros((M, N))
    for b in range(kb):
        cols = slice(b * 128, min(K, (b + 1) * 128))
        want += (sa[:, None, b].astype(np.float64) * np.repeat(sb[:, b], 128)[None]
                 * (qa[:, cols].double().numpy() @ qb[:, cols].double().numpy().T))
    got = Y.double().cpu().numpy()
    assert np.isinf(want).sum() == 2 * 128 + 256
    assert not np.isnan(got).any() and np.array_equal(got[np.isinf(want)], want[np.isinf(want)])
    fin = np.isfinite(want)                 # every product is positive: the sum is the sum of magnitudes
    tol = 1.2 * ((K + 8) * 2.0 ** -23 + (2.0 ** -15 + 2.0 ** -8 if out == torch.bfloat16 else 2.0 ** -24))
    assert (np.abs(got[fin] - want[fin]) <= tol * want[fin]).all()


def e4m3_of(x, m):
    """The e4m3 value of 448 x / m, of exact rationals, half to even."""
    from fractions import Fraction
    q = Fraction(448) * Fraction(float(x)) / Fraction(float(m))
    a, e = abs(q), -6
    while a >= Fraction(2) ** (e + 1):
        e += 1
    step = Fraction(2) ** (e - 3)
    return float(round(q / step) * step)            # Fraction rounds half to even


def halfway_block(rng, exact, n):
    """fp32 [n], led by its maximum m: the others make 448 x / m a halfway point
    of e4m3 exactly, or are the fp32 number nearest to that or next to it,
    nearer to the halfway point than an fp32 quotient can tell."""
    m = 7 * 8 * int(rng.integers(2 ** 17, 2 ** 18)) if exact else int(rng.integers(2 ** 23, 2 ** 24))
    scale = np.float32(2.0 ** int(rng.integers(-60, 60)))
    half = 2 * rng.integers(0, 16, n) + 1                                  # odd: in halves of a step
    e = np.where(half < 16, -10, rng.integers(-10, 4, n))                  # (below 2^-6 the step is 2^-9)
    x = (half * 2.0 ** e * m / 448.0).astype(np.float32)
    if not exact:
        x = np.nextafter(x, np.where(rng.random(n) < 0.3, 0, np.where(rng.random(n) < 0.5, x, 1e30)).astype(np.float32))
    x *= rng.choice([-1, 1], n).astype(np.float32)
    x[0] = m
    return x * scale


@pytest.mark.parametrize("br", [1, 128])
@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("inf", [False, True])
def test_quantize_fp32_halfway_points(ox, br, exact, inf):
    say("fp32 halfway points", br, exact, inf)
    rng = np.random.default_rng([13, br, exact, inf])
    if br == 1:
        X = np.stack([halfway_block(rng, exact, 128) for _ in range(128)])
    else:
        X = halfway_block(rng, exact, 128 * 128).reshape(128, 128)
    m = np.abs(X).max(axis=1) if br == 1 else np.full(128, np.abs(X).max())
    want = np.array([[e4m3_of(x, m[r]) for x in X[r]] for r in range(128)])
    if inf:
        X[:, 127] = np.inf
        want[:, 127] = 448.0
    Q, S = ox.ox_quantize_fp8(torch.from_numpy(X).cuda(), block_rows=br)
    np.testing.assert_array_equal(Q.float().cpu().numpy().astype(np.float64), want)


# Sums of n independent terms in fp32, each addition off by a rounding of about
# 2^-25.3 of the partial sum (0.29 of a step, at a magnitude between powers of
# two): the error of a chain of n grows as n * 2^-25.3 / sqrt(2) of a term's size.
# Chains of at most 256 k added up give sqrt(128 + K / 512) * 2^-25.3 of the norm of
# a random result (2.8e-7 at K = 4096, 2.9e-7 at 10240), one chain over K
# sqrt(K / 2) * 2^-25.3 (1.1e-6, 1.7e-6).  The bound lies between.
NORM = 5e-7


def off_norm(got, want):
    return float(((got.double() - want).norm() / want.norm()).item())


@pytest.mark.parametrize("variant", [""] + VARIANTS["f32"] + ["kn " + v for v in VARIANTS["f32 kn"]])
@pytest.mark.parametrize("K", [4096, 10240])
def test_fp32_sums_stay_short(ox, monkeypatch, variant, K):
    kn = variant.startswith("kn ")
    if variant:
        monkeypatch.setenv("OX_FORCE_KERNEL", variant.split()[-1])
    say("fp32 sums", variant, K)
    g = torch.Generator(device="cuda").manual_seed(K)
    A, B = torch.randn(48, K, device="cuda", generator=g), torch.randn(1, 256, K, device="cuda", generator=g)
    off = torch.tensor([0, 48], dtype=torch.int32, device="cuda")
    Y = ox.ox_gemm_grouped(A, B.transpose(1, 2).contiguous() if kn else B, off, transB=not kn)
    assert off_norm(Y, A.double() @ B[0].double().t().contiguous()) < NORM


@pytest.mark.parametrize("variant", [""] + VARIANTS["fp8x"])
def test_e4m3_to_fp32_keeps_small_products(ox, monkeypatch, variant):
    # one large product and one 2^-16 of it, side by side in every way that a
    # matrix instruction might group them: 448 * 448 + 4 * 1 exactly
    if variant:
        monkeypatch.setenv("OX_FORCE_KERNEL", variant)
    say("small products", variant)
    M, N, K = 96, 64, 256
    A, B = torch.zeros(M, K), torch.zeros(N, K)
    B[:, 0] = 448.0
    B[:, 1:] = 4.0
    for m in range(M):
        A[m, 0] = 448.0
        A[m, 1 + m] = 1.0
    one = torch.ones(2, M, device="cuda"), torch.ones(1, 2, device="cuda")
    Y = ox.ox_gemm_fp8(A.to(F8).cuda(), one[0], B.to(F8).cuda(), one[1], out_dtype=torch.float32)
    assert (Y == 448.0 * 448.0 + 4.0).all().item()


@pytest.mark.parametrize("variant", [""] + VARIANTS["fp8x"])
def test_e4m3_to_fp32_sums(ox, monkeypatch, variant):
    if variant:
        monkeypatch.setenv("OX_FORCE_KERNEL", variant)
    say("e4m3 to fp32 sums", variant)
    g = torch.Generator(device="cuda").manual_seed(14)
    K = 4096
    A, B = (torch.randn(n, K, device="cuda", generator=g).mul_(60).clamp_(-448, 448).to(F8) for n in (48, 256))
    sa, sb = torch.rand(K // 128, 48, device="cuda", generator=g) + 0.5, torch.rand(2, K // 128, device="cuda", generator=g) + 0.5
    Y = ox.ox_gemm_fp8(A, sa, B, sb, out_dtype=torch.float32)
    a = A.double() * sa.double().t().repeat_interleave(128, dim=1)
    b = B.double() * sb.double().repeat_interleave(128, dim=0).repeat_interleave(128, dim=1)
    assert off_norm(Y, a @ b.t().contiguous()) < NORM


@pytest.mark.parametrize("tokens,experts,width,hidden", [(5, 8, 256, 512), (100, 4, 384, 640)])
def test_example_layer_step_by_step(ox, tokens, experts, width, hidden):
    """Every step of the layer against 64 bits, from the buffers that it ran on."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py")
    spec = importlib.util.spec_from_file_location("expert_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    say("example layer", tokens, experts, width, hidden)
    g = torch.Generator(device="cuda").manual_seed(2)
    layer = mod.ExpertLayer(tokens, experts, width, hidden, g)
    X = torch.randn(tokens, width, generator=g, device="cuda").bfloat16()
    out = layer(X)
    weight, token, place, offsets = layer.route(X)
    off = offsets.tolist()
    bf16 = torch.bfloat16

    def wide64(t):
        return t.float().cpu().double().numpy()
    for e in range(experts):
        for W, q, s in ((layer.W1, layer.q1, layer.s1), (layer.W2, layer.q2, layer.s2)):
            Q, S, V = quantize_plain(wide64(W[e]), 128)
            check_codes(q[e], Q, V, bf16)
            np.testing.assert_array_equal(wide64(s[e]), S)
    for x, q, s in ((X[token.long()], layer.xq, layer.xs), (layer.h, layer.hq, layer.hs)):
        Q, S, V = quantize_plain(wide64(x), 1)
        check_codes(q, Q, V, bf16)
        np.testing.assert_array_equal(wide64(s), S.T)
    for a, sa, q, s, bias, act, y in ((layer.xq, layer.xs, layer.q1, layer.s1, wide64(layer.b1), "gelu", layer.h),
                                      (layer.hq, layer.hs, layer.q2, layer.s2, None, "none", layer.y)):
        ref, S = grouped_plain(wide(wide64(a), wide64(sa).T, 1), wide(wide64(q), wide64(s), 128), off, bias, act)
        check(y, ref, S, a.shape[1], bf16, act, "layer", e4m3=True)
    rows = wide64(layer.y)[place.cpu().numpy()].reshape(tokens, mod.TOP, -1) * wide64(weight)[:, :, None]
    # two products and a sum in fp32, rounded once to bf16
    tol = 2.0 ** -8 * np.abs(rows.sum(axis=1)) + 4 * 2.0 ** -24 * np.abs(rows).sum(axis=1)
    assert (np.abs(wide64(out) - rows.sum(axis=1)) <= tol).all()


@pytest.mark.parametrize("variant", [""] + VARIANTS["fp8"])
@pytest.mark.parametrize("kind", ["normal", "positive", "seven"])
def test_e4m3_to_bf16_loses_what_the_header_says(ox, monkeypatch, variant, kind):
    """A second block of K holds the negative of each eight's largest product, so
    that the small products, and what they lose beside it, are the result."""
    if variant:
        monkeypatch.setenv("OX_FORCE_KERNEL", variant)
    say("e4m3 to bf16", variant, kind)
    M, N = 40, 64
    rng = np.random.default_rng([15, len(kind)])
    if kind == "seven":                     # seven products just below the cut: all of them are lost
        a, b = np.full((M, 128), 1.875), np.full((N, 128), 3.75)
        a[:, ::8], b[:, ::8] = 256.0, 256.0
    else:
        a, b = (np.exp2(rng.integers(-2, 5, (n, 128))) * (1 + rng.integers(0, 8, (n, 128)) / 8) for n in (M, N))
        if kind == "normal":
            a *= rng.choice([-1, 1], a.shape)
        a[:, ::8] *= 8.0
        b[:, ::8] *= 8.0
    A, B = np.concatenate([a, np.zeros((M, 128))], axis=1), np.concatenate([b, np.zeros((N, 128))], axis=1)
    A[:, 128::8], B[:, 128::8] = -a[:, ::8], b[:, ::8]
    ta, tb = torch.from_numpy(A).float().to(F8), torch.from_numpy(B).float().to(F8)
    assert (ta.double().numpy() == A).all() and (tb.double().numpy() == B).all()

    def power(x):
        return np.exp2(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -30))))
    P = A[:, None] * B[None]                                                   # [M, N, 256]
    tops = (power(A)[:, None] * power(B)[None] * (P != 0)).reshape(M, N, 32, 8).max(axis=3, keepdims=True)
    cut = 2.0 ** -13 * np.maximum(tops, 2.0 ** -60)
    P8 = P.reshape(M, N, 32, 8)
    want, exact = (np.trunc(P8 / cut) * cut).sum(axis=(2, 3)), P.sum(axis=2)
    lost = np.abs(want - exact)
    assert (lost <= 7 * 2.0 ** -13 * np.abs(P8).max(axis=3).sum(axis=2)).all() and lost.max() > 0
    Y = ox.ox_gemm_fp8(ta.cuda(), torch.ones(2, M, device="cuda"), tb.cuda(), torch.ones(1, 2, device="cuda"))
    got = Y.double().cpu().numpy()
    # the additions between the eights (fp32, and exact up to 2^-23 of the sums) and the rounding to bf16
    tol = 2.0 ** -8 * np.abs(want) + 64 * 2.0 ** -23 * np.abs(P).sum(axis=2)
    assert (np.abs(got - want) <= tol).all()
