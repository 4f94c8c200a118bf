"""The RMS norm with 8-bit results, the int8 quantisation of rows and the int8
product with run-time scales on the GPU, against plain 64-bit forms on the CPU.

Tolerances, derived from the formulas.
- ox_quantize_i8: codes and scales are those of exact quotients: equal.
- ox_gemm_i8: the int32 sum is exact; its conversion, two multiplications and
  the addition of the bias are four roundings of 2^-24, of |scaled sum| +
  |bias|.  GELU's slope is below 1.13 and its own evaluation good to 2^-20 of
  |v|; the last rounding adds half a step of the type.
- ox_rmsnorm: s and z = s * gamma are a rounding each (2^-24).  The sum of
  squares is a chain of at most 64 additions a thread, 6 in the wave and 16
  over the waves, of squares that are off by 2 * 2^-24: below 90 * 2^-24 of
  itself, half of that in its root; the division, the addition of eps, the
  root and the reciprocal add four, y's product one more.  All of it is below
  2^-18 of |y|, before the last rounding.
- The codes of a norm are those of z / max|z|: z is off by 2 * 2^-24 on either
  side, the quotient by 2^-21 of itself at most (2^-14 of a code's step)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

F8 = torch.float8_e4m3fn
TINY = 2.0 ** -100


def say(*a):
    print("[case]", *a, flush=True)


@pytest.fixture(scope="module")
def ox():
    import conv_implicit_gemm_amd as ox
    return ox


def blocks(n):
    return -(-n // 128)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def round_e4m3(v):
    v = np.asarray(v, np.float64)
    a = np.maximum(np.abs(v), 2.0 ** -30)
    step = np.exp2(np.maximum(np.floor(np.log2(a)), -6.0) - 3.0)
    return np.clip(np.rint(v / step) * step, -448.0, 448.0)


def act64(v, act):
    if act == "relu":
        return np.maximum(v, 0)
    if act == "relu6":
        return np.clip(v, 0, 6)
    if act == "gelu":
        return (0.5 * torch.from_numpy(v) * torch.erfc(torch.from_numpy(-v / np.sqrt(2.0)))).numpy()
    return v


def guarded(shape, dtype, shift=0):
    """A tensor of `shape`, `shift` elements off a 256-byte border, between two
    guards; returns (tensor, check) -- check() fails if a guard was written."""
    n = int(np.prod(shape))
    whole = torch.full((n + 512 + shift,), 77, dtype=torch.uint8 if dtype == F8 else dtype, device="cuda")
    t = whole[256 + shift:256 + shift + n].view(shape)

    def intact():
        assert (whole[:256 + shift] == 77).all().item() and (whole[256 + shift + n:] == 77).all().item()
    return (t.view(F8) if dtype == F8 else t), intact


def shifted(x, shift):
    """A copy of x on the GPU that starts `shift` elements off an aligned address."""
    if shift == 0:
        return x.contiguous().cuda()
    size = x.element_size()
    raw = torch.empty(x.numel() + shift, dtype={1: torch.uint8, 2: torch.int16, 4: torch.int32}[size], device="cuda")
    raw[shift:] = x.contiguous().cuda().reshape(-1).view(raw.dtype)
    return raw[shift:].view(x.dtype).view(x.shape)


# ------------------------------------------------------- int8 quantisation --

def quantize_plain(X):
    """codes, scales (float32) of rows in 64 bits: 127 x is exact there, and no
    quotient of two floats is within 2^-40 of a halfway point without being it"""
    fin = np.isfinite(X)
    m = np.maximum(np.where(fin, np.abs(X), 0.0).max(axis=1, initial=0.0), TINY)
    q = np.rint(127.0 * np.where(fin, X, 0.0) / m[:, None])
    q = np.where(np.isinf(X), np.copysign(127.0, np.where(np.isnan(X), 0, X)), q)
    s = (m.astype(np.float32) / np.float32(127)).astype(np.float32)
    return q.astype(np.int8), np.where(np.isnan(X).any(axis=1), np.float32(np.nan), s)


ROWS_K = [(1, 1), (1, 7), (3, 8), (5, 127), (4, 130), (24, 512), (9, 520), (6, 1024), (7, 1031), (3, 2048), (24, 4096), (2, 4099),
          (5, 8192), (3, 9000), (2, 16384), (2, 20001), (2, 32768), (1, 65535), (2, 65536), (1030, 64)]


@pytest.mark.parametrize("dtype,shift", [(torch.bfloat16, 0), (torch.float32, 0), (torch.bfloat16, 1), (torch.float32, 3)])
@pytest.mark.parametrize("rows,K", ROWS_K)
def test_quantize(ox, rows, K, dtype, shift):
    say("quantize_i8", rows, K, dtype, shift)
    rng = np.random.default_rng([21, rows, K])
    X = torch.from_numpy(rng.standard_normal((rows, K)) * np.exp(rng.uniform(-20, 20, (rows, 1)))).to(dtype)
    Q, okq = guarded((rows, K), torch.int8, shift)
    S, oks = guarded((rows,), torch.float32)
    ox.ox_quantize_i8(shifted(X, shift), Q=Q, scales=S)
    torch.cuda.synchronize()
    okq(), oks()
    q, s = quantize_plain(X.double().numpy())
    np.testing.assert_array_equal(S.cpu().numpy(), s)
    np.testing.assert_array_equal(Q.cpu().numpy(), q)


def test_quantize_halfway_points_bf16(ox):
    # every bf16 significand under every one as the row's maximum, at eight magnitudes
    sig = torch.arange(128, 256, dtype=torch.float32)
    X = torch.cat([sig.repeat(128, 1) * 2.0 ** -e for e in range(8)], dim=1)
    X = torch.minimum(X, sig[:, None].expand_as(X))
    X[:, 0] = sig
    X = torch.cat([X, -X], dim=1).bfloat16()
    Q, S = ox.ox_quantize_i8(X.cuda())
    q, s = quantize_plain(X.double().numpy())
    v = 127.0 * X.double().numpy() / sig.double().numpy()[:, None]
    assert (np.abs(v - np.floor(v)) == 0.5).sum() > 500
    np.testing.assert_array_equal(Q.cpu().numpy(), q)
    np.testing.assert_array_equal(S.cpu().numpy(), s)


@pytest.mark.parametrize("top", [1.0, 3.0, 1.9999998807907104, 254.0, 3.4e38, 2.0 ** -99])
def test_quantize_next_to_halfway_points_fp32(ox, top):
    # the floats nearest to (n + 1/2) m / 127, and their neighbours
    m = np.float32(top)
    h = ((np.arange(-127, 127) + 0.5) * np.float64(m) / 127.0).astype(np.float32)
    X = np.concatenate([h, np.nextafter(h, np.float32(np.inf)), np.nextafter(h, np.float32(-np.inf)), [m, -m, 0.0]]).astype(np.float32)
    Q, S = ox.ox_quantize_i8(torch.from_numpy(X[None]).cuda())
    q, s = quantize_plain(X[None].astype(np.float64))
    np.testing.assert_array_equal(Q.cpu().numpy(), q)
    np.testing.assert_array_equal(S.cpu().numpy(), s)


@pytest.mark.parametrize("K", [256, 5000, 40000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_zeros_infinities_nans_and_tiny(ox, dtype, K):
    rng = np.random.default_rng(22)
    X = rng.standard_normal((7, K)).astype(np.float32)
    X[0] = 0
    X[1, 3], X[1, K - 1] = np.inf, -np.inf
    X[2, 100] = np.nan
    X[3] = 1e-38
    X[4] *= 1e37
    X[5] = np.inf
    X[6] = np.nan
    X = torch.from_numpy(X).to(dtype)
    Q, S = ox.ox_quantize_i8(X.cuda())
    q, s = quantize_plain(X.double().numpy())
    np.testing.assert_array_equal(S.cpu().numpy(), s)
    np.testing.assert_array_equal(Q.cpu().numpy(), q)


# ---------------------------------------------------------------- products --

M_N_K = [(1, 1, 1), (1, 64, 128), (2, 130, 256), (3, 17, 96), (5, 256, 1000), (16, 300, 640), (17, 128, 384), (24, 72, 2064),
         (33, 200, 77), (64, 96, 512), (100, 129, 257), (127, 256, 272), (130, 384, 400), (256, 256, 1024), (300, 520, 144),
         (513, 264, 640), (1, 2000, 4096), (16, 16, 2048)]


def i8_operands(rng, M, N, K):
    A = rng.integers(-128, 128, (M, K)).astype(np.int8)
    B = rng.integers(-128, 128, (N, K)).astype(np.int8)
    sa = np.exp(rng.uniform(-6, 0, M)).astype(np.float32)
    sb = np.exp(rng.uniform(-6, 0, N)).astype(np.float32)
    return A, sa, B, sb


def check_product(Y, A, sa, B, sb, bias, act, what):
    p = (A.astype(np.float64) @ B.astype(np.float64).T) * sa.astype(np.float64)[:, None] * sb.astype(np.float64)[None, :]
    b = 0.0 if bias is None else bias.double().cpu().numpy()
    ref = act64(p + b, act)
    mag = np.abs(p) + np.abs(b)
    tol = 4.1 * 2.0 ** -24 * mag * (1.13 if act == "gelu" else 1.0) + half_step(Y.dtype) * np.abs(ref) * 1.01 + 2.0 ** -126
    if act == "gelu":
        tol = tol + 2.0 ** -20 * mag
    got = Y.double().cpu().numpy()
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), "%s: %d of %d, first at %s" % (what, bad.sum(), bad.size, np.argwhere(bad)[0])


@pytest.mark.parametrize("M,N,K", M_N_K)
@pytest.mark.parametrize("out,act,shift", [(torch.bfloat16, "none", 0), (torch.float32, "gelu", 0), (torch.float32, "none", 1),
                                           (torch.bfloat16, "relu6", 3)])
def test_gemm_i8(ox, M, N, K, out, act, shift):
    say("gemm_i8", M, N, K, out, act, shift)
    rng = np.random.default_rng([23, M, N, K])
    A, sa, B, sb = i8_operands(rng, M, N, K)
    bias = torch.from_numpy(rng.standard_normal(N)).to(out).cuda() if act != "none" else None
    Y, ok = guarded((M, N), out, shift)
    ox.ox_gemm_i8(shifted(torch.from_numpy(A), shift), torch.from_numpy(sa).cuda(), shifted(torch.from_numpy(B), shift),
                  torch.from_numpy(sb).cuda(), bias=bias, act=act, Y=Y)
    torch.cuda.synchronize()
    ok()
    check_product(Y, A, sa, B, sb, bias, act, (M, N, K))


VARIANTS = ["32x64", "64x64", "128x128", "256x256", "32x32x4", "64x64x2", "128x128x2", "regs", "regs128", "stream"]


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("M,N,K", [(1, 48, 1040), (19, 77, 176), (130, 200, 1552), (300, 272, 4096)])
def test_every_variant(ox, variant, M, N, K, monkeypatch):
    say("gemm_i8", variant, M, N, K)
    monkeypatch.setenv("OX_FORCE_KERNEL", variant)
    rng = np.random.default_rng([24, M, N, K])
    A, sa, B, sb = i8_operands(rng, M, N, K)
    # the largest sums that fit: all -128 times -128 in one place
    A[0], B[0] = -128, -128
    Y, ok = guarded((M, N), torch.float32)
    ox.ox_gemm_i8(torch.from_numpy(A).cuda(), torch.from_numpy(sa).cuda(), torch.from_numpy(B).cuda(),
                  torch.from_numpy(sb).cuda(), Y=Y)
    torch.cuda.synchronize()
    ok()
    check_product(Y, A, sa, B, sb, None, "none", (variant, M, N, K))


@pytest.mark.parametrize("variant", [None, "32x32x4", "128x128x2"])
def test_longest_sums(ox, variant, monkeypatch):
    if variant:
        monkeypatch.setenv("OX_FORCE_KERNEL", variant)
    K = 131071 if variant is None else 131056
    A, B = torch.full((3, K), -128, dtype=torch.int8), torch.full((20, K), -128, dtype=torch.int8)
    A[1] = 127
    one = torch.ones(20, device="cuda")
    Y = ox.ox_gemm_i8(A.cuda(), one[:3].contiguous(), B.cuda(), one, out_dtype=torch.float32)
    want = torch.tensor([16384.0 * K, -127.0 * 128 * K, 16384.0 * K]).double()[:, None].expand(3, 20)
    assert (Y.double().cpu() - want).abs().max().item() <= 2.0 ** -24 * 2.0 ** 31      # the conversion to fp32


def test_gemm_i8_without_k_is_the_bias(ox):
    A, B = torch.empty((3, 0), dtype=torch.int8, device="cuda"), torch.empty((5, 0), dtype=torch.int8, device="cuda")
    b = torch.tensor([-1.0, 0.5, 2.0, -3.0, 7.0], device="cuda")
    Y = ox.ox_gemm_i8(A, torch.ones(3, device="cuda"), B, torch.ones(5, device="cuda"), bias=b, act="relu",
                      out_dtype=torch.float32)
    assert torch.equal(Y, b.clamp(min=0).expand(3, 5))


# -------------------------------------------------------------- RMS norm --

def norm_plain(X, R, g, eps):
    s = X if R is None else X + R
    z = s * (1.0 if g is None else g)
    return s, z / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps)


def check_norm(got, scales, X, R, g, eps, out):
    _, y = norm_plain(X, R, g, eps)
    rel = 2.0 ** -18
    if out == "same":
        tol = (rel + half_step(got.dtype) * (1 + rel)) * np.abs(y) + 2.0 ** -126
        assert (np.abs(got.double().cpu().numpy() - y) <= tol).all()
        return
    sc = scales.double().cpu().numpy()
    q = got.float().cpu().double().numpy()
    if out == "i8":
        m = np.maximum(np.abs(y).max(axis=1), TINY)
        np.testing.assert_allclose(sc, m / 127.0, rtol=rel)
        assert (np.abs(127.0 * y / m[:, None] - q) <= 0.5 + 2.0 ** -13).all()
        return
    for j in range(blocks(y.shape[1])):
        b = y[:, j * 128:(j + 1) * 128]
        m = np.maximum(np.abs(b).max(axis=1), TINY)
        np.testing.assert_allclose(sc[j], m / 448.0, rtol=rel)
        v = 448.0 * b / m[:, None]
        lo, hi = round_e4m3(v * (1 - 2.0 ** -21)), round_e4m3(v * (1 + 2.0 ** -21))
        c = q[:, j * 128:(j + 1) * 128]
        assert ((c == lo) | (c == hi)).all()


@pytest.mark.parametrize("out", ["same", "fp8", "i8"])
@pytest.mark.parametrize("dtype,shift", [(torch.bfloat16, 0), (torch.float32, 0), (torch.bfloat16, 1)])
@pytest.mark.parametrize("rows,K", ROWS_K)
def test_rmsnorm(ox, rows, K, dtype, shift, out):
    say("rmsnorm", rows, K, dtype, shift, out)
    rng = np.random.default_rng([25, rows, K])
    X = torch.from_numpy(rng.standard_normal((rows, K))).to(dtype)
    R = torch.from_numpy(rng.standard_normal((rows, K)) * np.exp(rng.uniform(-3, 3, (rows, 1)))).to(dtype)
    g = torch.from_numpy(1 + 0.2 * rng.standard_normal(K)).to(dtype)
    ydt = {"same": dtype, "fp8": F8, "i8": torch.int8}[out]
    for residual, gamma in ((True, True), (False, False), (False, True)):
        Y, oky = guarded((rows, K), ydt, shift)
        sc, oks = (None, None) if out == "same" else guarded((blocks(K), rows) if out == "fp8" else (rows,), torch.float32)
        S, okt = guarded((rows, K), dtype, shift) if residual else (None, None)
        got = ox.ox_rmsnorm(shifted(X, shift), shifted(g, shift) if gamma else None, residual=shifted(R, shift) if residual else None,
                            eps=1e-6, out=out, Y=Y, scales=sc, S=S)
        torch.cuda.synchronize()
        for ok in (oky, oks, okt):
            if ok:
                ok()
        assert got[0] is Y and got[1] is sc and got[2] is S
        x, r, gg = X.double().numpy(), R.double().numpy() if residual else None, g.double().numpy() if gamma else None
        if residual:
            assert torch.equal(S.cpu(), (X.float() + R.float()).to(dtype))
        check_norm(Y, sc, x, r, gg, 1e-6, out)


@pytest.mark.parametrize("out", ["same", "fp8", "i8"])
@pytest.mark.parametrize("K", [384, 6000])
def test_rmsnorm_in_place(ox, K, out):
    rng = np.random.default_rng([26, K])
    X, R = (torch.from_numpy(rng.standard_normal((9, K))).bfloat16().cuda() for _ in range(2))
    g = torch.from_numpy(1 + 0.2 * rng.standard_normal(K)).bfloat16().cuda()
    want = ox.ox_rmsnorm(X, g, residual=R, out=out)
    for where in ("X", "residual"):
        x, r = X.clone(), R.clone()
        y, sc, s = ox.ox_rmsnorm(x, g, residual=r, out=out, S=x if where == "X" else r,
                                 Y=(r if where == "X" else x) if out == "same" else None)
        assert torch.equal(s, want[2]) and torch.equal(y.view(torch.uint8), want[0].view(torch.uint8))
        if sc is not None:
            assert torch.equal(sc, want[1])


@pytest.mark.parametrize("K", [256, 3000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rmsnorm_zeros_infinities_nans_and_ends_of_the_range(ox, dtype, K):
    rng = np.random.default_rng(27)
    X = rng.standard_normal((8, K)).astype(np.float32)
    X[0] = 0
    X[1, 5] = np.inf            # finite values become 0, the infinity NaN
    X[2, 5] = np.nan            # the whole row
    X[3] *= 1e-30               # eps is all of the mean
    X[4] *= 3e37                # the sum of squares overflows: zeros
    X[5] *= 1e17
    X[6] = -np.inf
    X[7, 1:] = 0
    X = torch.from_numpy(X).to(dtype)
    x = X.double().numpy()
    y, _, _ = ox.ox_rmsnorm(X.cuda(), eps=1e-6)
    y = y.double().cpu().numpy()
    ref = norm_plain(x, None, None, 1e-6)[1]
    ref[1] = np.where(np.isinf(x[1]), np.nan, 0.0)
    ref[4] = 0.0
    ref[6] = np.nan
    assert np.array_equal(np.isnan(y), np.isnan(ref))
    tol = (2.0 ** -18 + half_step(dtype) * 1.01) * np.abs(ref) + 2.0 ** -126
    assert (np.abs(y - ref)[~np.isnan(ref)] <= tol[~np.isnan(ref)]).all()

    q, s, _ = ox.ox_rmsnorm(X.cuda(), eps=1e-6, out="i8")
    q, s = q.cpu().numpy(), s.double().cpu().numpy()
    assert np.isnan(s[[1, 2, 6]]).all() and np.isfinite(s[[0, 3, 4, 5, 7]]).all()
    assert (q[[0, 1, 2, 4, 6]] == 0).all()
    for r in (3, 5, 7):
        m = max(np.abs(ref[r]).max(), TINY)
        assert abs(s[r] - m / 127) <= 2.0 ** -18 * m / 127 and (np.abs(127 * ref[r] / m - q[r]) <= 0.5 + 2.0 ** -13).all()

    c, s, _ = ox.ox_rmsnorm(X.cuda(), eps=1e-6, out="fp8")
    c, s = c.float().cpu().double().numpy(), s.double().cpu().numpy()
    assert np.array_equal(np.isnan(c), np.isnan(ref)) and np.isfinite(s).all() and (s > 0).all()
    for r in (0, 3, 4, 5, 7):
        for j in range(blocks(K)):
            b = ref[r, j * 128:(j + 1) * 128]
            m = max(np.abs(b).max(), TINY)
            v = 448.0 * b / m
            got = c[r, j * 128:(j + 1) * 128]
            assert ((got == round_e4m3(v * (1 - 2.0 ** -21))) | (got == round_e4m3(v * (1 + 2.0 ** -21)))).all()


@pytest.mark.parametrize("gamma", [3e38, 1e-38, 0.0, np.inf, np.nan])
def test_rmsnorm_weights_at_the_ends_of_the_range(ox, gamma):
    # y leaves fp32, or is far below a scale's least magnitude, in one column
    X = torch.ones((3, 200), device="cuda")
    X[1, 7] = 3.0
    g = torch.ones(200, device="cuda")
    g[7] = gamma
    y, _, _ = ox.ox_rmsnorm(X, g, eps=1e-6)
    q, s, _ = ox.ox_rmsnorm(X, g, eps=1e-6, out="i8")
    c, cs, _ = ox.ox_rmsnorm(X, g, eps=1e-6, out="fp8")
    want_q, want_s = quantize_plain(y.double().cpu().numpy())
    np.testing.assert_allclose(s.cpu().numpy(), want_s, rtol=2.0 ** -20)
    fin = np.where(np.isfinite(y.cpu().numpy()), y.double().cpu().numpy(), 0.0)
    m = np.maximum(np.abs(fin).max(axis=1, keepdims=True), TINY)
    assert (np.abs(127 * fin / m - q.cpu().numpy())[np.isfinite(y.cpu().numpy())] <= 0.5 + 2.0 ** -13).all()
    k, ks = ox.ox_quantize_fp8(y)
    np.testing.assert_allclose(cs.cpu().numpy(), ks.cpu().numpy(), rtol=2.0 ** -20)
    a, b = c.float().cpu().numpy(), k.float().cpu().numpy()
    assert np.array_equal(np.isnan(a), np.isnan(b))
    assert (np.abs(a - b)[~np.isnan(b)] <= np.abs(b)[~np.isnan(b)] / 8 + 2.0 ** -9).all()


# --------------------------------------------------------------- together --

def test_a_feed_forward_layer_in_int8(ox):
    """norm with residual -> int8 -> product, GELU -> int8 -> product, eager and
    replayed from a HIP graph with other inputs, against the same codes in 64 bits."""
    rng = np.random.default_rng(28)
    T, D, H = 24, 512, 1200
    W1, W2 = (torch.from_numpy(rng.standard_normal(s) * s[1] ** -0.5).bfloat16().cuda() for s in ((H, D), (D, H)))
    b1 = torch.from_numpy(rng.standard_normal(H)).bfloat16().cuda()
    g = torch.from_numpy(1 + 0.1 * rng.standard_normal(D)).bfloat16().cuda()
    w1, s1 = ox.ox_quantize_i8(W1)
    w2, s2 = ox.ox_quantize_i8(W2)
    X, R = (torch.zeros((T, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def layer():
        q, sq, total = ox.ox_rmsnorm(X, g, residual=R, out="i8")
        h = ox.ox_gemm_i8(q, sq, w1, s1, bias=b1, act="gelu")
        p, sp = ox.ox_quantize_i8(h)
        return q, sq, total, h, p, sp, ox.ox_gemm_i8(p, sp, w2, s2)

    def fill(seed):
        r = np.random.default_rng([29, seed])
        X.copy_(torch.from_numpy(r.standard_normal((T, D))))
        R.copy_(torch.from_numpy(3 * r.standard_normal((T, D))))

    def check(outs):
        q, sq, total, h, p, sp, y = outs
        check_norm(q, sq, X.double().cpu().numpy(), R.double().cpu().numpy(), g.double().cpu().numpy(), 1e-6, "i8")
        n = lambda t: t.cpu().numpy()                                          # noqa: E731
        check_product(h, n(q), n(sq), n(w1), n(s1), b1, "gelu", "first")
        want = quantize_plain(h.double().cpu().numpy())
        np.testing.assert_array_equal(n(p), want[0])
        np.testing.assert_array_equal(n(sp), want[1])
        check_product(y, n(p), n(sp), n(w2), n(s2), None, "none", "second")

    fill(0)
    check(layer())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = layer()
    for seed in (1, 2, 3):
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        eager = layer()
        for a, b in zip(held, eager):
            assert torch.equal(a, b)
        check(held)


@pytest.mark.parametrize("M,N", [(70, 66), (5, 300), (130, 130)])
def test_every_end_of_a_row(ox, M, N):
    """K that ends everywhere inside a piece of 16 bytes and a block of 128: int8
    and bf16 products of small whole numbers, exact in fp32."""
    g = torch.Generator().manual_seed(M)
    for K in list(range(1, 35)) + list(range(111, 146)) + list(range(250, 275)):
        say("row ends", M, N, K)
        A, B = (torch.randint(-9, 10, (n, K), generator=g, dtype=torch.int8) for n in (M, N))
        want = A.double() @ B.double().T
        one = [torch.ones(n, device="cuda") for n in (M, N)]
        assert torch.equal(ox.ox_gemm_i8(A.cuda(), one[0], B.cuda(), one[1], out_dtype=torch.float32).double().cpu(), want)
        off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
        Y = ox.ox_gemm_grouped(A.bfloat16().cuda(), B.bfloat16().cuda()[None], off, transB=True)
        assert torch.equal(Y.cpu(), want.bfloat16())
