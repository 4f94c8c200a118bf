"""The e4m3 and expert-grouped products and the e4m3 quantisation on the GPU
against plain 64-bit forms on the CPU.

Tolerances.  A result is an fp32 sum of K products and is rounded once to its
type.  Any order of K additions (and the two multiplications by scales) in
fp32, each off by at most 2^-23 of the partial sums (rounding or truncation
inside the matrix unit), stays within (K + 8) * 2^-23 * S of the exact sum,
S = sum |a||b| (scaled) + |bias|.  ReLU does not widen it; GELU's slope is
below 1.13 and its own evaluation is good to 2^-20 of |v|.  The last rounding
adds eps/2 of the result (bf16 2^-8, fp32 2^-24).

e4m3 operands with bf16 results run on the matrix unit's e4m3 instruction,
which adds the products of neighbouring k with 15 bits below the largest
(448*448 + 4*1 gives 448*448): 2^-15 * S more for those."""
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


# ------------------------------------------------------------- plain forms --

def blocks(n):
    return -(-n // 128)


def round_e4m3(v):
    v = np.asarray(v, np.float64)
    a = np.maximum(np.abs(v), 2.0 ** -30)
    step = np.exp2(np.maximum(np.floor(np.log2(a)), -6.0) - 3.0)
    return np.clip(np.rint(v / step) * step, -448.0, 448.0)


def quantize_plain(X, block_rows):
    """(values of the codes, scales [row blocks, k-blocks], 448 x / m) in 64 bits"""
    R, K = X.shape
    rb, kb = -(-R // block_rows), blocks(K)
    Q, S, V = np.zeros((R, K)), np.zeros((rb, kb)), np.zeros((R, K))
    for i in range(rb):
        for j in range(kb):
            at = (slice(i * block_rows, min(R, (i + 1) * block_rows)), slice(j * 128, min(K, (j + 1) * 128)))
            x = X[at]
            fin = np.isfinite(x)
            m = max(np.abs(x[fin]).max(initial=0.0), 2.0 ** -100)
            S[i, j] = np.float32(m) / np.float32(448)
            V[at] = np.where(fin, x, 0.0) * 448.0 / m
            q = round_e4m3(V[at])
            q = np.where(np.isinf(x), np.copysign(448.0, np.where(np.isnan(x), 0, x)), q)
            Q[at] = np.where(np.isnan(x), np.nan, q)
    return Q, S, V


def check_codes(got, Q, V, dtype):
    """bf16: every code.  fp32: the quotient, taken in fp32, may be off by
    2^-23 of itself, which moves a code only if a halfway point is that near."""
    got = got.float().cpu().numpy().astype(np.float64)
    if dtype == torch.float32:
        near = round_e4m3(V * (1 + 2.0 ** -23)) != round_e4m3(V * (1 - 2.0 ** -23))
        got = np.where(near & (np.abs(got - Q) <= np.abs(Q) / 7 + 2.0 ** -9), Q, got)
    np.testing.assert_array_equal(got, Q)


def act64(v, act):
    if act == "relu":
        return np.maximum(v, 0)
    if act == "relu6":
        return np.clip(v, 0, 6)
    if act == "gelu":
        return (0.5 * torch.from_numpy(v) * torch.erfc(torch.from_numpy(-v / np.sqrt(2.0)))).numpy()
    return v


def grouped_plain(A, B, off, bias, act):
    """A [T, K], B [E, N, K] float64; returns (Y, S) with S the sum of magnitudes."""
    T, N = A.shape[0], B.shape[1]
    Y, S = np.zeros((T, N)), np.zeros((T, N))
    for e in range(B.shape[0]):
        lo, hi = off[e], off[e + 1]
        b = np.zeros(N) if bias is None else bias[e]
        Y[lo:hi] = act64(A[lo:hi] @ B[e].T + b, act)
        S[lo:hi] = np.abs(A[lo:hi]) @ np.abs(B[e].T) + np.abs(b)
    return Y, S


def check(got, ref, S, K, dtype, act, what, e4m3=False):
    got = got.double().cpu().numpy()
    eps = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    tol = 1.2 * (K + 8) * 2.0 ** -23 * S + eps * np.abs(ref) + 2.0 ** -126
    if e4m3 and dtype == torch.bfloat16:
        tol = tol + 1.2 * 2.0 ** -15 * S
    if act == "gelu":
        tol = tol + 2.0 ** -20 * S
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what
    bad = np.abs(got - ref) > tol
    assert not bad.any(), "%s: %d of %d, first at %s" % (what, bad.sum(), bad.size, np.argwhere(bad)[0])


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
    """A copy of x that starts `shift` elements off an aligned address."""
    if shift == 0:
        return x.contiguous().cuda()
    size = x.element_size()
    raw = torch.empty(x.numel() + shift, dtype={1: torch.uint8, 2: torch.int16, 4: torch.int32}[size], device="cuda")
    raw[shift:] = x.contiguous().cuda().reshape(-1).view(raw.dtype)
    return raw[shift:].view(x.dtype).view(x.shape)


def f8_weights(rng, E, N, K):
    """codes [E, N, K] and scales with every magnitude that a block can have"""
    q = round_e4m3(rng.standard_normal((E, N, K)) * 60)
    s = np.exp(rng.uniform(-3, 3, (E, blocks(N), blocks(K)))).astype(np.float32)
    return q, s


def wide(q, s, br):
    full = np.repeat(np.repeat(s.astype(np.float64), br, axis=-2), 128, axis=-1)
    return q * full[..., :q.shape[-2], :q.shape[-1]]


def codes(q):
    return torch.from_numpy(q).float().to(F8)


# ------------------------------------------------------------ quantisation --

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,K,br,shift", [
    (1, 128, 1, 0), (1, 1, 1, 0), (3, 127, 1, 0), (5, 130, 1, 0), (24, 4096, 1, 0), (17, 640, 1, 0), (9, 1040, 1, 0),
    (33, 513, 1, 0), (8, 256, 1, 1), (67, 384, 1, 0), (128, 128, 128, 0), (1, 64, 128, 0), (130, 300, 128, 0),
    (257, 272, 128, 0), (64, 256, 128, 1)])
def test_quantize(ox, rows, K, br, shift, dtype):
    say("quantize", rows, K, br, shift, dtype)
    rng = np.random.default_rng([5, rows, K, br])
    X = torch.from_numpy(rng.standard_normal((rows, K)) * np.exp(rng.uniform(-20, 20, (rows, 1)))).to(dtype)
    X[0, 0] = 0.0
    Q, okq = guarded((rows, K), F8, shift)
    S, oks = guarded((blocks(K), rows) if br == 1 else (blocks(rows), blocks(K)), torch.float32)
    ox.ox_quantize_fp8(shifted(X, shift), block_rows=br, Q=Q, scales=S)
    torch.cuda.synchronize()
    okq(), oks()
    q, s, v = quantize_plain(X.double().numpy(), br)
    np.testing.assert_array_equal(S.cpu().numpy(), (s.T if br == 1 else s).astype(np.float32))
    check_codes(Q, q, v, dtype)


@pytest.mark.parametrize("br", [1, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_zeros_infinities_nans_and_tiny(ox, dtype, br):
    rng = np.random.default_rng(6)
    X = rng.standard_normal((5, 256)).astype(np.float32)
    X[0] = 0
    X[1, :128] = np.nan
    X[1, 130] = np.inf
    X[2, 3], X[2, 200], X[2, 201] = -np.inf, np.inf, np.nan
    X[3, :128] = 1e-38                       # far below 2^-100
    X[3, 128:] = 3e38
    X[4, :128] = np.inf
    if br == 128:
        X[3] = 1.0
    X = torch.from_numpy(X).to(dtype)
    Q, S = ox.ox_quantize_fp8(X.cuda(), block_rows=br)
    q, s, v = quantize_plain(X.double().numpy(), br)
    np.testing.assert_array_equal(S.cpu().numpy(), (s.T if br == 1 else s).astype(np.float32))
    check_codes(Q, q, v, dtype)
    assert np.isfinite(S.cpu().numpy()).all() and (S > 0).all().item()


def test_quantize_rounds_ties_to_even(ox):
    # 448 in the block keeps the scale at 1; the rest are halfway points and their neighbours
    x = [448.0, 17.0, 19.0, 21.0, 0.0009765625, 0.0029296875, 0.5 / 512, 1.5 / 512, 2.5 / 512, -17.0, 464.0 - 16.0, 432.0]
    X = torch.tensor([x + [0.0] * (128 - len(x))])
    Q, S = ox.ox_quantize_fp8(X.cuda())
    assert S.item() == 1.0
    np.testing.assert_array_equal(Q.float().cpu().numpy(), round_e4m3(X.numpy()))


def test_quantize_bf16_halfway_points(ox):
    # every bf16 significand under every one as the block's maximum: the halfway
    # points among their quotients go to even
    sig = torch.arange(128, 256, dtype=torch.float32)
    X = torch.cat([sig.repeat(128, 1) * 2.0 ** -7, sig.repeat(128, 1) * 2.0 ** -12], dim=1)
    X[:, 0] = sig / 32
    X[:, 128] = sig / 32
    X = X.bfloat16()
    Q, S = ox.ox_quantize_fp8(X.cuda())
    q, s, v = quantize_plain(X.double().numpy(), 1)
    step = np.exp2(np.maximum(np.floor(np.log2(np.abs(v))), -6.0) - 3.0)
    assert (np.abs(v / step - np.floor(v / step) - 0.5) == 0).sum() > 100
    check_codes(Q, q, v, torch.bfloat16)


@pytest.mark.parametrize("K", [256, 200, 1024])
def test_quantize_gathers_rows(ox, K):
    rng = np.random.default_rng(7)
    X = torch.from_numpy(rng.standard_normal((11, K))).bfloat16()
    idx = np.array([3, 3, 0, 10, -1, 11, 7, 2 ** 31 - 1, -2 ** 31, 5, 5, 1, 9, 2, 4, 6, 8], np.int64)
    Q, S = ox.ox_quantize_fp8(X.cuda(), index=torch.from_numpy(idx.astype(np.int32)).cuda())
    inside = (idx >= 0) & (idx < 11)
    rows = np.where(inside[:, None], X.double().numpy()[np.where(inside, idx, 0)], 0.0)
    q, s, v = quantize_plain(rows, 1)
    np.testing.assert_array_equal(S.cpu().numpy(), s.T.astype(np.float32))
    check_codes(Q, q, v, torch.bfloat16)


# ---------------------------------------------------------------- products --

M_N_K = [(1, 1, 1), (1, 64, 128), (2, 130, 256), (3, 17, 96), (5, 256, 1000), (16, 300, 640), (17, 128, 384), (24, 72, 2064),
         (33, 200, 77), (64, 96, 512), (100, 129, 257), (127, 256, 272), (130, 384, 400), (256, 256, 1024), (300, 520, 144),
         (513, 264, 640)]


@pytest.mark.parametrize("M,N,K", M_N_K)
@pytest.mark.parametrize("out,act,shift", [(torch.bfloat16, "none", 0), (torch.float32, "gelu", 0),
                                           (torch.bfloat16, "relu6", 1)])
def test_gemm_fp8(ox, M, N, K, out, act, shift):
    say("gemm_fp8", M, N, K, out, act, shift)
    rng = np.random.default_rng([8, M, N, K])
    qa = round_e4m3(rng.standard_normal((M, K)) * 60)
    sa = np.exp(rng.uniform(-5, 0, (M, blocks(K)))).astype(np.float32)
    qb, sb = f8_weights(rng, 1, N, K)
    bias = torch.from_numpy(rng.standard_normal(N)).to(out) if act != "none" else None
    Y, ok = guarded((M, N), out, shift)
    ox.ox_gemm_fp8(shifted(codes(qa), shift), torch.from_numpy(sa.T.copy()).cuda(), shifted(codes(qb[0]), shift),
                   torch.from_numpy(sb[0]).cuda(), bias=None if bias is None else bias.cuda(), act=act, Y=Y)
    torch.cuda.synchronize()
    ok()
    ref, S = grouped_plain(wide(qa, sa, 1), wide(qb, sb, 128), [0, M],
                           None if bias is None else bias.double().numpy()[None], act)
    check(Y, ref, S, K, out, act, (M, N, K), e4m3=True)


# rows of each expert (after `skip` rows that belong to nobody, before `tail` more)
COUNTS = {"one": ([1], 0, 0), "empty": ([0, 0, 0], 0, 5), "edges": ([0, 3, 0, 0, 1, 0], 0, 0), "all_last": ([0, 0, 40], 0, 0),
          "mixed": ([17, 0, 1, 64, 5, 33], 0, 0), "gaps": ([5, 0, 20], 3, 11), "many": ([(7 * i) % 5 for i in range(70)], 0, 0),
          "large": ([150, 2, 300, 129], 0, 0), "hundreds": ([1 if i % 3 else 0 for i in range(200)], 1, 2)}


def offsets_of(name):
    counts, skip, tail = COUNTS[name]
    off = np.concatenate([[skip], skip + np.cumsum(counts)]).astype(np.int64)
    return off, int(off[-1]) + tail


def grouped_case(ox, fmt, name, N, K, transB, act, shift, out=None):
    off, T = offsets_of(name)
    E = len(off) - 1
    rng = np.random.default_rng([9, T, E, N, K])
    offd = torch.from_numpy(off.astype(np.int32)).cuda()
    if fmt == "fp8":
        out = out or torch.bfloat16
        qa = round_e4m3(rng.standard_normal((T, K)) * 60)
        sa = np.exp(rng.uniform(-5, 0, (T, blocks(K)))).astype(np.float32)
        qb, sb = f8_weights(rng, E, N, K)
        A64, B64 = wide(qa, sa, 1), wide(qb, sb, 128)
    else:
        out = torch.bfloat16 if fmt == "bf16" else torch.float32
        A = torch.from_numpy(rng.standard_normal((T, K))).to(out)
        B = torch.from_numpy(rng.standard_normal((E, N, K) if transB else (E, K, N)) / np.sqrt(K)).to(out)
        A64, B64 = A.double().numpy(), B.double().numpy()
        if not transB:
            B64 = B64.transpose(0, 2, 1)
    bias = torch.from_numpy(rng.standard_normal((E, N))).to(out) if act != "none" else None
    Y, ok = guarded((T, N), out, shift)
    Y.fill_(float("nan"))
    bd = None if bias is None else bias.cuda()
    if fmt == "fp8":
        call = lambda: ox.ox_gemm_grouped_fp8(a8, sad, b8, sbd, offd, bias=bd, act=act, Y=Y)   # noqa: E731
        a8, sad = shifted(codes(qa), shift), torch.from_numpy(sa.T.copy()).cuda()
        b8, sbd = shifted(codes(qb), shift), torch.from_numpy(sb).cuda()
    else:
        Ad, Bd = shifted(A, shift), shifted(B, shift)
        call = lambda: ox.ox_gemm_grouped(Ad, Bd, offd, bias=bd, transB=transB, act=act, Y=Y)   # noqa: E731
    call()
    torch.cuda.synchronize()
    ok()
    ref, S = grouped_plain(A64, B64, off, None if bias is None else bias.double().numpy(), act)
    check(Y, ref, S, K, out, act, (fmt, name, N, K, transB), e4m3=fmt == "fp8")
    first = Y.clone()
    call()
    assert torch.equal(first.view(torch.uint8), Y.view(torch.uint8)), "two runs differ"


@pytest.mark.parametrize("name", list(COUNTS))
@pytest.mark.parametrize("fmt,transB", [("f32", True), ("f32", False), ("bf16", True), ("bf16", False), ("fp8", True)])
def test_grouped_offsets(ox, fmt, transB, name):
    say("grouped", fmt, transB, name)
    grouped_case(ox, fmt, name, 136, 160, transB, "gelu", 0)


@pytest.mark.parametrize("N,K,act,shift", [(64, 64, "none", 0), (1, 1, "relu", 0), (33, 70, "none", 0), (128, 129, "relu", 0),
                                           (256, 512, "none", 1), (264, 1040, "relu6", 0), (520, 208, "none", 0)])
@pytest.mark.parametrize("fmt,transB", [("f32", True), ("f32", False), ("bf16", True), ("bf16", False), ("fp8", True)])
@pytest.mark.parametrize("name", ["mixed", "large"])
def test_grouped_sizes(ox, fmt, transB, name, N, K, act, shift):
    say("grouped", fmt, transB, name, N, K, act, shift)
    grouped_case(ox, fmt, name, N, K, transB, act, shift)


def test_grouped_fp8_to_f32(ox):
    grouped_case(ox, "fp8", "mixed", 200, 384, True, "relu", 0, out=torch.float32)


def test_no_reduction_leaves_the_bias(ox):
    off = torch.tensor([1, 3], dtype=torch.int32, device="cuda")
    bias = torch.randn(1, 40, device="cuda")
    Y = ox.ox_gemm_grouped(torch.empty(4, 0, device="cuda"), torch.empty(1, 40, 0, device="cuda"), off, bias=bias, act="relu")
    want = torch.zeros(4, 40)
    want[1:3] = bias.cpu().clamp(min=0)
    assert torch.equal(Y.cpu(), want)


def test_bad_offsets_stay_inside_the_tensors(ox):
    # decreasing, negative and too large offsets: Y is undefined, its neighbours are not
    A = torch.randn(40, 64, device="cuda").bfloat16()
    B = torch.randn(5, 72, 64, device="cuda").bfloat16()
    for off in ([0, 30, 10, 50, 20, 40], [-5, 7, 7, 2 ** 31 - 1, -2 ** 31, 41], [90, 80, 70, 60, 50, 45]):
        Y, ok = guarded((40, 72), torch.bfloat16)
        ox.ox_gemm_grouped(A, B, torch.tensor(off, dtype=torch.int32, device="cuda"), Y=Y)
        torch.cuda.synchronize()
        ok()


@pytest.mark.parametrize("M", [3, 40, 300])
def test_nan_codes_reach_their_rows_and_columns_only(ox, M):
    N, K = 200, 400
    rng = np.random.default_rng(10)
    qa, (qb, sb) = round_e4m3(rng.standard_normal((M, K)) * 60), f8_weights(rng, 1, N, K)
    sa = np.exp(rng.uniform(-5, 0, (M, blocks(K)))).astype(np.float32)
    qa[M // 2, 399] = np.nan
    qb[0, 7, 130] = np.nan
    Y = ox.ox_gemm_fp8(codes(qa).cuda(), torch.from_numpy(sa.T.copy()).cuda(), codes(qb[0]).cuda(),
                       torch.from_numpy(sb[0]).cuda())
    want = np.zeros((M, N), bool)
    want[M // 2] = True
    want[:, 7] = True
    np.testing.assert_array_equal(torch.isnan(Y).cpu().numpy(), want)


def test_other_stream_and_graph_replays(ox):
    """The whole expert layer recorded once and replayed with other tokens and
    other offsets, eager work between the replays."""
    T, E, N, K = 96, 6, 256, 384
    g = torch.Generator(device="cuda").manual_seed(3)
    X = torch.randn(40, K, device="cuda", generator=g).bfloat16()
    W, W2 = (torch.randn(E, a, b, device="cuda", generator=g).bfloat16() / 16 for a, b in ((N, K), (K, N)))
    w8 = [ox.ox_quantize_fp8(W[e], block_rows=128) for e in range(E)]
    B, sb = torch.stack([q.view(torch.uint8) for q, _ in w8]).view(F8), torch.stack([s for _, s in w8])
    index = torch.zeros(T, dtype=torch.int32, device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    Q, sa = torch.empty(T, K, dtype=F8, device="cuda"), torch.empty(3, T, device="cuda")
    H, Y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda"), torch.empty(T, K, dtype=torch.bfloat16, device="cuda")

    def layer():
        ox.ox_quantize_fp8(X, index=index, Q=Q, scales=sa)
        ox.ox_gemm_grouped_fp8(Q, sa, B, sb, off, act="gelu", Y=H)
        ox.ox_gemm_grouped(H, W2, off, Y=Y)

    def fill(seed):
        r = np.random.default_rng(seed)
        index.copy_(torch.from_numpy(r.integers(0, 40, T).astype(np.int32)))
        cut = np.sort(r.integers(0, T + 1, E + 1)).astype(np.int32)
        off.copy_(torch.from_numpy(cut))

    side = torch.cuda.Stream()
    fill(0)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.synchronize()
    eager = Y.clone()
    Y.zero_()
    layer()
    torch.cuda.synchronize()
    assert torch.equal(eager, Y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    for seed in (1, 2, 3, 4):
        fill(seed)
        layer()
        torch.cuda.synchronize()
        want = Y.clone()
        Y.fill_(float("nan"))
        H.fill_(float("nan"))
        (X.float() @ W[0].float().t()).sum().item()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(want, Y), seed


# every kernel of the products, forced, on experts with full, partial and no
# tiles, a last partial block of K (fp8 368 = 2 * 128 + 112) and more blocks
# than any tile keeps in flight
VARIANTS = {"fp8": ["regs", "regs128", "stream", "32x64", "64x64", "128x128", "256x256", "32x32x4", "64x64x2", "128x128x2"],
            "fp8x": ["regs", "regs128", "stream", "32x64", "64x64", "128x128", "128x256", "32x32x4", "64x64x2", "128x128x2"],
            "bf16": ["regs", "regs128", "stream", "32x64", "64x64", "128x128", "256x128", "256x256", "32x32x4", "64x64x2",
                     "128x128x2"],
            "bf16 kn": ["regs", "regs128", "32x64", "64x64", "64x128", "128x128", "256x128", "256x256", "32x32x4", "64x64x2",
                        "128x128x2"],
            "f32": ["regs", "regs128", "stream", "32x64", "64x64", "128x128", "64x64x2"],
            "f32 kn": ["regs", "regs128", "32x64", "64x64", "128x128", "64x64x2"]}


@pytest.mark.parametrize("fmt,variant", [(f, v) for f in VARIANTS for v in VARIANTS[f]])
@pytest.mark.parametrize("name,N,K", [("large", 264, 368), ("gaps", 304, 1040), ("mixed", 40, 32)])
def test_every_variant(ox, monkeypatch, fmt, variant, name, N, K):
    say("variant", fmt, variant, name, N, K)
    monkeypatch.setenv("OX_FORCE_KERNEL", variant)
    kind = {"fp8x": "fp8", "bf16 kn": "bf16", "f32 kn": "f32"}.get(fmt, fmt)
    grouped_case(ox, kind, name, N, K, not fmt.endswith("kn"), "relu", 0, out=torch.float32 if fmt == "fp8x" else None)


def test_forced_variants_that_do_not_apply_are_refused(ox, monkeypatch):
    A, B = torch.zeros(4, 64, device="cuda"), torch.zeros(1, 64, 64, device="cuda")
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    monkeypatch.setenv("OX_FORCE_KERNEL", "256x256")           # fp32 has none
    with pytest.raises(ox.OxError):
        ox.ox_gemm_grouped(A, B, off)
    monkeypatch.setenv("OX_FORCE_KERNEL", "stream")            # [K, N] weights are not streamed
    with pytest.raises(ox.OxError):
        ox.ox_gemm_grouped(A, B, off, transB=False)


@pytest.mark.parametrize("fmt,T,E,N,K,transB", [("fp8", 700, 1, 1600, 1088, True), ("bf16", 1500, 3, 1100, 704, True),
                                                ("bf16", 1500, 3, 1104, 704, False), ("f32", 600, 2, 520, 260, True),
                                                ("fp8", 3000, 2, 2100, 520, True)])
def test_larger_problems_as_chosen(ox, fmt, T, E, N, K, transB):
    COUNTS["tmp"] = ([T // E + (7 if e == 0 else 0) for e in range(E)], 0, 3)
    say("larger", fmt, T, E, N, K, transB)
    grouped_case(ox, fmt, "tmp", N, K, transB, "none", 0)


def check_gpu(got, A, B, K, dtype):
    """check() for one expert's rows, in 64 bits on the GPU."""
    ref, S = A.double() @ B.double().t(), A.double().abs() @ B.double().abs().t()
    eps = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    bad = (got.double() - ref).abs() > 1.2 * (K + 8) * 2.0 ** -23 * S + eps * ref.abs()
    assert not bad.any().item() and not torch.isnan(got).any().item()


@pytest.mark.parametrize("rows", [1, 40])
def test_weights_past_32_bits(ox, rows):
    # 7 x 16384 x 16384 fp32 weights: the last expert starts 6.4 GB in
    E, N = 7, 16384
    say("weights past 32 bits", rows)
    B = torch.empty(E, N, N, device="cuda")
    B[0].fill_(float("nan"))
    B[E - 1].normal_()
    A = torch.randn(rows, N, device="cuda")
    off = torch.tensor([0] * E + [rows], dtype=torch.int32, device="cuda")
    Y = ox.ox_gemm_grouped(A, B, off)
    check_gpu(Y[:, :2048], A, B[E - 1, :2048], N, torch.float32)
    check_gpu(Y[:, -2048:], A, B[E - 1, -2048:], N, torch.float32)


def test_rows_past_32_bits(ox):
    # 130000 x 16384 bf16 rows (4.3 GB) quantised, and as the left operand
    T, K, N = 130000, 16384, 72
    say("rows past 32 bits")
    A = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    A[-300:].normal_()
    B = torch.randn(1, N, K, device="cuda").bfloat16()
    Y = ox.ox_gemm_grouped(A, B, torch.tensor([0, T], dtype=torch.int32, device="cuda"))
    check_gpu(Y[-300:], A[-300:], B[0], K, torch.bfloat16)
    assert (Y[:-300] == 0).all().item()
    Q, S = ox.ox_quantize_fp8(A)
    q, s = ox.ox_quantize_fp8(A[-300:].contiguous())
    assert torch.equal(Q[-300:].view(torch.uint8), q.view(torch.uint8)) and torch.equal(S[:, -300:], s)
    assert (Q[:-300].view(torch.uint8) == 0).all().item()


@pytest.mark.parametrize("tokens,experts,width,hidden", [(5, 8, 256, 512), (200, 4, 384, 1024)])
def test_example_layer(tokens, experts, width, hidden):
    # two e4m3 roundings of 2^-4 relative at most (half a step) on either side of
    # each product: independent errors of a sum average out far below the 4 * 2^-4
    # that they could reach together
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py")
    spec = importlib.util.spec_from_file_location("expert_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    off, same = mod.main(["--tokens", str(tokens), "--experts", str(experts), "--width", str(width), "--hidden", str(hidden)])
    assert same and off < 4 * 2.0 ** -4
