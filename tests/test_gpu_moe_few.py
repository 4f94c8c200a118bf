"""The routed feed-forward layer of a few tokens on the GPU against a plain
64-bit form on the CPU.

Tolerances, element by element.  A product's fp32 sum of K products is within
(K + 8) * 2^-23 * S of the exact one in any order, S the sum of magnitudes (bias
among them).  The activations' slopes are below 1.13 and their own evaluation is
good to 2^-20 of |v|; a gate times a value carries both errors.  bf16: h passes
as two bf16 numbers, off by 2^-17 of it at most.  |W2| carries the error of h to
the result, beside the second product's own.  A softmax weight is off by
2^-24 * |score - best| + 2^-21 of itself (the subtraction; exp, sum and
division).  The sum over a token's experts adds (top + 8) * 2^-23 of the
magnitudes, and the last rounding half a step of the type."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

F8 = torch.float8_e4m3fn
BF, F32 = torch.bfloat16, torch.float32


def say(*a):
    print("[case]", *a, flush=True)


@pytest.fixture(scope="module")
def ox():
    import conv_implicit_gemm_amd as ox
    return ox


def blocks(n):
    return -(-n // 128)


def act64(v, act):
    v = torch.from_numpy(v)
    if act == "relu":
        return v.clamp(min=0).numpy()
    if act == "relu6":
        return v.clamp(0, 6).numpy()
    if act == "gelu":
        return (0.5 * v * torch.erfc(-v / np.sqrt(2.0))).numpy()
    if act == "silu":
        return (v * torch.sigmoid(v)).numpy()
    return v.numpy()


def chosen_plain(scores, top, renormalise):
    """experts [T, top] and weights, by the words of the definition"""
    T, E = scores.shape
    ids, w = np.full((T, top), -1), np.zeros((T, top))
    for t in range(T):
        s = np.minimum(np.where(np.isnan(scores[t]), -np.inf, scores[t]), np.finfo(np.float32).max)
        can = [e for e in range(E) if s[e] > -np.inf]
        best = sorted(can, key=lambda e: (-s[e], e))[:top]
        if not best:
            continue
        p = np.exp(s - s[best[0]])
        ids[t, :len(best)] = best
        w[t, :len(best)] = p[best] / (p[best].sum() if renormalise else p[can].sum())
    return ids, w


class Layer:
    """Operands on the GPU, and their values in 64 bits."""

    def __init__(self, seed, t, E, D, H, gated, bias, shift=0):
        rng = np.random.default_rng([31, seed])
        wide = 2 * H if gated else H
        self.E, self.D, self.H, self.gated = E, D, H, gated
        self.t = F32 if t == "f32" else BF
        self.scales = [None, None]
        self.W, self.w64 = [], []
        for i, (r, c) in enumerate(((wide, D), (D, H))):
            w = torch.from_numpy(rng.standard_normal((E, r, c)) * max(1, c) ** -0.5)
            if t == "fp8":
                s = torch.from_numpy(np.exp(rng.uniform(-4, -2, (E, blocks(r), blocks(c))))).float()
                q = (w * 60).float().to(F8)
                full = s.double().repeat_interleave(128, dim=1).repeat_interleave(128, dim=2)[:, :r, :c]
                self.scales[i] = s.cuda()
                self.W.append(shifted(q, shift))
                self.w64.append((q.double() * full).numpy())
            else:
                w = w.to(self.t)
                self.W.append(shifted(w, shift))
                self.w64.append(w.double().numpy())
        self.b = [torch.from_numpy(rng.standard_normal((E, n))).to(self.t).cuda() if bias else None for n in (wide, D)]
        self.b64 = [b.double().cpu().numpy() if b is not None else np.zeros((E, n)) for b, n in zip(self.b, (wide, D))]
        self.rng = rng

    def plain(self, X, ids, w, scores, act):
        """(Y, how far the kernel's may be before its last rounding)"""
        T, D = X.shape
        Y, tol = np.zeros((T, D)), np.zeros((T, D))
        for t in range(T):
            for e, wt in zip(ids[t], w[t]):
                if e < 0:
                    continue
                W1, W2, b1, b2 = self.w64[0][e], self.w64[1][e], self.b64[0][e], self.b64[1][e]
                v = W1 @ X[t] + b1
                dv = (D + 8) * 2.0 ** -23 * (np.abs(W1) @ np.abs(X[t]) + np.abs(b1))
                if self.gated:
                    g, u, dg, du = v[:self.H], v[self.H:], dv[:self.H], dv[self.H:]
                    ag = act64(g, act)
                    dag = 1.13 * dg + 2.0 ** -20 * np.abs(g)
                    h = ag * u
                    dh = np.abs(u) * dag + np.abs(ag) * du + dag * du + 2.0 ** -24 * np.abs(h)
                else:
                    h = act64(v, act)
                    dh = 1.13 * dv + 2.0 ** -20 * np.abs(v)
                if self.t is BF:
                    dh = dh + 2.0 ** -17 * (np.abs(h) + dh)
                y = W2 @ h + b2
                mag = np.abs(W2) @ np.abs(h) + np.abs(b2)
                dy = np.abs(W2) @ dh + (self.H + 8) * 2.0 ** -23 * mag
                best = np.max(np.where(np.isnan(scores[t]), -np.inf, scores[t]))
                rel = 2.0 ** -24 * abs(best - scores[t][e]) + 2.0 ** -21 if np.isfinite(best) else 2.0 ** -21
                Y[t] += wt * y
                tol[t] += wt * (dy + (rel + (len(ids[t]) + 8) * 2.0 ** -23) * (mag + dy))
        return Y, tol

    def check(self, got, X, ids, w, scores, act, what):
        ref, tol = self.plain(X, ids, w, scores, act)
        half = torch.finfo(self.t).eps / 2
        tol = 1.02 * tol + half * (np.abs(ref) + tol) * 1.01 + 2.0 ** -126
        got = got.double().cpu().numpy()
        bad = ~(np.abs(got - ref) <= tol)
        assert not bad.any(), "%s: %d of %d, first at %s" % (what, bad.sum(), bad.size, np.argwhere(bad)[0])


def shifted(x, shift):
    """A copy of x on the GPU that starts `shift` elements off an aligned address."""
    if shift == 0:
        return x.contiguous().cuda()
    size = x.element_size()
    raw = torch.empty(x.numel() + shift, dtype={1: torch.uint8, 2: torch.int16, 4: torch.int32}[size], device="cuda")
    raw[shift:] = x.contiguous().cuda().reshape(-1).view(raw.dtype)
    return raw[shift:].view(x.dtype).view(x.shape)


def guarded(shape, dtype, shift=0):
    n = int(np.prod(shape))
    whole = torch.full((n + 512 + shift,), 77, dtype=dtype, device="cuda")

    def intact():
        assert (whole[:256 + shift] == 77).all().item() and (whole[256 + shift + n:] == 77).all().item()
    return whole[256 + shift:256 + shift + n].view(shape), intact


def scratch(ox, T, D, H, E, top):
    """A workspace of exactly the bytes asked for, full of NaN, before a guard."""
    n = ox.ox_moe_few_workspace_bytes(T, D, H, E, top)
    assert n > 0
    whole = torch.full((n + 256,), 255, dtype=torch.uint8, device="cuda")

    def intact():
        assert (whole[n:] == 255).all().item()
    return whole[:n], intact


def run_case(ox, layer, T, top, act, scores, renormalise=True, shift=0, what=None):
    X = torch.from_numpy(layer.rng.standard_normal((T, layer.D))).to(layer.t)
    ids, w = chosen_plain(scores.double().numpy(), top, renormalise)
    Y, oky = guarded((T, layer.D), layer.t, shift)
    E, oke = guarded((T, top), torch.int32)
    W, okw = guarded((T, top), F32)
    ws, oks = scratch(ox, T, layer.D, layer.H, layer.E, top)
    out = ox.ox_moe_few(shifted(X, shift), scores.cuda(), layer.W[0], layer.W[1], top, w1_scales=layer.scales[0],
                        w2_scales=layer.scales[1], b1=layer.b[0], b2=layer.b[1], act=act, gated=layer.gated,
                        renormalise=renormalise, Y=Y, experts=E, weights=W, workspace=ws)
    torch.cuda.synchronize()
    assert out is Y
    for ok in (oky, oke, okw, oks):
        ok()
    np.testing.assert_array_equal(E.cpu().numpy(), ids)
    s = scores.double().numpy()
    far = np.nanmax(np.where(np.isfinite(s), s, np.nan)) - np.nanmin(np.where(np.isfinite(s), s, np.nan))
    np.testing.assert_allclose(W.double().cpu().numpy(), w, rtol=2.0 ** -24 * far + 2.0 ** -21, atol=1e-37)
    layer.check(Y, X.double().numpy(), ids, w, s, act, what)
    return X, Y


#        T, E, top, D, H
SIZES = [(1, 1, 1, 1, 1), (1, 8, 2, 64, 128), (2, 4, 4, 100, 33), (3, 8, 2, 129, 257), (5, 70, 3, 256, 96), (8, 16, 8, 320, 200),
         (13, 8, 2, 250, 490), (16, 2, 1, 1000, 72), (17, 3, 3, 130, 300), (33, 130, 2, 72, 40), (40, 2, 2, 144, 512),
         (64, 4, 2, 384, 160), (64, 300, 16, 40, 24), (64, 1, 1, 65, 129), (7, 512, 5, 16, 16)]


@pytest.mark.parametrize("t", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("gated,act,bias,shift", [(True, "silu", False, 0), (False, "gelu", True, 1), (True, "gelu", True, 0),
                                                  (False, "relu6", False, 3)])
@pytest.mark.parametrize("T,E,top,D,H", SIZES)
def test_layer(ox, T, E, top, D, H, gated, act, bias, shift, t):
    say("moe_few", T, E, top, D, H, gated, act, bias, shift, t)
    layer = Layer([T, E, D, H], t, E, D, H, gated, bias, shift)
    scores = torch.from_numpy(2 * layer.rng.standard_normal((T, E)))
    run_case(ox, layer, T, top, act, scores.to(F32 if gated else BF), renormalise=bias, shift=shift, what=(T, E, top, D, H, t))


@pytest.mark.parametrize("T", [6, 40])
@pytest.mark.parametrize("renormalise", [True, False])
def test_masks_ties_infinities_and_nans_among_the_scores(ox, T, renormalise):
    E, top = 12, 3
    layer = Layer(1, "bf16", E, 72, 48, True, True)
    scores = torch.from_numpy(layer.rng.standard_normal((T, E))).float()
    inf, nan = float("inf"), float("nan")
    scores[0] = -inf                                     # no expert: zeros
    scores[1] = nan                                      # likewise
    scores[2] = -inf
    scores[2, 5] = -3e38                                 # one
    scores[3] = 0.5                                      # ties: the lowest
    scores[3, 0], scores[3, 2] = -inf, nan
    scores[4, 7], scores[4, 3] = inf, inf                # two infinities share
    scores[5] = torch.tensor([0.0, -0.0] * (E // 2))     # one value
    X, Y = run_case(ox, layer, T, top, "silu", scores, renormalise=renormalise)
    assert (Y[:2] == 0).all().item()


def test_a_batch_without_any_expert_is_zeros(ox):
    layer = Layer(2, "fp8", 9, 130, 40, True, True)
    _, Y = run_case(ox, layer, 5, 2, "silu", torch.full((5, 9), float("-inf")).index_fill_(0, torch.tensor([4]), 0.0))
    assert (Y[:4] == 0).all().item()
    Y = ox.ox_moe_few(torch.ones((5, 130), dtype=BF, device="cuda"), torch.full((5, 9), float("nan"), device="cuda"), layer.W[0],
                      layer.W[1], 2, w1_scales=layer.scales[0], w2_scales=layer.scales[1], b1=layer.b[0], b2=layer.b[1])
    assert (Y == 0).all().item()


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["relu", "none"])
@pytest.mark.parametrize("T", [4, 24])
def test_infinities_and_nans_stay_with_their_tokens(ox, t, T, act):
    """Weights of one expert and the row of one token that are not finite (ReLU
    takes a NaN to 0, as in every call of the library)."""
    E, D, H = 4, 100, 60
    layer = Layer(3, t, E, D, H, False, False)
    layer.W[0][1], layer.W[1][1] = float("inf"), float("nan")
    layer.W[1][2, 7] = float("inf")
    X = torch.from_numpy(np.abs(layer.rng.standard_normal((T, D)))).to(layer.t)
    X[3] = float("nan")
    scores = torch.full((T, E), float("-inf"))
    for i in range(T):
        scores[i, (0, 1, 2, 0)[i % 4]] = 0.0
    Y = ox.ox_moe_few(X.cuda(), scores.cuda(), layer.W[0], layer.W[1], 1, act=act, gated=False).float().cpu()
    finite = [i for i in range(T) if i % 4 in (0, 3) and i != 3]
    assert torch.isfinite(Y[finite]).all() and torch.isnan(Y[1::4]).all()
    assert torch.isnan(Y[3]).all() if act == "none" else (Y[3] == 0).all()
    assert not torch.isfinite(Y[2::4, 7]).any() and torch.isfinite(Y[2::4, [c for c in range(D) if c != 7]]).all()


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_hidden_values_at_the_ends_of_the_range(ox, t):
    """h infinite, or above what bf16 holds: infinities, not NaN."""
    E, D, H = 1, 32, 16
    layer = Layer(4, t, E, D, H, False, False)
    layer.W[0].zero_()
    layer.W[0][0, :, 0] = 1.0
    layer.W[1].fill_(0.5)
    X = torch.zeros((3, D), dtype=layer.t)
    X[0, 0], X[1, 0], X[2, 0] = float("inf"), 3e38, 2.0
    Y = ox.ox_moe_few(X.cuda(), torch.zeros((3, 1), device="cuda"), layer.W[0], layer.W[1], 1, act="none", gated=False)
    assert (Y[:2] == float("inf")).all().item() and (Y[2] == 16.0).all().item()


def test_no_hidden_columns_leave_the_biases(ox):
    b2 = torch.arange(20, dtype=F32, device="cuda").view(2, 10)
    W1, W2 = torch.empty((2, 0, 10), device="cuda"), torch.empty((2, 10, 0), device="cuda")
    scores = torch.tensor([[0.0, -1e30], [-1e30, 0.0]], device="cuda")
    Y = ox.ox_moe_few(torch.ones((2, 10), device="cuda"), scores, W1, W2, 1, b2=b2, act="relu", gated=False)
    assert torch.equal(Y, b2)


def test_results_do_not_depend_on_what_ran_before(ox):
    """One workspace for calls of different sizes, in turn; the same bits each time."""
    ws = torch.full((8 << 20,), 255, dtype=torch.uint8, device="cuda")
    cases = []
    for seed, (T, E, top, D, H) in enumerate([(64, 8, 2, 512, 256), (1, 8, 2, 1024, 640), (20, 32, 4, 300, 100)]):
        layer = Layer([5, seed], "bf16", E, D, H, True, True)
        cases.append((layer, top, torch.from_numpy(layer.rng.standard_normal((T, D))).bfloat16().cuda(),
                      torch.from_numpy(layer.rng.standard_normal((T, E))).float().cuda()))

    def call(c):
        layer, top, X, scores = c
        return ox.ox_moe_few(X, scores, layer.W[0], layer.W[1], top, b1=layer.b[0], b2=layer.b[1], workspace=ws)
    first = [call(c) for c in cases]
    for _ in range(5):
        for c, y in zip(cases, first):
            assert torch.equal(call(c), y)


def test_a_decoding_step_norm_router_experts(ox):
    """ox_rmsnorm -> the router's ox_gemm_fused -> ox_moe_few, eager and replayed
    from a HIP graph with other inputs (a padded place among them)."""
    T, E, top, D, H = 12, 16, 2, 256, 320
    layer = Layer(6, "fp8", E, D, H, True, False)
    rng = layer.rng
    g = torch.from_numpy(1 + 0.1 * rng.standard_normal(D)).bfloat16().cuda()
    router = torch.from_numpy(rng.standard_normal((E, D)) * D ** -0.5).bfloat16().cuda()
    X, R = (torch.zeros((T, D), dtype=BF, device="cuda") for _ in range(2))
    pad = torch.zeros((T, 1), device="cuda")
    ws = torch.empty(ox.ox_moe_few_workspace_bytes(T, D, H, E, top), dtype=torch.uint8, device="cuda")

    def step():
        y, _, total = ox.ox_rmsnorm(X, g, residual=R)
        scores = ox.ox_gemm_fused(y, router, transB=True).float() + pad
        ids, w = torch.empty((T, top), dtype=torch.int32, device="cuda"), torch.empty((T, top), device="cuda")
        out = ox.ox_moe_few(y, scores, layer.W[0], layer.W[1], top, w1_scales=layer.scales[0], w2_scales=layer.scales[1],
                            experts=ids, weights=w, workspace=ws)
        return y, total, scores, ids, w, out

    def fill(seed):
        r = np.random.default_rng([32, seed])
        X.copy_(torch.from_numpy(r.standard_normal((T, D))))
        R.copy_(torch.from_numpy(r.standard_normal((T, D))))
        pad.zero_()
        pad[T - seed:] = float("-inf")

    def check(outs):
        y, total, scores, ids, w, out = (o.cpu() for o in outs)
        s = scores.double().numpy()
        want = chosen_plain(s, top, True)
        np.testing.assert_array_equal(ids.numpy(), want[0])
        layer.check(out, y.double().numpy(), want[0], want[1], s, "silu", "step")

    fill(0)
    check(step())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in (1, 2, 3, 4):
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        check(held)
        for a, b in zip(held, step()):
            assert torch.equal(a, b)
        assert (held[-1][T - seed:] == 0).all().item()


def test_on_another_stream(ox):
    layer = Layer(7, "bf16", 8, 512, 512, True, False)
    X = torch.from_numpy(layer.rng.standard_normal((9, 512))).bfloat16().cuda()
    scores = torch.from_numpy(layer.rng.standard_normal((9, 8))).float().cuda()
    want = ox.ox_moe_few(X, scores, layer.W[0], layer.W[1], 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    Y, ws = torch.empty_like(X), torch.empty(ox.ox_moe_few_workspace_bytes(9, 512, 512, 8, 2), dtype=torch.uint8, device="cuda")
    ox.ox_moe_few(X, scores, layer.W[0], layer.W[1], 2, Y=Y, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(Y, want)


@pytest.mark.parametrize("t,H,shift", [("bf16", 512, 0), ("fp8", 1000, 3), ("f32", 250, 0)])
def test_wide_rows_of_many_tokens(ox, t, H, shift):
    """Many steps to every wave of the second product: its other tile, with a last
    one of three columns, and an expert with more tokens than one pass takes."""
    T, E, top, D = 40, 8, 2, 8195
    say("moe_few wide", t, H, shift)
    layer = Layer([8, H], t, E, D, H, False, True, shift)
    scores = torch.from_numpy(layer.rng.standard_normal((T, E))).float()
    scores[:36, 5] += 9.0
    run_case(ox, layer, T, top, "relu", scores, shift=shift, what=("wide", t))


def test_weights_behind_four_gigabytes(ox):
    """The last of 130 experts, 4.5 GB behind the first, has the bits it has alone."""
    E, D, H = 130, 4096, 4224
    g = torch.Generator(device="cuda").manual_seed(9)
    W1 = torch.empty((E, H, D), dtype=BF, device="cuda")
    W2 = torch.empty((E, D, H), dtype=BF, device="cuda")
    for w in (W1, W2):
        w[0].zero_()
        w[E - 1].normal_(0, 0.02, generator=g)
    X = torch.randn((1, D), generator=g, device="cuda").bfloat16()
    scores = torch.full((1, E), float("-inf"), device="cuda")
    scores[0, E - 1] = 1.0
    Y = ox.ox_moe_few(X, scores, W1, W2, 1, act="silu", gated=False)
    alone = ox.ox_moe_few(X, torch.ones((1, 1), device="cuda"), W1[E - 1:], W2[E - 1:], 1, act="silu", gated=False)
    assert torch.equal(Y, alone) and (Y != 0).any().item()


def test_two_streams_at_once_with_a_workspace_each(ox):
    layer = Layer(10, "bf16", 16, 1024, 512, True, False)
    X = [torch.from_numpy(layer.rng.standard_normal((t, 1024))).bfloat16().cuda() for t in (30, 7)]
    scores = [torch.from_numpy(layer.rng.standard_normal((len(x), 16))).float().cuda() for x in X]
    want = [ox.ox_moe_few(x, s, layer.W[0], layer.W[1], 4) for x, s in zip(X, scores)]
    streams = [torch.cuda.Stream() for _ in X]
    ws = [torch.empty(ox.ox_moe_few_workspace_bytes(len(x), 1024, 512, 16, 4), dtype=torch.uint8, device="cuda") for x in X]
    Y = [[torch.empty_like(x) for _ in range(20)] for x in X]
    torch.cuda.synchronize()
    for i in range(20):
        for x, s, w, y, st in zip(X, scores, ws, Y, streams):
            ox.ox_moe_few(x, s, layer.W[0], layer.W[1], 4, Y=y[i], workspace=w, stream=st)
    torch.cuda.synchronize()
    for ys, y in zip(Y, want):
        assert all(torch.equal(one, y) for one in ys)


def test_the_result_in_place_of_the_tokens(ox):
    layer = Layer(11, "fp8", 6, 200, 90, True, True)
    X = torch.from_numpy(layer.rng.standard_normal((18, 200))).bfloat16().cuda()
    scores = torch.from_numpy(layer.rng.standard_normal((18, 6))).float().cuda()

    def call(x, y):
        return ox.ox_moe_few(x, scores, layer.W[0], layer.W[1], 2, w1_scales=layer.scales[0], w2_scales=layer.scales[1],
                             b1=layer.b[0], b2=layer.b[1], Y=y)
    want = call(X, None)
    assert torch.equal(call(X, X), want) and torch.equal(X, want)


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("T", [2, 64])
def test_the_widest_layers(ox, T, t):
    """D, then H, at their limit of 2^22, with values whose sums are exact in
    fp32 in any order (multiples of 2^-20 below 2^3) and results exact in bf16."""
    n, few = 1 << 22, 8
    x = torch.ones((T, 1), dtype=t, device="cuda")
    x[1::2] = 2.0
    route = torch.zeros((T, 1), device="cuda")
    say("moe_few widest", T, t)
    W1 = torch.full((1, few, n), 2.0 ** -20, dtype=t, device="cuda")      # h = x
    W1[..., 1::2] = 0
    W1 *= 0.5
    W2 = torch.zeros((1, n, few), dtype=t, device="cuda")
    d = torch.arange(n, device="cuda") % 7
    W2[0, :, 3] = d.to(t)
    Y = ox.ox_moe_few(x.expand(T, n).contiguous(), route, W1, W2, 1, act="none", gated=False)
    assert torch.equal(Y.float(), x.float() * d.float())
    W1 = torch.zeros((1, n, few), dtype=t, device="cuda")
    W1[0, :, 5] = (torch.arange(n, device="cuda") % 2).to(t)
    W2 = torch.full((1, few, n), 2.0 ** -20, dtype=t, device="cuda")      # 2^21 of them are met
    Y = ox.ox_moe_few(x.expand(T, few).contiguous(), route, W1, W2, 1, act="none", gated=False)
    assert torch.equal(Y, (2 * x).expand(T, few))
