"""Cases and plain forms of the RMS norm with 8-bit results, the int8 product
with scales found at run time, and the routed feed-forward layer of a few
tokens: what is measured, with real sizes, and what each result is.

Four operators of the package are called here:

  ox_rmsnorm      s = x + residual, y = s / sqrt(mean(s^2) + eps) * gamma, as
                  the type of x, as e4m3 codes with a scale per 1 x 128 block
                  (scales [ceil(K/128), rows]) or as int8 codes with a scale
                  per row; s comes back too, for the next residual
  ox_quantize_i8  int8 codes and one fp32 scale per row
  ox_gemm_i8      Y = act(a_scales[m] * b_scales[n] * (A B^T)[m, n] + bias[n])
  ox_moe_few      router scores -> the best experts of each token -> their
                  (gated) feed-forward layers -> the weighted sum, for up to 64
                  tokens

Where ``own`` is false, ``run`` computes the same in elementary torch
operations.  int8 codes of a norm go straight on to the product (``norm_i8``):
what comes back there is the product.
"""
import math

import torch

own = False

BLOCK = 128          # elements along K (and weight rows) that share an e4m3 scale
E4M3_MAX = 448.0
TINY = 2.0 ** -100   # the largest magnitude of a block or row is taken to be at least this
EPS = 1e-6
F8 = torch.float8_e4m3fn
F32_MAX = 3.4028234663852886e38
SCRATCH = 64 << 20   # bytes of the scratch memory that a serving program keeps for its calls


def listed():
    return [
        # 24 decoding requests between two layers: residual, norm, e4m3 rows for the next product
        dict(name="norm_rows24", op="norm", t="bf16", rows=24, K=4096, residual=True, out="fp8"),
        # a prompt's 8192 tokens, the same
        dict(name="norm_prompt", op="norm", t="bf16", rows=8192, K=4096, residual=True, out="fp8"),
        # 24 decoding requests of an int8 model: residual, norm, int8 rows, and the product that reads them
        dict(name="norm_i8_rows24", op="norm_i8", rows=24, K=1024, N=4096, residual=True, bias=True, act="gelu"),
        # the hidden rows of 24 decoding requests
        dict(name="quant_rows24", op="quantize_i8", t="bf16", rows=24, K=4096),
        # a prompt's hidden rows
        dict(name="quant_prompt", op="quantize_i8", t="bf16", rows=8192, K=8192),
        # one token through a 4096 x 4096 layer: a serving step of batch 1
        dict(name="i8_row1", op="gemm_i8", M=1, N=4096, K=4096, out="bf16", bias=False, act="none"),
        # a prompt of 1000 tokens, odd sizes, fp32 results (a head's logits)
        dict(name="i8_odd1000", op="gemm_i8", M=1000, N=1000, K=2000, out="f32", bias=True, act="none"),
        # a long prompt (or a batch of them): the compute-bound end
        dict(name="i8_8192", op="gemm_i8", M=8192, N=8192, K=8192, out="bf16", bias=False, act="none"),
        # one decoding token, 2 of 8 large experts
        dict(name="moe_row1", op="moe", t="bf16", T=1, E=8, top=2, D=1024, H=4096, gated=True, act="silu", bias=False, pad=0),
        # 8 decoding tokens, 8 of 128 small experts each, e4m3 weights
        dict(name="moe_rows8_fp8", op="moe", t="fp8", T=8, E=128, top=8, D=2048, H=1024, gated=True, act="silu", bias=False, pad=0),
        # 64 decoding tokens, 8 of 64 experts each: every expert is read
        dict(name="moe_rows64", op="moe", t="bf16", T=64, E=64, top=8, D=2048, H=1024, gated=True, act="silu", bias=False, pad=0),
        # an fp32 model with biases and odd widths, a batch of 13 whose last two places are empty
        dict(name="moe_f32_odd", op="moe", t="f32", T=13, E=8, top=2, D=1000, H=1998, gated=False, act="gelu", bias=True, pad=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _length(rng, lo, hi):
    """A length along N or K: whole blocks, whole 16-byte pieces, or any."""
    n = _log(rng, lo, hi)
    way = rng.random()
    if way < 0.5:
        return min(hi, max(lo, (n + 64) // 128 * 128))
    if way < 0.8:
        return min(hi, max(lo, (n + 8) // 16 * 16))
    return n


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_i8", "quantize_i8", "gemm_i8", "gemm_i8", "moe", "moe", "moe"])
    if op == "norm":
        return dict(op=op, t=rng.choice(["bf16", "bf16", "f32"]), rows=_log(rng, 1, 8192), K=_length(rng, 64, 8192),
                    residual=rng.random() < 0.7, out=rng.choice(["fp8", "fp8", "same"]))
    if op == "norm_i8":
        return dict(op=op, rows=_log(rng, 1, 2048), K=_length(rng, 64, 8192), N=_length(rng, 64, 4096),
                    residual=rng.random() < 0.7, bias=rng.random() < 0.5, act=rng.choice(["none", "relu", "gelu"]))
    if op == "quantize_i8":
        return dict(op=op, t=rng.choice(["bf16", "bf16", "f32"]), rows=_log(rng, 1, 8192), K=_length(rng, 64, 8192))
    if op == "gemm_i8":
        return dict(op=op, M=_log(rng, 1, 8192), N=_length(rng, 64, 8192), K=_length(rng, 64, 8192),
                    out=rng.choice(["bf16", "bf16", "f32"]), bias=rng.random() < 0.5,
                    act=rng.choice(["none", "relu", "gelu"]))
    t = rng.choice(["bf16", "fp8", "f32"])
    gated = rng.random() < 0.7
    E, D, H = _log(rng, 2, 128), _length(rng, 64, 4096), _length(rng, 64, 4096)
    while E > 2 and E * D * H * (3 if gated else 2) > (1 << 28 if t != "f32" else 1 << 26):   # weights: 512 MB in bf16 at most
        E = E // 2
    T = _log(rng, 1, 64)
    return dict(op=op, t=t, T=T, E=E, top=min(E, rng.choice([1, 2, 2, 4, 6, 8])), D=D, H=H, gated=gated,
                act=rng.choice(["silu", "silu", "gelu"] if gated else ["gelu", "relu", "silu"]),
                bias=rng.random() < 0.3, pad=T // 8 if rng.random() < 0.3 else 0)


def _blocks(n):
    return -(-n // BLOCK)


def _quantize_f8(X, block_rows):
    """(codes, scales [row blocks, k-blocks]) of a 2-D tensor, in 64 bits."""
    X = X.double()
    R, K = X.shape
    rb, kb = -(-R // block_rows), _blocks(K)
    P = torch.nn.functional.pad(X, (0, kb * BLOCK - K, 0, rb * block_rows - R)).reshape(rb, block_rows, kb, BLOCK)
    m = P.abs().amax(dim=(1, 3), keepdim=True).clamp(min=TINY)
    q = (P * (E4M3_MAX / m)).to(F8).reshape(rb * block_rows, kb * BLOCK)[:R, :K]
    return q.contiguous(), (m / E4M3_MAX).float().view(rb, kb)


def _quantize_i8(X):
    """(codes, scales [rows]) in 64 bits: a value next to a border has to fall on its side."""
    X = X.double()
    m = X.abs().amax(dim=1, keepdim=True).clamp(min=TINY)
    return torch.round(X * 127.0 / m).to(torch.int8), (m / 127.0).float().view(-1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda") * std

    def activations(rows, K):
        # a few channels are much larger than the rest, as in trained models
        big = 1.0 + 15.0 * (torch.rand((1, K), generator=g, device="cuda") < 0.01)
        return normal(rows, K) * big

    def empty(*shape, dtype):
        return torch.empty(shape, dtype=dtype, device="cuda")

    s = dict(case=dict(case))
    op = case["op"]
    if op in ("norm", "norm_i8"):
        R, K = case["rows"], case["K"]
        t = torch.float32 if case.get("t") == "f32" else torch.bfloat16
        # (the stream that the layers add to is the larger of the two)
        s["X"] = normal(R, K).to(t) if case["residual"] else activations(R, K).to(t)
        s["residual"] = activations(R, K).to(t) if case["residual"] else None
        s["S"] = empty(R, K, dtype=t) if case["residual"] else None
        s["gamma"] = (1.0 + normal(K, std=0.2)).to(t)
        out = case.get("out", "i8")
        s["Y"] = empty(R, K, dtype=F8 if out == "fp8" else torch.int8 if out == "i8" else t)
        s["scales"] = empty(_blocks(K), R, dtype=torch.float32) if out == "fp8" else empty(R, dtype=torch.float32) if out == "i8" else None
        if op == "norm_i8":
            N = case["N"]
            s["B"], s["b_scales"] = _quantize_i8(normal(N, K, std=K ** -0.5))
            s["bias"] = normal(N).bfloat16() if case["bias"] else None
            s["Z"] = empty(R, N, dtype=torch.bfloat16)
        return s
    if op == "quantize_i8":
        R, K = case["rows"], case["K"]
        s["X"] = activations(R, K).to(torch.bfloat16 if case["t"] == "bf16" else torch.float32)
        s["Q"], s["scales"] = empty(R, K, dtype=torch.int8), empty(R, dtype=torch.float32)
        return s
    if op == "gemm_i8":
        M, N, K = case["M"], case["N"], case["K"]
        s["A"], s["a_scales"] = _quantize_i8(activations(M, K))
        s["B"], s["b_scales"] = _quantize_i8(normal(N, K, std=K ** -0.5))
        t = torch.bfloat16 if case["out"] == "bf16" else torch.float32
        s["bias"] = normal(N).to(t) if case["bias"] else None
        s["Y"] = empty(M, N, dtype=t)
        return s
    T, E, D, H, top = case["T"], case["E"], case["D"], case["H"], case["top"]
    t = torch.float32 if case["t"] == "f32" else torch.bfloat16
    wide = 2 * H if case["gated"] else H
    s["X"] = activations(T, D).to(t)
    s["scores"] = normal(T, E)                       # the router's product, in fp32
    if case["pad"]:
        s["scores"][T - case["pad"]:] = -math.inf    # places without a request: no expert is to run for them
    s["W1_scales"] = s["W2_scales"] = None
    for name, rows, cols in (("W1", wide, D), ("W2", D, H)):
        if case["t"] == "fp8":
            s[name] = empty(E, rows, cols, dtype=F8)
            s[name + "_scales"] = empty(E, _blocks(rows), _blocks(cols), dtype=torch.float32)
            for e in range(E):
                s[name][e], s[name + "_scales"][e] = _quantize_f8(normal(rows, cols, std=cols ** -0.5), BLOCK)
        else:
            s[name] = normal(E, rows, cols, std=cols ** -0.5).to(t)
    s["b1"] = normal(E, wide, std=0.1).to(t) if case["bias"] else None
    s["b2"] = normal(E, D, std=0.1).to(t) if case["bias"] else None
    s["Y"], s["experts"], s["weights"] = empty(T, D, dtype=t), empty(T, top, dtype=torch.int32), empty(T, top, dtype=torch.float32)
    s["workspace"] = empty(SCRATCH, dtype=torch.uint8)
    return s


def _act(v, act):
    if act == "relu":
        return v.clamp(min=0)
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * 0.7071067811865476))
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    return v


def _norm(s):
    """(the sum in fp32, its norm in fp32)"""
    v = s["X"].float()
    if s["residual"] is not None:
        v = v + s["residual"].float()
    return v, v * torch.rsqrt((v * v).mean(dim=1, keepdim=True) + EPS) * s["gamma"].float()


def _product(A, a_scales, B, b_scales, bias, act, t):
    Y = torch.mm(A.float(), B.float().t()) * a_scales[:, None] * b_scales[None, :]
    if bias is not None:
        Y = Y + bias.float()
    return _act(Y, act).to(t)


def _moe_plain(s, case):
    T, E, top = case["T"], case["E"], case["top"]
    score = s["scores"].float()
    score = torch.where(score == score, score, torch.full_like(score, -math.inf)).clamp(max=F32_MAX)
    order = torch.argsort(score, dim=1, descending=True, stable=True)[:, :top]      # ties: the lowest index
    best = torch.gather(score, 1, order)
    chosen = best > -math.inf
    p = torch.where(chosen, torch.exp(best - best[:, :1].clamp(min=-F32_MAX)), torch.zeros_like(best))
    weights = torch.where(chosen, p / p.sum(dim=1, keepdim=True), torch.zeros_like(p))
    share = torch.zeros((T, E), device="cuda").scatter_(1, order, weights)          # [T, E]
    W1, W2 = s["W1"].float(), s["W2"].float()
    if case["t"] == "fp8":
        W1, W2 = W1 * _spread(s["W1_scales"], W1), W2 * _spread(s["W2_scales"], W2)
    # every expert for every token: with few tokens the weights are what counts
    h = torch.bmm(W1, s["X"].float().t().expand(E, -1, -1).contiguous())            # [E, wide, T]
    if s["b1"] is not None:
        h = h + s["b1"].float().unsqueeze(2)
    h = _act(h[:, :case["H"]], case["act"]) * h[:, case["H"]:] if case["gated"] else _act(h, case["act"])
    y = torch.bmm(W2, h)                                                            # [E, D, T]
    if s["b2"] is not None:
        y = y + s["b2"].float().unsqueeze(2)
    Y = (y * share.t().unsqueeze(1)).sum(dim=0).t().contiguous()
    return Y.to(s["Y"].dtype), torch.where(chosen, order, torch.full_like(order, -1)).to(torch.int32), weights


def _spread(scales, W):
    full = scales.repeat_interleave(BLOCK, dim=1).repeat_interleave(BLOCK, dim=2)
    return full[:, :W.shape[1], :W.shape[2]]


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import conv_implicit_gemm_amd as ox
        if op == "norm":
            return ox.ox_rmsnorm(s["X"], s["gamma"], residual=s["residual"], eps=EPS, out=case["out"], Y=s["Y"],
                                 scales=s["scales"], S=s["S"])
        if op == "norm_i8":
            q, scales, total = ox.ox_rmsnorm(s["X"], s["gamma"], residual=s["residual"], eps=EPS, out="i8", Y=s["Y"],
                                             scales=s["scales"], S=s["S"])
            return ox.ox_gemm_i8(q, scales, s["B"], s["b_scales"], bias=s["bias"], act=case["act"], Y=s["Z"]), scales, total
        if op == "quantize_i8":
            return ox.ox_quantize_i8(s["X"], Q=s["Q"], scales=s["scales"])
        if op == "gemm_i8":
            return ox.ox_gemm_i8(s["A"], s["a_scales"], s["B"], s["b_scales"], bias=s["bias"], act=case["act"], Y=s["Y"])
        Y = ox.ox_moe_few(s["X"], s["scores"], s["W1"], s["W2"], case["top"], w1_scales=s["W1_scales"],
                          w2_scales=s["W2_scales"], b1=s["b1"], b2=s["b2"], act=case["act"], gated=case["gated"],
                          Y=s["Y"], experts=s["experts"], weights=s["weights"], workspace=s["workspace"])
        return Y, s["experts"], s["weights"]
    if op == "norm":
        total, y = _norm(s)
        q, scales = y.to(s["X"].dtype), None
        if case["out"] == "fp8":
            q, scales = _quantize_f8(y, 1)
            scales = scales.t().contiguous()
        return q, scales, total.to(s["X"].dtype) if case["residual"] else None
    if op == "norm_i8":
        total, y = _norm(s)
        q, scales = _quantize_i8(y)
        return (_product(q, scales, s["B"], s["b_scales"], s["bias"], case["act"], torch.bfloat16), scales,
                total.to(s["X"].dtype) if case["residual"] else None)
    if op == "quantize_i8":
        return _quantize_i8(s["X"])
    if op == "gemm_i8":
        return _product(s["A"], s["a_scales"], s["B"], s["b_scales"], s["bias"], case["act"], s["Y"].dtype)
    return _moe_plain(s, case)


def _product_work(M, N, K, out, bias):
    return dict(bytes=M * K + N * K + 4 * (M + N) + M * N * out + (N * out if bias else 0), flops=2.0 * M * N * K)


def work(case):
    op = case["op"]
    if op in ("norm", "norm_i8"):
        R, K, size = case["rows"], case["K"], 4 if case.get("t") == "f32" else 2
        bytes_ = R * K * size * (3 if case["residual"] else 1) + K * size
        if op == "norm_i8":
            # (the codes between the two calls need not leave the chip, but the sum has to)
            w = _product_work(R, case["N"], K, 2, case["bias"])
            return dict(bytes=bytes_ + w["bytes"] - R * K, flops=w["flops"] + 8.0 * R * K)
        bytes_ += R * K + 4 * R * _blocks(K) if case["out"] == "fp8" else R * K * size
        return dict(bytes=bytes_, flops=8.0 * R * K)
    if op == "quantize_i8":
        R, K = case["rows"], case["K"]
        return dict(bytes=R * K * (3 if case["t"] == "bf16" else 5) + 4 * R, flops=3.0 * R * K)
    if op == "gemm_i8":
        return _product_work(case["M"], case["N"], case["K"], 2 if case["out"] == "bf16" else 4, case["bias"])
    T, E, D, H, top = case["T"] - case["pad"], case["E"], case["D"], case["H"], case["top"]
    parts = 3 if case["gated"] else 2
    size = {"f32": 4, "bf16": 2, "fp8": 1}[case["t"]]
    x = 4 if case["t"] == "f32" else 2
    active = E * (1.0 - (1.0 - top / E) ** T)         # experts that some token chooses, on average
    per = parts * D * H * size
    if case["t"] == "fp8":
        per += 4 * parts * _blocks(D) * _blocks(H)
    if case["bias"]:
        per += x * ((parts - 1) * H + D)
    return dict(bytes=active * per + 2 * case["T"] * D * x + 4 * case["T"] * E + 8 * case["T"] * top,
                flops=2.0 * T * top * parts * D * H)


def _round_e4m3(v):
    """float64 -> the nearest e4m3 value (ties to even), as float64: 3 mantissa
    bits, exponents from -6 up, steps of 2^-9 below."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -20))).clamp(min=-6.0)
    step = torch.exp2(e - 3.0)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _act64(v, act):
    if act == "gelu":
        return 0.5 * v * torch.erfc(-v / math.sqrt(2.0))
    if act == "silu":
        return v * torch.sigmoid(v)
    return torch.where(v > 0, v, torch.zeros_like(v)) if act == "relu" else v


def _norm64(s):
    v = s["X"].double()
    if s["residual"] is not None:
        v += s["residual"].double()
    rms = torch.sqrt(torch.linalg.vector_norm(v, dim=1).square() / v.shape[1] + EPS)
    return v, (v / rms[:, None]) * s["gamma"].double()


def _codes64(X):
    """int8 codes as float64, and the scales"""
    top = X.abs().max(dim=1).values
    top = torch.maximum(top, torch.full_like(top, TINY))
    return torch.round(127.0 * X / top[:, None]), top / 127.0


def _product64(A, a_scales, B, b_scales, bias, act):
    Y = A.double() @ B.double().t().contiguous()
    Y *= torch.outer(a_scales.double(), b_scales.double())
    if bias is not None:
        Y += bias.double()
    return _act64(Y, act)


def _moe64(s, case):
    T, top = case["T"], case["top"]
    X, scores = s["X"].double(), s["scores"].double().cpu()
    Y = torch.zeros(s["Y"].shape, dtype=torch.float64, device="cuda")
    experts, weights = torch.full((T, top), -1, dtype=torch.int32), torch.zeros((T, top), dtype=torch.float64)
    of = {}                                            # expert -> [(token, weight)]
    for t in range(T):
        row = scores[t].tolist()
        best = sorted((e for e, v in enumerate(row) if v > -math.inf), key=lambda e: (-row[e], e))[:top]
        part = [math.exp(row[e] - row[best[0]]) for e in best]
        for j, e in enumerate(best):
            experts[t, j], weights[t, j] = e, part[j] / sum(part)
            of.setdefault(e, []).append((t, part[j] / sum(part)))

    def matrix(name, e):
        W = s[name][e].double()
        if case["t"] != "fp8":
            return W
        r, c = (torch.arange(n, device="cuda") // BLOCK for n in W.shape)
        return W * s[name + "_scales"][e].double()[r][:, c]

    for e, users in sorted(of.items()):
        rows = torch.tensor([t for t, _ in users], device="cuda")
        h = X[rows] @ matrix("W1", e).t().contiguous()
        if s["b1"] is not None:
            h += s["b1"][e].double()
        if case["gated"]:
            gate, up = h.split(case["H"], dim=1)
            h = _act64(gate, case["act"]) * up
        else:
            h = _act64(h, case["act"])
        y = h @ matrix("W2", e).t().contiguous()
        if s["b2"] is not None:
            y += s["b2"][e].double()
        Y[rows] += y * torch.tensor([w for _, w in users], dtype=torch.float64, device="cuda")[:, None]
    return Y, experts.cuda(), weights.cuda()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gemm_i8":
        return _product64(s["A"], s["a_scales"], s["B"], s["b_scales"], s["bias"], case["act"])
    if op == "quantize_i8":
        q, scales = _codes64(s["X"].double())
        return q.to(torch.int8), scales
    if op == "moe":
        return _moe64(s, case)
    total, y = _norm64(s)
    total = total if case["residual"] else None
    if op == "norm_i8":
        q, scales = _codes64(y)
        return _product64(q, scales, s["B"], s["b_scales"], s["bias"], case["act"]), scales, total
    if case["out"] == "same":
        return y, None, total
    R, K = y.shape
    Q, S = torch.empty_like(y), torch.empty((_blocks(K), R), dtype=torch.float64, device="cuda")
    for j in range(_blocks(K)):
        cols = slice(j * BLOCK, min(K, (j + 1) * BLOCK))
        top = y[:, cols].abs().max(dim=1).values
        top = torch.maximum(top, torch.full_like(top, TINY))
        S[j] = top / E4M3_MAX
        Q[:, cols] = _round_e4m3(y[:, cols] * (E4M3_MAX / top)[:, None])
    return Q, S, total
