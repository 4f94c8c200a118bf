"""Cases and plain forms of the 8-bit floating-point and expert-grouped
matrix products: what is measured, with real sizes, and what each result is.

Three operators of the package are called here:

  ox_quantize_fp8      X -> e4m3 codes with one fp32 scale per block: 1 x 128
                       (activations; optionally gathering the rows in expert
                       order) or 128 x 128 (weights).  Activation scales are
                       stored k-block first, [ceil(K/128), rows]; weight
                       scales [ceil(N/128), ceil(K/128)].
  ox_gemm_fp8          Y = act(dequant(A) dequant(B)^T + bias)
  ox_gemm_grouped      the rows of A are sorted by expert, rows
  ox_gemm_grouped_fp8  offsets[e] .. offsets[e+1] - 1 times expert e's weights

Where ``own`` is false, ``run`` computes the same in elementary torch
operations.
"""
import math

import torch

own = False

BLOCK = 128          # elements along K (and weight rows) that share a scale
E4M3_MAX = 448.0
TINY = 2.0 ** -100   # a block's largest magnitude is taken to be at least this
F8 = torch.float8_e4m3fn


def listed():
    return [
        # one token through a 4096 x 4096 layer: a serving step of batch 1
        dict(name="fp8_row1", op="gemm_fp8", M=1, N=4096, K=4096, out="bf16", bias=False, act="none"),
        # a batch of 24 decoding requests through an expanding layer, fused GELU
        dict(name="fp8_rows24", op="gemm_fp8", M=24, N=4096, K=1024, out="bf16", bias=True, act="gelu"),
        # a prompt of 1000 tokens, with a last partial k-block and fp32 results (a head's logits)
        dict(name="fp8_odd1000", op="gemm_fp8", M=1000, N=1000, K=2000, out="f32", bias=True, act="none"),
        # a long prompt (or a batch of them): the compute-bound end
        dict(name="fp8_8192", op="gemm_fp8", M=8192, N=8192, K=8192, out="bf16", bias=False, act="none"),
        # 8 decoding tokens, 2 of 8 experts each: weights' bytes count
        dict(name="grp_bf16_decode", op="grouped", t="bf16", T=16, E=8, active=7, N=4096, K=1024, transB=True, bias=True, act="gelu"),
        # a prompt of 4096 tokens, 2 of 8 experts each
        dict(name="grp_bf16_prompt", op="grouped", t="bf16", T=8192, E=8, active=8, N=4096, K=4096, transB=True, bias=False, act="none"),
        # weights as an ONNX MatMul stores them ([K, N]), many small experts, some idle
        dict(name="grp_bf16_kn", op="grouped", t="bf16", T=4003, E=64, active=60, N=1024, K=2048, transB=False, bias=False, act="none"),
        # an fp32 model's experts
        dict(name="grp_f32", op="grouped", t="f32", T=1000, E=8, active=8, N=1024, K=1024, transB=True, bias=True, act="relu"),
        # 8 decoding tokens, 8 of 128 experts each
        dict(name="grp_fp8_decode", op="grouped", t="fp8", T=64, E=128, active=50, N=2048, K=1024, transB=True, bias=False, act="none"),
        # a prompt of 2048 tokens, 8 of 32 experts each
        dict(name="grp_fp8_prompt", op="grouped", t="fp8", T=16384, E=32, active=32, N=4096, K=2048, transB=True, bias=False, act="none"),
        # the activations of 24 decoding requests
        dict(name="quant_rows24", op="quantize", t="bf16", rows=24, K=4096, block_rows=1, index=False, R=24),
        # a prompt's activations, copied to their experts' order (2 experts a token) as they are quantised
        dict(name="quant_gather", op="quantize", t="bf16", rows=8192, K=4096, block_rows=1, index=True, R=16384),
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
    op = rng.choice(["gemm_fp8", "grouped", "grouped", "quantize"])
    if op == "gemm_fp8":
        return dict(op=op, M=_log(rng, 1, 8192), N=_length(rng, 64, 8192), K=_length(rng, 64, 8192),
                    out=rng.choice(["bf16", "bf16", "f32"]), bias=rng.random() < 0.5,
                    act=rng.choice(["none", "relu", "gelu"]))
    if op == "grouped":
        t = rng.choice(["bf16", "fp8", "f32"])
        E, N, K = _log(rng, 2, 128), _length(rng, 64, 4096), _length(rng, 64, 4096)
        while E > 2 and E * N * K > (1 << 28 if t != "f32" else 1 << 26):   # the weights: 512 MB in bf16 at most
            E = E // 2
        T = _log(rng, 1, 16384)
        most = 2.5e11 if t != "f32" else 1.6e10
        while 2.0 * T * N * K > most:
            T = T // 2 + 1
        return dict(op=op, t=t, T=T, E=E, active=max(1, int(E * rng.uniform(0.5, 1.0))), N=N, K=K,
                    transB=t == "fp8" or rng.random() < 0.6, bias=rng.random() < 0.5,
                    act=rng.choice(["none", "relu", "gelu"]))
    block_rows = rng.choice([1, 1, 128])
    rows = _log(rng, 1, 8192)
    index = block_rows == 1 and rng.random() < 0.5
    return dict(op=op, t=rng.choice(["bf16", "bf16", "f32"]), rows=rows, K=_length(rng, 64, 4096),
                block_rows=block_rows, index=index, R=min(16384, rows * rng.choice([1, 2])) if index else rows)


def _counts(case):
    """Rows of each expert, the busiest first: popularity falls with rank^-1/2,
    every active expert has a row at least."""
    T, E = case["T"], case["E"]
    active = min(case["active"], T, E)
    share = [(i + 1) ** -0.5 for i in range(active)]
    left = T - active
    got = [1 + int(left * s / sum(share)) for s in share]
    for i in range(T - sum(got)):
        got[i % active] += 1
    return got + [0] * (E - active)


def _blocks(n):
    return -(-n // BLOCK)


def _quantize64(X, block_rows):
    """(codes, scales [row blocks, k-blocks]) of a 2-D or 3-D tensor, in 64 bits."""
    X = X.double()
    R, K = X.shape[-2:]
    rb, kb = -(-R // block_rows), _blocks(K)
    P = torch.nn.functional.pad(X, (0, kb * BLOCK - K, 0, rb * block_rows - R))
    P = P.reshape(X.shape[:-2] + (rb, block_rows, kb, BLOCK))
    m = P.abs().amax(dim=(-3, -1), keepdim=True).clamp(min=TINY)
    q = (P * (E4M3_MAX / m)).to(F8)
    q = q.reshape(X.shape[:-2] + (rb * block_rows, kb * BLOCK))[..., :R, :K]
    return q.contiguous(), (m / E4M3_MAX).float().squeeze(-1).squeeze(-2)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda") * std

    def activations(rows, K):
        # a few channels are much larger than the rest, as in trained models
        big = 1.0 + 15.0 * (torch.rand((1, K), generator=g, device="cuda") < 0.01)
        return normal(rows, K) * big

    s = dict(case=dict(case))
    op = case["op"]
    if op == "quantize":
        t = torch.bfloat16 if case["t"] == "bf16" else torch.float32
        X = activations(case["rows"], case["K"]) if case["block_rows"] == 1 else normal(case["rows"], case["K"], std=case["K"] ** -0.5)
        s["X"] = X.to(t)
        s["index"] = None
        if case["index"]:
            s["index"] = torch.randint(0, case["rows"], (case["R"],), generator=g, device="cuda", dtype=torch.int32)
        s["Q"] = torch.empty((case["R"], case["K"]), dtype=F8, device="cuda")
        kb = _blocks(case["K"])
        s["scales"] = torch.empty((kb, case["R"]) if case["block_rows"] == 1 else (_blocks(case["R"]), kb), device="cuda")
        return s
    N, K = case["N"], case["K"]
    if op == "gemm_fp8":
        a, sa = _quantize64(activations(case["M"], K), 1)
        b, sb = _quantize64(normal(N, K, std=K ** -0.5), BLOCK)
        o = torch.bfloat16 if case["out"] == "bf16" else torch.float32
        s.update(A=a, a_scales=sa.t().contiguous(), B=b, b_scales=sb,
                 bias=normal(N).to(o) if case["bias"] else None,
                 Y=torch.empty((case["M"], N), dtype=o, device="cuda"))
        return s
    counts = _counts(case)
    order = torch.randperm(case["E"], generator=g, device="cuda").cpu().tolist()
    counts = [counts[i] for i in order]
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    s["cap"] = max(counts)   # the experts' capacity, which the plain form pads to
    s["offsets"] = torch.tensor(off, dtype=torch.int32, device="cuda")
    T, E = case["T"], case["E"]
    if case["t"] == "fp8":
        a, sa = _quantize64(activations(T, K), 1)
        s.update(A=a, a_scales=sa.t().contiguous())
        s["B"] = torch.empty((E, N, K), dtype=F8, device="cuda")
        s["b_scales"] = torch.empty((E, _blocks(N), _blocks(K)), device="cuda")
        for e in range(E):
            s["B"][e], s["b_scales"][e] = _quantize64(normal(N, K, std=K ** -0.5), BLOCK)
        t = torch.bfloat16
    else:
        t = torch.bfloat16 if case["t"] == "bf16" else torch.float32
        s["A"] = activations(T, K).to(t)
        s["B"] = (normal(E, N, K, std=K ** -0.5) if case["transB"] else normal(E, K, N, std=K ** -0.5)).to(t)
    s["bias"] = normal(E, N).to(t) if case["bias"] else None
    s["Y"] = torch.empty((T, N), dtype=t, device="cuda")
    return s


def _act(v, act):
    if act == "relu":
        return v.clamp(min=0)
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * 0.7071067811865476))
    return v


def _dequant_rows(q, scales):
    """codes [R, K], scales [k-blocks, R] -> fp32 [R, K]"""
    return q.float() * scales.t().repeat_interleave(BLOCK, dim=1)[:, :q.shape[1]]


def _dequant_weights(q, scales):
    """codes [..., N, K], scales [..., ceil(N/128), ceil(K/128)] -> fp32"""
    full = scales.repeat_interleave(BLOCK, dim=-2).repeat_interleave(BLOCK, dim=-1)
    return q.float() * full[..., :q.shape[-2], :q.shape[-1]]


def _grouped_plain(s, case):
    A, B = s["A"], s["B"]
    if case["t"] == "fp8":
        A, B = _dequant_rows(A, s["a_scales"]), _dequant_weights(B, s["b_scales"])
    A, B = A.float(), B.float()
    if case["transB"]:
        B = B.transpose(1, 2).contiguous()
    T, E, cap = case["T"], case["E"], s["cap"]
    off = s["offsets"].long()
    row = torch.arange(T, device="cuda")
    e = torch.searchsorted(off, row, right=True) - 1       # an idle expert's offsets are equal: the last one holds the row
    slot = e * cap + (row - off[e])
    P = torch.zeros((E * cap, A.shape[1]), device="cuda")
    P[slot] = A
    Y = torch.bmm(P.view(E, cap, -1), B).view(E * cap, -1)[slot]
    if s["bias"] is not None:
        Y = Y + s["bias"].float()[e]
    return _act(Y, case["act"]).to(s["Y"].dtype)


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import conv_implicit_gemm_amd as ox
        if op == "quantize":
            return ox.ox_quantize_fp8(s["X"], index=s["index"], block_rows=case["block_rows"], Q=s["Q"], scales=s["scales"])
        if op == "gemm_fp8":
            return ox.ox_gemm_fp8(s["A"], s["a_scales"], s["B"], s["b_scales"], bias=s["bias"], act=case["act"], Y=s["Y"])
        if case["t"] == "fp8":
            return ox.ox_gemm_grouped_fp8(s["A"], s["a_scales"], s["B"], s["b_scales"], s["offsets"], bias=s["bias"],
                                          act=case["act"], Y=s["Y"])
        return ox.ox_gemm_grouped(s["A"], s["B"], s["offsets"], bias=s["bias"], transB=case["transB"], act=case["act"], Y=s["Y"])
    if op == "quantize":
        X = s["X"] if s["index"] is None else s["X"][s["index"].long()]
        q, scales = _quantize64(X, case["block_rows"])
        return q, scales.t().contiguous() if case["block_rows"] == 1 else scales
    if op == "gemm_fp8":
        Y = torch.mm(_dequant_rows(s["A"], s["a_scales"]), _dequant_weights(s["B"], s["b_scales"]).t())
        if s["bias"] is not None:
            Y = Y + s["bias"].float()
        return _act(Y, case["act"]).to(s["Y"].dtype)
    return _grouped_plain(s, case)


def work(case):
    op = case["op"]
    K, kb = case["K"], _blocks(case["K"])
    if op == "quantize":
        size = 2 if case["t"] == "bf16" else 4
        R = case["R"]
        scales = R * kb if case["block_rows"] == 1 else _blocks(R) * kb
        # a gathered row that is asked for twice is read once; the index itself is read
        rows = min(case["rows"], R)
        if case["index"]:
            rows = case["rows"] * (1.0 - (1.0 - 1.0 / case["rows"]) ** R)
        return dict(bytes=rows * K * size + R * K + 4 * scales + (4 * R if case["index"] else 0), flops=3.0 * R * K)
    N = case["N"]
    if op == "gemm_fp8":
        M, size = case["M"], 2 if case["out"] == "bf16" else 4
        return dict(bytes=M * K + N * K + 4 * (M * kb + _blocks(N) * kb) + M * N * size + (N * size if case["bias"] else 0),
                    flops=2.0 * M * N * K)
    T, active = case["T"], min(case["active"], case["T"], case["E"])
    size = {"f32": 4, "bf16": 2, "fp8": 1}[case["t"]]
    out = 4 if case["t"] == "f32" else 2
    scales = 4 * (T * kb + active * _blocks(N) * kb) if case["t"] == "fp8" else 0
    return dict(bytes=T * K * size + active * N * K * size + scales + T * N * out + (active * N * out if case["bias"] else 0)
                + 4 * (case["E"] + 1), flops=2.0 * T * N * K)


def _round_e4m3(v):
    """float64 -> the nearest e4m3 value (ties to even), as float64: 3 mantissa
    bits, exponents from -6 up, steps of 2^-9 below."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -20))).clamp(min=-6.0)
    step = torch.exp2(e - 3.0)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _wide(q, scales, rows_per_scale):
    """codes [R, K] and scales [row blocks, k-blocks] -> float64 values"""
    r = torch.arange(q.shape[0], device=q.device) // rows_per_scale
    k = torch.arange(q.shape[1], device=q.device) // BLOCK
    return q.double() * scales.double()[r][:, k]


def _act64(v, act):
    if act == "gelu":
        return 0.5 * v * torch.erfc(-v / math.sqrt(2.0))
    return torch.where(v > 0, v, torch.zeros_like(v)) if act == "relu" else v


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        X = s["X"].double()
        if s["index"] is not None:
            X = X.index_select(0, s["index"].long())
        R, K = X.shape
        br = case["block_rows"]
        Q = torch.empty_like(X)
        S = torch.empty((-(-R // br), _blocks(K)), dtype=torch.float64, device="cuda")
        for j in range(_blocks(K)):
            cols = slice(j * BLOCK, min(K, (j + 1) * BLOCK))
            top = X[:, cols].abs().max(dim=1).values
            if br > 1:
                top = torch.stack([c.max() for c in top.split(br)])
            top = torch.maximum(top, torch.full_like(top, TINY))
            S[:, j] = top / E4M3_MAX
            Q[:, cols] = _round_e4m3(X[:, cols] * (E4M3_MAX / top).repeat_interleave(br)[:R, None])
        return Q, S.t().contiguous() if br == 1 else S
    if op == "gemm_fp8":
        Y = _wide(s["A"], s["a_scales"].t(), 1) @ _wide(s["B"], s["b_scales"], BLOCK).t().contiguous()
        if s["bias"] is not None:
            Y += s["bias"].double()
        return _act64(Y, case["act"])
    off = s["offsets"].cpu().tolist()
    Y = torch.zeros((case["T"], case["N"]), dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        if case["t"] == "fp8":
            a, b = _wide(s["A"][lo:hi], s["a_scales"][:, lo:hi].t(), 1), _wide(s["B"][e], s["b_scales"][e], BLOCK)
        else:
            a, b = s["A"][lo:hi].double(), s["B"][e].double()
        y = a @ (b.t().contiguous() if case["transB"] else b)
        if s["bias"] is not None:
            y += s["bias"][e].double()
        Y[lo:hi] = _act64(y, case["act"])
    return Y
