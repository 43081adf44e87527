"""The 8-bit linear layers around the quantized attention, as cases to measure.

Three operators, which a W8A8 layer uses one after the other:

``norm``      rms_norm_quant: the residual's addition, the root-mean-square norm and INT8 codes with one scale for
              each token, in one pass over the activations;
``quantize``  quantize_token: the same codes without a norm, for the attention's output and for weights (a weight's
              row is an output channel, so the same call gives its scale for each channel);
``matmul``    matmul_i8: the product of INT8 codes, exact in integers, with a scale for each token and each channel
              and a bias.

Definitions. With h = x, or x + residual rounded to x's type (what is stored is what is normalised), g = h * weight in
32 bits, a = max |g| over the row and s = max(a / 127, 2^-126) (1 where a is 0): codes = round_half_even(g / s), the
quotient rounded to 32 bits first, and scale = s / sqrt(mean(h^2) + eps) (1 where a is 0). The norm's factor is common
to a row, so the codes do not depend on it: they are the same whole numbers in whatever order its sum is taken.
quantize_token is this with h = x, weight 1 and no norm. matmul_i8: out[m, n] = (sum_k a[m, k] b[n, k]) * a_scale[m]
* b_scale[n] + bias[n].
"""

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6
MOST_VALUES = 65536 * 5120               # activations of the largest norm case
MOST_PRODUCTS = 32768 * 5120 * 5120      # multiplications of the largest matmul case


def listed():
    return [
        # one token of a serving step, hidden size 40 heads x 128: nothing but latency
        dict(name="norm 1x5120", op="norm", rows=1, width=5120, type="bf16", weight="bf16", residual=True),
        # a ragged batch of text tokens in fp16 at an odd width, weight kept in fp32, no residual
        dict(name="norm 333x1031 fp16", op="norm", rows=333, width=1031, type="fp16", weight="fp32", residual=False),
        # a prompt of 16384 tokens (three sequences of 1024, 5000 and 10360), hidden size 32 heads x 128
        dict(name="norm 16384x4096", op="norm", rows=16384, width=4096, type="bf16", weight="bf16", residual=True),
        # a video of 65536 tokens, hidden size 40 heads x 128
        dict(name="norm 65536x5120", op="norm", rows=65536, width=5120, type="bf16", weight="bf16", residual=True),
        # a small fp32 weight with odd row length, quantized for each channel
        dict(name="quantize 515x2047 fp32", op="quantize", rows=515, width=2047, type="fp32"),
        # the attention's output before the output projection, 16384 tokens x 40 heads x 128
        dict(name="quantize 16384x5120", op="quantize", rows=16384, width=5120, type="bf16"),
        # one token through the output projection: the weight is read once
        dict(name="matmul 1x5120x5120", op="matmul", m=1, n=5120, k=5120, type="bf16", bias=False),
        # a batch of 16 single tokens through the joint projection of 32 query and 2 x 8 key-value heads x 128
        dict(name="matmul 16x6144x4096", op="matmul", m=16, n=6144, k=4096, type="bf16", bias=False),
        # 77 text tokens, every size odd, fp16 output with a bias
        dict(name="matmul 77x5003x2047 fp16", op="matmul", m=77, n=5003, k=2047, type="fp16", bias=True),
        # a chunk of 512 tokens through a wide first feed-forward layer, fp32 output
        dict(name="matmul 512x20480x5120 fp32", op="matmul", m=512, n=20480, k=5120, type="fp32", bias=True),
        # a prompt of 16384 tokens through the joint projection of 32 query and 2 x 8 key-value heads x 128
        dict(name="matmul 16384x6144x4096", op="matmul", m=16384, n=6144, k=4096, type="bf16", bias=False),
        # 32768 video tokens through the output projection of 40 heads x 128
        dict(name="matmul 32768x5120x5120", op="matmul", m=32768, n=5120, k=5120, type="bf16", bias=True),
    ]


def _spread(rng, low, high):
    """A whole number from low to high, even over its logarithm; half of them multiples of 64 where that leaves any."""
    v = int(round(low * (high / low) ** rng.random()))
    if rng.random() < 0.5:
        v = (v + 63) // 64 * 64
    return min(max(v, low), high)


def draw(rng):
    op = rng.choice(["norm", "norm", "quantize", "matmul", "matmul", "matmul"])
    if op == "matmul":
        m, n, k = _spread(rng, 1, 32768), _spread(rng, 64, 20480), _spread(rng, 64, 20480)
        while m * n * k > MOST_PRODUCTS or m * n > 32768 * 10240:
            m = (m + 1) // 2
        return dict(op=op, m=m, n=n, k=k, type=rng.choice(["bf16", "bf16", "fp16", "fp32"]), bias=rng.random() < 0.5)
    rows, width = _spread(rng, 1, 65536), _spread(rng, 64, 20480)
    kind = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    while rows * width * SIZE[kind] > MOST_VALUES * 2:
        rows = (rows + 1) // 2
    if op == "quantize":
        return dict(op=op, rows=rows, width=width, type=kind)
    return dict(op=op, rows=rows, width=width, type=kind, weight=rng.choice([kind, "fp32"]), residual=rng.random() < 0.7)


def _codes(gen, rows, width):
    """INT8 codes as the quantizer lays them out: rows start at multiples of 16 bytes."""
    pitch = (width + 15) // 16 * 16
    x = torch.randn((rows, pitch), device="cuda", generator=gen).mul_(32.0).round_().clamp_(-127, 127)
    return x.to(torch.int8)[:, :width]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = dict(case=case)
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"], s["b"] = _codes(gen, m, k), _codes(gen, n, k)
        s["a_scale"] = torch.rand((m,), device="cuda", generator=gen).mul_(0.04).add_(0.01)
        s["b_scale"] = torch.rand((n,), device="cuda", generator=gen).mul_(8e-4).add_(2e-4)
        s["bias"] = torch.randn((n,), device="cuda", generator=gen) if case["bias"] else None
        return s
    rows, width, kind = case["rows"], case["width"], TYPES[case["type"]]
    # activations: a gain for each channel, and a few channels far above the others
    gain = torch.randn((width,), device="cuda", generator=gen).mul_(0.5).exp_()
    gain = torch.where(torch.rand((width,), device="cuda", generator=gen) < 0.005, gain * 20, gain).to(kind)
    s["x"] = torch.randn((rows, width), device="cuda", generator=gen, dtype=kind).mul_(gain)
    if case["op"] == "norm":
        w = torch.randn((width,), device="cuda", generator=gen).mul_(0.2).add_(1.0)
        s["weight"] = w.to(TYPES[case["weight"]])
        s["residual"] = (torch.randn((rows, width), device="cuda", generator=gen, dtype=kind).mul_(gain)
                         if case["residual"] else None)
    return s


def _plain_codes(g):
    """(codes, s) of rows g in 32 bits."""
    a = g.abs().amax(-1, keepdim=True)
    # a tensor divisor: a plain number would be turned into a multiplication by its reciprocal
    s = (a / torch.full_like(a, 127.0)).clamp_min(2.0 ** -126)
    s = torch.where(a == 0, torch.ones_like(s), s)
    return torch.round(g / s).clamp(-127, 127).to(torch.int8), s, a == 0


def run(state):
    case = state["case"]
    if case["op"] == "norm":
        if own:
            import quantized_block_sparse_attn_b200 as qb
            return qb.rms_norm_quant(state["x"], state["weight"], EPS, residual=state["residual"])
        x, residual = state["x"], state["residual"]
        h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
        f = h.float()
        codes, s, zero = _plain_codes(f * state["weight"].float())
        scale = s / torch.sqrt((f * f).mean(-1, keepdim=True) + EPS)
        scale = torch.where(zero, torch.ones_like(scale), scale).squeeze(-1)
        return codes, scale, None if residual is None else h
    if case["op"] == "quantize":
        if own:
            import quantized_block_sparse_attn_b200 as qb
            return qb.quantize_token(state["x"])
        codes, s, _ = _plain_codes(state["x"].float())
        return codes, s.squeeze(-1)
    kind = TYPES[case["type"]]
    if own:
        import quantized_block_sparse_attn_b200 as qb
        return qb.matmul_i8(state["a"], state["b"], state["a_scale"], state["b_scale"], bias=state["bias"],
                            out_dtype=kind)
    # sums of whole numbers: exact in 32 bits while they stay below 2^24, as they do for codes of this spread
    y = (state["a"].float() @ state["b"].float().t()) * state["a_scale"][:, None] * state["b_scale"]
    if state["bias"] is not None:
        y = y + state["bias"]
    return y.to(kind)


def work(case):
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k + n * k + m * n * SIZE[case["type"]] + 4 * (m + n) + (4 * n if case["bias"] else 0),
                "flops": 2 * m * n * k}
    rows, width, size = case["rows"], case["width"], SIZE[case["type"]]
    if case["op"] == "quantize":
        return {"bytes": rows * width * (size + 1) + 4 * rows, "flops": 2 * rows * width}
    tensors = 3 if case["residual"] else 1          # x, and the residual read and written
    return {"bytes": rows * width * (size * tensors + 1) + width * SIZE[case["weight"]] + 4 * rows,
            "flops": (5 if case["residual"] else 4) * rows * width}


def exact(case, seed):
    """The definitions in 64 bits. The codes are whole numbers, fixed by their definition in 32 bits: no value here."""
    s = prepare(case, seed)
    if case["op"] == "matmul":
        out = torch.empty((case["m"], case["n"]), dtype=torch.float64, device="cuda")
        bt = s["b"].double().t() * s["b_scale"].double()
        for at in range(0, case["m"], 4096):
            out[at:at + 4096] = (s["a"][at:at + 4096].double() * s["a_scale"][at:at + 4096, None].double()) @ bt
        return out if s["bias"] is None else out.add_(s["bias"].double())
    scales, sums = [], []
    for at in range(0, case["rows"], 8192):
        h = s["x"][at:at + 8192].double()
        if case["op"] == "norm":
            if s["residual"] is not None:
                h = h + s["residual"][at:at + 8192].double()
                sums.append(h)
                h = h.to(TYPES[case["type"]]).double()
            top = (h * s["weight"].double()).abs().amax(-1)
            scale = top / 127 / (h.square().mean(-1) + EPS).sqrt()
        else:
            top = h.abs().amax(-1)
            scale = top / 127
        scales.append(torch.where(top == 0, torch.ones_like(scale), scale))
    scales = torch.cat(scales)
    if case["op"] == "quantize":
        return None, scales
    return None, scales, torch.cat(sums) if sums else None
