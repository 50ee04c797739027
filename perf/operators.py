"""Timed cases of the operators that answer with quantized weights: the mixture-of-experts layer over
packed codes, the block-scaled 8-bit floating-point product, and the two ways to its operands (rounding
a matrix to e4m3 with a scale per block of 128, and turning packed codes into e4m3 integers).

``own`` False: the operators in their plain form (elementary torch operations in fp32).  ``own`` True:
the calls a user makes of the library.
"""
import math

import torch

own = False

F8 = torch.float8_e4m3fn
F8_MAX = 448.0
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # one token through a small square layer: latency only
        {"name": "fp8_matmul_1x768x768", "op": "matmul", "m": 1, "n": 768, "k": 768, "rows": 1, "y": "fp16"},
        # one token through a 4096-wide layer with 128x128 weight blocks: the weights' bytes
        {"name": "fp8_matmul_1x4096x4096", "op": "matmul", "m": 1, "n": 4096, "k": 4096, "rows": 128, "y": "bf16"},
        # a ragged batch against GPTQ codes (a scale per weight row and group), odd output width, fp32 result
        {"name": "fp8_matmul_333x4099x11008", "op": "matmul", "m": 333, "n": 4099, "k": 11008, "rows": 1, "y": "fp32"},
        # a prompt batch through an up projection: the tensor cores
        {"name": "fp8_matmul_8192x11008x4096", "op": "matmul", "m": 8192, "n": 11008, "k": 4096, "rows": 128,
         "y": "bf16"},
        # the activations of a few tokens before a product
        {"name": "fp8_quantize_7x4096", "op": "quantize", "m": 7, "k": 4096, "rows": 1, "x": "fp16"},
        # a prompt batch's activations before a down projection
        {"name": "fp8_quantize_16384x11008", "op": "quantize", "m": 16384, "k": 11008, "rows": 1, "x": "bf16"},
        # a weight matrix once, in 128x128 blocks
        {"name": "fp8_quantize_w_11008x4096", "op": "quantize", "m": 11008, "k": 4096, "rows": 128, "x": "fp16"},
        # a 3-bit grouped layer made ready for the tensor cores
        {"name": "fp8_from_packed_4096x4096_3bit", "op": "packed", "m": 4096, "k": 4096, "bits": 3, "group": 128},
        # a 4-bit layer with a grid per row
        {"name": "fp8_from_packed_11008x4096_4bit", "op": "packed", "m": 11008, "k": 4096, "bits": 4, "group": 0},
        # a few tokens through small relu experts: latency
        {"name": "moe_5tok_4x768x768_2bit", "op": "moe", "t": 5, "e": 4, "top": 1, "d": 768, "f": 768, "bits": 2,
         "group": 0, "x": "fp32", "y": "fp32", "act": "relu", "renorm": False},
        # one token, two of eight wide gated experts: the ordinary decoding step
        {"name": "moe_1tok_8x4096x11008_4bit", "op": "moe", "t": 1, "e": 8, "top": 2, "d": 4096, "f": 11008,
         "bits": 4, "group": 128, "x": "bf16", "y": "bf16", "act": "silu", "renorm": True},
        # a decoding batch over many narrow experts: nearly every expert is read
        {"name": "moe_32tok_32x4096x1408_3bit", "op": "moe", "t": 32, "e": 32, "top": 6, "d": 4096, "f": 1408,
         "bits": 3, "group": 128, "x": "fp16", "y": "fp32", "act": "silu", "renorm": True},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of ``step`` between lo and hi, spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, round(v / step) * step)) if step == 1 else max(step, int(v / step) * step)


def draw(rng):
    op = rng.choice(["matmul", "moe", "quantize", "packed", "matmul", "moe"])
    while True:
        if op == "matmul":
            c = {"op": op, "m": _log(rng, 1, 8192), "n": _log(rng, 64, 12288), "k": _log(rng, 128, 16384, 16),
                 "rows": rng.choice([1, 128]), "y": rng.choice(list(DT))}
            fits = c["m"] * c["n"] * c["k"] <= 2 ** 38
        elif op == "quantize":
            c = {"op": op, "m": _log(rng, 1, 16384), "k": _log(rng, 128, 16384, 16), "rows": rng.choice([1, 128]),
                 "x": rng.choice(list(DT))}
            fits = c["m"] * c["k"] * SIZE[c["x"]] <= 3 * 10 ** 8
        elif op == "packed":
            c = {"op": op, "m": _log(rng, 16, 12288), "k": _log(rng, 128, 12288, 32), "bits": rng.choice([2, 3, 4])}
            c["group"] = rng.choice([0, 128] if c["k"] % 128 == 0 else [0])
            fits = c["m"] * c["k"] <= 5 * 10 ** 7
        else:
            e = rng.choice([2, 4, 8, 16, 32, 64])
            c = {"op": op, "t": _log(rng, 1, 64), "e": e, "top": rng.randint(1, min(e, 8)),
                 "d": _log(rng, 256, 4096, 32), "f": _log(rng, 256, 12288, 32), "bits": rng.choice([2, 3, 4]),
                 "x": rng.choice(list(DT)), "y": rng.choice(list(DT)), "act": rng.choice(["silu", "relu"]),
                 "renorm": rng.random() < 0.5}
            groups = [g for g in (32, 64, 128) if c["d"] % g == 0 and c["f"] % g == 0]
            c["group"] = rng.choice([0] + groups)
            fits = c["e"] * c["d"] * c["f"] <= 36 * 10 ** 7
        if fits:
            return c


def _blocks(n, b):
    return (n + b - 1) // b


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _activations(rows, k, dtype, g):
    """Normal values with one channel in a hundred twenty times as large, as calibration inputs have."""
    x = torch.randn(rows, k, generator=g, device="cuda")
    big = torch.rand(k, generator=g, device="cuda") < 0.01
    return torch.where(big, x * 20.0, x).to(dtype)


def _packed(lead, k, bits, group, g):
    """Uniform codes, zero points near the middle of the grid, scales that give weights of size 1/sqrt(k)."""
    ng = k // group if group else 1
    words = torch.randint(-2 ** 31, 2 ** 31, (*lead, k * bits // 32), generator=g, device="cuda", dtype=torch.int64)
    size = 1.0 / math.sqrt(k * (4 ** bits - 1) / 12.0)
    scales = (torch.rand(*lead, ng, generator=g, device="cuda") + 0.5) * size
    zeros = torch.randint(2 ** (bits - 1) - 1, 2 ** (bits - 1) + 1, (*lead, ng), generator=g, device="cuda",
                          dtype=torch.int32)
    return words.to(torch.int32), scales, zeros


def prepare(case, seed):
    g = _gen(seed)
    c = case
    s = {"case": dict(case)}
    if c["op"] == "matmul":
        kb = _blocks(c["k"], 128)
        s["a"] = (torch.randn(c["m"], c["k"], generator=g, device="cuda") * 100.0).clamp_(-F8_MAX, F8_MAX).to(F8)
        s["sa"] = torch.exp2(torch.randint(-9, -5, (c["m"], kb), generator=g, device="cuda").float())
        if c["rows"] == 1:  # GPTQ codes: small integers, a grid scale per row and group
            s["b"] = torch.randint(-8, 8, (c["n"], c["k"]), generator=g, device="cuda", dtype=torch.int8).to(F8)
            s["sb"] = (torch.rand(c["n"], kb, generator=g, device="cuda") + 0.5) * (0.2 / math.sqrt(c["k"]))
        else:
            s["b"] = (torch.randn(c["n"], c["k"], generator=g, device="cuda") * 100.0).clamp_(-F8_MAX, F8_MAX).to(F8)
            s["sb"] = torch.exp2(torch.randint(-14, -11, (_blocks(c["n"], 128), kb), generator=g, device="cuda").float())
    elif c["op"] == "quantize":
        s["x"] = _activations(c["m"], c["k"], DT[c["x"]], g)
        if c["m"] > 64:
            s["x"][c["m"] - c["m"] // 64:] = 0  # the padding rows of a batch
    elif c["op"] == "packed":
        s["w"] = _packed((c["m"],), c["k"], c["bits"], c["group"], g)
    else:
        s["x"] = _activations(c["t"], c["d"], DT[c["x"]], g)
        s["router"] = (torch.randn(c["e"], c["d"], generator=g, device="cuda") / math.sqrt(c["d"])).to(DT[c["x"]])
        s["up"] = _packed((c["e"], c["f"]), c["d"], c["bits"], c["group"], g)
        s["gate"] = _packed((c["e"], c["f"]), c["d"], c["bits"], c["group"], g) if c["act"] == "silu" else None
        s["down"] = _packed((c["e"], c["d"]), c["f"], c["bits"], c["group"], g)
    return s


# ------------------------------------------------------------------------------------- plain forms
def _spread(scales, k, rows=1, n=None):
    """Scales per (block of rows, block of 128 columns) as one per value."""
    s = scales.repeat_interleave(128, dim=1)[:, :k]
    return s if rows == 1 else s.repeat_interleave(rows, dim=0)[:n]


def _plain_matmul(s, c):
    a = s["a"].float() * _spread(s["sa"], c["k"])
    b = s["b"].float() * _spread(s["sb"], c["k"], c["rows"], c["n"])
    return (a @ b.t()).to(DT[c["y"]])


def _plain_quantize(s, c):
    m, k, r = c["m"], c["k"], c["rows"]
    x = s["x"].float()
    mb, kb = _blocks(m, r), _blocks(k, 128)
    padded = torch.nn.functional.pad(x, (0, kb * 128 - k, 0, mb * r - m))
    amax = padded.view(mb, r, kb, 128).abs().amax(dim=(1, 3))
    frac, exp = torch.frexp(amax)  # amax = frac 2^exp, frac in [0.5, 1); 448 = 0.875 * 2^9
    k2 = torch.where(frac <= 0.875, exp - 9, exp - 8).clamp(min=-126)
    scales = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), k2), torch.ones_like(amax))
    return (x / _spread(scales, k, r, m)).to(F8), scales


def _plain_codes(words, bits):
    """Codes [..., k] of the packed words: code j is bits [bits j, bits j + bits) of the row's stream."""
    unit = words.view(*words.shape[:-1], -1, bits)
    at = torch.arange(32, device=words.device, dtype=torch.int32) * bits
    word, off = (at >> 5).long(), at & 31
    low = (unit[..., word] >> off) & ((1 << bits) - 1)
    keep = torch.clamp(32 - off, max=bits)  # bits of the code inside its first word
    low = low & ((1 << keep) - 1)
    high = (unit[..., (word + 1).clamp(max=bits - 1)] << keep) & ((1 << bits) - 1)
    code = torch.where(keep < bits, low | high, low)
    return code.flatten(-2)


def _plain_weights(w, bits, group):
    words, scales, zeros = w
    q = _plain_codes(words, bits)
    g = group or q.shape[-1]
    q = q.view(*q.shape[:-1], -1, g)
    return (scales[..., None] * (q - zeros[..., None]).float()).flatten(-2)


def _plain_packed(s, c):
    words, scales, zeros = s["w"]
    q = _plain_codes(words, c["bits"])
    g = c["group"] or c["k"]
    q = (q.view(c["m"], -1, g) - zeros[..., None]).float().view(c["m"], c["k"])
    of = torch.arange(0, c["k"], 128, device=q.device) // g
    return q.to(F8), scales[:, of]


def _plain_moe(s, c):
    x = s["x"].float()
    p = torch.softmax(x @ s["router"].float().t(), dim=-1)
    w, ids = torch.sort(p, dim=-1, descending=True, stable=True)
    w, ids = w[:, :c["top"]], ids[:, :c["top"]]
    if c["renorm"]:
        w = w / w.sum(dim=-1, keepdim=True)
    pairs = c["t"] * c["top"] <= c["e"]  # few tokens: only the chosen experts, pair by pair; else all of them

    def product(v, name, eq):
        t = s[name]
        if pairs:
            t = tuple(z[ids] for z in t)
        return torch.einsum(eq, v, _plain_weights(t, c["bits"], c["group"]))

    up_eq, down_eq = ("td,tkfd->tkf", "tkf,tkdf->tkd") if pairs else ("td,efd->etf", "etf,edf->etd")
    h = product(x, "up", up_eq)
    if c["act"] == "silu":
        gate = product(x, "gate", up_eq)
        h = gate / (1 + torch.exp(-gate)) * h
    else:
        h = torch.clamp(h, min=0)
    y = product(h, "down", down_eq)
    if pairs:
        y = (w[:, :, None] * y).sum(dim=1)
    else:
        dense = torch.zeros_like(p).scatter_(1, ids, w)
        y = (dense.t()[:, :, None] * y).sum(dim=0)
    return y.to(DT[c["y"]]), ids.to(torch.int32), w


# ------------------------------------------------------------------------------------- the library's calls
def _own_buffers(s, c):
    """What a user's program keeps from call to call: outputs, status words, workspace."""
    import post_weight_quantization_21_b200 as gptq

    dev = torch.device("cuda")
    st = torch.zeros(2, dtype=torch.int32, device=dev)
    b = {"gptq": gptq, "status": st}
    if c["op"] == "matmul":
        b["y"] = torch.empty(c["m"], c["n"], dtype=DT[c["y"]], device=dev)
        need = gptq.gptq_fp8_matmul_workspace_size(c["m"], c["n"], c["k"])
    elif c["op"] == "moe":
        b["y"] = torch.empty(c["t"], c["d"], dtype=DT[c["y"]], device=dev)
        b["ids"] = torch.empty(c["t"], c["top"], dtype=torch.int32, device=dev)
        b["w"] = torch.empty(c["t"], c["top"], dtype=torch.float32, device=dev)
        need = gptq.gptq_moe_workspace_size(c["t"], c["d"], c["f"], c["e"], c["top"])
        b["act"] = gptq.GPTQ_ACT_SILU_GATED if c["act"] == "silu" else gptq.GPTQ_ACT_RELU
        b["flags"] = gptq.GPTQ_MOE_RENORMALIZE if c["renorm"] else 0
    else:
        rows = c["rows"] if c["op"] == "quantize" else 1
        b["q"] = torch.empty(c["m"], c["k"], dtype=F8, device=dev)
        b["scales"] = torch.empty(_blocks(c["m"], rows), _blocks(c["k"], 128), dtype=torch.float32, device=dev)
        need = 0
    b["ws"] = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    return b


def _own_run(s, c):
    if "own" not in s:
        s["own"] = _own_buffers(s, c)
    b = s["own"]
    gptq = b["gptq"]
    if c["op"] == "matmul":
        gptq.gptq_fp8_matmul(s["a"], s["sa"], s["b"], s["sb"], c["rows"], b["y"], b["status"], b["ws"])
        return b["y"]
    if c["op"] == "quantize":
        gptq.gptq_fp8_quantize(s["x"], b["q"], b["scales"], c["rows"])
        return b["q"], b["scales"]
    if c["op"] == "packed":
        gptq.gptq_fp8_from_packed(*s["w"], c["bits"], c["group"], b["q"], b["scales"])
        return b["q"], b["scales"]
    gptq.gptq_moe_layer(s["x"], s["router"], s["up"], s["gate"], s["down"], b["ids"], b["w"], b["y"], b["status"],
                        b["ws"], c["bits"], c["group"], b["act"], b["flags"])
    return b["y"], b["ids"], b["w"]


def run(state):
    c = state["case"]
    if own:
        return _own_run(state, c)
    if c["op"] == "matmul":
        return _plain_matmul(state, c)
    if c["op"] == "quantize":
        return _plain_quantize(state, c)
    if c["op"] == "packed":
        return _plain_packed(state, c)
    return _plain_moe(state, c)


def work(case):
    c = case
    if c["op"] == "matmul":
        m, n, k, kb = c["m"], c["n"], c["k"], _blocks(c["k"], 128)
        return {"bytes": m * k + n * k + 4 * kb * (m + _blocks(n, c["rows"])) + m * n * SIZE[c["y"]],
                "flops": 2 * m * n * k}
    if c["op"] == "quantize":
        m, k = c["m"], c["k"]
        return {"bytes": m * k * (SIZE[c["x"]] + 1) + 4 * _blocks(m, c["rows"]) * _blocks(k, 128), "flops": 2 * m * k}
    if c["op"] == "packed":
        m, k, ng = c["m"], c["k"], (c["k"] // c["group"] if c["group"] else 1)
        return {"bytes": m * k * c["bits"] / 8 + 8 * m * ng + m * k + 4 * m * _blocks(k, 128), "flops": m * k}
    t, e, top, d, f = (c[n] for n in ("t", "e", "top", "d", "f"))
    mats = 3 if c["act"] == "silu" else 2
    grids = 8 * (mats - 1) * f * (d // c["group"] if c["group"] else 1) + 8 * d * (f // c["group"] if c["group"] else 1)
    experts = e * (1.0 - (1.0 - top / e) ** t)  # distinct experts that t tokens choose, on average
    return {"bytes": experts * (mats * d * f * c["bits"] / 8 + grids) + (t + e) * d * SIZE[c["x"]]
            + t * d * SIZE[c["y"]] + 8 * t * top,
            "flops": 2 * t * (top * mats * d * f + e * d)}


# ------------------------------------------------------------------------------------- 64-bit definitions
def _exact_codes(words, bits):
    """Codes from the stream's single bits."""
    shift = torch.arange(32, device=words.device, dtype=torch.int32)
    stream = ((words.unsqueeze(-1) >> shift) & 1).to(torch.uint8).flatten(-2)
    stream = stream.view(*stream.shape[:-1], -1, bits)
    code = stream[..., 0].to(torch.int16)
    for b in range(1, bits):
        code += stream[..., b].to(torch.int16) << b
    return code


def _exact_weights(w, e, bits, group):
    words, scales, zeros = (z[e] for z in w)
    q = _exact_codes(words, bits).double()
    g = group or q.shape[-1]
    rep = lambda z: z.double().repeat_interleave(g, dim=-1)
    return rep(scales) * (q - rep(zeros))


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "matmul":
        y = torch.zeros(c["m"], c["n"], dtype=torch.float64, device="cuda")
        for i, k0 in enumerate(range(0, c["k"], 128)):
            part = s["a"][:, k0:k0 + 128].double() @ s["b"][:, k0:k0 + 128].double().t()
            sb = s["sb"][:, i].double().repeat_interleave(c["rows"])[:c["n"]]
            y += s["sa"][:, i].double()[:, None] * sb[None, :] * part
        return y
    if c["op"] == "quantize":
        x, r = s["x"].double(), c["rows"]
        q = torch.empty_like(x)
        scales = torch.empty(_blocks(c["m"], r), _blocks(c["k"], 128), dtype=torch.float64, device="cuda")
        for i, k0 in enumerate(range(0, c["k"], 128)):
            blk = x[:, k0:k0 + 128]
            amax = blk.abs().amax(dim=1)
            amax = torch.nn.functional.pad(amax, (0, _blocks(c["m"], r) * r - c["m"])).view(-1, r).amax(dim=1)
            step = torch.where(amax > 0, torch.exp2(torch.ceil(torch.log2(amax / F8_MAX))), 1.0)
            step = torch.where(step * F8_MAX < amax, step * 2, step)  # a logarithm that was rounded down
            step = torch.where((amax > 0) & (step * F8_MAX / 2 >= amax), step / 2, step)  # or up
            scales[:, i] = step
            v = blk / step.repeat_interleave(r)[:c["m"], None]
            _, e = torch.frexp(v)
            ulp = torch.exp2(torch.clamp(e - 1, min=-6).double() - 3)  # e4m3: three bits after the first, down to 2^-9
            q[:, k0:k0 + 128] = torch.round(v / ulp) * ulp  # ties to even
        return q, scales
    if c["op"] == "packed":
        words, scales, zeros = s["w"]
        g = c["group"] or c["k"]
        q = _exact_codes(words, c["bits"]).double() - zeros.double().repeat_interleave(g, dim=-1)
        return q, scales.double().repeat_interleave(g, dim=-1)[:, ::128]
    x = s["x"].double()
    logits = x @ s["router"].double().t()
    p = torch.exp(logits - logits.amax(dim=1, keepdim=True))
    p = p / p.sum(dim=1, keepdim=True)
    ids = torch.argsort(p, dim=1, descending=True, stable=True)[:, :c["top"]]
    w = torch.gather(p, 1, ids)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    y = torch.zeros_like(x)
    for e in range(c["e"]):
        tok, slot = torch.nonzero(ids == e, as_tuple=True)
        if tok.numel():
            h = x[tok] @ _exact_weights(s["up"], e, c["bits"], c["group"]).t()
            if c["act"] == "silu":
                gate = x[tok] @ _exact_weights(s["gate"], e, c["bits"], c["group"]).t()
                h = h * gate * torch.sigmoid(gate)
            else:
                h = torch.relu(h)
            y.index_add_(0, tok, w[tok, slot][:, None] * (h @ _exact_weights(s["down"], e, c["bits"], c["group"]).t()))
    return y, None, w
