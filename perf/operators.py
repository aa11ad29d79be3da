"""Workloads of the MXFP4 operators and of MoE routing with its balance loss.

Five operators of mixture-of-experts inference and training:

* ``route``       softmax over the experts' logits, the top-k experts of each token
                  with their weights, the tokens per expert and the balance loss;
                  training cases also take the gradient of the logits;
* ``quantize``    1 x 32 microscaled FP4 (E2M1 codes, UE8M0 scales) of an FP32 or
                  BF16 matrix, or of its transpose, and the values read back;
* ``gemm``        D = A B^T of two MXFP4 operands, BF16 out;
* ``contiguous``  the same per expert, the experts' tokens concatenated in segments
                  padded to 128 rows;
* ``masked``      the same per expert, a fixed [G, M_max, K] buffer with a count per
                  expert on the device.

``listed()`` and ``draw(rng)`` give the cases, ``prepare`` makes what a program holds
before the call, ``run`` is one pass: the library's kernels where ``own`` is true,
else elementary torch operations in 32 bits.  ``exact`` states the operators in 64
bits, apart from both.

Sizes are those of the library's own workload table (the DeepSeek-V3/R1 inference
shapes) and generic odd ones.  Activations are N(0, 1) with each entry multiplied by
50 with probability 0.001, weights N(0, 0.02), router logits N(0, 1.5).
"""

import torch

own = False

# The values of the 16 E2M1 codes (sign, two exponent bits, one mantissa bit).
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
E2M1 = E2M1 + [-v for v in E2M1]


def listed():
    return [
        # one decode step's routing: latency
        dict(name="route_step", op="route", tokens=64, experts=32, top_k=8, dtype="fp32",
             normalize=True, masked=0.0, dead=0.0, backward=False),
        # a training step's routing, padded batch: forward and gradient
        dict(name="route_train", op="route", tokens=32768, experts=256, top_k=8, dtype="bf16",
             normalize=True, masked=0.05, dead=0.0, backward=True),
        # an odd number of experts, some of them closed to some tokens (logit -inf)
        dict(name="route_odd", op="route", tokens=5001, experts=72, top_k=6, dtype="fp32",
             normalize=False, masked=0.02, dead=0.4, backward=True),
        # activations of a prefill before an expert layer
        dict(name="quantize_rows", op="quantize", rows=4096, cols=7168, dtype="bf16",
             transpose=False),
        # an operand of a backward product, quantized along its other axis
        dict(name="quantize_transposed", op="quantize", rows=4096, cols=2112, dtype="fp32",
             transpose=True),
        # a single token through a projection: latency
        dict(name="gemm_one", op="gemm", m=1, n=2112, k=7168),
        # a decode batch: the weights' bytes
        dict(name="gemm_decode", op="gemm", m=64, n=7168, k=16384),
        # a prefill: the tensor cores' rate
        dict(name="gemm_prefill", op="gemm", m=4096, n=7168, k=16384),
        # prefill through the experts
        dict(name="contiguous_prefill", op="contiguous", groups=8, tokens=32768, n=4096, k=7168),
        # ragged: experts with few tokens or none, N and K off the tiles
        dict(name="contiguous_odd", op="contiguous", groups=13, tokens=1500, n=1448, k=1056),
        # decode through the experts, fixed buffers and counts on the device
        dict(name="masked_decode", op="masked", groups=32, m_max=256, n=7168, k=2048),
        dict(name="masked_odd", op="masked", groups=7, m_max=100, n=1000, k=544),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = lo * (hi / lo) ** rng.random()
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["route", "quantize", "gemm", "contiguous", "masked"])
    if op == "route":
        experts = _log(rng, 4, 512)
        tokens = _log(rng, 1, min(32768, 32768 * 256 // experts))
        return dict(op=op, tokens=tokens, experts=experts,
                    top_k=rng.randint(1, min(16, experts)), dtype=rng.choice(["fp32", "bf16"]),
                    normalize=rng.random() < 0.5, masked=rng.choice([0.0, 0.1]),
                    dead=rng.choice([0.0, 0.5]), backward=rng.random() < 0.7)
    if op == "quantize":
        k = _log(rng, 32, 16384, 32)
        m = _log(rng, 8, min(8192, 4096 * 7168 // k), 8)
        transpose = rng.random() < 0.4
        return dict(op=op, rows=k if transpose else m, cols=m if transpose else k,
                    dtype=rng.choice(["fp32", "bf16"]), transpose=transpose)
    if op == "gemm":
        k, n = _log(rng, 32, 16384, 32), _log(rng, 8, 24576, 8)
        return dict(op=op, m=_log(rng, 1, max(1, min(4096, 4096 * 7168 * 16384 // (n * k)))),
                    n=n, k=k)
    groups = rng.randint(1, 32)
    if op == "contiguous":
        k, n = _log(rng, 64, 7168, 32), _log(rng, 64, 4096, 8)
        groups = min(groups, max(1, 8 * 4096 * 7168 // (n * k)))
        return dict(op=op, groups=groups, tokens=_log(rng, 8, 16384), n=n, k=k)
    k, n = _log(rng, 64, 4096, 32), _log(rng, 64, 7168, 8)
    groups = min(groups, max(1, 32 * 7168 * 2048 // (n * k)))
    return dict(op=op, groups=groups, m_max=_log(rng, 1, 256), n=n, k=k)


# --------------------------------------------------------------------------- inputs
def _dtype(case):
    return {"fp32": torch.float32, "bf16": torch.bfloat16}[case["dtype"]]


def _activations(gen, *shape):
    x = torch.randn(shape, generator=gen, device="cuda")
    x.mul_(torch.where(torch.rand(shape, generator=gen, device="cuda") < 0.001, 50.0, 1.0))
    return x


def _scale_exponent(amax):
    """The smallest e with 6 * 2^e >= amax, at least -127 (amax FP32, finite)."""
    frac, e = torch.frexp(amax)  # amax = frac * 2^e, frac in [0.5, 1)
    e = e - 3 + (frac > 0.75).to(e.dtype)
    return torch.where(amax > 0, e.clamp(min=-127), torch.full_like(e, -127))


def _nearest_code(v):
    """E2M1 codes (no sign) of FP32 magnitudes up to 6, to nearest, ties to even:
    a magnitude on a border goes to the even code of its two neighbours."""
    code = torch.zeros(v.shape, dtype=torch.uint8, device=v.device)
    for border, up_on_tie in ((0.25, False), (0.75, True), (1.25, False), (1.75, True),
                              (2.5, False), (3.5, True), (5.0, False)):
        code += (v >= border) if up_on_tie else (v > border)
    return code


def _quantize(x):
    """x FP32 [.., R, K] -> (codes uint8 [.., R, K/2], scale bytes uint8 [.., R, K/32])."""
    g = x.unflatten(-1, (-1, 32))
    e = _scale_exponent(g.abs().amax(-1))
    # two steps, so that neither factor leaves FP32's range
    half = torch.div(-e, 2, rounding_mode="floor")
    v = g * _pow2(half)[..., None] * _pow2(-e - half)[..., None]
    code = _nearest_code(v.abs()) | (torch.signbit(v).to(torch.uint8) << 3)
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8)


def _pow2(e):
    """2^e in FP32 for whole e in [-126, 127], from the bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _block_scales(sb):
    """Scale bytes [.., R, K/32] -> the library's int32 words [.., R/128, K/128, 32, 4]:
    word [b, p, r, c] holds groups 4p .. 4p+3 of row 128 b + 32 c + r, the lowest group in
    the lowest byte; rows and groups past the operand are zero."""
    r, kg = sb.shape[-2:]
    rb, kw = -(-r // 128), -(-kg // 4)
    full = torch.zeros(sb.shape[:-2] + (rb * 128, kw * 4), dtype=torch.uint8, device=sb.device)
    full[..., :r, :kg] = sb
    full = full.unflatten(-1, (kw, 4)).unflatten(-3, (rb, 4, 32))  # [.., rb, c, r, kw, 4]
    full = full.movedim(-2, -4)                                    # [.., rb, kw, c, r, 4]
    return full.transpose(-2, -3).contiguous().view(torch.int32).squeeze(-1)


def _operand(gen, kind, *shape):
    """An MXFP4 operand as a program holds it: codes and scale words."""
    x = _activations(gen, *shape) if kind == "a" else \
        torch.randn(shape, generator=gen, device="cuda") * 0.02
    q, sb = _quantize(x)
    return q.contiguous(), _block_scales(sb)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case)
    op = case["op"]
    if op == "route":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        x = torch.randn((t, e), generator=gen, device="cuda") * 1.5
        if case["dead"]:
            # some tokens may only use part of the experts, a few none at all
            some = torch.rand((t, 1), generator=gen, device="cuda") < case["dead"]
            shut = torch.rand((t, e), generator=gen, device="cuda") < 0.5
            none = torch.rand((t, 1), generator=gen, device="cuda") < 0.01
            x = torch.where((some & shut) | none, float("-inf"), x)
        s["logits"] = x.to(_dtype(case))
        s["mask"] = None
        if case["masked"]:
            s["mask"] = torch.rand(t, generator=gen, device="cuda") >= case["masked"]
        if case["backward"]:
            s["dweights"] = torch.randn((t, k), generator=gen, device="cuda")
            s["dloss"] = torch.full((1,), 0.01, device="cuda")
        return s
    if op == "quantize":
        x = _activations(gen, case["rows"], case["cols"])
        x[:, : case["cols"] // 16] *= 1e-3  # groups of other sizes
        s["x"] = x.to(_dtype(case))
        return s
    n, k = case["n"], case["k"]
    if op == "gemm":
        s["a"], s["sfa"] = _operand(gen, "a", case["m"], k)
        s["b"], s["sfb"] = _operand(gen, "b", n, k)
        s["d"] = torch.zeros((case["m"], n), dtype=torch.bfloat16, device="cuda")
        return s
    g = case["groups"]
    s["b"], s["sfb"] = _operand(gen, "b", g, n, k)
    if op == "masked":
        s["masked_m"] = torch.randint(0, case["m_max"] + 1, (g,), generator=gen, device="cuda",
                                      dtype=torch.int32)
        s["a"], s["sfa"] = _operand(gen, "a", g, case["m_max"], k)
        s["d"] = torch.zeros((g, case["m_max"], n), dtype=torch.bfloat16, device="cuda")
        return s
    pick = torch.randint(0, g, (case["tokens"],), generator=gen, device="cuda")
    counts = torch.bincount(pick, minlength=g).tolist()
    padded = [-(-c // 128) * 128 for c in counts]
    rows = -(-(case["tokens"] + 127 * g) // 128) * 128  # room for any split of the tokens
    idx = torch.full((rows,), -1, dtype=torch.int32)
    row = 0
    for e, (c, p) in enumerate(zip(counts, padded)):
        idx[row:row + c] = e
        row += p
    s["m_indices"] = idx.cuda()
    s["a"], s["sfa"] = _operand(gen, "a", rows, k)
    s["d"] = torch.zeros((rows, n), dtype=torch.bfloat16, device="cuda")
    return s


# --------------------------------------------------------------------------- one pass
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import moe_grouped_gemm_act_b200 as dg
    op = s["op"]
    if op == "route":
        idx, w, counts, loss, n = dg.dg_moe_route(s["logits"], s["top_k"],
                                                  normalize=s["normalize"],
                                                  token_mask=s["mask"])
        out = dict(idx=idx, weights=w, counts=counts, loss=loss)
        if s["backward"]:
            out["dlogits"] = dg.dg_moe_route_backward(
                s["logits"], idx, w, counts, n, s["dweights"], s["dloss"],
                normalize=s["normalize"])
        return out
    if op == "quantize":
        q, sf = dg.dg_quantize_mxfp4(s["x"], transpose=s["transpose"])
        return dg.dg_dequantize_mxfp4(q, sf, torch.bfloat16)
    if op == "gemm":
        return dg.dg_mxfp4_gemm_nt(s["a"], s["sfa"], s["b"], s["sfb"], s["d"])
    if op == "contiguous":
        return dg.dg_m_grouped_mxfp4_gemm_nt_contiguous(s["a"], s["sfa"], s["b"], s["sfb"],
                                                        s["d"], s["m_indices"])
    return dg.dg_m_grouped_mxfp4_gemm_nt_masked(s["a"], s["sfa"], s["b"], s["sfb"], s["d"],
                                                s["masked_m"])


def _read(q, words):
    """The FP32 values of an MXFP4 operand (codes and scale words)."""
    kg = q.shape[-1] // 16
    table = torch.tensor([[E2M1[c & 15], E2M1[c >> 4]] for c in range(256)], device=q.device)
    v = table[q.to(torch.int32)].flatten(-2)
    sb = words.unsqueeze(-1).view(torch.uint8).transpose(-2, -3)   # [.., rb, kw, c, r, 4]
    sb = sb.movedim(-4, -2).flatten(-2).flatten(-4, -2)            # [.., R, groups]
    e = sb[..., : q.shape[-2], :kg].to(torch.int32)
    scale = torch.where(e > 0, e << 23, 1 << 22).view(torch.float32)  # 2^-127 is subnormal
    return (v.unflatten(-1, (kg, 32)) * scale[..., None]).flatten(-2)


def _plain(s):
    op = s["op"]
    if op == "route":
        return _plain_route(s)
    if op == "quantize":
        x = s["x"].float()
        x = (x.t() if s["transpose"] else x).contiguous()
        q, sb = _quantize(x)
        return _read(q, _block_scales(sb)).to(torch.bfloat16)
    a, b, d = _read(s["a"], s["sfa"]), _read(s["b"], s["sfb"]), s["d"]
    if op == "gemm":
        d.copy_(a @ b.t())
    elif op == "masked":
        live = torch.arange(d.shape[1], device=d.device) < s["masked_m"][:, None]
        d.copy_(torch.where(live[..., None], torch.bmm(a, b.transpose(1, 2)), d.float()))
    else:
        for e in range(b.shape[0]):
            rows = (s["m_indices"] == e).nonzero().flatten()
            d[rows] = (a[rows] @ b[e].t()).to(d.dtype)
    return d


def _plain_route(s):
    x = s["logits"].float()
    t, e = x.shape
    k = s["top_k"]
    live = (x > float("-inf")).any(1)
    if s["mask"] is not None:
        live = live & s["mask"]
    x = torch.where(live[:, None], x, float("-inf"))
    top = torch.where(live, x.amax(1), 0.0)
    p = torch.exp(x - top[:, None])
    p = p / torch.where(live, p.sum(1), 1.0)[:, None]
    value, idx = torch.sort(x, dim=1, descending=True, stable=True)
    value, idx = value[:, :k], idx[:, :k]
    used = value > float("-inf")
    w = torch.where(used, p.gather(1, idx), 0.0)
    if s["normalize"]:
        w = w / torch.where(live, w.sum(1), 1.0)[:, None]
    counts = torch.zeros(e, device=x.device).index_add_(
        0, idx.flatten(), used.flatten().float())
    n = live.sum().clamp(min=1).float()
    factor = e / (k * n * n)
    out = dict(idx=torch.where(used, idx, -1).to(torch.int32), weights=w,
               counts=counts.to(torch.int32), loss=(factor * (counts * p.sum(0)).sum()).view(1))
    if s["backward"]:
        c = s["dloss"] * factor * counts
        dw = torch.where(used, s["dweights"], 0.0)
        grad = p * (c - (p * c).sum(1, keepdim=True))
        if s["normalize"]:
            dv = w * (dw - (w * dw).sum(1, keepdim=True))
            grad = grad.scatter_add(1, idx, dv)
        else:
            dv = w * dw
            grad = grad.scatter_add(1, idx, dv) - p * dv.sum(1, keepdim=True)
        out["dlogits"] = grad.to(s["logits"].dtype)
    return out


# --------------------------------------------------------------------------- the work
def _operand_bytes(r, k):
    return r * k / 2 + r * k / 32


def work(case):
    op = case["op"]
    if op == "route":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        size = 4 if case["dtype"] == "fp32" else 2
        moved = t * e * size + t * k * 8 + e * 4
        flops = 5 * t * e
        if case["backward"]:
            moved += 2 * t * e * size + t * k * 12
            flops += 7 * t * e
        return {"bytes": moved, "flops": flops}
    if op == "quantize":
        size = 4 if case["dtype"] == "fp32" else 2
        r, c = case["rows"], case["cols"]
        # the input, the codes and scales written and read back, the values
        return {"bytes": r * c * size + 2 * _operand_bytes(r, c) + r * c * 2, "flops": 4 * r * c}
    n, k = case["n"], case["k"]
    if op == "gemm":
        m, g = case["m"], 1
    elif op == "contiguous":
        m, g = case["tokens"], case["groups"]
    else:
        m, g = case["groups"] * case["m_max"] // 2, case["groups"]  # counts are uniform
    return {"bytes": _operand_bytes(m, k) + g * _operand_bytes(n, k) + m * n * 2,
            "flops": 2 * m * n * k}


# --------------------------------------------------------------------------- in 64 bits
def _exact_values(q, words):
    """The operand in FP64, from the formats' definitions: a code's sign bit, two exponent
    bits (bias 1, subnormal at 0) and one mantissa bit; a scale byte e is 2^(e - 127)."""
    code = torch.stack([q & 15, q >> 4], -1).flatten(-2)
    expo, man = ((code >> 1) & 3).double(), (code & 1).double()
    mag = torch.where(expo == 0, man / 2, (1 + man / 2) * torch.exp2(expo - 1))
    v = torch.where(code >= 8, -mag, mag)
    rows, k = v.shape[-2:]
    r = torch.arange(rows, device=q.device)[:, None]
    g = torch.arange(k // 32, device=q.device)[None, :]
    word = words[..., r // 128, g // 4, r % 32, (r % 128) // 32].long()
    byte = (word >> (8 * (g % 4))) & 255
    return v * torch.exp2(byte.double() - 127).repeat_interleave(32, -1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(s)
    if op == "quantize":
        x = s["x"].double()
        g = (x.t() if case["transpose"] else x).unflatten(-1, (-1, 32))
        amax = g.abs().amax(-1, keepdim=True)
        e = torch.ceil(torch.log2(amax / 6)).clamp(min=-127)
        # log2 may be off by its last bit next to a power of two
        e = torch.where(6 * torch.exp2(e - 1) >= amax, e - 1, e)
        e = torch.where(6 * torch.exp2(e) < amax, e + 1, e).clamp(min=-127)
        v = g / torch.exp2(e)
        # spacing of the code grid at |v|: 0.5 below 2, 1 below 4, 2 above
        step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0)).double()
        return (torch.round(v / step) * step * torch.exp2(e)).flatten(-2)
    d = s["d"].double()
    if op == "gemm":
        return _exact_values(s["a"], s["sfa"]) @ _exact_values(s["b"], s["sfb"]).t()
    if op == "masked":
        for e, m in enumerate(s["masked_m"].tolist()):
            a = _exact_values(s["a"][e], s["sfa"][e])[:m]
            d[e, :m] = a @ _exact_values(s["b"][e], s["sfb"][e]).t()
        return d
    a = _exact_values(s["a"], s["sfa"])
    for e in range(case["groups"]):
        rows = s["m_indices"] == e
        d[rows] = a[rows] @ _exact_values(s["b"][e], s["sfb"][e]).t()
    return d


def _exact_route(s):
    x = s["logits"].double()
    t, e = x.shape
    k = s["top_k"]
    live = torch.isfinite(x).any(1)
    if s["mask"] is not None:
        live &= s["mask"]
    p = torch.zeros_like(x)
    p[live] = torch.softmax(x[live], 1)
    # the place of each expert in its token's order: larger logits, then lower indices
    score = torch.where(live[:, None], x, float("-inf"))
    order = torch.argsort(-score, dim=1, stable=True)[:, :k]
    used = torch.isfinite(score.gather(1, order))
    idx = torch.where(used, order, -1)
    sel = torch.zeros_like(x).scatter_add_(1, order, used.double())
    z = (p * sel).sum(1, keepdim=True)
    scale = 1 / torch.where(z > 0, z, 1) if s["normalize"] else torch.ones_like(z)
    w = p.gather(1, order) * used * scale
    counts = sel.sum(0)
    n = max(1, int(live.sum()))
    factor = e / (k * n * n)
    out = dict(idx=idx.to(torch.int32), weights=w, counts=counts.to(torch.int32),
               loss=(factor * (counts * p.sum(0)).sum()).view(1))
    if s["backward"]:
        # d/dp of both results, then through the softmax
        dw = torch.zeros_like(x).scatter_add_(1, order, s["dweights"].double() * used)
        dp = dw * scale * sel
        if s["normalize"]:
            dp = dp - sel * (dw * p * sel).sum(1, keepdim=True) * scale * scale
        dp = dp + s["dloss"].double() * factor * counts
        out["dlogits"] = p * (dp - (p * dp).sum(1, keepdim=True))
    return out
