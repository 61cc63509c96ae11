"""Measured cases of microscaled 4-bit rows (MXFP4: E2M1 codes in blocks of 32 with one E8M0
scale each) and of the router's balance: quantization and its inverse (``moe_quantize_mxfp4``,
``moe_dequantize_mxfp4``), the products by expert on such rows (``moe_grouped_gemm_mxfp4``),
the balance loss with the experts' counts (``moe_balance_loss``) and its gradient
(``moe_balance_loss_grad``).

``own`` chooses between the plain form (elementary torch operations in 32 bits) and the
library's calls.  A case's ``op`` names the operator; its other fields are sizes and options.
"""

import math

import torch

own = False

BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
E8M0 = torch.float8_e8m0fnu
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
COEF = 0.01


# ---------------------------------------------------------------------------------------
# Cases.
# ---------------------------------------------------------------------------------------
def listed():
    return [
        # a decode batch's tokens into 4 bits, with blocks that fill no whole dword of scales
        _quantize("quantize_decode", 37, 2912),
        # a prefill batch's tokens into 4 bits
        _quantize("quantize_prefill", 16384, 3584),
        # one token's first product over the experts it is routed to
        _grouped("first_token", 1, 896, 16, 384, 3584, situ=True, gather=True),
        # first product of a decode batch with the activation, most experts without rows
        _grouped("first_decode", 16, 896, 16, 384, 3584, situ=True, gather=True),
        # a dense projection of a decode batch: one matrix, a row count that no tile divides
        _grouped("projection_decode", 16, 1, 1, 7181, 7168),
        # second product of a mid batch, experts of very different popularity
        _grouped("second_mid_zipf", 1024, 896, 16, 3584, 384, zipf=1.0),
        # first product of a prefill batch, rows gathered from the tokens
        _grouped("first_prefill", 4096, 896, 16, 384, 3584, situ=True, gather=True),
        # few experts and many rows each: bound by the matrix units
        _grouped("dense_prefill", 16384, 8, 2, 3584, 4096, gather=True),
        # the load of a decode batch
        _balance("balance_decode", 64, 896, 16),
        # a training batch whose last tokens are padding
        _balance("balance_batch", 16384, 896, 16, mask=True),
        # gradient for a small batch of an odd number of experts, BF16 logits
        _balance("gradient_small", 211, 130, 4, bf16=True, grad=True),
        # gradient of a training batch, added to what the logits already have
        _balance("gradient_batch", 16384, 896, 16, mask=True, add=True, grad=True),
    ]


def _quantize(name, T, K):
    return _named(name, {"op": "quantize", "T": T, "K": K})


def _grouped(name, T, E, k, N, K, situ=False, gather=False, zipf=0.0):
    return _named(name, {"op": "grouped", "T": T, "E": E, "k": k, "N": N, "K": K, "situ": situ,
                         "gather": gather, "zipf": zipf})


def _balance(name, T, E, k, bf16=False, mask=False, add=False, grad=False):
    return _named(name, {"op": "gradient" if grad else "balance", "T": T, "E": E, "k": k,
                         "bf16": bf16, "mask": mask, "add": add})


def _named(name, case):
    return dict(case, name=name) if name else case


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], its logarithm uniform."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(max(step * round(v / step), lo), hi)


def draw(rng):
    op = rng.choice(["quantize", "grouped", "grouped", "balance", "gradient"])
    flip = lambda: rng.random() < 0.5  # noqa: E731
    if op == "quantize":
        K = _log(rng, 32, 16384, 32)
        return _quantize(None, _log(rng, 1, min(16384, 16384 * 3584 // K)), K)
    if op != "grouped":
        E = _log(rng, 2, 4096)
        k = min(E, _log(rng, 1, 16))
        T = _log(rng, 1, min(65536, 16384 * 896 // E))
        return _balance(None, T, E, k, bf16=flip(), mask=flip(), add=flip() and op == "gradient",
                        grad=op == "gradient")
    while True:
        situ, gather, zipf = flip(), flip(), rng.choice([0.0, 1.0])
        E = _log(rng, 1, 896)
        k = min(E, _log(rng, 1, 16))
        N, K, T = _log(rng, 16, 8192), _log(rng, 128, 7168, 32), _log(rng, 1, 16384)
        rows, weights = N * (2 if situ else 1), E * N * (2 if situ else 1) * K
        # the work of the listed cases, and padded 32-bit rows of the plain form that fit
        if (weights <= 1 << 31 and T * k * rows * K <= 1 << 38
                and min(E, T * k) * T * (rows + K) <= 1 << 32):
            return _grouped(None, T, E, k, N, K, situ=situ, gather=gather, zipf=zipf)


# ---------------------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    return {"quantize": _prepare_quantize, "grouped": _prepare_grouped,
            "balance": _prepare_balance, "gradient": _prepare_balance}[case["op"]](case, g)


def _empty(*shape, dtype=BF16):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _normal(g, *shape, std=1.0, dtype=BF16):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def _uniform(g, lo, hi, *shape):
    return torch.empty(shape, dtype=F32, device="cuda").uniform_(lo, hi, generator=g)


def _tokens(g, T, H):
    """BF16 token rows with one channel in a hundred twenty times larger."""
    x = _normal(g, T, H)
    return x.mul_(1.0 + 19.0 * (_uniform(g, 0, 1, H) < 0.01).to(BF16))


def _stride(K):
    """Bytes between two rows of scales: whole dwords."""
    return (K + 127) // 128 * 4


def _prepare_quantize(c, g):
    T, K = c["T"], c["K"]
    return dict(c, x=_tokens(g, T, K), codes=_empty(T, K // 2, dtype=torch.uint8),
                scales=_empty(T, _stride(K), dtype=torch.uint8), out=_empty(T, K))


def _microscale(x):
    """(rounded values before the scale, scale bytes, scales) of rows [T, K] in blocks of 32: the
    scale is the power of two that brings the block's largest magnitude into [4, 8), the values go
    to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6, ties to the even code."""
    v = x.float().view(x.shape[0], -1, 32)
    byte = (((v.abs().amax(2).view(I32) >> 23) & 255) - 2).clamp_(min=0)
    v = v * ((254 - byte) << 23).view(F32)[:, :, None]
    m = v.abs()
    step = 0.5 + 0.5 * (m >= 2).float() + (m >= 4).float()
    m = ((m / step).round() * step).clamp_(max=6.0)
    return torch.copysign(m, v), byte, (byte << 23).view(F32)


def _pack(v, byte):
    """Codes [T, K/2] and scales [T, stride] of _microscale's values."""
    T = v.shape[0]
    m = v.abs().view(T, -1)
    code = (2 * m).to(torch.uint8)                                      # 0, 0.5, 1, 1.5, 2
    code = code - (m >= 3).to(torch.uint8) - (m >= 4).to(torch.uint8) - 3 * (m >= 6).to(torch.uint8)
    code = (code + 8 * torch.signbit(v).view(T, -1).to(torch.uint8)).view(T, -1, 2)
    scales = torch.zeros((T, _stride(m.shape[1])), dtype=torch.uint8, device=v.device)
    scales[:, :byte.shape[1]] = byte.to(torch.uint8)
    return code[:, :, 0] + 16 * code[:, :, 1], scales


def _prepare_grouped(c, g):
    T, E, k, N, K = (c[n] for n in ("T", "E", "k", "N", "K"))
    Nw, R = N * (2 if c["situ"] else 1), T * k
    # experts drawn without replacement from popularities (e + 1)^-zipf
    logp = -c["zipf"] * torch.arange(1, E + 1, device="cuda", dtype=F32).log()
    gumbel = -(-_uniform(g, 1e-7, 1.0, T, E).log()).log()
    ids = (logp + gumbel).topk(k, dim=1).indices.reshape(-1)
    order = torch.sort(ids, stable=True).indices
    counts = torch.bincount(ids, minlength=E)
    rows = T if c["gather"] else R
    x = torch.empty((rows, K // 2), dtype=torch.uint8, device="cuda")
    xs = torch.empty((rows, _stride(K)), dtype=torch.uint8, device="cuda")
    channels = 1.0 + 19.0 * (_uniform(g, 0, 1, K) < 0.01).to(BF16)
    for r in range(0, rows, 32768):
        n = min(32768, rows - r)
        v, byte, _ = _microscale(_normal(g, n, K) * channels)
        x[r:r + n], xs[r:r + n] = _pack(v, byte)
    w = torch.empty((E * Nw, K // 2), dtype=torch.uint8, device="cuda")
    ws = torch.empty((E * Nw, _stride(K)), dtype=torch.uint8, device="cuda")
    at = max(1, (1 << 27) // K)
    for r in range(0, E * Nw, at):
        n = min(at, E * Nw - r)
        v, byte, _ = _microscale(_normal(g, n, K, std=0.02))
        w[r:r + n], ws[r:r + n] = _pack(v, byte)
    s = dict(c, R=R, x_rows=rows, cumsum=counts.cumsum(0).to(I32), x=x, x_scales=xs,
             w=w.view(E, Nw, K // 2), w_scales=ws.view(E, Nw, -1),
             row_idx=order.to(I32) if c["gather"] else None,
             beta=_uniform(g, 3, 5, E) if c["situ"] else None,
             lam=_uniform(g, 20, 30, E) if c["situ"] else None, out=_empty(R, N))
    # the plan a program makes from the routing: experts with rows, the largest number of them
    s["present"], s["most"] = counts.nonzero().reshape(-1), int(counts.max())
    return s


def _prepare_balance(c, g):
    T, E, k = c["T"], c["E"], c["k"]
    dtype = BF16 if c["bf16"] else F32
    # logits of a router in training: some experts are liked more than others
    logits = (_normal(g, T, E, std=1.5, dtype=F32) + _normal(g, E, std=0.5, dtype=F32)).to(dtype)
    ids = logits.float().topk(k, dim=1).indices.to(I32)
    s = dict(c, logits=logits, ids=ids, mask=None)
    if c["mask"]:                                    # about a tenth of the batch is padding
        s["mask"] = torch.arange(T, device="cuda") < T - T // 10
    if c["op"] == "balance":
        s.update(counts=_empty(E, dtype=I32), sums=_empty(E, dtype=F32), tokens=_empty(1, dtype=I32),
                 loss=_empty(1, dtype=F32), workspace=None)
        return s
    live = ids if s["mask"] is None else ids[s["mask"]]
    s.update(counts=torch.bincount(live.reshape(-1), minlength=E).to(I32),
             tokens=torch.tensor([live.shape[0]], dtype=I32, device="cuda"),
             grad_loss=torch.tensor([0.25], dtype=F32, device="cuda"),
             # as large as the balance's own gradient
             more=_normal(g, T, E, std=0.25 * COEF / (T * E), dtype=F32).to(dtype) if c["add"] else None,
             grad=_empty(T, E, dtype=dtype))
    return s


# ---------------------------------------------------------------------------------------
# One pass.
# ---------------------------------------------------------------------------------------
def run(state):
    return (_own if own else _plain)[state["op"]](state)


def _plain_quantize(s):
    T, K = s["T"], s["K"]
    v, byte, scale = _microscale(s["x"])
    scales = torch.zeros((T, _stride(K)), dtype=torch.uint8, device="cuda")
    scales[:, :K // 32] = byte.to(torch.uint8)
    return {"values": (v * scale[:, :, None]).view(T, K).to(BF16), "scales": scales.view(E8M0)}


def _decode(codes, scales):
    """FP32 values [..., K] of codes [..., K/2] and scales [..., stride]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=F32, device="cuda")
    K = codes.shape[-1] * 2
    v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1)
    scale = (scales[..., :K // 32].int() << 23).view(F32)
    return (v.view(*codes.shape[:-1], K // 32, 32) * scale[..., None]).view(*codes.shape[:-1], K)


def _plain_grouped(s):
    R, N, most, present = s["R"], s["N"], s["most"], s["present"]
    ends = s["cumsum"].long()[present]
    starts = torch.cat((torch.zeros_like(ends[:1]), ends[:-1]))
    rows = starts[:, None] + torch.arange(most, device="cuda")          # [experts, most]
    there = rows < ends[:, None]
    rows = rows.clamp(max=R - 1)
    src = s["row_idx"].long()[rows] // s["k"] if s["gather"] else rows
    x = _decode(s["x"], s["x_scales"])
    w = _decode(s["w"][present], s["w_scales"][present])
    h = torch.bmm(x[src], w.transpose(1, 2).contiguous())
    if s["situ"]:
        beta, lam = s["beta"][present][:, None, None], s["lam"][present][:, None, None]
        gate, up = h[:, :, :N], h[:, :, N:]
        h = (beta * torch.tanh(gate / beta) * torch.sigmoid(gate)) * (lam * torch.tanh(up / lam))
    return h[there].to(BF16)


def _probabilities(s):
    z = s["logits"].float()
    p = torch.exp(z - z.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True)
    return p if s["mask"] is None else torch.where(s["mask"][:, None], p, 0.0)


def _plain_balance(s):
    T, E = s["T"], s["E"]
    ids = s["ids"].long()
    if s["mask"] is not None:
        ids = torch.where(s["mask"][:, None], ids, E)
    ones = torch.ones(ids.numel(), dtype=I32, device="cuda")
    counts = torch.zeros(E + 1, dtype=I32, device="cuda").index_add_(0, ids.reshape(-1), ones)[:E]
    sums = _probabilities(s).sum(0)
    tokens = torch.full((1,), T, dtype=I32, device="cuda")
    if s["mask"] is not None:
        tokens = s["mask"].sum(dtype=I32).reshape(1)
    share = counts.float() / counts.sum().clamp(min=1)
    loss = COEF * E * (share * sums).sum().reshape(1) / tokens.clamp(min=1)
    return {"counts": counts, "sums": sums, "tokens": tokens, "loss": loss}


def _plain_gradient(s):
    E = s["E"]
    p = _probabilities(s)
    # a constant takes nothing from the gradient: the mean goes first, in 64 bits, so that nearly
    # equal counts keep their differences and equal ones give zeros
    counts = s["counts"].double()
    share = ((counts - counts.mean()) / counts.sum().clamp(min=1)).float()
    scale = s["grad_loss"] * (COEF * E) / s["tokens"].clamp(min=1)
    grad = scale * p * (share - (p * share).sum(1, keepdim=True))
    if s["more"] is not None:
        grad = grad + s["more"].float()
    return grad.to(s["logits"].dtype)


_plain = {"quantize": _plain_quantize, "grouped": _plain_grouped, "balance": _plain_balance,
          "gradient": _plain_gradient}


def _own_quantize(s):
    import routed_moe_layer_amd as rm
    rm.moe_quantize_mxfp4(s["x"], s["T"], s["K"], s["codes"], s["scales"])
    rm.moe_dequantize_mxfp4(s["codes"], s["scales"], s["T"], s["K"], s["out"])
    return {"values": s["out"], "scales": s["scales"].view(E8M0)}


def _own_grouped(s):
    import routed_moe_layer_amd as rm
    rm.moe_grouped_gemm_mxfp4(s["R"], s["N"], s["K"], s["E"], s["x"], s["x_scales"], s["cumsum"],
                              s["w"], s["w_scales"], s["out"], x_rows=s["x_rows"],
                              row_idx=s["row_idx"], row_div=s["k"], situ=s["situ"],
                              situ_beta=s["beta"], situ_linear_beta=s["lam"])
    return s["out"]


def _own_balance(s):
    import routed_moe_layer_amd as rm
    if s["workspace"] is None:                       # kept from the first pass on
        s["workspace"] = _empty(rm.moe_balance_workspace_size(s["T"], s["E"]), dtype=torch.uint8)
    rm.moe_balance_loss(s["T"], s["E"], s["k"], s["logits"], s["ids"], COEF, s["counts"], s["sums"],
                        s["tokens"], s["loss"], s["workspace"], token_mask=s["mask"],
                        logits_bf16=s["bf16"])
    return {"counts": s["counts"], "sums": s["sums"], "tokens": s["tokens"], "loss": s["loss"]}


def _own_gradient(s):
    import routed_moe_layer_amd as rm
    rm.moe_balance_loss_grad(s["T"], s["E"], s["logits"], s["counts"], s["tokens"], COEF, s["grad"],
                             grad_loss=s["grad_loss"], token_mask=s["mask"], add=s["more"],
                             logits_bf16=s["bf16"])
    return s["grad"]


_own = {"quantize": _own_quantize, "grouped": _own_grouped, "balance": _own_balance,
        "gradient": _own_gradient}


# ---------------------------------------------------------------------------------------
# What one pass cannot do without.
# ---------------------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "quantize":                        # the rows, their codes and scales, the values
        T, K = c["T"], c["K"]
        return {"bytes": T * (2 * K + K / 2 + _stride(K) + 2 * K), "flops": 4 * T * K}
    if c["op"] in ("balance", "gradient"):
        T, E, k, size = c["T"], c["E"], c["k"], 2 if c["bf16"] else 4
        live = T - T // 10 if c["mask"] else T
        if c["op"] == "balance":
            return {"bytes": live * (E * size + 4 * k) + T * c["mask"] + 8 * E, "flops": 4 * live * E}
        return {"bytes": live * E * size + T * E * size * (2 if c["add"] else 1) + T * c["mask"],
                "flops": 8 * live * E}
    T, E, k, N, K = (c[n] for n in ("T", "E", "k", "N", "K"))
    Nw, R = N * (2 if c["situ"] else 1), T * k
    # expected number of experts with rows: popularities p, T independent tokens of k picks
    p = [(e + 1) ** -c["zipf"] for e in range(E)]
    total = sum(p)
    used = sum(1.0 - (1.0 - min(1.0, v / total * k)) ** T for v in p)
    rows = T if c["gather"] else R
    return {"bytes": (used * Nw + rows) * (K / 2 + _stride(K)) + R * N * 2,
            "flops": 2.0 * R * Nw * K}


# ---------------------------------------------------------------------------------------
# The definitions in 64 bits.
# ---------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"quantize": _exact_quantize, "grouped": _exact_grouped, "balance": _exact_balance,
            "gradient": _exact_gradient}[case["op"]](s)


def _exact_quantize(s):
    T, K = s["T"], s["K"]
    values, scales = [], torch.full((T, _stride(K)), 2.0 ** -127, dtype=F64, device="cuda")
    for lo in range(0, T, 2048):
        v = s["x"][lo:lo + 2048].double().view(-1, K // 32, 32)
        top = v.abs().max(2).values
        shared = torch.frexp(top).exponent.double() - 1.0 - 2.0      # floor(log2) - 2
        scale = torch.exp2(torch.where(top == 0, -127.0, shared.clamp(min=-127.0)))
        m = (v / scale[:, :, None]).abs()
        # borders between neighbours; one whose lower neighbour has the even code keeps it
        got = torch.zeros_like(m)
        for lower, upper, keeps in zip(E2M1, E2M1[1:], (True, False) * 4):
            border = (lower + upper) / 2
            got += (upper - lower) * ((m > border) if keeps else (m >= border)).double()
        values.append((torch.sign(v) * got * scale[:, :, None]).view(-1, K))
        scales[lo:lo + 2048, :K // 32] = scale
    return {"values": torch.cat(values), "scales": scales}


def _exact_decode(codes, scales):
    K = codes.shape[1] * 2
    v = torch.empty((codes.shape[0], K), dtype=F64, device="cuda")
    for half in (0, 1):
        nib = (codes.int() >> (4 * half)) & 15
        e, m = (nib >> 1) & 3, nib & 1
        mag = torch.where(e == 0, 0.5 * m.double(), (1.0 + 0.5 * m) * torch.exp2(e.double() - 1))
        v[:, half::2] = torch.where(nib >= 8, -mag, mag)
    return v * torch.exp2(scales[:, :K // 32].double() - 127.0).repeat_interleave(32, dim=1)


def _exact_grouped(s):
    if 2.0 * s["R"] * s["w"].shape[1] * s["K"] > 5e14:
        return None
    out = torch.zeros((s["R"], s["N"]), dtype=F64, device="cuda")
    ends, at = s["cumsum"].tolist(), 0
    for e, end in enumerate(ends):
        if end > at:
            src = s["row_idx"][at:end].long() // s["k"] if s["gather"] else slice(at, end)
            x = _exact_decode(s["x"][src], s["x_scales"][src])
            h = x @ _exact_decode(s["w"][e], s["w_scales"][e]).t().contiguous()
            if s["situ"]:
                b, m = s["beta"][e].double(), s["lam"][e].double()
                gate, up = h[:, :s["N"]], h[:, s["N"]:]
                h = b * torch.tanh(gate / b) / (1.0 + torch.exp(-gate)) * m * torch.tanh(up / m)
            out[at:end] = h
        at = end
    return out


def _exact_balance(s):
    E = s["E"]
    live = slice(None) if s["mask"] is None else s["mask"]
    z, ids = s["logits"][live].double(), s["ids"][live].long()
    sums = torch.exp(z - torch.logsumexp(z, 1, keepdim=True)).sum(0)
    counts = torch.bincount(ids.reshape(-1), minlength=E)
    loss = COEF * E * (counts.double() / max(1, ids.numel()) * sums).sum() / max(1, z.shape[0])
    return {"counts": None, "sums": sums, "tokens": None, "loss": loss.reshape(1)}


def _exact_gradient(s):
    E = s["E"]
    grad = torch.zeros((s["T"], E), dtype=F64, device="cuda")
    live = torch.ones(s["T"], dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
    z = s["logits"][live].double()
    p = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
    n = s["counts"].long().sum()
    f = (E * s["counts"].long() - n).double() / (E * n.clamp(min=1)).double()
    f = f * (s["grad_loss"].double() * COEF * E / s["tokens"].double().clamp(min=1))
    grad[live] = p * f - p * (p @ f[:, None])
    return grad if s["more"] is None else grad + s["more"].double()
