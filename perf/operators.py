"""Measured cases of the operators that take a token batch through an expert layer whose
weights are BF16 or 8 bits wide, stage by stage: the norm before it (``moe_rmsnorm``), the
dense projection that makes the router's logits (``moe_matvec_nvfp4``), the products by
expert (``moe_grouped_gemm``) and the weighted sum back into tokens (``moe_combine``).

``own`` chooses between the plain form (elementary torch operations in 32 bits) and the
library's calls.  A case's ``op`` names the operator; its other fields are sizes and options.
"""

import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
EPS = 1e-6
CODE_MAX = {"int8": 127.0, "e4m3": 448.0}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------------------
# Cases.
# ---------------------------------------------------------------------------------------
def listed():
    return [
        # one decoded token: the residual's addition, the norm for the router, 8-bit rows
        _norm("norm_token", 1, 3584, "e4m3", residual=True, y=True),
        # a decode batch whose rows go on in int8 only
        _norm("norm_decode_int8", 64, 7168, "int8", residual=True, y=False),
        # a prefill batch, every output
        _norm("norm_prefill", 16384, 3584, "e4m3", residual=True, y=True),
        # the router's logits of one token: few weight rows, FP32 out
        _matvec("logits_token", 1, 896, 3584, f32=True),
        # a wide projection of one token: the weight stream alone
        _matvec("projection_token", 1, 16384, 7168),
        # the same kind of projection for a decode batch, a row count that no tile divides
        _matvec("projection_decode", 16, 7181, 7168),
        # first product of a decode batch with the activation, most experts without rows
        _grouped("first_decode", 16, 896, 16, 384, 3584, "bf16", situ=True, gather=True),
        # second product of a mid batch, experts of very different popularity
        _grouped("second_mid_zipf", 1024, 896, 16, 3584, 384, "bf16", zipf=1.0),
        # first product of a prefill batch in int8, rows gathered from the tokens
        _grouped("first_prefill_int8", 4096, 896, 16, 384, 3584, "int8", situ=True, gather=True),
        # few experts and many rows each: bound by the matrix units
        _grouped("dense_prefill_e4m3", 16384, 8, 2, 3584, 4096, "e4m3", gather=True),
        # a decode batch's rows back into its tokens
        _combine("combine_decode", 16, 16, 3584, add=True),
        # a prefill batch's rows, some of them dropped at an expert's capacity
        _combine("combine_prefill", 16384, 16, 3584, drop=True),
    ]


def _norm(name, T, H, q, residual=True, y=True):
    return _named(name, {"op": "rmsnorm", "T": T, "H": H, "q": q, "residual": residual, "y": y})


def _matvec(name, T, N, K, f32=False):
    return _named(name, {"op": "matvec", "T": T, "N": N, "K": K, "f32": f32})


def _grouped(name, T, E, k, N, K, q, situ=False, gather=False, zipf=0.0):
    return _named(name, {"op": "grouped", "T": T, "E": E, "k": k, "N": N, "K": K, "q": q,
                         "situ": situ, "gather": gather, "zipf": zipf})


def _combine(name, T, k, H, add=False, drop=False):
    return _named(name, {"op": "combine", "T": T, "k": k, "H": H, "add": add, "drop": drop})


def _named(name, case):
    return dict(case, name=name) if name else case


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], its logarithm uniform."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(max(step * round(v / step), lo), hi)


def draw(rng):
    op = rng.choice(["rmsnorm", "matvec", "grouped", "grouped", "combine"])
    flip = lambda: rng.random() < 0.5  # noqa: E731
    if op == "rmsnorm":
        H = _log(rng, 128, 16384, 8)
        T = _log(rng, 1, min(16384, 16384 * 3584 // H))
        q = rng.choice(["none", "int8", "e4m3"])
        return _norm(None, T, H, q, residual=flip(), y=q == "none" or flip())
    if op == "matvec":
        K = _log(rng, 128, 16384, 16)
        N = _log(rng, 16, min(32768, 16384 * 7168 // K))
        return _matvec(None, _log(rng, 1, 64), N, K, f32=flip())
    if op == "combine":
        H, k = _log(rng, 128, 16384, 8), _log(rng, 1, 64)
        T = _log(rng, 1, min(16384, 16384 * 16 * 3584 // (H * k)))
        return _combine(None, T, k, H, add=flip(), drop=flip())
    while True:
        q, situ, gather, zipf = rng.choice(["bf16", "int8", "e4m3"]), flip(), flip(), rng.choice([0.0, 1.0])
        E = _log(rng, 1, 896)
        k = min(E, _log(rng, 1, 16))
        N, K, T = _log(rng, 16, 4096), _log(rng, 128, 7168, 16), _log(rng, 1, 16384)
        rows, weights = N * (2 if situ else 1), E * N * (2 if situ else 1) * K
        # the work of the listed cases, and padded 32-bit rows of the plain form that fit
        if (weights <= 1 << 30 and T * k * rows * K <= 1 << 37
                and min(E, T * k) * T * (rows + K) <= 1 << 32):
            return _grouped(None, T, E, k, N, K, q, situ=situ, gather=gather, zipf=zipf)


# ---------------------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    return {"rmsnorm": _prepare_norm, "matvec": _prepare_matvec, "grouped": _prepare_grouped,
            "combine": _prepare_combine}[case["op"]](case, g)


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


def _code_dtype(q):
    return {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}[q]


def _prepare_norm(c, g):
    T, H, q = c["T"], c["H"], c["q"]
    s = dict(c, x=_tokens(g, T, H), weight=(1.0 + 0.1 * _normal(g, H, dtype=F32)).to(BF16))
    s["res"] = _normal(g, T, H, std=2.0) if c["residual"] else None
    s["res_out"] = _empty(T, H) if c["residual"] else None
    s["out"] = _empty(T, H) if c["y"] else None
    s["codes"] = s["scales"] = s["values"] = None
    if q != "none":
        s["codes"], s["scales"] = _empty(T, H, dtype=_code_dtype(q)), _empty(T, dtype=F32)
    if q == "int8":
        s["values"] = _empty(T, H)
    return s


def _prepare_matvec(c, g):
    T, N, K = c["T"], c["N"], c["K"]
    w = _normal(g, N, K, std=0.02, dtype=F32)
    amax = w.abs().amax()
    q = (448.0 * 6.0 / amax).reshape(1)
    blocks = w.view(N, K // 16, 16)
    s8 = (blocks.abs().amax(2) * q / 6.0).clamp_(max=448.0).to(torch.float8_e4m3fn)
    s = s8.float()
    enc = torch.where(s == 0, torch.zeros_like(s), q / s)
    v = (blocks * enc[:, :, None]).view(N, K)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    code = (torch.bucketize(v.abs(), edges) + 8 * (v < 0)).to(torch.uint8).view(N, K // 2, 2)
    return dict(c, x=_tokens(g, T, K), codes=(code[:, :, 0] + 16 * code[:, :, 1]).contiguous(),
                scales=s8.view(torch.uint8).contiguous(), alpha=1.0 / q,
                out=_empty(T, N, dtype=F32 if c["f32"] else BF16))


def _prepare_grouped(c, g):
    T, E, k, N, K, q = (c[n] for n in ("T", "E", "k", "N", "K", "q"))
    Nw, R = N * (2 if c["situ"] else 1), T * k
    # experts drawn without replacement from popularities (e + 1)^-zipf
    logp = -c["zipf"] * torch.arange(1, E + 1, device="cuda", dtype=F32).log()
    gumbel = -(-_uniform(g, 1e-7, 1.0, T, E).log()).log()
    ids = (logp + gumbel).topk(k, dim=1).indices.reshape(-1)
    order = torch.sort(ids, stable=True).indices
    counts = torch.bincount(ids, minlength=E)
    rows = T if c["gather"] else R
    x = _tokens(g, rows, K)
    w = _empty(E, Nw, K)
    for e in range(0, E, 64):
        w[e:e + 64].normal_(0.0, 0.02, generator=g)
    s = dict(c, R=R, x_rows=rows, cumsum=counts.cumsum(0).to(torch.int32), x=x, w=w,
             row_idx=order.to(torch.int32) if c["gather"] else None, x_scale=None, w_scale=None,
             beta=_uniform(g, 3, 5, E) if c["situ"] else None,
             lam=_uniform(g, 20, 30, E) if c["situ"] else None, out=_empty(R, N))
    # the plan a program makes from the routing: experts with rows, the largest number of them
    s["present"], s["most"] = counts.nonzero().reshape(-1), int(counts.max())
    if q != "bf16":
        s["x"], s["x_scale"] = _quantize_rows(x, q)
        s["w"], s["w_scale"] = _empty(E, Nw, K, dtype=_code_dtype(q)), _empty(E, Nw, dtype=F32)
        for e in range(0, E, 64):
            s["w"][e:e + 64], s["w_scale"][e:e + 64] = _quantize_rows(w[e:e + 64], q)
    return s


def _quantize_rows(x, q):
    v = x.float()
    scale = v.abs().amax(-1) / CODE_MAX[q]
    v = v / scale.clamp(min=1e-30)[..., None]
    return (v.round() if q == "int8" else v).to(_code_dtype(q)), scale


def _prepare_combine(c, g):
    T, k, H = c["T"], c["k"], c["H"]
    R = T * k
    idx = torch.randperm(R, generator=g, device="cuda").to(torch.int32)
    if c["drop"]:
        idx = torch.where(_uniform(g, 0, 1, R) < 0.02, torch.full_like(idx, -1), idx)
    rows = _empty(R, H)
    for r in range(0, R, 65536):
        rows[r:r + 65536].normal_(0.0, 1.0, generator=g)
    return dict(c, R=R, rows=rows, idx=idx, weights=_normal(g, T, k, dtype=F32).softmax(1).to(BF16),
                add=_normal(g, T, H) if c["add"] else None, out=_empty(T, H))


# ---------------------------------------------------------------------------------------
# One pass.
# ---------------------------------------------------------------------------------------
def run(state):
    return (_own if own else _plain)[state["op"]](state)


def _plain_norm(s):
    h = s["x"].float()
    if s["residual"]:
        h = h + s["res"].float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["weight"].float()
    got = {"res": h.to(BF16) if s["residual"] else None, "y": y.to(BF16) if s["y"] else None}
    q = s["q"]
    if q != "none":
        scale = y.abs().amax(1) / CODE_MAX[q]
        v = torch.where(scale[:, None] == 0, torch.zeros_like(y), y / scale[:, None])
        got["scales"] = scale
        if q == "int8":
            got["values"] = (v.round().clamp(-127, 127) * scale[:, None]).to(BF16)
        else:
            got["codes"] = v.clamp(-448, 448).to(torch.float8_e4m3fn)
    return got


def _plain_matvec(s):
    T, N, K = s["T"], s["N"], s["K"]
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=F32, device="cuda")
    c = s["codes"]
    v = torch.stack((table[(c & 15).int()], table[(c >> 4).int()]), 2).view(N, K // 16, 16)
    w = (v * s["scales"].view(torch.float8_e4m3fn).float()[:, :, None]).view(N, K)
    out = (s["x"].float() @ w.t()) * s["alpha"]
    return out if s["f32"] else out.to(BF16)


def _plain_grouped(s):
    R, N, most, present = s["R"], s["N"], s["most"], s["present"]
    ends = s["cumsum"].long()[present]
    starts = torch.cat((torch.zeros_like(ends[:1]), ends[:-1]))
    rows = starts[:, None] + torch.arange(most, device="cuda")          # [experts, most]
    there = rows < ends[:, None]
    rows = rows.clamp(max=R - 1)
    src = s["row_idx"].long()[rows] // s["k"] if s["gather"] else rows
    x = s["x"].float()
    w = s["w"][present].float()
    if s["q"] != "bf16":
        x = x * s["x_scale"][:, None]
        w = w * s["w_scale"][present][:, :, None]
    h = torch.bmm(x[src], w.transpose(1, 2).contiguous())
    if s["situ"]:
        beta, lam = s["beta"][present][:, None, None], s["lam"][present][:, None, None]
        gate, up = h[:, :, :N], h[:, :, N:]
        h = (beta * torch.tanh(gate / beta) * torch.sigmoid(gate)) * (lam * torch.tanh(up / lam))
    return h[there].to(BF16)


def _plain_combine(s):
    T, k, H = s["T"], s["k"], s["H"]
    idx = s["idx"].long()
    w = torch.where(idx < 0, 0.0, s["weights"].float().reshape(-1)).view(T, 1, k)
    out = torch.bmm(w, s["rows"][idx.clamp(min=0)].float().view(T, k, H)).view(T, H)
    if s["add"] is not None:
        out = out + s["add"].float()
    return out.to(BF16)


_plain = {"rmsnorm": _plain_norm, "matvec": _plain_matvec, "grouped": _plain_grouped,
          "combine": _plain_combine}


def _quant(q):
    import routed_moe_layer_amd as rm
    return {"none": rm.MOE_QUANT_NONE, "bf16": rm.MOE_QUANT_NONE,
            "int8": rm.MOE_QUANT_INT8_ROW_DYNAMIC, "e4m3": rm.MOE_QUANT_E4M3_ROW_DYNAMIC}[q]


def _own_norm(s):
    import routed_moe_layer_amd as rm
    rm.moe_rmsnorm(s["T"], s["H"], s["x"], s["res"], s["weight"], EPS, _quant(s["q"]),
                   s["res_out"], s["out"], s["codes"], s["scales"])
    got = {"res": s["res_out"], "y": s["out"]}
    if s["q"] != "none":
        got["scales"] = s["scales"]
        if s["q"] == "int8":
            got["values"] = torch.mul(s["codes"], s["scales"][:, None], out=s["values"])
        else:
            got["codes"] = s["codes"]
    return got


def _own_matvec(s):
    import routed_moe_layer_amd as rm
    rm.moe_matvec_nvfp4(s["T"], s["N"], s["K"], s["x"], s["codes"], s["scales"], s["alpha"],
                        s["out"], out_f32=s["f32"])
    return s["out"]


def _own_grouped(s):
    import routed_moe_layer_amd as rm
    rm.moe_grouped_gemm(s["R"], s["N"], s["K"], s["E"], s["x"], s["cumsum"], s["w"], s["out"],
                        quant=_quant(s["q"]), x_scale=s["x_scale"], w_scale=s["w_scale"],
                        x_rows=s["x_rows"], row_idx=s["row_idx"], row_div=s["k"], situ=s["situ"],
                        situ_beta=s["beta"], situ_linear_beta=s["lam"])
    return s["out"]


def _own_combine(s):
    import routed_moe_layer_amd as rm
    rm.moe_combine(s["T"], s["H"], s["k"], s["R"], s["rows"], s["idx"], s["weights"], s["add"],
                   s["out"])
    return s["out"]


_own = {"rmsnorm": _own_norm, "matvec": _own_matvec, "grouped": _own_grouped,
        "combine": _own_combine}


# ---------------------------------------------------------------------------------------
# What one pass cannot do without.
# ---------------------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "rmsnorm":
        per = 2 + 2 * c["y"] + (4 if c["residual"] else 0) + (0 if c["q"] == "none" else 1)
        return {"bytes": c["T"] * c["H"] * per + 2 * c["H"] + 4 * c["T"], "flops": 6 * c["T"] * c["H"]}
    if c["op"] == "matvec":
        T, N, K = c["T"], c["N"], c["K"]
        return {"bytes": N * K * 9 / 16 + 2 * T * K + T * N * (4 if c["f32"] else 2),
                "flops": 2 * T * N * K}
    if c["op"] == "combine":
        T, k, H = c["T"], c["k"], c["H"]
        return {"bytes": T * k * (2 * H + 6) + 2 * T * H * (2 if c["add"] else 1),
                "flops": 2 * T * k * H}
    T, E, k, N, K = (c[n] for n in ("T", "E", "k", "N", "K"))
    size, Nw, R = (2 if c["q"] == "bf16" else 1), N * (2 if c["situ"] else 1), T * k
    # expected number of experts with rows: popularities p, T independent tokens of k picks
    p = [(e + 1) ** -c["zipf"] for e in range(E)]
    total = sum(p)
    used = sum(1.0 - (1.0 - min(1.0, v / total * k)) ** T for v in p)
    rows = T if c["gather"] else R
    return {"bytes": used * Nw * K * size + rows * K * size + R * N * 2,
            "flops": 2.0 * R * Nw * K}


# ---------------------------------------------------------------------------------------
# The definitions in 64 bits.
# ---------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"rmsnorm": _exact_norm, "matvec": _exact_matvec, "grouped": _exact_grouped,
            "combine": _exact_combine}[case["op"]](s)


def _exact_norm(s):
    got = {"res": [], "y": [], "scales": [], "values": [], "codes": []}
    for lo in range(0, s["T"], 2048):
        h = s["x"][lo:lo + 2048].double()
        if s["res"] is not None:
            h = h + s["res"][lo:lo + 2048].double()
        got["res"].append(h)
        rms = ((h ** 2).sum(1) / s["H"] + EPS).sqrt()
        y = h / rms[:, None] * s["weight"].double()
        got["y"].append(y)
        if s["q"] != "none":
            step = y.abs().max(1).values / CODE_MAX[s["q"]]
            got["scales"].append(step)
            v = y / step.clamp(min=1e-300)[:, None]
            got["values"].append(torch.round(v) * step[:, None])
            # nearest E4M3 value: 4 significant bits, steps of 2^-9 below 2^-6
            exp = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
            grid = torch.exp2(exp - 3)
            got["codes"].append(torch.round(v / grid) * grid)
    want = {"res": s["residual"], "y": s["y"], "scales": s["q"] != "none",
            "values": s["q"] == "int8", "codes": s["q"] == "e4m3"}
    return {n: torch.cat(got[n]) if keep else None for n, keep in want.items()
            if keep or n in ("res", "y")}


def _exact_matvec(s):
    T, N, K = s["T"], s["N"], s["K"]
    out = torch.empty((T, N), dtype=F64, device="cuda")
    x = s["x"].double()
    for lo in range(0, N, 4096):
        c = s["codes"][lo:lo + 4096].int()
        n = c.shape[0]
        w = torch.empty((n, K), dtype=F64, device="cuda")
        for half in (0, 1):
            nib = (c >> (4 * half)) & 15
            e, m = (nib >> 1) & 3, nib & 1
            mag = torch.where(e == 0, 0.5 * m.double(), (1.0 + 0.5 * m) * torch.exp2(e.double() - 1))
            w[:, half::2] = torch.where(nib >= 8, -mag, mag)
        b = s["scales"][lo:lo + 4096].int()
        e, m = (b >> 3) & 15, (b & 7).double()
        sc = torch.where(e == 0, m * 2.0 ** -9, (1.0 + m / 8) * torch.exp2(e.double() - 7))
        w = w * sc.repeat_interleave(16, dim=1)
        out[:, lo:lo + n] = (w @ x.t().contiguous()).t() * s["alpha"].double()
    return out


def _exact_grouped(s):
    if 2.0 * s["R"] * s["w"].shape[1] * s["K"] > 5e14:
        return None
    out = torch.zeros((s["R"], s["N"]), dtype=F64, device="cuda")
    ends, at = s["cumsum"].tolist(), 0
    for e, end in enumerate(ends):
        if end > at:
            src = s["row_idx"][at:end].long() // s["k"] if s["gather"] else slice(at, end)
            x, w = s["x"][src].double(), s["w"][e].double()
            if s["x_scale"] is not None:
                x, w = x * s["x_scale"][src].double()[:, None], w * s["w_scale"][e].double()[:, None]
            h = x @ w.t().contiguous()
            if s["situ"]:
                b, m = s["beta"][e].double(), s["lam"][e].double()
                gate, up = h[:, :s["N"]], h[:, s["N"]:]
                h = b * torch.tanh(gate / b) / (1.0 + torch.exp(-gate)) * m * torch.tanh(up / m)
            out[at:end] = h
        at = end
    return out


def _exact_combine(s):
    T, k = s["T"], s["k"]
    out = torch.zeros((T, s["H"]), dtype=F64, device="cuda")
    idx = s["idx"].long().view(T, k)
    for j in range(k):
        i = idx[:, j]
        out += torch.where(i < 0, 0.0, s["weights"][:, j].double())[:, None] * s["rows"][i.clamp(min=0)].double()
    return out if s["add"] is None else out + s["add"].double()
