"""Plain definitions in 64 bits of the microscaled FP4 operators (moe_quantize_mxfp4,
moe_dequantize_mxfp4, moe_grouped_gemm_mxfp4) and of the router's balance loss with its gradient
(moe_balance_loss, moe_balance_loss_grad), with bounds of the rounding errors the fp32 kernels
may make.  One rounding to BF16 is off by at most 2^-8 of the value, one to fp32 by 2^-24."""

import torch

from tests import expert_ops as ref

BF16_HALF_STEP, F32_HALF_STEP = ref.BF16_HALF_STEP, ref.F32_HALF_STEP


def stride(K):
    return (K + 127) // 128 * 4


def quantize(x):
    """(codes [rows, K/2], scales [rows, stride]) of BF16 rows: every step exact in doubles."""
    rows, K = x.shape
    v = x.double().view(rows, K // 32, 32)
    bad = ~v.isfinite().all(2)
    v = torch.where(bad[:, :, None], 0.0, v)
    top = v.abs().amax(2)
    byte = (torch.frexp(top).exponent.long() - 1 - 2 + 127).clamp(min=0)
    byte = torch.where(top == 0, 0, byte)
    m = v.abs() * torch.exp2(127.0 - byte.double())[:, :, None]
    # borders between neighbours; at a border the even code (0, 2, 4, 6) wins
    code = torch.zeros_like(m, dtype=torch.long)
    for i, (lo, hi) in enumerate(zip(ref.E2M1, ref.E2M1[1:])):
        code += (m > (lo + hi) / 2) if i % 2 == 0 else (m >= (lo + hi) / 2)
    code += 8 * torch.signbit(v)
    code = torch.where(bad[:, :, None], 0, code).view(rows, K // 2, 2)
    scales = torch.zeros((rows, stride(K)), dtype=torch.uint8, device=x.device)
    scales[:, :K // 32] = torch.where(bad, 255, byte).to(torch.uint8)
    return (code[:, :, 0] + 16 * code[:, :, 1]).to(torch.uint8), scales


def decode(codes, scales):
    """[rows, K] doubles of codes [rows, K/2] and scales [rows, stride]; NaN where the byte is 255."""
    table = torch.tensor(ref.E2M1 + tuple(-v for v in ref.E2M1), dtype=torch.float64,
                         device=codes.device)
    c = codes.long()
    v = torch.stack((table[c & 15], table[c >> 4]), 2).reshape(codes.shape[0], -1)
    b = scales[:, :v.shape[1] // 32].double()
    s = torch.where(b == 255, float("nan"), torch.exp2(b - 127.0))
    return v * s.repeat_interleave(32, dim=1)


def grouped(x, src, cumsum, w, N, beta=None, lam=None, situ=False):
    """(rows, bound, written) of the products by expert of decoded rows x [x_rows, K] and weights
    w(e) [Nw, K]; src: [R] source row of each sorted row, -1 for zeros.

    The matrix unit adds a block's 32 products exactly (multiples of 1/4 up to 36 times one power
    of two) and the blocks' sums in fp32, each addition off by less than a step, 2^-23, of a sum
    that the magnitudes' sum bounds: K / 32 of them, and up to four for what it takes together."""
    R, K = src.numel(), x.shape[1]
    out = torch.zeros((R, N), dtype=torch.float64, device=x.device)
    tol = torch.zeros_like(out)
    sum_err = (K / 32 + 4) * 2 * F32_HALF_STEP
    at = 0
    for e, end in enumerate(cumsum.tolist()):
        if end > at:
            s = src[at:end].long()
            xe = torch.where((s >= 0)[:, None], x[s.clamp(min=0)], 0.0)
            h, mag = ref.product(xe, w(e))
            err = sum_err * mag
            if situ:
                b, m = float(beta[e]), float(lam[e])
                a, c = ref.situ_parts(h[:, :N], h[:, N:], b, m)
                # |d(a)/dg| <= 1.1 and |d(c)/du| <= 1; the functions themselves 2^-20, and
                # exp(-g) = exp2(fl(-g / ln 2)) is off by |g| * 2^-24 of its value more
                own = 2.0 ** -20 + h[:, :N].abs() * F32_HALF_STEP
                err = 1.1 * err[:, :N] * c.abs() + a.abs() * err[:, N:] + own * (a * c).abs()
                h = a * c
            out[at:end], tol[at:end] = h, err + BF16_HALF_STEP * 1.001 * h.abs() + 1e-38
        at = max(at, end)
    written = torch.arange(R, device=x.device) < at
    return out, tol, written


# ---------------------------------------------------------------------------------------
# Balance.
# ---------------------------------------------------------------------------------------
def probabilities(logits, mask):
    """(p, relative error bound of the kernel's p): exp2((z - m) log2 e) has an argument off by
    2.5 half steps of |z - m| (times ln 2, which its scale cancels) and is itself off by a step;
    the sum of a row carries its terms' errors, weighted, and up to 64 + 6 additions; then a
    division and two products."""
    z = logits.double()
    m = z.amax(1, keepdim=True)
    m = torch.where(m == -float("inf"), 0.0, m)
    e = torch.exp(z - m)
    s = e.sum(1, keepdim=True)
    p = torch.where(s == 0, 0.0, e / s)
    far = torch.where(p > 0, (z - m).abs(), 0.0)
    rel = F32_HALF_STEP * (2.5 * (far + (p * far).sum(1, keepdim=True)) + 2 + 2 + 70 + 6)
    if mask is not None:
        live = mask.bool()[:, None]
        p, rel = torch.where(live, p, 0.0), torch.where(live, rel, 0.0)
    return p, rel


def balance(logits, ids, mask, coef):
    """(counts, sums, its bound, tokens, loss, its bound)."""
    T, E = logits.shape
    live = torch.ones(T, dtype=torch.bool, device=logits.device) if mask is None else mask.bool()
    i = ids.view(T, -1)[live].reshape(-1).long()
    counts = torch.bincount(i[(i >= 0) & (i < E)], minlength=E)
    p, rel = probabilities(logits, mask)
    sums = p.sum(0)
    # at most T / 8 additions in a lane where one workgroup takes all, fewer than 2^12 in every
    # case; then 8 over wavefronts and a rounding behind the sum in doubles
    adds = min(T, 4096) + 16
    tol = (rel * p).sum(0) + adds * F32_HALF_STEP * sums + T * 2.0 ** -126
    tokens, routed = int(live.sum()), int(counts.sum())
    f = coef * E / (max(1, tokens) * max(1, routed))
    loss = f * float((counts.double() * sums).sum())
    return counts, sums, tol, tokens, loss, f * float((counts.double() * tol).sum()) + 4 * F32_HALF_STEP * abs(loss)


def balance_grad(logits, mask, counts, tokens, coef, g, add):
    """(gradient, bound before its last rounding)."""
    T, E = logits.shape
    p, rel = probabilities(logits, mask)
    c = counts.double()
    routed = float(c.sum())
    f = 0.0 if tokens <= 0 or routed <= 0 else g * coef * E / (tokens * routed)
    d = c - c.mean()
    dot = (p * d).sum(1, keepdim=True)
    grad = f * p * (d - dot)
    # the centred counts are rounded once; the dot product carries p's errors and 64 + 8 additions
    off = F32_HALF_STEP * d.abs() + (p * d.abs() * (rel + 80 * F32_HALF_STEP)).sum(1, keepdim=True)
    tol = abs(f) * p * (off + (d - dot).abs() * (rel + 6 * F32_HALF_STEP))
    tol = tol + abs(f) * (d - dot).abs() * 2.0 ** -126 + 2.0 ** -140
    if mask is not None:
        grad = torch.where(mask.bool()[:, None], grad, 0.0)
    if add is not None:
        grad = grad + add.double()
        tol = tol + F32_HALF_STEP * grad.abs()
    return grad, tol
