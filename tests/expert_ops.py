"""Plain definitions in 64 bits of the expert-stage operators (moe_rmsnorm, moe_matvec_nvfp4,
moe_grouped_gemm, moe_combine), with bounds of the rounding errors the fp32 kernels may make.

Each function returns the reference and, where the result is a sum, the sum of the terms'
magnitudes: a sum of n terms accumulated in fp32 in any order is off by at most about
n * 2^-24 times that.  One rounding to BF16 is off by at most 2^-8 of the value.
"""

import torch

BF16_HALF_STEP = 2.0 ** -8
F32_HALF_STEP = 2.0 ** -24
CODE_MAX = {"int8": 127.0, "e4m3": 448.0}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def rmsnorm(x, res, weight, eps):
    """(h, y) of the norm."""
    h = x.double() if res is None else x.double() + res.double()
    return h, h / (h.square().mean(1, keepdim=True) + eps).sqrt() * weight.double()


def norm_rel(H):
    """Relative error of the kernel's fp32 y: the sum of H squares (at most 64 in a row per
    lane, then 6 + 16 partial sums) enters under a root, and 8 more roundings follow."""
    return (0.5 * (H / 8 / 64 + 8 + 22) + 8) * F32_HALF_STEP


def nvfp4_weights(codes, scales):
    """[N, K] doubles: code times block scale."""
    c = codes.long()
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=codes.device)
    v = torch.stack((table[c & 15], table[c >> 4]), 2).reshape(codes.shape[0], -1)
    b = scales.long()
    e, m = (b >> 3) & 15, (b & 7).double()
    s = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2(e.double() - 7))
    return v * s.repeat_interleave(16, dim=1)


def product(x, w):
    """(x @ w^T, |x| @ |w|^T) in doubles."""
    wt = w.double().t().contiguous()
    return x.double() @ wt, x.double().abs() @ wt.abs()


def situ_parts(g, u, beta, lam):
    """The two factors of SiTU."""
    return beta * torch.tanh(g / beta) * torch.sigmoid(g), lam * torch.tanh(u / lam)


# The matrix unit's E4M3 products: it adds the eight products of one lane group after
# shifting each to the largest of them, and bits below 2^-13 of that one are cut.  So of the
# other seven each is off by less than 2^-13 of the largest, and a whole sum by less than
# 7 * 2^-13 * (sum over the groups of the largest product), which is at most 7 * 2^-13 times
# the sum of the products' magnitudes.  (A product of two E4M3 values rounded from 32-bit
# numbers is itself off by up to 2^-3 of its value.)
E4M3_SUM = 7 * 2.0 ** -13


def grouped(x, x_scale, src, cumsum, w, w_scale, N, beta=None, lam=None, situ=False):
    """(rows, bound, written): the products by expert, the allowed error and which rows are
    written.  src: [R] source row of each sorted row, -1 for zeros."""
    R, K = src.numel(), x.shape[1]
    out = torch.zeros((R, N), dtype=torch.float64, device=x.device)
    tol = torch.zeros_like(out)
    sum_err = 0.0 if x.dtype == torch.int8 else K * F32_HALF_STEP
    if x.dtype == torch.float8_e4m3fn:
        sum_err += E4M3_SUM
    at = 0
    for e, end in enumerate(cumsum.tolist()):
        if end > at:
            s = src[at:end].long()
            xe = torch.where((s >= 0)[:, None], x[s.clamp(min=0)].double(), 0.0)
            h, mag = product(xe, w[e])
            err = sum_err * mag
            if x_scale is not None:
                f = torch.where(s >= 0, x_scale[s.clamp(min=0)].double(), 0.0)[:, None] * w_scale[e].double()
                h, err = h * f, err * f + 3 * F32_HALF_STEP * (h * f).abs()
            if situ:
                b, m = float(beta[e]), float(lam[e])
                a, c = situ_parts(h[:, :N], h[:, N:], b, m)
                # |d(a)/dg| <= 1.1 and |d(c)/du| <= 1; the functions themselves 2^-20, and
                # exp(-g) = exp2(fl(-g / ln 2)) is off by |g| * 2^-24 of its value more
                own = 2.0 ** -20 + h[:, :N].abs() * F32_HALF_STEP
                err = 1.1 * err[:, :N] * c.abs() + a.abs() * err[:, N:] + own * (a * c).abs()
                h = a * c
            out[at:end], tol[at:end] = h, err + BF16_HALF_STEP * 1.001 * h.abs() + 1e-38
        at = max(at, end)
    written = torch.arange(R, device=x.device) < at
    return out, tol, written


def combine(rows, idx, weights, add):
    """(out, bound) of the weighted sum."""
    T, k = weights.shape
    i = idx.long().view(T, k)
    keep = (i >= 0) & (i < rows.shape[0])
    picked = torch.where(keep[:, :, None], rows[torch.where(keep, i, 0)].double(), 0.0)
    terms = weights.double()[:, :, None] * picked
    out, mag = terms.sum(1), terms.abs().sum(1)
    if add is not None:
        out, mag = out + add.double(), mag + add.double().abs()
    return out, (k + 1) * F32_HALF_STEP * mag + BF16_HALF_STEP * 1.001 * out.abs() + 1e-38


def e4m3_nearest(v):
    """Nearest E4M3 value (ties to even), |v| <= 448."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step
