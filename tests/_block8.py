"""Plain forms of the e4m3 block-scaled operators for the tests: the
quantiser in the fp32 steps that its definition names (compared bit for bit),
norms and products in 64 bits, and the tolerances that follow from counting
roundings."""
import torch

GROUP = 128
TINY = 2.0 ** -100


def groups(k):
    return -(-k // GROUP)


def spread(s, K):
    """[M, G] to [M, K]: each group's value for each of its columns."""
    return s.repeat_interleave(GROUP, dim=1)[:, :K]


def group_amax(x):
    """max |x| per group; a group that holds NaN or Inf gives that."""
    K = x.shape[1]
    return torch.stack([x[:, g * GROUP:(g + 1) * GROUP].abs().amax(1) for g in range(groups(K))], 1)


def factors(a):
    """(scale, 448 / a) of group maxima in fp32."""
    a = a.float()
    a = torch.where(a == 0, a, torch.where(a < TINY, torch.full_like(a, TINY), a))
    top = torch.full_like(a, 448.0)  # 448.0 / a would be a reciprocal and a product: two roundings
    return a / top, torch.where(a == 0, torch.zeros_like(a), top / a)


def quantise(x):
    """codes (float8_e4m3fn) and scales of 16-bit rows, on the CPU."""
    x = x.float().cpu()
    s, r = factors(group_amax(x))
    return (x * spread(r, x.shape[1])).to(torch.float8_e4m3fn), s


def quantise_blocks(w):
    """codes [N, K] and scales of a 16-bit weight W [K, N], on the CPU."""
    w = w.float().cpu().t().contiguous()
    a = group_amax(group_amax(w).t().contiguous()).t().contiguous()
    s, r = factors(a)
    rr = spread(r, w.shape[1]).repeat_interleave(GROUP, dim=0)[:w.shape[0]]
    return (w * rr).to(torch.float8_e4m3fn), s


def values(codes, scales):
    return codes.double() * spread(scales.double(), codes.shape[1])


def weight_values(codes, scales):
    N, K = codes.shape
    return codes.double() * spread(scales.double(), K).repeat_interleave(GROUP, dim=0)[:N]


def product(codes, scales, wcodes, wscales, bias=None):
    """(Y, sum of the absolute products) in 64 bits."""
    x, w = values(codes, scales), weight_values(wcodes, wscales)
    y, a = x @ w.t(), x.abs() @ w.abs().t()
    if bias is not None:
        y, a = y + bias.double(), a + bias.double().abs()
    return y, a


def product_tolerance(y, a, K, dtype):
    """Each product of two e4m3 numbers is exact in fp32.  A group's sum makes
    at most 128 additions, the groups' sums at most G more with two roundings
    of the scales' product and one of the bias: each is off by at most 2^-23
    of the absolute sum (the tensor cores may cut where others round).  Then
    one rounding to 16 bits, half a step: eps / 2 relative, and in fp16 half
    the subnormal step 2^-24 absolute."""
    half = torch.finfo(dtype).eps / 2
    t = (GROUP + groups(K) + 3) * 2.0 ** -23 * a
    return t + half * (y.abs() + t) + (2.0 ** -25 if dtype == torch.float16 else 0.0)


def check_product(Y, codes, scales, wcodes, wscales, bias, K):
    y, a = product(codes, scales, wcodes, wscales, bias)
    top = torch.finfo(Y.dtype).max
    assert (y.abs() < top).all(), "the case overflows the output type"
    off = (Y.double() - y).abs() - product_tolerance(y, a, K, Y.dtype)
    assert (off <= 0).all(), f"off by {off.max().item():.3g} more than allowed, {(off > 0).sum().item()} places"


def norm(x, residual, weight, eps):
    """(h in the type of x, y in 64 bits)."""
    h = x if residual is None else (x.double() + residual.double()).to(x.dtype)
    d = h.double()
    return h, d / torch.sqrt(d.square().mean(1, keepdim=True) + eps) * weight.double()


# A norm's fp32 steps: the mean of squares is a sum of positive terms in
# runs of at most 64 with a tree of at most 10 + 32 more, so off by at most
# 110 x 2^-24 relative, half of that after the root; the root, two products
# and the division add 5 more.  60 x 2^-24 < 2^-18.
NORM_REL = 2.0 ** -18


def check_normed(Y, y):
    half = torch.finfo(Y.dtype).eps / 2
    tol = y.abs() * (NORM_REL + half * (1 + NORM_REL)) + (2.0 ** -25 if Y.dtype == torch.float16 else 0.0)
    assert ((Y.double() - y).abs() <= tol).all()


def check_quantised(codes, scales, y):
    """Codes and scales of the 64-bit rows y known to NORM_REL: the scale to
    that and two fp32 roundings, a value to half an e4m3 step (2^-4 of it, or
    2^-10 of the scale below e4m3's normal numbers) and a little more for the
    error of y itself."""
    a = group_amax(y)
    a = torch.where((a > 0) & (a < TINY), torch.full_like(a, TINY), a)
    s = a / 448.0
    assert ((scales.double() - s).abs() <= s * (NORM_REL + 2.0 ** -22)).all()
    v = values(codes, scales)
    tol = torch.maximum(y.abs() * 2.0 ** -4, spread(s, y.shape[1]) * 2.0 ** -10) * (1 + 2.0 ** -10)
    tol = tol + y.abs() * NORM_REL
    assert ((v - y).abs() <= tol).all()
