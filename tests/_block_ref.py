"""Plain 64-bit forms of the operators around the experts (fp8 quantizer and
products, balance loss, norms) for the tests; torch float64 on any device."""
import torch

U32 = 2.0 ** -24    # half a step of fp32, relative
BF16 = 2.0 ** -8    # of bfloat16
TINY = 2.0 ** -126  # smallest normal fp32 (and bfloat16) number


def half_step(dtype):
    return BF16 if dtype == torch.bfloat16 else U32


def e4m3(v):
    """v (float64) rounded to the nearest e4m3 value, ties to even, saturating."""
    a = v.abs().clamp(max=448.0)
    e = (torch.frexp(a).exponent - 1).clamp(min=-6).double()
    step = torch.exp2(e - 3)
    return torch.sign(v) * torch.round(a / step) * step


def codes_value(codes):
    return codes.view(torch.float8_e4m3fn).double()


def group_scale(amax, qmax=448.0):
    s = torch.where(amax > 0, (amax / qmax).clamp(min=TINY), torch.ones_like(amax))
    return torch.where(torch.isfinite(amax), s, torch.full_like(s, float("nan")))


def pad_to(v, n, dim):
    short = n - v.shape[dim]
    if short == 0:
        return v
    z = v.new_zeros([short if d == dim else s for d, s in enumerate(v.shape)])
    return torch.cat([v, z], dim)


def up128(n):
    return (n + 127) // 128 * 128


def wide(codes, scale, block=False):
    """Values of codes [M, K] with scale [K/128, M], or [ceil(M/128), K/128]
    with block."""
    M, K = codes.shape
    s = scale.double()
    s = s.repeat_interleave(128, 0)[:M] if block else s.t()
    return (codes_value(codes).view(M, K // 128, 128) * s.unsqueeze(2)).view(M, K)


def silu_mul(x):
    g, u = x.double().chunk(2, 1)
    return g / (1 + torch.exp(-g)) * u


def softmax(z):
    z = z.double()
    m = z.max(1, keepdim=True).values
    m = torch.where(m == -float("inf"), torch.zeros_like(m), m)
    e = torch.exp(z - m)
    s = e.sum(1, keepdim=True)
    return torch.where(s == 0, torch.zeros_like(e), e / s)


def balance(z, ids, mask, coef):
    """(loss, counts, probs, tokens) in float64 / int64."""
    T, E = z.shape
    k = ids.shape[1]
    keep = torch.ones(T, dtype=torch.bool, device=z.device) if mask is None else mask.bool()
    n = int(keep.sum())
    picked = ids[keep].reshape(-1).long()
    picked = picked[(picked >= 0) & (picked < E)]
    counts = torch.bincount(picked, minlength=E)
    if n == 0:
        return z.new_zeros((), dtype=torch.float64), counts, z.new_zeros(E, dtype=torch.float64), 0
    probs = softmax(z[keep]).sum(0) / n
    return coef * E * (counts.double() / (k * n) * probs).sum(), counts, probs, n


def norm(v, w, eps):
    return v / torch.sqrt((v * v).mean(1, keepdim=True) + eps) * w
