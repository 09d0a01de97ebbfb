"""Plain 64-bit forms of cross attention and softmax cross entropy, each value with a bound on
how far the library's may be from it.

The bounds follow the library's arithmetic on the same inputs, term by term:
- a sum of K products in fp32 (CUDA cores or tensor cores) is off by at most
  (K + 4) 2^-23 of the sum of its terms' sizes;
- exponentials by 2^-21 relative, a stored fp32 statistic by 2^-23 of its size;
- bf16 inputs: P, dS and dz are rounded to bf16 for their products (half a
  step, 2^-8 relative), and so are the outputs.
- underflow: a weight, or a weight times its gradient factor, below the least
  normal number 2^-126 (fp32 and bf16 alike) may become zero or lose bits, an
  absolute error of at most 2^-126 for the weight (so 2^-126 of the factor it
  multiplies) and 2^-126 for the product.  Relative bounds alone would ask for
  weights like 1e-206 that no such number holds.
First-order errors are added up in absolute value; a factor 1.05 covers the
products of errors.
"""
import math

import torch

U = 2.0 ** -23  # a unit of fp32 arithmetic (twice a rounding's half step)
EXP = 2.0 ** -21
BF = torch.finfo(torch.bfloat16).eps / 2
SLACK = 1.05
MASK = -1e30
TINY = 2.0 ** -126


def _half(dtype):
    """Relative size of rounding an operand of a product, and of rounding an output."""
    return (BF, BF) if dtype == torch.bfloat16 else (0.0, 2.0 ** -24)


def _heads(t, heads):
    """[batch, token, kv_heads, w] -> [batch, heads, token, w] in 64 bits, key heads repeated."""
    t = t.double().permute(0, 2, 1, 3)
    return t.repeat_interleave(heads // t.shape[1], dim=1)


def attention(q, k, v, k_len=None, bias=None, scale=None, dout=None, out=None):
    """Returns {name: (value, bound)} for out and lse, and with dout for dq, dk, dv."""
    B, n, H, d = q.shape
    m, Hk, dv = k.shape[1], k.shape[2], v.shape[3]
    scale = d ** -0.5 if scale is None else scale
    rnd, rout = _half(q.dtype)
    dev = q.device
    live = torch.ones(B, m, dtype=torch.bool, device=dev)
    if k_len is not None:
        live &= torch.arange(m, device=dev)[None] < k_len.clamp(0, m)[:, None]
    b64 = torch.zeros(B, m, dtype=torch.float64, device=dev)
    if bias is not None:
        live &= ~(bias <= MASK)
        b64 = torch.where(live, bias.double(), b64)
    keep = live[:, None, :, None]
    Q = _heads(q, H)
    K = torch.where(keep, _heads(k, H), torch.zeros((), dtype=torch.float64, device=dev))
    V = torch.where(keep, _heads(v, H), torch.zeros((), dtype=torch.float64, device=dev))
    S = torch.einsum("bhid,bhjd->bhij", Q, K) * scale
    aS = torch.einsum("bhid,bhjd->bhij", Q.abs(), K.abs()) * scale
    z = S + b64[:, None, None, :]
    z = z.masked_fill(~live[:, None, None, :], -math.inf)
    eS = (d + 4) * U * aS + 3 * U * (S.abs() + b64[:, None, None, :].abs())
    lse = torch.logsumexp(z, dim=-1) if m else torch.full((B, H, n), -math.inf, dtype=torch.float64, device=dev)
    empty = torch.isinf(lse) & (lse < 0)
    P = torch.exp(z - torch.where(empty, torch.zeros_like(lse), lse)[..., None])
    P = torch.where(empty[..., None], torch.zeros_like(P), P)
    # exponents against the running maximum, whose own size adds a rounding
    top = z.amax(dim=-1, keepdim=True) if m else torch.zeros(B, H, n, 1, dtype=torch.float64, device=dev)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    eP = eS + 3 * U * (top.abs() + torch.where(P > 0, z, torch.zeros_like(z)).abs()) + EXP
    aPV = torch.einsum("bhij,bhjd->bhid", P, V.abs())
    O = torch.einsum("bhij,bhjd->bhid", P, V)
    sumerr = (m + 64) * U
    w = torch.einsum("bhij->bhi", P * eP)
    eO = torch.einsum("bhij,bhjd->bhid", P * eP + TINY, V.abs()) + (w + 2 * sumerr + 4 * U)[..., None] * aPV + rnd * aPV \
        + rout * O.abs()
    elog = w + sumerr + 3 * U * torch.where(empty, torch.zeros_like(lse), lse).abs() + 4 * U
    res = {"out": (O.permute(0, 2, 1, 3), SLACK * eO.permute(0, 2, 1, 3)), "lse": (lse, SLACK * elog)}
    if dout is None:
        return res
    G = _heads(dout, H)
    eP = eS + (elog + 3 * U * torch.where(empty, torch.zeros_like(lse), lse).abs())[..., None] \
        + 3 * U * torch.where(P > 0, z, torch.zeros_like(z)).abs() + EXP
    dP = torch.einsum("bhid,bhjd->bhij", G, V)
    adP = torch.einsum("bhid,bhjd->bhij", G.abs(), V.abs())
    D = torch.einsum("bhij,bhij->bhi", P, dP)
    aGO = torch.einsum("bhid,bhid->bhi", G.abs(), O.abs())
    # D comes from the stored out: its error and its rounding enter
    eD = torch.einsum("bhid,bhid->bhi", G.abs(), eO) + (dv + 8) * U * aGO
    dS = P * (dP - D[..., None])
    edS = P * ((dP - D[..., None]).abs() * eP + (dv + 4) * U * adP + eD[..., None]
               + 2 * U * (dP.abs() + D.abs()[..., None]))
    edS = edS + rnd * (dS.abs() + edS) + TINY * (1 + (dP - D[..., None]).abs())

    def fold(t):  # heads that share a key head
        return t.reshape(B, Hk, H // Hk, m, t.shape[-1]).sum(dim=2).permute(0, 2, 1, 3)

    rows = (n * (H // Hk) + 64) * U
    dQ = scale * torch.einsum("bhij,bhjd->bhid", dS, K)
    edQ = scale * (torch.einsum("bhij,bhjd->bhid", edS, K.abs())
                   + sumerr * torch.einsum("bhij,bhjd->bhid", dS.abs(), K.abs())) + rout * dQ.abs()
    dK = fold(scale * torch.einsum("bhij,bhid->bhjd", dS, Q))
    edK = fold(scale * (torch.einsum("bhij,bhid->bhjd", edS, Q.abs())
                        + rows * torch.einsum("bhij,bhid->bhjd", dS.abs(), Q.abs()))) + rout * dK.abs()
    dV = fold(torch.einsum("bhij,bhid->bhjd", P, G))
    edV = fold(torch.einsum("bhij,bhid->bhjd", P * eP + TINY, G.abs())
               + (rnd * (1 + BF) + rows) * torch.einsum("bhij,bhid->bhjd", P, G.abs())) + rout * dV.abs()
    res["dq"] = (dQ.permute(0, 2, 1, 3), SLACK * edQ.permute(0, 2, 1, 3))
    res["dk"], res["dv"] = (dK, SLACK * edK), (dV, SLACK * edV)
    return res


def cross_entropy(x, w, target, scale=1.0, ignore=-100, dloss=None, dlse=None):
    """Returns {name: (value, bound)} for loss and lse, and with dloss for dx and dw."""
    n, d = x.shape
    V = w.shape[0]
    rnd, rout = _half(x.dtype)
    X, W = x.double(), w.double()
    z = scale * X @ W.t()
    ez = (d + 4) * U * scale * (X.abs() @ W.abs().t()) + 3 * U * z.abs()
    lse = torch.logsumexp(z, dim=1)
    counted = target != ignore
    idx = target.clamp(0, V - 1)[:, None]
    p = torch.exp(z - lse[:, None])
    top = z.amax(dim=1, keepdim=True)
    sumerr = (min(V, 256) + V / 128 + 16) * U
    elog = (p * (ez + 3 * U * (top.abs() + z.abs()) + EXP)).sum(dim=1) + sumerr + 3 * U * lse.abs()
    zero = torch.zeros_like(lse)
    hit = z.gather(1, idx)[:, 0]
    res = {"lse": (lse, SLACK * elog),
           "loss": (torch.where(counted, lse - hit, zero),
                    SLACK * torch.where(counted, elog + ez.gather(1, idx)[:, 0] + 3 * U * hit.abs(), zero))}
    if dloss is None:
        return res
    g = torch.where(counted, dloss.double(), zero)
    gs = g + (dlse.double() if dlse is not None else 0.0)
    hot = torch.zeros_like(z).scatter_(1, idx, g[:, None])
    dz = p * gs[:, None] - hot
    edz = p * gs.abs()[:, None] * (ez + elog[:, None] + 3 * U * (lse.abs()[:, None] + z.abs()) + EXP) \
        + 3 * U * (p * gs.abs()[:, None] + hot.abs())
    edz = edz + rnd * (dz.abs() + edz) + TINY * (1 + gs.abs()[:, None])
    dx = scale * dz @ W
    edx = scale * (edz @ W.abs() + (V + 64) * U * (dz.abs() @ W.abs())) + rout * dx.abs()
    dw = scale * dz.t() @ X
    edw = scale * (edz.t() @ X.abs() + (n + 64) * U * (dz.abs().t() @ X.abs())) + rout * dw.abs()
    res["dx"], res["dw"] = (dx, SLACK * edx), (dw, SLACK * edw)
    return res


def check(got, ref, names=None):
    """Every value within its bound (equal where either is infinite); returns the worst ratio."""
    worst = 0.0
    for name in names or got:
        value, bound = ref[name]
        g = got[name].double()
        assert g.shape == value.shape, (name, g.shape, value.shape)
        inf = torch.isinf(value)
        assert torch.equal(g[inf], value[inf]), name
        err, lim = (g - value)[~inf].abs(), bound[~inf] + 1e-37
        assert not torch.isnan(err).any(), f"{name}: NaN"
        if err.numel():
            ratio = (err / lim).max().item()
            assert ratio <= 1.0, f"{name}: {ratio:.3g} of the bound, max error {err.max().item():.3g}"
            worst = max(worst, ratio)
    return worst
