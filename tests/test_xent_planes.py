"""fp32 cross entropy as three bf16 planes a factor and six products: inputs whose every dropped product shows, and sums
long enough to show an accumulator that is not cut.

The bounds count what the arithmetic does.  U = 2^-23.
- A product's sum runs on the tensor core in steps of 16 terms, each of which truncates the accumulator by at most U of
  its size: (terms / 16) U of the sum of the terms' sizes, and 8 U for the planes that are left out (3 x 2^-24 of a term
  and more where they are small), the smaller products and the rounding of the result.
- dz: the exponent's roundings (|lse| up to 10: 2^-21 = 4 U at most), ex2.approx 2 U, two products U: 8 U relative.
"""
import itertools
import math

import pytest
import torch

U = 2.0 ** -23
PAIRS = [(0, 0), (0, 1), (1, 0), (0, 2), (2, 0), (1, 1)]


def plane_values(*shape, seed):
    """fp32 numbers 1 + m + l whose bf16 planes are 1, m and l, all of them positive and near the largest they can be: m a
    multiple of 2^-16 below 2^-8, l one of 2^-23 below 2^-17.  A product left out then adds up instead of averaging out."""
    g = torch.Generator().manual_seed(seed)
    m = torch.randint(210, 251, shape, generator=g).double() * 2.0 ** -16
    low = torch.randint(52, 63, shape, generator=g).double() * 2.0 ** -23
    return (1.0 + m + low).float()


def planes(t):
    out, rest = [], t.double()
    for _ in range(3):
        out.append(rest.float().bfloat16().double())
        rest = rest - out[-1]
    return out


def product(a, b, left_out=None):
    """a b^T of fp32 matrices over the plane pairs, but for one."""
    pa, pb = planes(a), planes(b)
    return sum(pa[i] @ pb[j].t() for i, j in PAIRS if (i, j) != left_out)


def logit_bound(x, w, scale):
    d = x.shape[1]
    # a single class: lse is its logit, a rounding each for the scaled maximum and the result
    return scale * (d / 16 + 8) * U * (x.double().abs() @ w.double().abs().t()) + 4 * U


def sum_bound(terms, size):
    return (min(terms, 2048) / 16 + math.ceil(terms / 2048) + 8 + 8) * U * size


LOGITS = [(5, 32), (40, 64), (300, 96)]  # rows, width


def logit_inputs(n, d):
    return plane_values(n, d, seed=n), plane_values(1, d, seed=d)


def grad_inputs(n, v, d):
    """Logits of next to nothing (a scale of 2^-40), so every weight is 1 / v, times a gradient that makes dz such numbers
    too: dz = (1 + m + l) scale but for the roundings of the exponential."""
    x, w = plane_values(n, d, seed=n + v), plane_values(v, d, seed=v + 7 * d)
    return x, w, v * plane_values(n, seed=n + d)


def grad_reference(x, w, lse, dlse, scale):
    z = scale * (x.double() @ w.double().t())
    dz = scale * torch.exp(z - lse.double()[:, None]) * dlse.double()[:, None]
    return dz, dz @ w.double(), dz.t() @ x.double()


GRADS = [(64, 64, 40), (33, 96, 64), (80, 16, 24)]  # rows, classes, width
SCALE = 2.0 ** -40


@pytest.mark.parametrize("left_out", PAIRS)
def test_a_product_left_out_would_show(left_out):
    for n, d in LOGITS:
        x, w = logit_inputs(n, d)
        scale = 1.0 / d
        z = scale * (x.double() @ w.double().t())
        assert ((scale * product(x, w) - z).abs() <= logit_bound(x, w, scale)).all()
        assert ((scale * product(x, w, left_out) - z).abs() > logit_bound(x, w, scale)).all()
    for n, v, d in GRADS:
        x, w, dlse = grad_inputs(n, v, d)
        lse = torch.full((n,), math.log(v))
        dz, dx, dw = grad_reference(x, w, lse, dlse, SCALE)
        for got, want, terms in [(lambda out: product(dz.float(), w.t().contiguous(), out), dx, v),
                                 (lambda out: product(dz.float().t().contiguous(), x.t().contiguous(), out), dw, n)]:
            assert ((got(None) - want).abs() <= sum_bound(terms, want)).all()
            assert ((got(left_out) - want).abs() > sum_bound(terms, want)).all()


def test_the_inputs_are_what_they_are_said_to_be():
    x = plane_values(50, 20, seed=1)
    h, m, low = planes(x)
    assert (h == 1).all() and (m > 0).all() and (low > 0).all() and torch.equal(h + m + low, x.double())
    assert set(PAIRS) == {(i, j) for i, j in itertools.product(range(3), repeat=2) if i + j <= 2}


def _fs():
    import log_domain_sinkhorn_updates_b200 as fs
    return fs


@pytest.mark.gpu
@pytest.mark.parametrize("n,d", LOGITS)
def test_logits_hold_every_product(n, d):
    x, w = (t.cuda() for t in logit_inputs(n, d))
    target = torch.zeros(n, dtype=torch.long, device="cuda")
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    _fs().fs_cross_entropy(x, w, target, loss, lse, scale=1.0 / d)
    z = (x.double() @ w.double().t()) / d
    assert ((lse.double() - z[:, 0]).abs() <= logit_bound(x, w, 1.0 / d)[:, 0]).all()
    assert (loss.abs() <= 4 * U).all()


def _gradient(x, w, lse, dlse, scale):
    n = x.shape[0]
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    target = torch.zeros(n, dtype=torch.long, device="cuda")
    _fs().fs_cross_entropy_grad(x, w, target, lse, torch.zeros(n, device="cuda"), dx, dw, dlse=dlse, scale=scale)
    return dx, dw


@pytest.mark.gpu
@pytest.mark.parametrize("n,v,d", GRADS)
def test_gradients_hold_every_product(n, v, d):
    x, w, dlse = (t.cuda() for t in grad_inputs(n, v, d))
    lse = torch.full((n,), math.log(v), device="cuda")
    dx, dw = _gradient(x, w, lse, dlse, SCALE)
    _, want_x, want_w = grad_reference(x, w, lse, dlse, SCALE)
    assert ((dx.double() - want_x).abs() <= sum_bound(v, want_x)).all()
    assert ((dw.double() - want_w).abs() <= sum_bound(n, want_w)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("n,v,d", [(8, 16384, 16), (3, 40001, 24), (5000, 40, 24), (16384, 70, 8), (2049, 2049, 40)])
def test_long_sums_of_one_sign_are_cut(n, v, d):
    """Sums over more than 2048 classes and more than 2048 rows: in one accumulator they would drift by half of terms / 16
    truncations (16384 terms: 460 U against a bound of 152)."""
    g = torch.Generator().manual_seed(v)
    x, w, dlse = torch.rand(n, d, generator=g) + 0.5, torch.rand(v, d, generator=g) + 0.5, torch.rand(n, generator=g) + 0.5
    x, w, dlse = x.cuda(), w.cuda(), dlse.cuda()
    lse = torch.full((n,), math.log(v), device="cuda")
    dx, dw = _gradient(x, w, lse, dlse, SCALE)
    _, want_x, want_w = grad_reference(x, w, lse, dlse, SCALE)
    assert ((dx.double() - want_x).abs() <= sum_bound(v, want_x)).all()
    assert ((dw.double() - want_w).abs() <= sum_bound(n, want_w)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("signs", [False, True])
@pytest.mark.parametrize("n,v,d", [(100, 300, 2048), (20, 70, 16384), (8, 5, 65536)])
def test_wide_rows_keep_the_stated_bound(n, v, d, signs, dtype):
    """The logits' sum is not cut: d / 16 truncations of terms of one sign, as the header states for wide rows."""
    g = torch.Generator(device="cuda").manual_seed(d)
    x, w = (torch.rand(k, d, device="cuda", generator=g) + 0.5 for k in (n, v))
    if signs:
        x, w = (t * (torch.randint(0, 2, t.shape, device="cuda", generator=g) * 2 - 1) for t in (x, w))
    x, w = x.to(dtype), w.to(dtype)
    scale = 2.0 / d
    target = torch.arange(n, device="cuda") % v
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    _fs().fs_cross_entropy(x, w, target, loss, lse, scale=scale)
    z = scale * (x.double() @ w.double().t())
    want = torch.logsumexp(z, dim=1)
    most = (scale * (d / 16 + 8) * U * (x.double().abs() @ w.double().abs().t())).amax(dim=1)
    # beside the logits: exponentials 4 U, their sum (v / 8 additions in each of its parts) and the statistic's roundings
    rest = (4 + min(v, 128) / 8 + 16 + 3 * want.abs()) * U
    assert ((lse.double() - want).abs() <= most + rest).all()
    assert ((loss.double() - (want - z.gather(1, target[:, None])[:, 0])).abs() <= 2 * most + rest + 4 * U).all()


@pytest.mark.gpu
@pytest.mark.parametrize("n,v,d", [(300, 4099, 256), (3000, 5000, 128), (1000, 16384, 64)])
def test_normal_inputs_in_the_norm(n, v, d):
    """Relative 2-norms against 64 bits.  Terms of mixed signs: an accumulator of K terms of size s is of size s sqrt(k)
    after k of them, so its K / 16 truncations of at most U of it come to at most (2/3) (K / 16) U of the result's own
    size, in the mean half of that; with the logits' absolute error in the exponent (d / 16 + 8) U |z| of size up to 10,
    8 U for dz, 16 U for planes and roundings."""
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randn(n, d, device="cuda", generator=g)
    w = torch.randn(v, d, device="cuda", generator=g) * 2 / d ** 0.5
    target = torch.randint(0, v, (n,), device="cuda", generator=g)
    dloss = torch.randn(n, device="cuda", generator=g)
    fs = _fs()
    loss, lse, dx, dw = torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty_like(x), torch.empty_like(w)
    fs.fs_cross_entropy(x, w, target, loss, lse)
    fs.fs_cross_entropy_grad(x, w, target, lse, dloss, dx, dw)
    z = x.double() @ w.double().t()
    dz = torch.exp(z - torch.logsumexp(z, 1)[:, None])
    dz[torch.arange(n), target] -= 1
    dz *= dloss.double()[:, None]
    for got, want, terms in [(dx, dz @ w.double(), v), (dw, dz.t() @ x.double(), n)]:
        off = ((got.double() - want).norm() / want.norm()).item()
        assert off <= (min(terms, 2048) / 48 + (d / 16 + 8) / 3 + 24) * U, off / U
