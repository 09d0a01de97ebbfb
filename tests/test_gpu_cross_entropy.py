"""Softmax cross entropy, forward and gradient, against the 64-bit form with derived bounds
(tests/ops_reference.py)."""
import math

import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def _fs():
    import log_domain_sinkhorn_updates_b200 as fs
    return fs


def make(n, v, d, dtype, seed=0, ignored=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(n, d, device="cuda", generator=g).to(dtype)
    w = (torch.randn(v, d, device="cuda", generator=g) * 2 / d ** 0.5).to(dtype)
    target = torch.randint(0, v, (n,), device="cuda", generator=g)
    if ignored and n > 2:
        target[torch.rand(n, device="cuda", generator=g) < 0.2] = -100
    return x, w, target, torch.randn(n, device="cuda", generator=g)


def run(x, w, target, dloss, dlse=None, **kw):
    fs = _fs()
    loss, lse = (torch.full((x.shape[0],), 7.0, device="cuda") for _ in range(2))
    fs.fs_cross_entropy(x, w, target, loss, lse, **kw)
    dx, dw = (torch.full(t.shape, 7.0, dtype=t.dtype, device="cuda") for t in (x, w))
    fs.fs_cross_entropy_grad(x, w, target, lse, dloss, dx, dw, dlse=dlse, **kw)
    fs.fs_check()
    return {"loss": loss, "lse": lse, "dx": dx, "dw": dw}


SIZES = [(1, 1, 1), (1, 5, 8), (1, 3000, 64), (2, 257, 1000), (63, 1000, 72), (128, 256, 64), (129, 513, 128),
         (300, 4099, 256), (257, 128, 520), (1000, 70, 96), (40, 301, 33), (5, 20000, 16), (700, 2048, 1024)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size", SIZES)
def test_against_64_bits(size, dtype):
    x, w, target, dloss = make(*size, dtype, seed=sum(size))
    ref.check(run(x, w, target, dloss), ref.cross_entropy(x, w, target, dloss=dloss))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scale_and_lse_gradient(dtype):
    x, w, target, dloss = make(150, 700, 64, dtype, seed=3)
    dlse = torch.linspace(-1, 1, 150, device="cuda")
    for scale in (0.01, 2.5):
        got = run(x, w, target, dloss, dlse, scale=scale)
        ref.check(got, ref.cross_entropy(x, w, target, scale=scale, dloss=dloss, dlse=dlse))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_all_ignored_and_another_ignore_index(dtype):
    x, w, target, dloss = make(140, 300, 64, dtype, seed=4)
    got = run(x, w, torch.full_like(target, -100), dloss)
    assert (got["loss"] == 0).all() and (got["dx"] == 0).all() and (got["dw"] == 0).all()
    t = target.clamp(min=0)
    ref.check(run(x, w, t, dloss, ignore_index=5),
              ref.cross_entropy(x, w, t, ignore=5, dloss=dloss))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_targets_out_of_range_are_loud_and_stay_in_their_row(dtype):
    x, w, target, dloss = make(140, 300, 64, dtype, seed=5, ignored=False)
    good = run(x, w, target, dloss)
    bad = target.clone()
    bad[3], bad[70], bad[139] = 300, -1, 2 ** 40
    got = run(x, w, bad, dloss)
    hit = torch.zeros(140, dtype=torch.bool, device="cuda")
    hit[[3, 70, 139]] = True
    assert torch.isnan(got["loss"][hit]).all() and torch.equal(got["loss"][~hit], good["loss"][~hit])
    assert torch.isnan(got["dx"][hit]).all() and torch.equal(got["dx"][~hit], good["dx"][~hit])
    assert torch.isnan(got["dw"]).any()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_large_logits(dtype):
    """Logits of hundreds: a softmax on one class, the loss exact where the target has it."""
    x, w, target, dloss = make(130, 520, 128, dtype, seed=6, ignored=False)
    x = x * 8
    target[:60] = (x[:60].float() @ w.float().t()).argmax(dim=1)
    got = run(x, w, target, dloss, scale=4.0)
    ref.check(got, ref.cross_entropy(x, w, target, scale=4.0, dloss=dloss))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides(dtype):
    """Rows inside wider buffers, one row for all (stride 0), an odd offset, gradients into parts of buffers."""
    fs = _fs()
    n, v, d = 150, 333, 64
    x, w, target, dloss = make(n, v, d, dtype, seed=7)
    want = ref.cross_entropy(x, w, target, dloss=dloss)
    xs = torch.full((n, d + 8), math.nan, dtype=dtype, device="cuda")
    ws = torch.full((v, 3 * d), math.nan, dtype=dtype, device="cuda")
    xs[:, :d], ws[:, d:2 * d] = x, w
    xv, wv = xs[:, :d], ws[:, d:2 * d]
    ref.check(run(xv, wv, target, dloss), want)
    odd = torch.full((n, d + 1), math.nan, dtype=dtype, device="cuda")
    odd[:, 1:] = x
    ref.check(run(odd[:, 1:], w, target, dloss), want)
    oddw = torch.full((v * (d + 1) + 1,), math.nan, dtype=dtype, device="cuda")[1:].view(v, d + 1)
    oddw[:, :d] = w
    ref.check(run(x, oddw[:, :d], target, dloss), want)
    xe = x[:1].expand(n, -1)
    ref.check(run(xe, w, target, dloss), ref.cross_entropy(xe, w, target, dloss=dloss))
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    fs.fs_cross_entropy(x, w, target, loss, lse)
    bx = torch.full((n + 1, d + 8), 3.0, dtype=dtype, device="cuda")
    bw = torch.full((v + 1, d + 1), 3.0, dtype=dtype, device="cuda")
    fs.fs_cross_entropy_grad(x, w, target, lse, dloss, bx[:n, :d], bw[:v, 1:])
    ref.check({"dx": bx[:n, :d], "dw": bw[:v, 1:]}, want)
    assert (bx[n] == 3).all() and (bx[:, d:] == 3).all() and (bw[v] == 3).all() and (bw[:, 0] == 3).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_same_bits_again_on_another_stream_and_in_a_graph(dtype):
    fs = _fs()
    x, w, target, dloss = make(200, 3000, 128, dtype, seed=8)
    a = run(x, w, target, dloss)
    b = run(x, w, target, dloss)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c = run(x, w, target, dloss, stream=s)
    s.synchronize()
    outs, graphs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        bufs = {k: torch.zeros_like(a[k]) for k in a}
        with torch.cuda.graph(g):
            fs.fs_cross_entropy(x, w, target, bufs["loss"], bufs["lse"])
            fs.fs_cross_entropy_grad(x, w, target, bufs["lse"], dloss, bufs["dx"], bufs["dw"])
        outs.append(bufs)
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for other in (b, c, *outs):
        for name in a:
            assert torch.equal(a[name], other[name]), name


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_several_pieces_of_the_vocabulary(dtype):
    """Enough rows that the gradient takes the classes in more than one piece, checked on samples."""
    n, v, d = 66000, 2500, 64
    x, w, target, dloss = make(n, v, d, dtype, seed=9)
    got = run(x, w, target, dloss)
    pick = torch.randperm(n, device="cuda")[:500]
    want = ref.cross_entropy(x[pick], w, target[pick], dloss=dloss[pick])
    ref.check({k: got[k][pick] for k in ("loss", "lse", "dx")}, want)
    # dw sums over every row: the 64-bit form in slices of the rows, their bounds added
    val, bound = 0.0, 0.0
    for a in range(0, n, 4000):
        s = slice(a, a + 4000)
        r = ref.cross_entropy(x[s], w, target[s], dloss=dloss[s])["dw"]
        val, bound = val + r[0], bound + r[1]
    # the fp32 sum runs over n terms, not 4000: at most (n + 64) U of the terms' sizes, of which a slice's bound
    # counts (4000 + 64) U
    bound = bound * ((n + 64) / 4064 if dtype == F32 else 1.5)
    ref.check({"dw": got["dw"]}, {"dw": (val, bound)})


@pytest.mark.parametrize("size", [(3, 1500, 40000, F32), (2, 5000, 40001, BF16)])
def test_wide_rows_copied_in_several_pieces(size):
    n, v, d, dtype = size
    x, w, target, dloss = make(n, v, d, dtype, seed=14, ignored=False)
    target[0] = v - 1
    ref.check(run(x, w, target, dloss), ref.cross_entropy(x, w, target, dloss=dloss))


def test_offsets_past_32_bits():
    """More than 2^31 class weights.  The classes but the last few repeat one row, so the 64-bit sums are short."""
    fs = _fs()
    v, d, tail, n = 1_100_000, 2048, 300, 3
    g = torch.Generator(device="cuda").manual_seed(2)
    row = torch.randn(1, d, device="cuda", generator=g).to(BF16) / 32
    w = row.expand(v, d).contiguous()
    w[-tail:] = (torch.randn(tail, d, device="cuda", generator=g) / 32).to(BF16)
    x = torch.randn(n, d, device="cuda", generator=g).to(BF16)
    target = torch.tensor([v - 1, v - tail, 5], device="cuda")
    dloss = torch.ones(n, device="cuda")
    got = run(x, w, target, dloss)
    z0, zt = x.double() @ row[0].double(), x.double() @ w[-tail:].double().t()
    lse = torch.logaddexp(z0 + math.log(v - tail), torch.logsumexp(zt, 1))
    hit = torch.stack([zt[0, -1], zt[1, 0], z0[2]])
    # the sum over 4297 tiles of 256: (256 + 4297 + 16) U; logits below 8 of 2048 terms of size below 60 together
    tol = (256 + 4297 + 16) * ref.U + 2 * (d + 8) * ref.U * 60
    assert (got["lse"] - lse).abs().max() <= tol and (got["loss"] - (lse - hit)).abs().max() <= 2 * tol
    pt = torch.exp(zt - lse[:, None])
    pt[0, -1] -= 1.0
    pt[1, 0] -= 1.0
    p0 = torch.exp(z0 - lse)
    want = pt.t() @ x.double()
    lim = (4 * ref.BF + 2 * tol) * (pt.abs().t() @ x.double().abs()) + 1e-9
    assert ((got["dw"][-tail:].double() - want).abs() <= lim).all()
    one = p0 @ x.double()
    lim0 = (4 * ref.BF + 2 * tol) * (p0 @ x.double().abs())
    assert ((got["dw"][6:-tail:1000].double() - one).abs() <= lim0).all()
    dx = pt @ w[-tail:].double() + ((v - tail) * p0)[:, None] * row.double()
    dx[2] -= row[0].double()
    # every p is rounded to bf16, and the fp32 sums run over at most 1.1e6 terms of one sign a column in parts
    size = pt.abs() @ w[-tail:].double().abs() + ((v - tail) * p0 + 1)[:, None] * row.double().abs()
    assert ((got["dx"].double() - dx).abs() <= (4 * ref.BF + 2 * tol + v / 16 * ref.U) * size).all()


def test_no_rows():
    fs = _fs()
    x, w, target, dloss = make(0, 100, 64, BF16)
    dw = torch.ones_like(w)
    loss = torch.empty(0, device="cuda")
    fs.fs_cross_entropy(x, w, target, loss, loss)
    fs.fs_cross_entropy_grad(x, w, target, loss, dloss, torch.empty_like(x), dw)
    assert (dw == 0).all()


def test_gradient_against_differences():
    x, w, target, dloss = make(20, 130, 24, F32, seed=12)
    dlse = torch.linspace(0, 1, 20, device="cuda")
    got = run(x, w, target, dloss, dlse)
    want = ref.cross_entropy(x, w, target, dloss=dloss, dlse=dlse)
    gen = torch.Generator(device="cuda").manual_seed(1)
    for i, name in enumerate(["dx", "dw"]):
        u = torch.randn(got[name].shape, device="cuda", generator=gen).double()
        f = []
        for e in (1e-5, -1e-5):
            t = [y + e * u if j == i else y for j, y in enumerate([x.double(), w.double()])]
            r = ref.cross_entropy(*t, target)
            f.append((r["loss"][0] * torch.where(target != -100, dloss, 0.0).double()).sum()
                     + (r["lse"][0] * dlse.double()).sum())
        slope = (f[0] - f[1]) / 2e-5
        assert (slope - (got[name].double() * u).sum()).abs() <= (want[name][1] * u.abs()).sum() + 1e-6


def test_a_scale_given_as_a_tensor_is_read_at_every_call():
    x, w = (torch.randn(s, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(s)) for s in (9, 300))
    target = torch.arange(9, device="cuda")
    scale, got = torch.tensor(0.1), []
    for value in (0.1, 0.5):
        scale.fill_(value)
        for sc in (scale, float(scale)):
            got.append((torch.empty(9, device="cuda"), torch.empty(9, device="cuda")))
            _fs().fs_cross_entropy(x, w, target, *got[-1], scale=sc)
    assert torch.equal(got[2][0], got[3][0]) and torch.equal(got[2][1], got[3][1])
    assert not torch.equal(got[1][1], got[3][1])


def test_refusals():
    fs = _fs()
    x, w, target, dloss = make(20, 30, 64, BF16)
    loss, lse = torch.empty(20, device="cuda"), torch.empty(20, device="cuda")
    for args in [(x.half(), w, target, loss, lse), (x, w.float(), target, loss, lse),
                 (x[:, :32], w, target, loss, lse), (x, w, target.int(), loss, lse), (x, w, target[:5], loss, lse),
                 (x, w, target, loss.double(), lse), (x, w, target, loss, lse[:10]), (x[None], w, target, loss, lse),
                 (x.t(), w, target, loss, lse), (x, w.cpu(), target, loss, lse), (x, w, target.cpu(), loss, lse)]:
        with pytest.raises(ValueError):
            fs.fs_cross_entropy(*args)
    for scale in (0.0, -2.0, math.nan, math.inf):
        with pytest.raises(fs.FsError):
            fs.fs_cross_entropy(x, w, target, loss, lse, scale=scale)
    with pytest.raises(fs.FsError):  # no classes
        fs.fs_cross_entropy(x, w[:0], target, loss, lse)
    with pytest.raises(fs.FsError):  # an output row on top of the next
        fs.fs_cross_entropy_grad(x, w, target, lse, dloss, torch.empty_like(x), w[:1].expand(30, -1))
    with pytest.raises(fs.FsError):
        need = fs.fs_cross_entropy_workspace(x, w)
        fs.fs_cross_entropy(x, w, target, loss, lse,
                            workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    fs.fs_check()
