"""Cross attention, forward and gradient, against the 64-bit form with derived bounds
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


def make(B, n, m, H, Hk, d, dv, dtype, seed=0, fused=False):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*s):
        return torch.randn(*s, device="cuda", generator=g)

    q = (1.5 * r(B, n, H, d)).to(dtype)
    if fused and d == dv:
        kv = r(B, m, 2, Hk, d).to(dtype)
        k, v = kv[:, :, 0], kv[:, :, 1]
    else:
        k, v = r(B, m, Hk, d).to(dtype), r(B, m, Hk, dv).to(dtype)
    return q, k, v, r(B, n, H, dv).to(dtype)


def forward(q, k, v, **kw):
    B, n, H, _ = q.shape
    out = torch.full((B, n, H, v.shape[3]), 7.0, dtype=q.dtype, device=q.device)
    lse = torch.full((B, H, n), 7.0, device=q.device)
    _fs().fs_cross_attn(q, k, v, out, lse, **kw)
    return out, lse


def gradient(q, k, v, out, lse, dout, **kw):
    grads = [torch.full(t.shape, 7.0, dtype=t.dtype, device=t.device) for t in (q, k, v)]
    _fs().fs_cross_attn_grad(q, k, v, out, lse, dout, *grads, **kw)
    return grads


def run(q, k, v, dout, **kw):
    out, lse = forward(q, k, v, **kw)
    dq, dk, dv = gradient(q, k, v, out, lse, dout, **kw)
    _fs().fs_check()
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


# batch, n, m, heads, kv heads, d, dv
SIZES = [
    (1, 1, 1, 1, 1, 8, 8),
    (2, 1, 129, 4, 2, 64, 64),
    (1, 1, 5000, 8, 1, 128, 128),
    (2, 1, 777, 6, 2, 96, 96),
    (3, 2, 640, 32, 2, 128, 64),
    (1, 7, 63, 3, 1, 40, 24),
    (2, 65, 128, 4, 4, 64, 64),
    (2, 130, 257, 6, 2, 128, 128),
    (1, 300, 1021, 5, 1, 80, 80),
    (1, 129, 130, 2, 2, 16, 128),
    (2, 33, 31, 2, 1, 33, 7),
    (1, 20, 70, 2, 1, 256, 256),
    (1, 400, 20, 2, 2, 128, 96),
    (1, 513, 384, 7, 7, 72, 72),
    (1, 30, 100, 2, 1, 64, 200),
    (1, 140, 200, 2, 1, 128, 8),
    (2, 100, 90, 3, 3, 8, 64),
    # enough heads that one CTA walks many tiles: one row block a CTA, and two
    (1, 128, 650, 100, 100, 32, 32),
    (2, 40, 900, 60, 60, 128, 128),
    (2, 150, 1300, 80, 80, 128, 64),
    (3, 260, 700, 64, 32, 96, 96),
    # more units than SMs: those behind the last full wave are split over their keys
    (2, 300, 1100, 64, 64, 64, 64),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size", SIZES)
def test_against_64_bits(size, dtype):
    q, k, v, dout = make(*size, dtype, seed=sum(size), fused=True)
    got = run(q, k, v, dout)
    ref.check(got, ref.attention(q, k, v, dout=dout))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [1, 50, 200])
@pytest.mark.parametrize("poison", [math.nan, math.inf])
def test_lengths_and_masks_with_anything_in_masked_places(dtype, n, poison):
    """Lengths of 0, 1, past the end and below zero; masks by -inf, by the type's lowest
    value, holes, a row without a key; NaN or infinity in every masked key."""
    B, m, H, Hk, d = 8, 421, 4, 2, 64
    q, k, v, dout = make(B, n, m, H, Hk, d, d, dtype, seed=5)
    g = torch.Generator(device="cuda").manual_seed(9)
    k_len = torch.tensor([0, 1, m, m + 50, -3, 128, 129, 300], dtype=torch.int32, device="cuda")
    bias = torch.randn(B, m, device="cuda", generator=g)
    bias[torch.rand(B, m, device="cuda", generator=g) < 0.2] = -math.inf
    bias[2, 10:140] = torch.finfo(F32).min
    bias[5] = -1e30  # masked everywhere
    bias[7, :299] = -math.inf
    bias[7, 299] = 0.25
    dead = (torch.arange(m, device="cuda")[None] >= k_len.clamp(0, m)[:, None]) | (bias <= -1e30)
    k[dead], v[dead] = poison, -poison
    for kw in ({"k_len": k_len, "bias": bias}, ):
        got = run(q, k, v, dout, **kw)
        ref.check(got, ref.attention(q, k, v, dout=dout, **kw))
    assert (got["out"][[0, 4, 5]] == 0).all() and torch.isneginf(got["lse"][[0, 4, 5]]).all()
    assert (got["dq"][[0, 4, 5]] == 0).all()
    assert (got["dk"][dead] == 0).all() and (got["dv"][dead] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_no_keys_no_queries(dtype):
    q, k, v, dout = make(2, 5, 0, 2, 1, 64, 64, dtype)
    out, lse = forward(q, k, v)
    assert (out == 0).all() and torch.isneginf(lse).all()
    dq, dk, dv = gradient(q, k, v, out, lse, dout)
    assert (dq == 0).all() and dk.numel() == 0
    q, k, v, dout = make(2, 0, 200, 2, 1, 64, 64, dtype)
    out, lse = forward(q, k, v)
    dq, dk, dv = gradient(q, k, v, out, lse, dout)
    assert (dk == 0).all() and (dv == 0).all()
    q, k, v, dout = make(0, 4, 6, 2, 1, 64, 64, dtype)
    out, lse = forward(q, k, v)
    gradient(q, k, v, out, lse, dout)
    _fs().fs_check()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [1, 140])
def test_strides(dtype, n):
    """Keys shared by the batch (stride 0) or by heads, transposed layouts, an odd offset, outputs into
    parts of larger buffers whose other parts stay as they were."""
    B, m, H, Hk, d = 3, 260, 4, 2, 64
    q, k, v, dout = make(B, n, m, H, Hk, d, d, dtype, seed=3)
    want = ref.attention(q, k, v, dout=dout)
    # [batch, head, token, width] memory
    qt, kt, vt = (t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for t in (q, k, v))
    ref.check(run(qt, kt, vt, dout), want)
    # one element off the natural alignment
    def shifted(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
        s = flat[1:].view(t.shape)
        s.copy_(t)
        return s
    ref.check(run(shifted(q), shifted(k), shifted(v), shifted(dout)), want)
    # broadcast over the batch, and over key heads
    k1, v1 = k[:1].expand(B, -1, -1, -1), v[:1].expand(B, -1, -1, -1)
    ref.check(run(q, k1, v1, dout), ref.attention(q, k1, v1, dout=dout))
    k2 = k[:, :, :1].expand(-1, -1, Hk, -1)
    ref.check(run(q, k2, v, dout), ref.attention(q, k2, v, dout=dout))
    # a token repeated (stride 0 along the keys)
    k3 = k[:, :1].expand(-1, m, -1, -1)
    ref.check(run(q, k3, v, dout), ref.attention(q, k3, v, dout=dout))
    # outputs inside larger buffers
    big = torch.full((B, n + 2, H + 1, d + 8), 3.0, dtype=dtype, device="cuda")
    out = big[:, 1:n + 1, :H, :d]
    lse = torch.empty(B, H, n, device="cuda")
    _fs().fs_cross_attn(q, k, v, out, lse)
    bigkv = torch.full((B, m + 1, 2, Hk, d), 3.0, dtype=dtype, device="cuda")
    dk, dv = bigkv[:, :m, 0], bigkv[:, :m, 1]
    bigq = torch.full((B, n + 1, H, d), 3.0, dtype=dtype, device="cuda")
    _fs().fs_cross_attn_grad(q, k, v, out, lse, dout, bigq[:, :n], dk, dv)
    ref.check({"out": out, "lse": lse, "dq": bigq[:, :n], "dk": dk, "dv": dv}, want)
    assert (big[:, 0] == 3).all() and (big[:, n + 1] == 3).all() and (big[:, :, H] == 3).all()
    assert (big[..., d:] == 3).all() and (bigkv[:, m] == 3).all() and (bigq[:, n] == 3).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scales_and_large_scores(dtype):
    """Scores of thousands: one key takes all; and a scale of its own."""
    q, k, v, dout = make(1, 70, 200, 2, 2, 64, 64, dtype, seed=11)
    for scale in (1e-4, 3.0, 40.0):
        got = run(q, k, v, dout, scale=scale)
        ref.check(got, ref.attention(q, k, v, dout=dout, scale=scale))


def test_nan_in_a_query_stays_in_its_row():
    q, k, v, dout = make(1, 140, 200, 2, 2, 64, 64, BF16, seed=2)
    want, _ = forward(q, k, v)
    q[0, 17, 1, 3] = math.nan
    out, lse = forward(q, k, v)
    assert torch.isnan(out[0, 17, 1]).all() and torch.isnan(lse[0, 1, 17])
    out[0, 17, 1] = want[0, 17, 1]
    assert torch.equal(out, want)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [1, 90])
def test_same_bits_again_on_another_stream_and_in_a_graph(dtype, n):
    fs = _fs()
    q, k, v, dout = make(2, n, 700, 4, 2, 64, 64, dtype, seed=8)
    k_len = torch.tensor([700, 333], dtype=torch.int32, device="cuda")
    a = run(q, k, v, dout, k_len=k_len)
    b = run(q, k, v, dout, k_len=k_len)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c = run(q, k, v, dout, k_len=k_len, stream=s)
    s.synchronize()
    # two graphs, captured with workspaces of their own, replayed at the same time
    outs, graphs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        bufs = {x: torch.zeros_like(a[x]) for x in a}
        with torch.cuda.graph(g):
            fs.fs_cross_attn(q, k, v, bufs["out"], bufs["lse"], k_len=k_len)
            fs.fs_cross_attn_grad(q, k, v, bufs["out"], bufs["lse"], dout, bufs["dq"], bufs["dk"], bufs["dv"],
                                  k_len=k_len)
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


@pytest.mark.parametrize("m", [100, 3000])
def test_without_lse_and_with_a_workspace_of_its_own(m):
    fs = _fs()
    q, k, v, _ = make(2, 1, m, 8, 2, 64, 64, BF16, seed=31)
    want, _ = forward(q, k, v)
    out = torch.zeros_like(q)
    need = fs.fs_cross_attn_workspace(q, k, v, out)
    ws = torch.full((need + 1024,), 255, dtype=torch.uint8, device="cuda")
    fs.fs_cross_attn(q, k, v, out, workspace=ws)
    assert torch.equal(out, want)
    assert (ws[need:] == 255).all()  # nothing behind it
    if need:
        with pytest.raises(fs.FsError):  # not on 256 bytes
            fs.fs_cross_attn(q, k, v, out, workspace=ws[8:])


def test_calls_at_once_on_two_streams():
    fs = _fs()
    sets = [make(2, 70, 900, 8, 4, 64, 64, BF16, seed=s) for s in (1, 2)]
    want = [run(*t) for t in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, (t, s) in enumerate(zip(sets, streams)):
            with torch.cuda.stream(s):
                out, lse = forward(*t[:3])
                got[i].append([out, lse, *gradient(*t[:3], out, lse, t[3])])
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        for r in runs:
            assert all(torch.equal(a, b) for a, b in zip(w.values(), r))


def test_offsets_past_32_bits():
    """Keys and values of more than 2^31 elements each; only the last ones count, so a wrong offset shows."""
    m, Hk, d = 1_100_000, 16, 128
    k = torch.zeros(1, m, Hk, d, dtype=BF16, device="cuda")
    v = torch.full_like(k, math.nan)
    g = torch.Generator(device="cuda").manual_seed(1)
    tail = 300
    k[:, -tail:] = torch.randn(1, tail, Hk, d, device="cuda", generator=g).to(BF16)
    v[:, -tail:] = torch.randn(1, tail, Hk, d, device="cuda", generator=g).to(BF16)
    q = torch.randn(1, 1, 2 * Hk, d, device="cuda", generator=g).to(BF16)
    bias = torch.full((1, m), -math.inf, device="cuda")
    bias[:, -tail:] = 0.0
    out, lse = forward(q, k, v, bias=bias)
    ref.check({"out": out, "lse": lse}, ref.attention(q, k[:, -tail:], v[:, -tail:]))
    dout = torch.randn(q.shape, device="cuda", generator=g).to(BF16)
    dq, dk, dv = gradient(q, k, v, out, lse, dout, bias=bias)
    want = ref.attention(q, k[:, -tail:], v[:, -tail:], dout=dout)
    ref.check({"dq": dq, "dk": dk[:, -tail:], "dv": dv[:, -tail:]}, want)
    assert (dk[:, :-tail] == 0).all() and (dv[:, :-tail] == 0).all()


FIRST_IN_CAPTURE = """
import torch
import log_domain_sinkhorn_updates_b200 as fs
q = torch.randn(1, 3, 2, 64, device="cuda", dtype=torch.bfloat16)
k = torch.randn(1, 500, 2, 64, device="cuda", dtype=torch.bfloat16)
out, lse = torch.zeros_like(q), torch.zeros(1, 2, 3, device="cuda")
x, w = torch.randn(5, 64, device="cuda"), torch.randn(70, 64, device="cuda")
t, loss, z = torch.zeros(5, dtype=torch.long, device="cuda"), torch.zeros(5, device="cuda"), torch.zeros(5, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    fs.fs_cross_attn(q, k, k, out, lse)
    fs.fs_cross_entropy(x, w, t, loss, z)
g.replay()
torch.cuda.synchronize()
want = torch.softmax(torch.einsum("bihd,bjhd->bhij", q.float(), k.float()) / 8, -1)
want = torch.einsum("bhij,bjhd->bihd", want, k.float())
assert (out.float() - want).abs().max() < 0.05 and (z - torch.logsumexp(x @ w.t(), 1)).abs().max() < 1e-3
print("captured")
"""


def test_the_first_calls_of_a_process_may_be_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_IN_CAPTURE], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout[-500:] + r.stderr[-1500:]


def test_gradient_against_differences():
    """fp32: d/de <dout, out(inputs + e u)> by central differences in 64 bits of the plain form equals
    <grad, u> of the library's gradient."""
    q, k, v, dout = make(2, 9, 37, 4, 2, 24, 16, F32, seed=21)
    k_len = torch.tensor([37, 20], dtype=torch.int32, device="cuda")
    got = run(q, k, v, dout, k_len=k_len)
    gen = torch.Generator(device="cuda").manual_seed(1)
    for i, name in enumerate(["dq", "dk", "dv"]):
        u = torch.randn(got[name].shape, device="cuda", generator=gen).double()
        ins = [q.double(), k.double(), v.double()]
        f = []
        for e in (1e-5, -1e-5):
            t = [x + e * u if j == i else x for j, x in enumerate(ins)]
            f.append((ref.attention(*t, k_len=k_len)["out"][0] * dout.double()).sum())
        slope = (f[0] - f[1]) / 2e-5
        bound = (ref.attention(q, k, v, k_len=k_len, dout=dout)[name][1] * u.abs()).sum()
        # central difference: third derivative times e^2, about 1e-10 of terms of order 1 to 100
        assert (slope - (got[name].double() * u).sum()).abs() <= bound + 1e-6


def test_equals_the_barycentric_map():
    """The barycentric map of the library at the same potentials: q = x, k = v = y, scale 2/eps and bias
    (g - |y|^2)/eps + log b; and lse is its f-update."""
    fs = _fs()
    gen = torch.Generator(device="cuda").manual_seed(4)
    n, m, d, eps = 300, 260, 32, 0.3
    X = torch.randn(1, n, d, device="cuda", generator=gen) / d ** 0.5
    Y = torch.randn(1, m, d, device="cuda", generator=gen) / d ** 0.5
    g = 0.1 * torch.randn(1, m, device="cuda", generator=gen)
    h = fs.fs_create(X, Y, eps=eps)
    f = torch.empty(1, n, device="cuda")
    fs.fs_update_f(h, g, f)
    T = torch.empty(1, n, d, device="cuda")
    fs.fs_barycentric_map(h, f, g, Y, T)
    bias = ((g.double() - (Y.double() ** 2).sum(-1)) / eps - math.log(m)).float()
    out, lse = forward(X[:, :, None], Y[:, :, None], Y[:, :, None], bias=bias, scale=2 / eps)
    want = ref.attention(X[:, :, None], Y[:, :, None], Y[:, :, None], bias=bias, scale=2 / eps)
    ref.check({"out": out, "lse": lse}, want)
    # the map: both sides are within 2^-14 of the exact map (the handle's derived bound), |y| <= 1.5
    assert (out[:, :, 0] - T).abs().max() <= 2 * 2.0 ** -14 * Y.abs().max()
    f2 = (X.double() ** 2).sum(-1) - eps * lse[:, 0].double()
    assert (f2 - f).abs().max() <= 1e-4 * ((X.unsqueeze(2) - Y.unsqueeze(1)) ** 2).sum(-1).max()
    fs.fs_destroy(h)


@pytest.mark.parametrize("dtype,d,dv", [(F32, 64, 64), (F32, 128, 36), (F32, 20, 128), (BF16, 36, 20), (BF16, 64, 64)])
@pytest.mark.parametrize("n,H,Hk", [(1, 3, 1), (4, 1, 1), (1, 5, 1), (2, 8, 2), (3, 6, 2), (3, 3, 1)])
def test_few_rows(n, H, Hk, dtype, d, dv):
    """1 to 9 rows a key head, lengths that leave parts and problems without a key."""
    for m in (0, 1, 31, 33, 2500):
        q, k, v, dout = make(3, n, m, H, Hk, d, dv, dtype, seed=m + n)
        k_len = torch.tensor([m, 0, m // 3 + 1], dtype=torch.int32, device="cuda")
        for kw in ({}, {"k_len": k_len}):
            out, lse = forward(q, k, v, **kw)
            ref.check({"out": out, "lse": lse}, ref.attention(q, k, v, **kw))
    _fs().fs_check()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size", [(2, 600, 64, 8, 1, 64, 128), (3, 5, 1300, 4, 2, 128, 64), (2, 1, 900, 2, 2, 32, 32)])
def test_gradient_of_few_heads_and_ragged_lengths(size, dtype):
    """Few enough CTAs that the gradient's streamed tiles are split; lengths that leave parts without a key."""
    q, k, v, dout = make(*size, dtype, seed=11)
    m = size[2]
    for lens in ([m, 0, 1], [m // 2 + 3, m, m - 1]):
        kw = {"k_len": torch.tensor(lens[:size[0]], dtype=torch.int32, device="cuda")}
        ref.check(run(q, k, v, dout, **kw), ref.attention(q, k, v, dout=dout, **kw))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size", [(1, 4, 5000, 8, 1, 128, 128), (1, 1, 9000, 4, 2, 64, 32), (1, 300, 260, 4, 4, 200, 130),
                                  (2, 200, 300, 4, 2, 40, 40), (1, 2000, 10, 1, 1, 64, 63)])
def test_gradient_split_over_its_streamed_rows(size, dtype):
    """Few rows against many keys, many rows against few, with a mask; outputs into parts of larger buffers."""
    q, k, v, dout = make(*size, dtype, seed=23)
    B, n, m, H, Hk, d, dv = size
    bias = torch.randn(B, m, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    bias[:, 3::7] = -math.inf
    want = ref.attention(q, k, v, dout=dout, bias=bias)
    got = run(q, k, v, dout, bias=bias)
    ref.check(got, want)
    bigk = torch.full((B, Hk, m + 1, d + 8), 3.0, dtype=dtype, device="cuda")
    bigq = torch.full((B, n + 1, H, d), 3.0, dtype=dtype, device="cuda")
    dk, dq, gv = bigk[:, :, :m, :d].transpose(1, 2), bigq[:, :n], torch.empty_like(v)
    _fs().fs_cross_attn_grad(q, k, v, got["out"], got["lse"], dout, dq, dk, gv, bias=bias)
    assert torch.equal(dq, got["dq"]) and torch.equal(dk, got["dk"]) and torch.equal(gv, got["dv"])
    assert (bigk[:, :, m] == 3).all() and (bigk[..., d:] == 3).all() and (bigq[:, n] == 3).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_more_problems_than_are_ordered_by_length(dtype):
    B, n, m = 41, 3, 700
    q, k, v, dout = make(B, n, m, 4, 2, 64, 64, dtype, seed=13)
    g = torch.Generator().manual_seed(3)
    kw = {"k_len": torch.randint(-5, m + 20, (B,), dtype=torch.int32, generator=g).cuda()}
    ref.check(run(q, k, v, dout, **kw), ref.attention(q, k, v, dout=dout, **kw))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [1, 6, 200])
def test_anything_in_the_queries_of_a_problem_without_keys(dtype, n):
    """Padding of a batch: length 0, NaN in q, k, v and the gradient; the other problems keep their bits."""
    q, k, v, dout = make(3, n, 400, 4, 2, 64, 64, dtype, seed=17)
    kw = {"k_len": torch.tensor([400, 0, 77], dtype=torch.int32, device="cuda")}
    clean = run(q, k, v, dout, **kw)
    for t in (q, k, v, dout):
        t[1] = math.nan
    got = run(q, k, v, dout, **kw)
    for name in got:
        assert torch.equal(got[name], clean[name]), name
    assert (got["out"][1] == 0).all() and (got["dk"][1] == 0).all() and (got["dv"][1] == 0).all()


def test_a_scale_given_as_a_tensor_is_read_at_every_call():
    q, k, v, _ = make(1, 4, 50, 2, 2, 64, 64, F32, seed=19)
    scale = torch.tensor(0.1)
    forward(q, k, v, scale=scale)
    scale.fill_(0.4)
    out, lse = forward(q, k, v, scale=scale)
    want_out, want_lse = forward(q, k, v, scale=0.4000000059604645)
    assert torch.equal(out, want_out) and torch.equal(lse, want_lse)


def test_refusals():
    fs = _fs()
    q, k, v, dout = make(2, 5, 9, 4, 2, 64, 64, BF16)
    out, lse = torch.empty_like(q), torch.empty(2, 4, 5, device="cuda")
    for bad in [dict(k_len=torch.ones(2, device="cuda")), dict(k_len=torch.ones(3, dtype=torch.int32, device="cuda")),
                dict(bias=torch.ones(2, 8, device="cuda")), dict(bias=torch.ones(2, 9, device="cuda", dtype=BF16)),
                dict(bias=torch.ones(2, 9)), dict(workspace=torch.empty(0, dtype=torch.uint8))]:
        with pytest.raises(ValueError):
            fs.fs_cross_attn(q, k, v, out, lse, **bad)
    for args in [(q.half(), k, v, out), (q, k.float(), v, out), (q, k[:, :, :, :32], v, out), (q, k, v[:, :8], out),
                 (q, k, v, out[:, :4]), (q[0], k, v, out), (q, k.cpu(), v, out),
                 (q.transpose(1, 3), k, v, out), (q, k.transpose(2, 3).contiguous().transpose(2, 3), v, out)]:
        with pytest.raises(ValueError):
            fs.fs_cross_attn(*args, lse)
    with pytest.raises(ValueError):
        fs.fs_cross_attn(q, k, v, out, lse[:, :, :4])
    for scale in (0.0, -1.0, math.nan, math.inf):
        with pytest.raises(fs.FsError):
            fs.fs_cross_attn(q, k, v, out, lse, scale=scale)
    with pytest.raises(fs.FsError):  # heads not a multiple
        fs.fs_cross_attn(q[:, :, :3], k, v, out[:, :, :3])
    with pytest.raises(fs.FsError):  # an output whose elements overlap
        fs.fs_cross_attn(q, k, v, out[:1].expand(2, -1, -1, -1), lse)
    with pytest.raises(fs.FsError):
        fs.fs_cross_attn_grad(q, k, v, out, lse, dout, torch.empty_like(q), k[:, :1].expand(-1, 9, -1, -1),
                              torch.empty_like(v))
    with pytest.raises(fs.FsError):  # workspace too small
        need = fs.fs_cross_attn_workspace(q, k, v, out, dout, q, k, v)
        assert need > 0
        fs.fs_cross_attn_grad(q, k, v, out, lse, dout, torch.empty_like(q), torch.empty_like(k), torch.empty_like(v),
                              workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    forward(q, k, v)
    gradient(q, k, v, *forward(q, k, v), dout, workspace=ws)
    fs.fs_check()
