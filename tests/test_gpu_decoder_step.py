"""Cross attention and cross entropy together, as a decoder uses them: queries read an encoder's states
(keys and values side by side in one projection's output), the read rows are scored against a vocabulary, and the
loss's gradient runs back through both.  Every stage is checked against its 64-bit form on what the stage before
really gave, with the bounds of tests/ops_reference.py; the whole against differences of the loss."""
import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def _fs():
    import log_domain_sinkhorn_updates_b200 as fs
    return fs


def make(B, n, m, H, Hk, d, V, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*s):
        return torch.randn(*s, device="cuda", generator=g)

    kv = r(B, m, 2, Hk, d).to(dtype)
    t = dict(q=r(B, n, H, d).to(dtype), kv=kv, k=kv[:, :, 0], v=kv[:, :, 1],
             w=(r(V, H * d) / (H * d) ** 0.5).to(dtype),
             target=torch.randint(0, V, (B * n,), device="cuda", generator=g))
    t["k_len"] = torch.randint(1, m + 1, (B,), device="cuda", generator=g).int()
    t["target"][torch.rand(B * n, device="cuda", generator=g) < 0.15] = -100
    t["dloss"] = (t["target"] != -100).float() / max(1, int((t["target"] != -100).sum()))
    return t


def buffers(t):
    B, n, H, d = t["q"].shape
    dev = t["q"].device
    o = dict(out=torch.empty_like(t["q"]), lse=torch.empty(B, H, n, device=dev), loss=torch.empty(B * n, device=dev),
             zlse=torch.empty(B * n, device=dev), dq=torch.empty_like(t["q"]), dkv=torch.empty_like(t["kv"]),
             dw=torch.empty_like(t["w"]))
    o["dout"] = torch.empty_like(o["out"])
    return o


def step(t, o):
    fs = _fs()
    rows = o["out"].view(-1, t["w"].shape[1])
    fs.fs_cross_attn(t["q"], t["k"], t["v"], o["out"], o["lse"], k_len=t["k_len"])
    fs.fs_cross_entropy(rows, t["w"], t["target"], o["loss"], o["zlse"])
    fs.fs_cross_entropy_grad(rows, t["w"], t["target"], o["zlse"], t["dloss"], o["dout"].view_as(rows), o["dw"])
    fs.fs_cross_attn_grad(t["q"], t["k"], t["v"], o["out"], o["lse"], o["dout"], o["dq"], o["dkv"][:, :, 0],
                          o["dkv"][:, :, 1], k_len=t["k_len"])


def check(t, o):
    a = ref.attention(t["q"], t["k"], t["v"], k_len=t["k_len"], dout=o["dout"])
    ref.check({"out": o["out"], "lse": o["lse"], "dq": o["dq"], "dk": o["dkv"][:, :, 0], "dv": o["dkv"][:, :, 1]}, a)
    rows = o["out"].reshape(-1, t["w"].shape[1])
    c = ref.cross_entropy(rows, t["w"], t["target"], dloss=t["dloss"])
    ref.check({"loss": o["loss"], "lse": o["zlse"], "dx": o["dout"].reshape(rows.shape), "dw": o["dw"]}, c)
    return a, c


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size", [(2, 1, 300, 8, 2, 64, 1000), (3, 33, 129, 4, 4, 32, 777), (2, 150, 400, 6, 3, 64, 3000),
                                  (1, 5, 2000, 2, 1, 128, 513)])
def test_a_step_and_its_replays(size, dtype):
    t = make(*size, dtype, seed=sum(size))
    o = buffers(t)
    step(t, o)
    check(t, o)
    # captured, then replayed on other inputs in the same buffers
    g = torch.cuda.CUDAGraph()
    p = buffers(t)
    with torch.cuda.graph(g):
        step(t, p)
    for seed in (1, 2):
        new = make(*size, dtype, seed=seed)
        for name in ("q", "kv", "w", "target", "k_len", "dloss"):
            t[name].copy_(new[name])
        g.replay()
        check(t, p)
    _fs().fs_check()


def test_loss_against_differences():
    """fp32: the loss's slope along a direction of every input, by central differences of the whole chain in 64
    bits, against the gradients.  What the stages' bounds allow is added up: the attention's gradients at the dout
    it was given, and dout's own distance from the exact chain's, carried by the derivative of out."""
    t = make(2, 9, 37, 4, 2, 24, 130, F32, seed=5)
    o = buffers(t)
    step(t, o)
    a, _ = check(t, o)
    keys = ["q", "k", "v", "w"]
    base = {x: t[x].double() for x in keys}

    def chain(ins):
        out = ref.attention(ins["q"], ins["k"], ins["v"], k_len=t["k_len"])["out"][0]
        r = ref.cross_entropy(out.reshape(-1, ins["w"].shape[1]), ins["w"], t["target"], dloss=t["dloss"])
        return out, (r["loss"][0] * t["dloss"].double()).sum(), r

    out0, _, exact = chain(base)
    gen = torch.Generator(device="cuda").manual_seed(3)
    e = 1e-5
    off = (o["dout"].double() - exact["dx"][0].reshape(out0.shape)).abs()
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("w", "dw")):
        u = torch.randn(base[name].shape, device="cuda", generator=gen).double()
        hi = chain({**base, name: base[name] + e * u})
        lo = chain({**base, name: base[name] - e * u})
        slope = (hi[1] - lo[1]) / (2 * e)
        if name == "w":
            got, bound = o["dw"].double(), exact["dw"][1].abs() + (o["dw"].double() - exact["dw"][0]).abs()
            allowed = (bound * u.abs()).sum()
        else:
            got = {"dq": o["dq"], "dk": o["dkv"][:, :, 0], "dv": o["dkv"][:, :, 1]}[grad].double()
            carried = (hi[0] - lo[0]).abs() / (2 * e)
            allowed = (a[grad][1] * u.abs()).sum() + (off * carried).sum()
        assert (slope - (got * u).sum()).abs() <= allowed + 1e-7, name
        # and the gradients are near the exact chain's as a whole, so that what was allowed above is small
        assert allowed <= 1e-3 * (got.abs() * u.abs()).sum(), name
