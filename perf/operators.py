"""Measured cases of the language-model operators: cross attention and softmax cross entropy.

Both are row softmaxes of a streamed score product with a per-column term, the
family of the library's log-domain updates and transport applications:

  cross attention   S_ij = scale q_i.k_j + bias_j,  out_i = sum_j softmax_j(S_i) v_j
  cross entropy     z_ij = scale x_i.w_j,  loss_i = log sum_j exp z_ij - z_{i, target_i}

`run` computes a case in elementary torch operations in 32 bits (`own` false)
or through the library's entry points (`own` true); `exact` is the definition
in 64 bits.
"""
import math

import torch

own = False

IGNORE = -100
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

CASES = [
    # --- cross attention: single tokens (serving) ---
    # one decoder step of one request over a short encoder output; latency is what counts
    dict(name="xattn_token_short", op="xattn", mode="token", dtype="bf16", batch=1, n=1, m=1500, heads=8,
         kv_heads=8, d=64, ragged=False, masked=False, fused_kv=False),
    # one step of a serving batch: requests with encoder outputs of different lengths, shared heads
    dict(name="xattn_token_batch", op="xattn", mode="token", dtype="bf16", batch=32, n=1, m=4096, heads=32,
         kv_heads=8, d=128, ragged=True, masked=False, fused_kv=True),
    # one request over a very long document: few rows, a long axis to split
    dict(name="xattn_token_long", op="xattn", mode="token", dtype="bf16", batch=1, n=1, m=131072, heads=32,
         kv_heads=8, d=128, ragged=False, masked=False, fused_kv=False),
    # --- cross attention: whole sequences ---
    # a decoder prompt against its encoder output, inference
    dict(name="xattn_prompt", op="xattn", mode="forward", dtype="bf16", batch=4, n=2048, m=4096, heads=16,
         kv_heads=16, d=128, ragged=False, masked=False, fused_kv=True),
    # a small training batch of odd lengths: padded encoder outputs, dropped positions, shared heads
    dict(name="xattn_train_ragged", op="xattn", mode="train", dtype="bf16", batch=3, n=333, m=1021, heads=12,
         kv_heads=4, d=64, ragged=True, masked=True, fused_kv=True),
    # a large training step
    dict(name="xattn_train_large", op="xattn", mode="train", dtype="bf16", batch=2, n=4096, m=8192, heads=32,
         kv_heads=8, d=128, ragged=False, masked=False, fused_kv=False),
    # full precision, a small model's step
    dict(name="xattn_train_f32", op="xattn", mode="train", dtype="f32", batch=2, n=200, m=300, heads=4,
         kv_heads=4, d=40, ragged=True, masked=True, fused_kv=False),
    # --- cross entropy over a vocabulary ---
    # the score of one token (perplexity of one step): one pass over the vocabulary's weights
    dict(name="xent_token", op="xent", mode="forward", dtype="bf16", n=1, m=65536, d=1024, ignored=False),
    # evaluation of one sequence
    dict(name="xent_eval", op="xent", mode="forward", dtype="bf16", n=2048, m=65536, d=2048, ignored=True),
    # a training step of odd sizes
    dict(name="xent_train_ragged", op="xent", mode="train", dtype="bf16", n=1021, m=50021, d=1000, ignored=True),
    # a training step with a large vocabulary
    dict(name="xent_train_large", op="xent", mode="train", dtype="bf16", n=8192, m=131072, d=2048, ignored=True),
    # full precision, a small model's step
    dict(name="xent_train_f32", op="xent", mode="train", dtype="f32", n=1024, m=16384, d=256, ignored=True),
]


def listed():
    return [dict(c) for c in CASES]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        if rng.random() < 0.55:
            mode = rng.choice(["token", "forward", "train"])
            dtype = "f32" if rng.random() < 0.2 else "bf16"
            kv_heads = rng.choice([1, 2, 4, 8])
            case = dict(op="xattn", mode=mode, dtype=dtype, heads=kv_heads * rng.choice([1, 2, 3, 4, 8]),
                        kv_heads=kv_heads, d=rng.choice([32, 40, 64, 80, 96, 128]), ragged=rng.random() < 0.6,
                        masked=rng.random() < 0.4, fused_kv=rng.random() < 0.5)
            if mode == "token":
                case.update(batch=_log_int(rng, 1, 32), n=1, m=_log_int(rng, 16, 65536))
            else:
                case.update(batch=rng.randint(1, 4), n=_log_int(rng, 2, 4096), m=_log_int(rng, 16, 8192))
            limit = 3e10 if dtype == "f32" else 1.1e12
        else:
            dtype = "f32" if rng.random() < 0.2 else "bf16"
            case = dict(op="xent", mode=rng.choice(["forward", "train"]), dtype=dtype, n=_log_int(rng, 1, 8192),
                        m=_log_int(rng, 1000, 131072), d=8 * _log_int(rng, 8, 512), ignored=rng.random() < 0.7)
            limit = 3e10 if dtype == "f32" else 4.0e12
        w = work(case)
        if w["flops"] <= limit and w["bytes"] <= 2.0e9:
            return case


def _lengths(case):
    """The valid encoder positions of each request: spread over (0, m], the longest m."""
    m, batch = case["m"], case["batch"]
    if not case["ragged"]:
        return [m] * batch
    return [max(1, m - (m * ((5 * b) % 8)) // 9) for b in range(batch)]


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    n, m, d = case["n"], case["m"], case["d"]
    if case["op"] == "xent":
        flops, byts = 2.0 * n * m * d, (n + m) * d * size + 16 * n
        if case["mode"] == "train":  # scores again, and one product for each gradient
            flops, byts = 4 * flops, 2 * (n + m) * d * size + 20 * n
        return {"bytes": float(byts), "flops": flops}
    heads, kv_heads, batch, keys = case["heads"], case["kv_heads"], case["batch"], sum(_lengths(case))
    pair = 2.0 * n * keys * heads * d
    q_bytes, kv_bytes = batch * n * heads * d * size, 2 * keys * kv_heads * d * size
    flops, byts = 2 * pair, 2 * q_bytes + kv_bytes
    if case["mode"] == "train":  # five products backward; q, k, v, out, dout in, the three gradients out
        flops, byts = 7 * pair, 4 * q_bytes + 2 * kv_bytes
    if case["mode"] != "token":
        byts += 4 * batch * n * heads
    if case["masked"]:
        byts += 4 * batch * m
    return {"bytes": float(byts), "flops": flops}


def _normal(gen, *shape):
    return torch.randn(*shape, device="cuda", generator=gen)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = TYPES[case["dtype"]]
    n, m, d = case["n"], case["m"], case["d"]
    if case["op"] == "xent":
        # class weights whose logits spread by about 2; each row leans to its target by a different amount
        w = _normal(gen, m, d).mul_(2.0 / math.sqrt(d))
        target = torch.randint(0, m, (n,), device="cuda", generator=gen)
        x = _normal(gen, n, d)
        x += torch.rand(n, 1, device="cuda", generator=gen) * 3.0 * w[target]
        if case["ignored"]:  # prompt or padding positions
            target[torch.rand(n, device="cuda", generator=gen) < 0.1] = IGNORE
        state = {"case": case, "x": x.to(t), "w": w.to(t), "target": target}
        if case["mode"] == "train":  # gradient of the mean over the counted rows
            keep = target != IGNORE
            state["dloss"] = keep.float() / keep.sum().clamp(min=1).float()
        return state
    batch, heads, kv_heads = case["batch"], case["heads"], case["kv_heads"]
    q = (2.0 * _normal(gen, batch, n, heads, d)).to(t)
    if case["fused_kv"]:  # one projection's output, keys and values side by side
        kv = _normal(gen, batch, m, 2, kv_heads, d).to(t)
        k, v = kv[:, :, 0], kv[:, :, 1]
    else:
        k, v = _normal(gen, batch, m, kv_heads, d).to(t), _normal(gen, batch, m, kv_heads, d).to(t)
    state = {"case": case, "q": q, "k": k, "v": v, "k_len": None, "bias": None}
    if case["ragged"]:
        state["k_len"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
    if case["masked"]:  # a tenth of the positions is dropped; the rest carries a small additive term
        bias = 0.5 * _normal(gen, batch, m)
        bias[torch.rand(batch, m, device="cuda", generator=gen) < 0.1] = -math.inf
        bias[:, 0] = 0.0
        state["bias"] = bias
    if case["mode"] == "train":
        state["dout"] = _normal(gen, batch, n, heads, d).to(t)
    return state


# ------------------------------------------------------------------ plain forms (32 bits)
def _plain_xent(state):
    case, target = state["case"], state["target"]
    x, w = state["x"].float(), state["w"].float()
    keep = target != IGNORE
    idx = target.clamp(min=0)[:, None]
    z = x @ w.t()
    top = z.amax(dim=1, keepdim=True)
    lse = top + (z - top).exp().sum(dim=1, keepdim=True).log()
    loss = torch.where(keep, (lse - z.gather(1, idx))[:, 0], 0.0)
    if case["mode"] == "forward":
        return loss, lse[:, 0]
    scale = torch.where(keep, state["dloss"], 0.0)[:, None]
    dz = z.sub_(lse).exp_().mul_(scale)
    dz.scatter_add_(1, idx, -scale)
    return loss, lse[:, 0], (dz @ w).to(state["x"].dtype), (dz.t() @ x).to(state["w"].dtype)


def _plain_scores(state):
    case = state["case"]
    batch, n, heads, d = state["q"].shape
    m, kv_heads = case["m"], case["kv_heads"]
    # [batch, kv head, group, ...]
    q = state["q"].float().reshape(batch, n, kv_heads, heads // kv_heads, d).permute(0, 2, 3, 1, 4)
    k = state["k"].float().permute(0, 2, 1, 3)[:, :, None]
    v = state["v"].float().permute(0, 2, 1, 3)[:, :, None]
    s = (q @ k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d))
    if state["bias"] is not None:
        s += state["bias"][:, None, None, None, :]
    if state["k_len"] is not None:
        out_of = torch.arange(m, device="cuda")[None, :] >= state["k_len"][:, None]
        s.masked_fill_(out_of[:, None, None, None, :], -math.inf)
    return q, k, v, s


def _plain_xattn(state):
    case = state["case"]
    batch, n, heads, d = state["q"].shape
    t = state["q"].dtype
    q, k, v, s = _plain_scores(state)
    top = s.amax(dim=-1, keepdim=True)
    p = s.sub_(top).exp_()
    total = p.sum(dim=-1, keepdim=True)
    p.div_(total)
    o = p @ v
    out = o.permute(0, 3, 1, 2, 4).reshape(batch, n, heads, d).to(t)
    if case["mode"] == "token":
        return out
    lse = (top + total.log()).reshape(batch, heads, n)
    if case["mode"] == "forward":
        return out, lse
    do = state["dout"].float().reshape(batch, n, case["kv_heads"], -1, d).permute(0, 2, 3, 1, 4)
    dv = (p.transpose(-1, -2) @ do).sum(dim=2)
    ds = do @ v.transpose(-1, -2)
    ds = ds.sub_((do * o).sum(dim=-1, keepdim=True)).mul_(p).mul_(1.0 / math.sqrt(d))
    dq = (ds @ k).permute(0, 3, 1, 2, 4).reshape(batch, n, heads, d)
    dk = (ds.transpose(-1, -2) @ q).sum(dim=2)
    return out, lse, dq.to(t), dk.permute(0, 2, 1, 3).to(t).contiguous(), dv.permute(0, 2, 1, 3).to(t).contiguous()


# ------------------------------------------------------------------ the library's calls
def _own_xent(state):
    import log_domain_sinkhorn_updates_b200 as fs
    x, w, target = state["x"], state["w"], state["target"]
    loss = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
    lse = torch.empty_like(loss)
    fs.fs_cross_entropy(x, w, target, loss, lse, ignore_index=IGNORE)
    if state["case"]["mode"] == "forward":
        return loss, lse
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    fs.fs_cross_entropy_grad(x, w, target, lse, state["dloss"], dx, dw, ignore_index=IGNORE)
    return loss, lse, dx, dw


def _own_xattn(state):
    import log_domain_sinkhorn_updates_b200 as fs
    q, k, v, mode = state["q"], state["k"], state["v"], state["case"]["mode"]
    batch, n, heads, _ = q.shape
    out = torch.empty_like(q)
    lse = None if mode == "token" else torch.empty(batch, heads, n, dtype=torch.float32, device=q.device)
    fs.fs_cross_attn(q, k, v, out, lse, k_len=state["k_len"], bias=state["bias"])
    if mode == "token":
        return out
    if mode == "forward":
        return out, lse
    dq = torch.empty_like(q)
    dk, dv = torch.empty(k.shape, dtype=k.dtype, device=k.device), torch.empty(v.shape, dtype=v.dtype, device=v.device)
    fs.fs_cross_attn_grad(q, k, v, out, lse, state["dout"], dq, dk, dv, k_len=state["k_len"], bias=state["bias"])
    return out, lse, dq, dk, dv


def run(state):
    if state["case"]["op"] == "xent":
        return _own_xent(state) if own else _plain_xent(state)
    return _own_xattn(state) if own else _plain_xattn(state)


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_xent(case, st):
    n, m = case["n"], case["m"]
    x, target = st["x"].double(), st["target"]
    piece = max(1, min(m, (1 << 28) // max(n, 1)))
    edges = [(a, min(a + piece, m)) for a in range(0, m, piece)]
    rows = torch.arange(n, device="cuda")
    lse = torch.full((n,), -math.inf, dtype=torch.float64, device="cuda")
    hit = torch.zeros(n, dtype=torch.float64, device="cuda")
    for a, b in edges:
        z = x @ st["w"][a:b].double().t()
        lse = torch.logaddexp(lse, torch.logsumexp(z, dim=1))
        here = (target >= a) & (target < b)
        hit[here] = z[rows[here], target[here] - a]
    counted = target != IGNORE
    loss = torch.where(counted, lse - hit, torch.zeros_like(lse))
    if case["mode"] == "forward":
        return loss, lse
    g = torch.where(counted, st["dloss"].double(), torch.zeros_like(lse))
    dx, dw = torch.zeros_like(x), []
    for a, b in edges:
        wp = st["w"][a:b].double()
        dz = torch.exp(x @ wp.t() - lse[:, None])
        here = (target >= a) & (target < b)
        dz[rows[here], target[here] - a] -= 1.0
        dz *= g[:, None]
        dx += dz @ wp
        dw.append(dz.t() @ x)
    return loss, lse, dx, torch.cat(dw)


def _exact_xattn(case, st):
    batch, n, heads, d = st["q"].shape
    m, kv_heads = case["m"], case["kv_heads"]
    group = heads // kv_heads
    out = torch.zeros(batch, n, heads, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(batch, heads, n, dtype=torch.float64, device="cuda")
    train = case["mode"] == "train"
    if train:
        dq = torch.zeros_like(out)
        dk = torch.zeros(batch, m, kv_heads, d, dtype=torch.float64, device="cuda")
        dv = torch.zeros_like(dk)
    for b, length in enumerate(_lengths(case)):
        for h in range(heads):
            c = h // group
            q, k, v = st["q"][b, :, h].double(), st["k"][b, :length, c].double(), st["v"][b, :length, c].double()
            s = torch.einsum("id,jd->ij", q, k) / math.sqrt(d)
            if st["bias"] is not None:
                s = s + st["bias"][b, :length].double()
            lse[b, h] = torch.logsumexp(s, dim=1)
            p = torch.exp(s - lse[b, h][:, None])
            out[b, :, h] = torch.einsum("ij,jd->id", p, v)
            if train:
                g = st["dout"][b, :, h].double()
                dp = torch.einsum("id,jd->ij", g, v)
                ds = p * (dp - (p * dp).sum(dim=1, keepdim=True)) / math.sqrt(d)
                dq[b, :, h] = torch.einsum("ij,jd->id", ds, k)
                dk[b, :length, c] += torch.einsum("ij,id->jd", ds, q)
                dv[b, :length, c] += torch.einsum("ij,id->jd", p, g)
    if case["mode"] == "token":
        return out
    return (out, lse, dq, dk, dv) if train else (out, lse)


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_xent(case, st) if case["op"] == "xent" else _exact_xattn(case, st)
