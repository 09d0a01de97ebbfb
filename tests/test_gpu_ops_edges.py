"""Cross attention and cross entropy where inputs are not finite, biases huge, or sizes past what the calls take."""
import math

import pytest
import torch

import ops_reference as ref
import test_gpu_cross_attn as attn
import test_gpu_cross_entropy as xent

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def _fs():
    import log_domain_sinkhorn_updates_b200 as fs
    return fs


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [1, 9, 300])
@pytest.mark.parametrize("first,count", [(0, 128), (128, 128), (256, 128), (0, 256), (512, 256), (896, 104), (0, 1000),
                                         (200, 128), (999, 1)])
def test_nan_class_rows_reach_loss_and_lse(dtype, n, first, count):
    """A corrupt shard of the vocabulary: whole blocks of NaN logits, aligned with a tile or not."""
    x, w, target, dloss = xent.make(n, 1000, 64, dtype, seed=first + n, ignored=False)
    target[:] = (first + count) % 1000 if count < 1000 else 0
    w[first:first + count] = math.nan
    got = xent.run(x, w, target, dloss)
    for name in got:
        assert torch.isnan(got[name]).all(), name


@pytest.mark.parametrize("first", [0, 256, 300])
def test_infinite_logits(first):
    """bf16: a class of -inf logits weighs nothing, one of +inf makes the row NaN, a row of -inf alone has lse -inf."""
    x, w, target, _ = xent.make(40, 700, 64, BF16, seed=first, ignored=False)
    x, target[:] = x.abs() + 0.5, 699
    w[first:first + 256] = -math.inf
    loss, lse = torch.empty(40, device="cuda"), torch.empty(40, device="cuda")
    _fs().fs_cross_entropy(x, w, target, loss, lse)
    kept = torch.cat([w[:first], w[first + 256:]])
    ref.check({"loss": loss, "lse": lse}, ref.cross_entropy(x, kept, target - 256))
    w[first] = math.inf
    _fs().fs_cross_entropy(x, w, target, loss, lse)
    assert torch.isnan(loss).all() and torch.isnan(lse).all()
    w[:] = -math.inf
    _fs().fs_cross_entropy(x, w, target, loss, lse)
    assert torch.isnan(loss).all() and torch.isneginf(lse).all()


def _shifted(q, k, v, dout, bias, k_len=None):
    """The 64-bit form with every problem's largest kept bias taken off: softmax and gradients are the same, and the
    bounds are those of biases of the remaining size.  Returns the form and those largest biases."""
    live = ~(bias <= ref.MASK)
    if k_len is not None:
        live &= torch.arange(bias.shape[1], device="cuda")[None] < k_len.clamp(0, bias.shape[1])[:, None]
    top = torch.where(live, bias.double(), -math.inf).amax(dim=1)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    rest = torch.where(live, bias.double() - top[:, None], -math.inf)
    return ref.attention(q, k, v, dout=dout, bias=rest, k_len=k_len), top


def _check_shifted(got, want, top):
    ref.check(got, want, [name for name in got if name != "lse"])
    lse, bound = want["lse"]
    full = lse + top[:, None, None]
    some = ~torch.isinf(full)
    assert torch.equal(torch.isneginf(got["lse"]), ~some)
    off = (got["lse"].double() - full).abs()
    assert (off[some] <= (bound + ref.U * full.abs())[some]).all()


BIG = [-1e9, -1e8, -65504.0, -1e4, -65.0, 1e6, 1e9, -9e29]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,d", [(1, 64), (9, 128), (150, 64), (40, 200)])
@pytest.mark.parametrize("size", BIG)
def test_biases_of_any_size_on_every_key(dtype, n, d, size):
    """A sample masked with a finite constant: its scores still decide, forward and gradient.  Beside it one with
    ordinary biases, one with the constant on all keys but a few, and one that is masked altogether."""
    m = 700
    q, k, v, dout = attn.make(5, n, m, 4, 2, d, d, dtype, seed=n)
    g = torch.Generator(device="cuda").manual_seed(7)
    step = max(0.25, 2.0 ** (math.floor(math.log2(abs(size))) - 23))
    bias = torch.full((5, m), size, device="cuda")
    bias[0, torch.rand(m, device="cuda", generator=g) < 0.3] += step
    bias[1] = 0.5 * torch.randn(m, device="cuda", generator=g)
    bias[2, 100:130] = 0.0
    bias[3] = -math.inf
    bias[4, ::3] = -math.inf
    k_len = torch.tensor([m, 333, m, m, 70], dtype=torch.int32, device="cuda")
    for lens in (None, k_len):
        got = attn.run(q, k, v, dout, bias=bias, k_len=lens)
        _check_shifted(got, *_shifted(q, k, v, dout, bias, lens))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size", [(2, 1, 9000, 4, 2, 64, 64), (2, 5, 6000, 8, 1, 128, 128), (2, 3, 4000, 1, 1, 40, 200)])
def test_parts_with_biases_of_different_sizes(dtype, size):
    """Keys split over CTAs whose largest biases are far apart, or nearly the same at 1e9."""
    q, k, v, dout = attn.make(*size, dtype, seed=5)
    m = size[2]
    for first, rest in [(-1e9, 0.0), (0.0, -1e9), (-1e9, -1e9 + 64), (1e9, 1e9), (-1e5, -1e5 - 3.0)]:
        bias = torch.full((2, m), rest, device="cuda")
        bias[:, :m // 2] = first
        bias[1, m - 3:] = max(first, rest)
        got = attn.run(q, k, v, dout, bias=bias)
        _check_shifted(got, *_shifted(q, k, v, dout, bias))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size", [(2, 50, 300, 4, 2, 64, 64), (2, 900, 300, 4, 2, 128, 96), (1, 3, 4000, 2, 1, 64, 64),
                                  (1, 70, 200, 2, 2, 200, 72)])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_masked_keys_get_zeros_beside_rows_that_are_not_finite(dtype, size, value):
    """A NaN or infinity in one query, or in its gradient, reaches every key that takes part and no other."""
    q, k, v, dout = attn.make(*size, dtype, seed=29)
    B, n, m = size[:3]
    bias = torch.zeros(B, m, device="cuda")
    bias[:, 20:25] = -math.inf
    bias[:, 30] = torch.finfo(F32).min
    k_len = torch.full((B,), m - 130, dtype=torch.int32, device="cuda")
    dead = (bias <= -1e30) | (torch.arange(m, device="cuda")[None] >= k_len[:, None])
    clean = attn.run(q, k, v, dout, bias=bias, k_len=k_len)
    for t in (q, dout):
        kept = t[:, n // 2].clone()
        t[:, n // 2] = value
        got = attn.run(q, k, v, dout, bias=bias, k_len=k_len)
        t[:, n // 2] = kept
        assert (got["dk"][dead] == 0).all() and (got["dv"][dead] == 0).all()
        assert not torch.isfinite(got["dk"][~dead]).all()
        others = torch.arange(n, device="cuda") != n // 2
        assert torch.equal(got["dq"][:, others], clean["dq"][:, others])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,m", [(1, 400), (6, 3000), (200, 400)])
def test_anything_in_the_queries_of_a_problem_whose_keys_are_all_masked(dtype, n, m):
    """Padding of a batch by masks: NaN in q, k, v and the gradient; the other problems keep their bits."""
    q, k, v, dout = attn.make(4, n, m, 4, 2, 64, 64, dtype, seed=17)
    bias = torch.zeros(4, m, device="cuda")
    bias[1] = -math.inf
    bias[2] = torch.finfo(F32).min
    bias[3, 5:] = -1e30
    for k_len in (None, torch.tensor([m, m, m, 77], dtype=torch.int32, device="cuda")):
        kw = {"bias": bias, "k_len": k_len}
        clean = attn.run(q, k, v, dout, **kw)
        bad = [t.clone() for t in (q, k, v, dout)]
        for t in bad:
            t[1:3] = math.nan
        got = attn.run(*bad, **kw)
        for name in got:
            assert torch.equal(got[name], clean[name]), name
        assert all((got[name][1:3] == 0).all() for name in ("out", "dq", "dk", "dv"))
        assert torch.isneginf(got["lse"][1:3]).all()


def test_a_wait_that_runs_out_is_reported_once_and_the_calls_stay_usable():
    fs = _fs()
    fs.fs_check()
    fs.fs_selftest_check(20)
    with pytest.raises(fs.FsError, match="FS_ERR_TIMEOUT"):
        fs.fs_check()
    fs.fs_check()
    with pytest.raises(fs.FsError, match="FS_ERR_INVALID_ARG"):
        fs.fs_selftest_check(0)
    q, k, v, dout = attn.make(1, 9, 50, 2, 1, 64, 64, BF16)
    ref.check(attn.run(q, k, v, dout), ref.attention(q, k, v, dout=dout))


def test_checks_on_one_stream_miss_nothing_that_another_raises():
    """A thread checks one stream without a pause, another raises errors on a second stream: each is reported once."""
    import threading
    import time
    fs = _fs()
    fs.fs_check()
    mine, other = torch.cuda.Stream(), torch.cuda.Stream()
    rounds, seen, stop, failures = 400, [0], threading.Event(), []

    def checks():
        while not stop.is_set():
            try:
                fs.fs_check(mine)
            except fs.FsError as e:
                if "FS_ERR_TIMEOUT" not in str(e):
                    failures.append(e)
                    return
                seen[0] += 1

    t = threading.Thread(target=checks)
    t.start()
    try:
        for i in range(rounds):
            fs.fs_selftest_check(1, other)
            other.synchronize()
            until = time.monotonic() + 1.0
            while seen[0] <= i and time.monotonic() < until and not failures:
                time.sleep(0)
            if seen[0] != i + 1:
                break
    finally:
        stop.set()
        t.join()
    assert not failures and seen[0] == rounds, (failures, seen[0])


def test_arguments_that_only_the_call_holds():
    """Lengths, masks, targets and statistics made in the call's own argument list live until its work is enqueued: the
    workspace that the call takes from the allocator is not theirs."""
    fs = _fs()
    # cross entropy: a temporary of the size class of the workspace
    for n, v in [(1, 1), (3, 200), (70, 5000), (900, 300)]:
        x, w, target, dloss = xent.make(n, v, 64, BF16, seed=n)
        want = xent.run(x, w, target, dloss)
        need = fs.fs_cross_entropy_workspace(x, w)
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        pad = torch.empty(max(0, need // 8 - n), dtype=torch.long, device="cuda")  # so that blocks of that size exist
        del pad
        fs.fs_cross_entropy(x, w, target.clone(), loss, lse)
        assert torch.equal(loss, want["loss"]) and torch.equal(lse, want["lse"])
        fs.fs_cross_entropy(x, w, torch.cat([target, target.new_zeros(max(0, need // 8 - n))])[:n], loss, lse)
        assert torch.equal(loss, want["loss"]) and torch.equal(lse, want["lse"])
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        fs.fs_cross_entropy_grad(x, w, target.clone(), lse.clone(), dloss.clone(), dx, dw)
        assert torch.equal(dx, want["dx"]) and torch.equal(dw, want["dw"])
    # attention: few rows, so the keys are split and the call has a workspace
    for dtype, m in [(BF16, 3000), (F32, 3000), (F32, 200)]:
        q, k, v, dout = attn.make(2, 1, m, 4, 2, 64, 64, dtype, seed=m)
        k_len = torch.tensor([m, m // 2], dtype=torch.int32, device="cuda")
        bias = torch.randn(2, m, device="cuda")
        want = attn.run(q, k, v, dout, k_len=k_len, bias=bias)
        need = fs.fs_cross_attn_workspace(q, k, v, q)
        out, lse = torch.empty_like(q), torch.empty(2, 4, 1, device="cuda")
        for size in (0, need // 4):
            big = torch.zeros(size + 2 * m, device="cuda")
            big[:2 * m] = bias.flatten()
            lens = torch.zeros(size + 2, dtype=torch.int32, device="cuda")
            lens[:2] = k_len
            torch.cuda.synchronize()
            fs.fs_cross_attn(q, k, v, out, lse, k_len=lens.clone()[:2], bias=big.clone()[:2 * m].view(2, m))
            assert torch.equal(out, want["out"]) and torch.equal(lse, want["lse"])
            grads = [torch.empty_like(t) for t in (q, k, v)]
            fs.fs_cross_attn_grad(q, k, v, out, lse.clone(), dout, *grads, k_len=lens.clone()[:2],
                                  bias=big.clone()[:2 * m].view(2, m))
            assert all(torch.equal(g, want[name]) for g, name in zip(grads, ("dq", "dk", "dv")))


def test_sizes_past_the_descriptors_are_refused():
    """Tensors expanded to more tokens, rows or classes than a C int holds, and an ignore_index past 64 bits."""
    fs = _fs()
    big = 2 ** 32 + 1
    q, one = torch.randn(1, 1, 1, 8, device="cuda"), torch.randn(1, 1, 1, 8, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((1, 1, 1), 7.0, device="cuda")
    many = one.expand(1, big, 1, 8)
    with pytest.raises(ValueError):
        fs.fs_cross_attn(q, many, many, out, lse)
    with pytest.raises(ValueError):
        fs.fs_cross_attn(many, one, one, many)
    with pytest.raises(ValueError):
        fs.fs_cross_attn_grad(q, many, many, out, lse, q, out, many, many)
    with pytest.raises(ValueError):
        fs.fs_cross_attn_workspace(q, many, many, out)
    x, loss, target = one.view(1, 8), torch.full((1,), 7.0, device="cuda"), torch.zeros(1, dtype=torch.long, device="cuda")
    with pytest.raises(ValueError):
        fs.fs_cross_entropy(x, x.expand(big, 8), target, loss, loss.clone())
    with pytest.raises(ValueError):
        fs.fs_cross_entropy(x.expand(big, 8), x, target, loss, loss.clone())
    for ignore in (2 ** 64 - 100, 2 ** 63, -2 ** 63 - 1):
        with pytest.raises(ValueError):
            fs.fs_cross_entropy(x, x, target, loss, loss.clone(), ignore_index=ignore)
        with pytest.raises(ValueError):
            fs.fs_cross_entropy_grad(x, x, target, loss, loss, x.clone(), x.clone(), ignore_index=ignore)
    assert (out == 7).all() and (lse == 7).all() and (loss == 7).all()
    # the ends of the range are taken
    for ignore in (2 ** 63 - 1, -2 ** 63):
        fs.fs_cross_entropy(x, x, torch.full_like(target, ignore), loss, loss.clone(), ignore_index=ignore)
        assert (loss == 0).all()
    m = 2 ** 30 - 1  # the most keys that the header allows, one row of memory behind them
    with pytest.raises(fs.FsError, match="FS_ERR_UNSUPPORTED"):
        fs.fs_cross_attn(q, one.expand(1, m + 1, 1, 8), one.expand(1, m + 1, 1, 8), out, lse)
    fs.fs_cross_attn(q, one.expand(1, m, 1, 8), one.expand(1, m, 1, 8), out, lse)
    want = math.log(m) + (q.double() * one.double()).sum().item() * 8 ** -0.5
    # equal scores: every weight is 1, their sums are exact; a group of lanes adds at most 2^30 / (64 parts x 32) = 2^19
    # equal values, each addition off by half a unit of the sum
    assert (out - one).abs().max() <= 2.0 ** 19 * 2.0 ** -24 * one.abs().max()
    assert abs(lse.item() - want) <= 16 * ref.U * 30
    fs.fs_check()


def test_width_zero_is_refused_like_other_sizes():
    fs = _fs()
    for d, dv in [(0, 8), (8, 0), (0, 0)]:
        q, v = torch.zeros(1, 2, 1, d, device="cuda"), torch.zeros(1, 2, 1, dv, device="cuda")
        with pytest.raises(fs.FsError, match="FS_ERR_INVALID_ARG"):
            fs.fs_cross_attn(q, q, v, v)
        with pytest.raises(fs.FsError, match="FS_ERR_INVALID_ARG"):
            fs.fs_cross_attn_grad(q, q, v, v, torch.zeros(1, 1, 2, device="cuda"), v, q, q, v)
        assert fs.fs_cross_attn_workspace(q, q, v, v) == 0
    x = torch.zeros(3, 0, device="cuda")
    with pytest.raises(fs.FsError, match="FS_ERR_INVALID_ARG"):
        fs.fs_cross_entropy(x, x, torch.zeros(3, dtype=torch.long, device="cuda"), *torch.zeros(2, 3, device="cuda"))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [1, 9, 150])
def test_scores_that_are_not_finite_and_take_part(dtype, n):
    """A key of infinite or NaN width makes the rows whose score with it is +inf or NaN NaN; where it is -inf, it weighs
    nothing, and rows of such scores alone have no key."""
    m = 300
    q, k, v, _ = attn.make(1, n, m, 2, 1, 64, 64, dtype, seed=n)
    q = q.abs() + 0.25
    want = ref.attention(q, torch.cat([k[:, :140], k[:, 141:]], 1), torch.cat([v[:, :140], v[:, 141:]], 1))
    k[0, 140, 0, 5] = -math.inf
    out, lse = attn.forward(q, k, v)
    ref.check({"out": out, "lse": lse}, want)
    for value in (math.inf, math.nan):
        k[0, 140, 0, 5] = value
        out, lse = attn.forward(q, k, v)
        assert torch.isnan(out).all() and torch.isnan(lse).all()
    k[..., 5] = -math.inf
    out, lse = attn.forward(q, k, v)
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [1, 90])
def test_a_captured_masked_step_replayed_on_other_masks(dtype, n):
    """What the biases are measured from is found by the kernels, so a graph captured on ordinary masks holds for a sample
    masked with -1e9, for one without a key, and back."""
    fs = _fs()
    m = 700
    q, k, v, dout = attn.make(2, n, m, 4, 2, 64, 64, dtype, seed=n)
    k_len = torch.tensor([m, 333], dtype=torch.int32, device="cuda")
    ordinary = torch.randn(2, m, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    bias, lens = ordinary.clone(), k_len.clone()
    names = ("out", "lse", "dq", "dk", "dv")
    bufs = dict(zip(names, (torch.zeros_like(q), torch.zeros(2, 4, n, device="cuda"), *(torch.zeros_like(t) for t in (q, k, v)))))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fs.fs_cross_attn(q, k, v, bufs["out"], bufs["lse"], k_len=lens, bias=bias)
        fs.fs_cross_attn_grad(q, k, v, bufs["out"], bufs["lse"], dout, bufs["dq"], bufs["dk"], bufs["dv"], k_len=lens,
                              bias=bias)
    for value in (None, -1e9, -math.inf, 1e6, None):
        bias.copy_(ordinary)
        if value is not None:
            bias[1] = value
        lens.copy_(k_len if value != 1e6 else k_len.flip(0))
        graph.replay()
        want = attn.run(q, k, v, dout, bias=bias.clone(), k_len=lens.clone())
        for name in names:
            assert torch.equal(bufs[name], want[name]), (value, name)


def test_calls_from_several_threads():
    """Threads with streams of their own, first calls of new geometries among them: the same bits as one after the other."""
    import threading
    fs = _fs()
    jobs = []
    for i, (n, m, d, dtype) in enumerate([(1, 2100, 64, BF16), (70, 300, 136, F32), (33, 500, 200, BF16), (5, 90, 24, F32)]):
        q, k, v, dout = attn.make(2, n, m, 4, 2, d, d, dtype, seed=i)
        x, w, target, dloss = xent.make(50 + i, 300 + i, 64, dtype, seed=i)
        bias = torch.randn(2, m, device="cuda")
        bias[1] = -1e9
        jobs.append((q, k, v, dout, bias, x, w, target, dloss))

    def work(q, k, v, dout, bias, x, w, target, dloss):
        out, lse = torch.empty_like(q), torch.empty(2, 4, q.shape[1], device="cuda")
        grads = [torch.empty_like(t) for t in (q, k, v, x, w)]
        fs.fs_cross_attn(q, k, v, out, lse, bias=bias)
        fs.fs_cross_attn_grad(q, k, v, out, lse, dout, *grads[:3], bias=bias)
        loss, z = torch.empty(x.shape[0], device="cuda"), torch.empty(x.shape[0], device="cuda")
        fs.fs_cross_entropy(x, w, target, loss, z)
        fs.fs_cross_entropy_grad(x, w, target, z, dloss, *grads[3:])
        return [out, lse, loss, z, *grads]

    got, errors = [[] for _ in jobs], []
    torch.cuda.synchronize()

    def thread(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    got[i].append(work(*jobs[i]))
            stream.synchronize()
        except Exception as e:  # noqa: BLE001 - reported by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=thread, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for job, runs in zip(jobs, got):
        want = work(*job)
        for run in runs:
            assert all(torch.equal(a, b) for a, b in zip(run, want))
    fs.fs_check()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,v,ignored", [(1000, 8192, 0), (300, 9000, 200), (2, 8192, 1), (5000, 8200, 1500)])
def test_a_factor_common_to_all_rows_is_not_rounded_with_the_logit_gradients(dtype, n, v, ignored):
    """The gradient of a mean: 1 / n, and the scale, here with significands that bf16 rounds by 0.45 of 2^-7, stay out of
    dz.  What is left of an error along the gradient: a target's dz is 1 - p short of 1, rounded to it (p < 2^-12 here), the
    other classes' sum is a hundredth of a gradient's size and rounds by 2^-8 at most, and where the outputs' roundings are
    even in sign, 2^-8 / sqrt(elements) x 4.  They are not altogether: a target's row of dw is x_i times one number, and of
    x_i's 8 bits times 1.0035 more round down than up.  The exact result's own rounding has that share too, and it is
    allowed for, with the 2^-12 / 2^-8 of the values that an error of 2^-12 before it makes round the other way, 2^-8 each.
    With the factors inside it is 0.45 x 2^-7 (14 x 2^-12)."""
    g = torch.Generator(device="cuda").manual_seed(n)
    d = 64
    x = torch.randn(n, d, device="cuda", generator=g).to(dtype)
    w = torch.randn(v, d, device="cuda", generator=g).to(dtype)
    target = torch.randint(0, v, (n,), device="cuda", generator=g)
    dloss = torch.full((n,), (1 + 0.45 * 2.0 ** -7) * 2.0 ** -10, device="cuda")
    target[:ignored], dloss[:ignored] = -100, math.nan  # rows before the first counted one; their dloss is not used
    for scale in (2.0 ** -7, (1 + 0.45 * 2.0 ** -7) * 2.0 ** -7):
        got = xent.run(x, w, target, dloss, scale=scale)
        z = scale * (x.double() @ w.double().t())
        dz = torch.softmax(z, 1)
        assert dz.max() < 2.0 ** -12
        dz[torch.arange(n), target.clamp(min=0)] -= 1
        dz = scale * dz * torch.where(target == -100, 0.0, dloss.double())[:, None]
        for name, want in (("dx", dz @ w.double()), ("dw", dz.t() @ x.double())):
            def along(t):
                return (((t.double() - want) * want).sum() / (want * want).sum()).abs().item()

            count = (n - ignored) * d  # the rows of dw that targets give, and those of dx
            most = 2 * 2.0 ** -12 + 2.0 ** -8 / 50 + 4 * 2.0 ** -8 / count ** 0.5 + along(want.to(dtype))
            assert along(got[name]) <= most, (name, along(got[name]) * 2 ** 12, most * 2 ** 12)
