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
