"""Argument checks of the handle-less operators answer on the host, before any device work
(no GPU needed), and the binding mirrors the header's structs."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    from log_domain_sinkhorn_updates_b200 import build, binding
    build.build()
    return binding.lib()


def _attn(**kw):
    from log_domain_sinkhorn_updates_b200.binding import FsAttnDesc, FsView
    a = dict(batch=2, n=5, m=9, heads=4, kv_heads=2, d=64, dv=64, dtype=1, scale=0.125)
    a.update({k: v for k, v in kw.items() if not isinstance(v, tuple)})
    q, k = FsView(5 * 4 * 64, 4 * 64, 64), FsView(9 * 2 * 64, 2 * 64, 64)
    views = dict(q=q, k=k, v=k, out=q, dout=q, dq=q, dk=k, dvw=k)
    views.update({n: FsView(*v) for n, v in kw.items() if isinstance(v, tuple)})
    return FsAttnDesc(*[a[n] for n in ("batch", "n", "m", "heads", "kv_heads", "d", "dv", "dtype", "scale")],
                      *[views[n] for n in ("q", "k", "v", "out", "dout", "dq", "dk", "dvw")])


BAD_ATTN = [dict(batch=-1), dict(n=-1), dict(m=-1), dict(heads=0), dict(kv_heads=0), dict(heads=3), dict(d=0),
            dict(d=257), dict(dv=0), dict(dv=300), dict(dtype=2), dict(dtype=-1), dict(scale=0.0), dict(scale=-1.0),
            dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=3e38), dict(k=(-1, 64, 64)), dict(q=(0, -8, 64))]
# of the forward's out, and of the gradient's dq, dk and dv: elements on top of one another
BAD_VIEWS = [(0, 256, 64), (1280, 0, 64), (1280, 256, 0), (1280, 256, 63), (1279, 256, 64), (1280, 255, 64)]


def _forward(L, desc, null=None):
    p = [ctypes.c_void_p(4096)] * 3 + [None, None, ctypes.c_void_p(4096), None]
    if null is not None:
        p[null] = None
    return L.fs_cross_attn(ctypes.byref(desc) if desc else None, *p, None, 0, None)


def _grad(L, desc, null=None):
    p = [ctypes.c_void_p(4096)] * 3 + [None, None] + [ctypes.c_void_p(4096)] * 6
    if null is not None:
        p[null] = None
    return L.fs_cross_attn_grad(ctypes.byref(desc) if desc else None, *p, None, 0, None)


def test_attention_descriptors(L):
    from log_domain_sinkhorn_updates_b200.binding import FS_ERR_INVALID_ARG, FS_ERR_UNSUPPORTED
    assert _forward(L, None) == FS_ERR_INVALID_ARG and _grad(L, None) == FS_ERR_INVALID_ARG
    for kw in BAD_ATTN:
        assert _forward(L, _attn(**kw)) == FS_ERR_INVALID_ARG, kw
        assert _grad(L, _attn(**kw)) == FS_ERR_INVALID_ARG, kw
        assert L.fs_cross_attn_workspace(ctypes.byref(_attn(**kw)), 0) == 0
        assert L.fs_last_error(None)
    for view in BAD_VIEWS:
        assert _forward(L, _attn(out=view)) == FS_ERR_INVALID_ARG, view
        assert _grad(L, _attn(dq=view)) == FS_ERR_INVALID_ARG, view
    for view in [(0, 128, 64), (1152, 64, 64), (1152, 128, 63), (1151, 128, 64)]:
        assert _grad(L, _attn(dk=view)) == FS_ERR_INVALID_ARG, view
        assert _grad(L, _attn(dvw=view)) == FS_ERR_INVALID_ARG, view
    for kw in (dict(batch=20000), dict(n=1 << 25), dict(m=1 << 30)):
        big = (1 << 50, 256, 64)
        assert _forward(L, _attn(out=big, **kw)) == FS_ERR_UNSUPPORTED, kw
    for null in (0, 1, 2, 5):
        assert _forward(L, _attn(), null) == FS_ERR_INVALID_ARG
    for null in (0, 1, 2, 5, 6, 7, 8, 9, 10):
        assert _grad(L, _attn(), null) == FS_ERR_INVALID_ARG


def test_nothing_to_do_is_not_an_error(L):
    assert _forward(L, _attn(batch=0)) == 0 and _forward(L, _attn(n=0)) == 0
    assert _grad(L, _attn(batch=0)) == 0 and _grad(L, _attn(n=0, m=0)) == 0


def _xent(**kw):
    from log_domain_sinkhorn_updates_b200.binding import FsXentDesc
    a = dict(n=5, v=9, d=64, dtype=1, scale=1.0, ldx=64, ldw=64, lddx=64, lddw=64, ignore_index=-100)
    a.update(kw)
    return FsXentDesc(*[a[k] for k in ("n", "v", "d", "dtype", "scale", "ldx", "ldw", "lddx", "lddw", "ignore_index")])


def test_cross_entropy_descriptors(L):
    from log_domain_sinkhorn_updates_b200.binding import FS_ERR_INVALID_ARG, FS_ERR_UNSUPPORTED

    def forward(desc, null=None):
        p = [ctypes.c_void_p(4096)] * 5
        if null is not None:
            p[null] = None
        return L.fs_cross_entropy(ctypes.byref(desc) if desc else None, *p, None, 0, None)

    def grad(desc, null=None):
        p = [ctypes.c_void_p(4096)] * 8
        if null is not None:
            p[null] = None
        return L.fs_cross_entropy_grad(ctypes.byref(desc) if desc else None, *p, None, 0, None)

    assert forward(None) == FS_ERR_INVALID_ARG and grad(None) == FS_ERR_INVALID_ARG
    for kw in [dict(n=-1), dict(v=0), dict(d=0), dict(dtype=5), dict(scale=0.0), dict(scale=-2.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=3e38), dict(ldx=-1), dict(ldw=-64)]:
        assert forward(_xent(**kw)) == FS_ERR_INVALID_ARG, kw
        assert grad(_xent(**kw)) == FS_ERR_INVALID_ARG, kw
        assert L.fs_cross_entropy_workspace(ctypes.byref(_xent(**kw)), None, None, 1) == 0
    for kw in [dict(lddx=63), dict(lddw=0)]:
        assert grad(_xent(**kw)) == FS_ERR_INVALID_ARG, kw
    for kw in [dict(v=(1 << 22) + 1), dict(d=65537), dict(n=(1 << 24) + 1)]:
        assert forward(_xent(lddx=1 << 17, lddw=1 << 17, **kw)) == FS_ERR_UNSUPPORTED, kw
    for null in range(5):
        assert forward(_xent(), null) == FS_ERR_INVALID_ARG
    for null in (0, 1, 2, 3, 4, 6, 7):
        assert grad(_xent(), null) == FS_ERR_INVALID_ARG
    assert forward(_xent(n=0)) == 0


def test_binding_refuses_on_the_host():
    import torch
    import log_domain_sinkhorn_updates_b200 as fs
    q = torch.zeros(1, 2, 2, 8)
    with pytest.raises(ValueError):  # host tensors
        fs.fs_cross_attn(q, q, q, q)
    with pytest.raises(ValueError):
        fs.fs_cross_entropy(q[0, 0], q[0, 0], torch.zeros(2, dtype=torch.long), torch.zeros(2), torch.zeros(2))


@pytest.mark.parametrize("cname,pyname", [("fs_view", "FsView"), ("fs_attn_desc", "FsAttnDesc"),
                                          ("fs_xent_desc", "FsXentDesc")])
def test_ctypes_structs_match_header(cname, pyname):
    from log_domain_sinkhorn_updates_b200 import binding
    txt = open(os.path.join(ROOT, "include", "flashsinkhorn.h")).read()
    txt = re.sub(r"/\*.*?\*/", "", txt, flags=re.S)
    body = re.search(r"typedef struct \{([^{}]*)\}\s*" + cname + r"\s*;", txt).group(1)
    fields = [v.strip().split()[-1] for decl in body.split(";") if decl.strip()
              for v in decl.strip().split(",")]
    assert [f for f, _ in getattr(binding, pyname)._fields_] == fields
