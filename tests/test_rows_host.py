"""What the calls over rows of tokens refuse, on the host alone (no GPU: every
case comes back before any HIP call), and their workspace sizes."""
import ctypes
import math

import pytest

ddp = pytest.importorskip("gradient_allreduce_averaging_amd")

OK, INVALID, UNSUPPORTED, OVERFLOW, ALIAS, CAPACITY = 0, 1, 2, 3, 4, 7
F32, BF16, I8, E4M3 = 0, 1, 2, 3
MB = 1 << 20


def _rows(*n):
    return (ctypes.c_int64 * len(n))(*n)


class _RowsC(ctypes.Structure):
    """ddp_rows_t."""
    _fields_ = [("rank", ctypes.c_void_p), ("stride", ctypes.c_int64)]


class Matrix:
    """A ddp_rows_t over made-up addresses."""

    def __init__(self, stride, *addr):
        self.arr = (ctypes.c_void_p * len(addr))(*addr)
        self.rows = _RowsC(ctypes.addressof(self.arr), stride)
        self.c = ctypes.addressof(self.rows)


def _vec(*addr):
    return (ctypes.c_void_p * len(addr))(*addr)


def norm(rows=(4, 4), width=256, x=(256, 1 * MB, 2 * MB), res=(256, 3 * MB, 4 * MB), dt=BF16,
         w=9 * MB, wdt=BF16, eps=1e-6, total=(256, 5 * MB, 6 * MB), y=(256, 7 * MB, 8 * MB), ydt=BF16,
         scale=None, n=None):
    m = [None if v is None else Matrix(*v) for v in (x, res, total, y)]
    c = [None if v is None else v.c for v in m]
    return ddp.lib.ddp_rms_norm(None if rows is None else _rows(*rows), len(rows or ()) if n is None else n,
                                width, c[0], c[1], dt, w, wdt, eps, c[2], c[3], ydt,
                                None if scale is None else _vec(*scale), None)


def test_norm_refuses():
    assert norm(rows=None, n=2) == INVALID
    assert norm(n=0) == INVALID
    assert norm(rows=(1,) * 65, n=65) == UNSUPPORTED
    assert norm(rows=(4, -1)) == INVALID
    assert norm(width=0) == INVALID
    assert norm(width=1 << 60) == OVERFLOW
    assert norm(rows=(1 << 52, 1), width=1 << 10) == OVERFLOW
    assert norm(dt=I8) == INVALID and norm(dt=9) == INVALID
    assert norm(wdt=I8) == INVALID
    assert norm(ydt=4) == INVALID
    assert norm(ydt=F32) == UNSUPPORTED                       # bf16 -> f32
    for eps in (-1e-6, math.nan, math.inf):
        assert norm(eps=eps) == INVALID
    assert norm(x=None) == INVALID
    assert norm(y=None) == INVALID
    assert norm(x=(256, 1 * MB, 0)) == INVALID                # a null address with rows
    assert norm(x=(256, 1 * MB + 1, 2 * MB)) == INVALID       # off the elements' alignment
    assert norm(x=(255, 1 * MB, 2 * MB)) == INVALID           # rows that overlap one another
    assert norm(x=(0, 1 * MB, 2 * MB)) == INVALID             # one row for all
    assert norm(ydt=I8) == INVALID                            # 8 bits without scales
    assert norm(scale=(10 * MB, 11 * MB)) == INVALID          # scales without 8 bits
    assert norm(ydt=I8, scale=(10 * MB, 10 * MB + 2)) == INVALID
    assert norm(x=(1 << 59, 1 * MB, 2 * MB)) == OVERFLOW


def test_norm_refuses_overlaps():
    assert norm(y=(256, 7 * MB, 7 * MB)) == ALIAS             # both ranks' outputs
    assert norm(y=(256, 5 * MB, 8 * MB)) == ALIAS             # y and the sum
    assert norm(y=(256, 2 * MB, 8 * MB)) == ALIAS             # another rank's input
    assert norm(y=(256, 1 * MB + 512, 8 * MB)) == ALIAS       # shifted by a row
    assert norm(y=(512, 1 * MB, 8 * MB)) == ALIAS             # another stride
    assert norm(y=(256, 9 * MB - 2, 8 * MB)) == ALIAS         # the weight
    assert norm(ydt=I8, y=(256, 1 * MB, 8 * MB), scale=(10 * MB, 11 * MB)) == ALIAS   # other size
    assert norm(ydt=E4M3, scale=(10 * MB, 10 * MB + 4)) == ALIAS
    assert norm(total=(256, 9 * MB, 6 * MB)) == ALIAS
    # rows of one buffer that interleave share no byte; by one element more they do
    assert norm(x=(512, 1 * MB, 2 * MB), y=(512, 1 * MB + 510, 8 * MB)) == ALIAS
    assert norm(x=(512, 1 * MB, 2 * MB), y=(512, 1 * MB + 514, 8 * MB)) == ALIAS


def test_norm_without_rows_does_nothing():
    assert norm(rows=(0, 0)) == OK
    assert norm(rows=(0,), x=None, y=None, res=None, total=None, w=None) == OK


def grad(rows=(4, 4), width=256, s=(256, 1 * MB, 2 * MB), dt=BF16, w=9 * MB, wdt=F32, eps=1e-6,
         dy=(256, 3 * MB, 4 * MB), ydt=BF16, dsum=(256, 5 * MB, 6 * MB), dx=(256, 7 * MB, 8 * MB),
         dw=(10 * MB, 11 * MB), dwdt=F32, ws=12 * MB, size=64 * MB, n=None):
    m = [None if v is None else Matrix(*v) for v in (s, dy, dsum, dx)]
    c = [None if v is None else v.c for v in m]
    return ddp.lib.ddp_rms_norm_grad(None if rows is None else _rows(*rows),
                                     len(rows or ()) if n is None else n, width, c[0], dt, w, wdt, eps,
                                     c[1], ydt, c[2], c[3], None if dw is None else _vec(*dw), dwdt, 0, ws,
                                     size, None)


def test_norm_grad_refuses():
    assert grad(rows=None, n=1) == INVALID
    assert grad(n=0) == INVALID
    assert grad(rows=(1,) * 65) == UNSUPPORTED
    assert grad(width=0) == INVALID
    assert grad(dt=E4M3) == INVALID and grad(ydt=I8) == INVALID and grad(dwdt=I8) == INVALID
    assert grad(ydt=F32) == UNSUPPORTED                       # f32 dy of a bf16 sum
    assert grad(eps=-1.0) == INVALID
    for k in ("s", "dy", "dx"):
        assert grad(**{k: None}) == INVALID
        assert grad(**{k: (256, 0, 20 * MB)}) == INVALID
        assert grad(**{k: (128, 20 * MB, 21 * MB)}) == INVALID
    assert grad(dw=(10 * MB, 0)) == INVALID
    assert grad(dw=(10 * MB, 11 * MB + 2)) == INVALID
    assert grad(ws=None) == INVALID
    assert grad(ws=12 * MB + 8) == INVALID
    need = ddp.rms_norm_grad_workspace((4, 4), 256)
    assert grad(size=need - 1) == CAPACITY
    assert grad(size=0) == CAPACITY


def test_norm_grad_refuses_overlaps():
    assert grad(dx=(256, 2 * MB, 8 * MB)) == ALIAS            # rank 1's sum
    assert grad(dx=(256, 1 * MB + 2, 8 * MB)) == ALIAS
    assert grad(dw=(10 * MB, 10 * MB)) == ALIAS
    assert grad(dw=(10 * MB, 1 * MB)) == ALIAS
    assert grad(dw=(9 * MB, 11 * MB)) == ALIAS                # the weight
    assert grad(ws=1 * MB - 16) == ALIAS
    assert grad(dw=(12 * MB + 16, 11 * MB)) == ALIAS          # the workspace


def test_norm_grad_without_rows_or_weight_does_nothing():
    assert grad(rows=(0, 0), dw=None, ws=None, size=0) == OK


def distill(rows=(4, 4), vocab=1000, z=(1000, 1 * MB, 2 * MB), dt=BF16, top=8,
            t=(8, 3 * MB, 4 * MB), tdt=F32, i=(8, 5 * MB, 6 * MB), ib=8, tw=None, tau=1.0,
            dz=(1000, 7 * MB, 8 * MB), loss=9 * MB, rl=(10 * MB, 11 * MB), ws=12 * MB, size=64 * MB,
            n=None, grad_call=True):
    m = [None if v is None else Matrix(*v) for v in (z, t, i, dz)]
    c = [None if v is None else v.c for v in m]
    head = [None if rows is None else _rows(*rows), len(rows or ()) if n is None else n, vocab, c[0], dt, top,
            c[1], tdt, c[2], ib, None if tw is None else _vec(*tw), tau]
    tail = [loss, None if rl is None else _vec(*rl), ws, size, None]
    if grad_call:
        return ddp.lib.ddp_distill_grad(*head, 1.0, c[3], *tail)
    return ddp.lib.ddp_distill_loss(*head, *tail)


@pytest.mark.parametrize("g", [True, False])
def test_distill_refuses(g):
    def f(**k):
        return distill(grad_call=g, **k)
    assert f(rows=None, n=1) == INVALID
    assert f(n=0) == INVALID
    assert f(rows=(1,) * 65) == UNSUPPORTED
    assert f(rows=(-1, 4)) == INVALID
    assert f(vocab=0) == INVALID
    assert f(dt=I8) == INVALID and f(tdt=E4M3) == INVALID
    assert f(top=0) == INVALID
    assert f(top=1025, t=(1025, 3 * MB, 4 * MB), i=(1025, 5 * MB, 6 * MB)) == UNSUPPORTED
    assert f(ib=2) == INVALID
    for tau in (0.0, -1.0, math.nan, math.inf):
        assert f(tau=tau) == INVALID
    for tau in (9e-7, 2e6):
        assert f(tau=tau) == UNSUPPORTED
    assert f(vocab=1 << 31, z=(1 << 31, 1 << 40, 1 << 50), dz=(1 << 31, 1 << 41, 1 << 51)) == UNSUPPORTED
    assert f(loss=None) == INVALID
    assert f(loss=9 * MB + 2) == INVALID
    for k in ("z", "t", "i"):
        assert f(**{k: None}) == INVALID
        assert f(**{k: (4096, 0, 20 * MB)}) == INVALID
    assert f(i=(8, 5 * MB + 4, 6 * MB)) == INVALID
    assert f(i=(7, 5 * MB, 6 * MB)) == INVALID
    assert f(tw=(0, 13 * MB)) == INVALID
    assert f(rl=(0, 13 * MB)) == INVALID
    assert f(ws=None) == INVALID and f(ws=12 * MB + 4) == INVALID
    need = ddp.distill_workspace((4, 4), 1000, 8)
    assert f(size=need - 1) == CAPACITY
    # overlaps
    assert f(loss=10 * MB) == ALIAS
    assert f(rl=(10 * MB, 10 * MB + 8)) == ALIAS
    assert f(rl=(3 * MB, 11 * MB)) == ALIAS
    assert f(ws=1 * MB) == ALIAS
    assert f(tw=(10 * MB, 13 * MB)) == ALIAS


def test_distill_grad_refuses_its_output():
    assert distill(dz=None) == INVALID
    assert distill(dz=(1000, 0, 8 * MB)) == INVALID
    assert distill(dz=(1000, 2 * MB, 8 * MB)) == ALIAS        # another rank's logits
    assert distill(dz=(1000, 1 * MB + 2, 8 * MB)) == ALIAS
    assert distill(dz=(1000, 3 * MB, 8 * MB)) == ALIAS        # the teacher
    # an index as wide and large as the gradient is no place for it
    assert distill(dt=F32, vocab=8, z=(8, 1 * MB, 2 * MB), i=(8, 5 * MB, 6 * MB), ib=4,
                   dz=(8, 5 * MB, 8 * MB)) == ALIAS


def test_workspace_sizes():
    L = ddp.lib
    assert L.ddp_rms_norm_grad_workspace(None, 1, 8) == -1
    assert L.ddp_rms_norm_grad_workspace(_rows(1), 0, 8) == -1
    assert L.ddp_rms_norm_grad_workspace(_rows(1), 1, 0) == -1
    assert L.ddp_rms_norm_grad_workspace(_rows(0), 1, 8) > 0
    assert L.ddp_distill_workspace(None, 1, 8, 1) == -1
    assert L.ddp_distill_workspace(_rows(0), 1, 8, 1) > 0
    assert L.ddp_distill_workspace(_rows(1), 1, 8, 0) == -1 and L.ddp_distill_workspace(_rows(1), 1, 8, 1025) == -1
    assert L.ddp_distill_workspace(_rows(1), 1, 2 ** 31, 1) == -1
    with pytest.raises(ddp.DDPError):
        ddp.distill_workspace([-1], 8, 1)
    with pytest.raises(ddp.DDPError):
        ddp.rms_norm_grad_workspace([1], 0)


def test_marshalling_refuses_what_is_no_list_of_gpu_tensors():
    import torch
    R = ddp._rows
    x = torch.zeros(2, 8)

    def pack(ts, more=None):
        rest = () if more is None else ((more, "y", R.F32, R.LIKE),)
        return R.pack(0, (ts, "x", R.F32, R.LIKE), *rest)

    for bad in (x.to_sparse(), x):
        with pytest.raises(ValueError, match="x: tensor is not on a GPU"):
            pack([bad])
    with pytest.raises(ValueError, match="no ranks"):
        pack([])
    with pytest.raises(ValueError, match="y: one tensor per rank"):
        pack([x, x], [x])
    for bad in ([1.0], [None], None, 3):
        with pytest.raises(TypeError):
            pack(bad)
    for bad in ((), (0,), (0, 1), (0, (1, 2)), ("x", ([x], "x", 1, -1))):
        with pytest.raises(TypeError):
            R.pack(*bad)
    assert R.span(0, None, "w", R.F32, 8) == (0, None, 0)
    with pytest.raises(ValueError, match="w: tensor is not on a GPU"):
        R.span(0, x, "w", R.F32, 8)
    with pytest.raises(TypeError):
        R.span(0, 1.0, "w", R.F32, 8)
    with pytest.raises(TypeError):
        R.span(0, x)
