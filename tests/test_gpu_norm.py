"""ddp_rms_norm and ddp_rms_norm_grad on the GPU against their definitions in
64 bits (bounds derived in rows_util.py), at widths from 1 past every
vector and block, ragged ranks, gaps and odd alignments, in place, every dtype,
rows of zeros, tiny values, infinities and NaN, offsets past 32 bits, captured
and on two streams."""
import math

import pytest
import torch

from gpu_util import torch_cuda
from rows_util import U, chain, check_norm, check_norm_grad, gaps_untouched, matrix, norm_64, norm_grad_64, norm_rel, norm_sum

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "i8": torch.int8, "e4m3": torch.float8_e4m3fn}
EPS = 1e-6


@pytest.fixture(scope="module")
def ddp():
    torch_cuda()
    import gradient_allreduce_averaging_amd as ddp
    return ddp


def _rand(seed, rows, width, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    t = torch.randn(rows, width, generator=g) * scale
    t *= torch.exp(0.7 * torch.randn(1, width, generator=g))
    return t.to(DT[dtype])


def _weight(seed, width, dtype):
    g = torch.Generator().manual_seed(seed)
    return (1 + 0.3 * torch.randn(width, generator=g)).to(DT[dtype]).cuda()


def _empty(rows, width, dtype, pad=0, shift=0):
    return matrix(torch.zeros(rows, width).to(DT[dtype]), pad, shift)


WIDTHS = [1, 2, 3, 7, 8, 9, 63, 64, 65, 255, 257, 511, 513, 1000, 1024, 2047, 2048, 2051, 4096, 4097, 5003, 8192,
          8200, 11008, 16384, 16411, 40009]


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_widths(ddp, width, dtype):
    """Every output type, with and without residual and kept sum, ragged ranks (one without
    rows), gaps between rows and odd first elements."""
    rows = [3, 0, 1, 5]
    outs = ["f32", "bf16", "i8", "e4m3"] if dtype == "f32" else ["bf16", "i8", "e4m3"]
    for k, out in enumerate(outs):
        pad, shift = [(0, 0), (5, 1), (8, 3), (1, 7)][(k + width) % 4]
        x = [matrix(_rand(10 * k + r, n, width, dtype), pad, shift) for r, n in enumerate(rows)]
        res = [matrix(_rand(90 + 10 * k + r, n, width, dtype, 3.0), pad, shift) for r, n in enumerate(rows)]
        w = _weight(k, width, "bf16" if k % 2 else "f32") if k != 2 else None
        for with_res, with_sum in ((True, True), (True, False), (False, False), (False, True)):
            y = [_empty(n, width, out, pad, shift) for n in rows]
            kept = [_empty(n, width, dtype, pad, shift) for n in rows] if with_sum else None
            scale = [torch.full((n,), math.nan, device="cuda") for n in rows] if out in ("i8", "e4m3") else None
            ddp.rms_norm(x, w, y, residual=res if with_res else None, sum_out=kept, scale=scale, eps=EPS)
            torch.cuda.synchronize()
            for r, n in enumerate(rows):
                if n == 0:
                    continue
                s = norm_sum(x[r], res[r] if with_res else None)
                what = (width, dtype, out, with_res, with_sum, r)
                check_norm(y[r], s, w, EPS, None if scale is None else scale[r], what)
                assert gaps_untouched(y[r]), what
                if with_sum:
                    assert torch.equal(kept[r].contiguous().view(torch.uint8), s.contiguous().view(torch.uint8)), what
                    assert gaps_untouched(kept[r]), what


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("dtype,dy", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
def test_norm_grad_widths(ddp, width, dtype, dy):
    for k, rows in enumerate(([3, 0, 1, 5], [37], [1])):
        pad, shift = [(0, 0), (5, 1), (8, 3), (1, 7)][(k + width) % 4]
        s = [matrix(_rand(10 * k + r, n, width, dtype), pad, shift) for r, n in enumerate(rows)]
        d = [matrix(_rand(40 + 10 * k + r, n, width, dy, 0.1), pad, shift) for r, n in enumerate(rows)]
        extra = [matrix(_rand(70 + 10 * k + r, n, width, dtype, 0.1), pad, shift) for r, n in enumerate(rows)]
        w = _weight(k, width, "bf16" if k % 2 else "f32") if k != 2 else None
        for with_sum, dwt, acc in ((True, "f32", False), (False, "bf16", True), (True, "bf16", False),
                                   (False, "f32", True), (False, None, False)):
            dx = [_empty(n, width, dtype, pad, shift) for n in rows]
            # the weight's place in a flat gradient, off any alignment but its own
            dw = old = None
            if dwt:
                dw = [_rand(k + r, 1, width + 9, dwt, 0.2).cuda()[0, 3:3 + width] for r in range(len(rows))]
                old = [t.clone() for t in dw]
            ddp.rms_norm_grad(s, w, d, dx, dsum=extra if with_sum else None, dweight=dw, accumulate=acc, eps=EPS)
            torch.cuda.synchronize()
            for r, n in enumerate(rows):
                what = (width, dtype, dy, with_sum, dwt, acc, rows, r)
                check_norm_grad(dx[r], None if dw is None else dw[r], s[r], w, d[r],
                                extra[r] if with_sum else None, EPS, old[r] if acc else None, what)
                assert gaps_untouched(dx[r]), what
                if dw is not None:   # nothing around the weight's place
                    whole = _rand(k + r, 1, width + 9, dwt, 0.2).cuda()[0]
                    assert torch.equal(dw[r]._base.view(-1)[:3], whole[:3])
                    assert torch.equal(dw[r]._base.view(-1)[3 + width:], whole[3 + width:])


@pytest.mark.parametrize("n_ranks", [1, 2, 8, 64])
def test_many_ranks_and_rows(ddp, n_ranks):
    """More rows than one grid's blocks hold at once, more ranks than one pass of them."""
    width = 136
    rows = [(700 if n_ranks <= 8 else 40) + 3 * r for r in range(n_ranks)]
    x = [_rand(r, n, width, "bf16").cuda() for r, n in enumerate(rows)]
    d = [_rand(100 + r, n, width, "bf16").cuda() for r, n in enumerate(rows)]
    w = _weight(1, width, "f32")
    y = [torch.empty_like(t) for t in x]
    dx = [torch.empty_like(t) for t in x]
    dw = [torch.empty(width, device="cuda") for _ in rows]
    ddp.rms_norm(x, w, y, eps=EPS)
    ddp.rms_norm_grad(x, w, d, dx, dweight=dw, eps=EPS)
    torch.cuda.synchronize()
    for r in range(n_ranks):
        check_norm(y[r], x[r], w, EPS, what=r)
        check_norm_grad(dx[r], dw[r], x[r], w, d[r], None, EPS, what=r)


@pytest.mark.parametrize("width", [9, 15, 513, 4095, 4097, 8191, 16377, 16384])
@pytest.mark.parametrize("first", [0, 1])
@pytest.mark.parametrize("pad", [0, 1])
def test_bf16_rows_on_and_off_a_word(ddp, width, first, pad):
    """Rows that start on a 4-byte boundary, off one, or in turn, in ranks of 1 to many rows: every
    element of the sums, and the weight gradient of both kinds of rows together."""
    rows = [1, 2, 0, 600]
    x = [matrix(_rand(r, n, width, "bf16"), pad, first + r % 2) for r, n in enumerate(rows)]
    d = [matrix(_rand(9 + r, n, width, "bf16"), pad, first) for r, n in enumerate(rows)]
    w = _weight(1, width, "f32")
    y = [_empty(n, width, "bf16", pad, 3) for n in rows]
    dx = [_empty(n, width, "bf16", pad, first) for n in rows]
    dw = [torch.full((width,), math.nan, device="cuda") for _ in rows]
    ddp.rms_norm(x, w, y, eps=EPS)
    ddp.rms_norm_grad(x, w, d, dx, dweight=dw, eps=EPS)
    torch.cuda.synchronize()
    for r, n in enumerate(rows):
        if n:
            check_norm(y[r], x[r], w, EPS, what=r)
            check_norm_grad(dx[r], dw[r], x[r], w, d[r], None, EPS, what=r)
            assert gaps_untouched(y[r]) and gaps_untouched(dx[r])
        else:
            assert (dw[r] == 0).all()


def test_more_rows_than_a_grid(ddp):
    rows, width = 70001, 9
    x = _rand(0, rows, width, "f32").cuda()
    d = _rand(1, rows, width, "f32").cuda()
    y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(width, device="cuda")
    ddp.rms_norm([x], None, [y], eps=EPS)
    ddp.rms_norm_grad([x], None, [d], [dx], dweight=[dw], eps=EPS)
    check_norm(y, x, None, EPS)
    check_norm_grad(dx, dw, x, None, d, None, EPS)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width", [5, 257, 513, 2048, 2051, 4097, 5003, 8195, 8200, 40009])
def test_in_place(ddp, dtype, width):
    """Among the widths those whose last, partial vector is the first of a wave."""
    rows = 600
    x0, r0 = _rand(0, rows, width, dtype).cuda(), _rand(1, rows, width, dtype).cuda()
    w = _weight(0, width, dtype)
    s0 = norm_sum(x0, r0)
    # the stream is updated where it lies, and the norm overwrites its input
    for y_in_x in (True, False):
        x, r = x0.clone(), r0.clone()
        y, kept = (x, r) if y_in_x else (r, x)
        ddp.rms_norm([x], w, [y], residual=[r], sum_out=[kept], eps=EPS)
        assert torch.equal(kept, s0)
        check_norm(y, s0, w, EPS)
    x, r = x0.clone(), r0.clone()
    ddp.rms_norm([x], w, [r], residual=[r], eps=EPS)      # nothing kept
    check_norm(r, s0, w, EPS)
    d0, e0 = _rand(2, rows, width, dtype).cuda(), _rand(3, rows, width, dtype).cuda()
    for which in range(3):
        t = [s0.clone(), d0.clone(), e0.clone()]
        dw = torch.empty(width, device="cuda")
        ddp.rms_norm_grad([t[0]], w, [t[1]], [t[which]], dsum=[t[2]], dweight=[dw], eps=EPS)
        check_norm_grad(t[which], dw, s0, w, d0, e0, EPS, what=which)


def test_interleaved_columns_of_one_buffer(ddp):
    buf = _rand(0, 7, 300, "bf16").cuda()
    want = buf[:, :100].clone()
    ddp.rms_norm([buf[:, :100]], None, [buf[:, 200:]], sum_out=[buf[:, 100:200]], eps=EPS)
    assert torch.equal(buf[:, :100], want) and torch.equal(buf[:, 100:200], want)
    check_norm(buf[:, 200:], want, None, EPS)


@pytest.mark.parametrize("width", [7, 513, 4096, 40009])
@pytest.mark.parametrize("out", ["bf16", "f32", "i8", "e4m3"])
def test_unusual_values(ddp, width, out):
    """Rows of zeros, of one huge element, of tiny ones (with eps 0 and not), with a NaN, with
    an infinity; the rows beside them keep their results."""
    x = _rand(0, 9, width, "f32")
    x[1] = 0.0
    x[2] = 0.0
    x[2, width // 2] = 3e18
    x[3] *= 1e-18
    x[4, width // 3] = math.nan
    x[5, width - 1] = math.inf
    x[6] *= 1e-30
    x[7] = -2.5
    x = x.cuda()
    for eps in (1e-6, 1e-30):
        y = torch.empty(9, width, device="cuda", dtype=DT[out])
        scale = [torch.empty(9, device="cuda")] if out in ("i8", "e4m3") else None
        ddp.rms_norm([x], None, [y], scale=scale, eps=eps)
        sc = None if scale is None else scale[0]
        # squares of the values in row 6 underflow, and in row 3 are far below eps = 1e-6
        good = [0, 1, 2, 7, 8] + ([3, 6] if eps == 1e-6 else [])
        check_norm(y[good], x[good], None, eps, None if sc is None else sc[good], (width, out, eps))
        if sc is None:
            assert torch.isnan(y[4].float()).all()
            assert torch.isnan(y[5, width - 1].float()) and (y[5, :width - 1].float() == 0).all()
        else:
            assert torch.isnan(sc[4]) and torch.isnan(sc[5]) and sc[1] == 0
            assert (y[1].float() == 0).all()


@pytest.mark.parametrize("width", [9, 16, 31, 33, 64, 120, 128, 129, 193, 256, 257, 505, 512])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_narrow_rows(ddp, width, dtype):
    """Several rows to a wave: one row to many, on and off a 4-byte boundary, in place, and few of
    them on one rank beside many on another."""
    for k, rows in enumerate(([1, 2], [2], [3, 0, 1000], [7, 9000])):
        pad, shift = [(0, 0), (1, 1), (3, 0), (0, 1)][k]
        x = [matrix(_rand(k + r, n, width, dtype), pad, shift) for r, n in enumerate(rows)]
        res = [matrix(_rand(k + r + 9, n, width, dtype), pad, shift) for r, n in enumerate(rows)]
        dy = [matrix(_rand(k + r + 20, n, width, dtype), pad, shift) for r, n in enumerate(rows)]
        w = _weight(k, width, dtype).cuda()
        old = [a.clone() for a in x]
        codes = [torch.empty(n, width, device="cuda", dtype=torch.int8) for n in rows]
        scale = [torch.empty(n, device="cuda") for n in rows]
        ddp.rms_norm(x, w, codes, residual=res, scale=scale, eps=EPS)
        ddp.rms_norm(x, w, res, residual=res, sum_out=x, eps=EPS)   # both in place
        fresh = [matrix(_rand(k + r + 9, n, width, dtype), pad, shift) for r, n in enumerate(rows)]
        for r, n in enumerate(rows):
            if not n:
                continue
            s = norm_sum(old[r], fresh[r])
            assert torch.equal(x[r], s), (width, rows)
            check_norm(res[r], s, w, EPS, what=(width, rows, r))
            check_norm(codes[r], s, w, EPS, scale[r], (width, rows, r))
        s = [a.clone() for a in x]
        dw = [torch.full((width,), math.nan, device="cuda") for _ in rows]
        d0 = [a.clone() for a in dy]
        ddp.rms_norm_grad(x, w, dy, dy, dsum=x, dweight=dw, eps=EPS)
        for r, n in enumerate(rows):
            if n:
                check_norm_grad(dy[r], dw[r], s[r], w, d0[r], s[r], EPS, what=(width, rows, r))
            else:
                assert (dw[r] == 0).all()
        assert all(gaps_untouched(a) for a, n in zip(x + res + dy, rows * 3) if n)


@pytest.mark.parametrize("width", [7, 48, 4096, 40009])
def test_tiny_rows_without_eps(ddp, width):
    """Rows whose mean square lies below the least normal float, forward and backward."""
    s = _rand(0, 5, width, "f32").cuda() * 2.0 ** -64
    dy, w = _rand(1, 5, width, "f32").cuda(), _weight(2, width, "f32")
    w = w.cuda()
    s[0] = 2.0 ** -66
    s[1] *= 2.0 ** 30   # an ordinary one
    y, dx, dw = torch.empty_like(s), torch.empty_like(s), torch.empty(width, device="cuda")
    ddp.rms_norm([s], w, [y], eps=0.0)
    ddp.rms_norm_grad([s], w, [dy], [dx], dweight=[dw], eps=0.0)
    want, _ = norm_64(s, w, 0.0)
    # a square, a partial sum and the mean are each off by at most half a step of 2^-149, so the mean
    # of squares of 2^-134 or more by (chain + 2) 2^-150 / width, and 2^-150 for its own rounding; the
    # root has half of that, beside the errors of ordinary rows
    mean = s.double().square().mean(1, keepdim=True)
    assert float(mean.min()) > 2.0 ** -134
    low = ((width + 2 * chain(width)) / width + 1) * 2.0 ** -150 / mean
    rel = norm_rel(width) + low
    assert ((y.double() - want).abs() <= want.abs() * (rel + 2 * U)).all()
    wdx, wdw = norm_grad_64(s, w, dy, None, 0.0)
    h, g = s.double(), dy.double() * w.double()
    rho = mean.rsqrt()
    big = rho * (g.abs() + (h * rho).abs() * rho * (g * h).abs().mean(1, keepdim=True))
    # the products g s are off by 2^-150 too, which rho ~ 2^64 leaves far below U
    assert ((dx.double() - wdx).abs() <= big * (4 * rel + (chain(width) + 16) * U)).all()
    assert ((dw.double() - wdw).abs() <= ((dy.double() * h * rho).abs() * (rel + 16 * U)).sum(0)).all()


def test_weight_that_is_zero_or_not_finite(ddp):
    width = 600
    x = _rand(0, 3, width, "bf16").cuda()
    w = torch.zeros(width, device="cuda")
    y, sc = torch.empty(3, width, device="cuda", dtype=torch.int8), torch.empty(3, device="cuda")
    ddp.rms_norm([x], w, [y], scale=[sc], eps=EPS)
    assert (y == 0).all() and (sc == 0).all()
    w[:] = 1e-36      # so small that top / most would overflow
    ddp.rms_norm([x], w, [y], scale=[sc], eps=EPS)
    check_norm(y, x, w, EPS, sc)
    w[5] = math.nan
    ddp.rms_norm([x], w, [y], scale=[sc], eps=EPS)
    assert torch.isnan(sc).all()
    z = torch.empty(3, width, device="cuda", dtype=torch.bfloat16)
    ddp.rms_norm([x], w, [z], eps=EPS)
    assert torch.isnan(z[:, 5]).all() and torch.isfinite(z[:, :5]).all() and torch.isfinite(z[:, 6:]).all()


def test_grad_keeps_a_bad_row_to_itself(ddp):
    width = 1030
    s, d = _rand(0, 4, width, "f32").cuda(), _rand(1, 4, width, "f32").cuda()
    s[2, 17] = math.nan
    dx = torch.empty_like(s)
    ddp.rms_norm_grad([s], None, [d], [dx], eps=EPS)
    good = [0, 1, 3]
    check_norm_grad(dx[good], None, s[good], None, d[good], None, EPS)
    assert torch.isnan(dx[2]).all()


@pytest.mark.parametrize("width", [48, 2048])
def test_grad_matches_differences(ddp, width):
    """dx and dweight against differences of the library's own forward pass in f32: the
    quotient over a step of h is off by a term in h^2, and by the forward's error over h."""
    rows = 3
    s, d = _rand(0, rows, width, "f32").cuda(), _rand(1, rows, width, "f32").cuda()
    w = _weight(2, width, "f32")
    dx, dw = torch.empty_like(s), torch.empty(width, device="cuda")
    ddp.rms_norm_grad([s], w, [d], [dx], dweight=[dw], eps=1e-3)
    y = torch.empty_like(s)

    def objective(s_, w_):
        ddp.rms_norm([s_], w_, [y], eps=1e-3)
        return (y.double() * d.double()).sum()

    g = torch.Generator().manual_seed(5)
    for _ in range(4):
        v = torch.randn(rows, width, generator=g).cuda()
        u = torch.randn(width, generator=g).cuda()
        h = 2.0 ** -7
        num = (objective(s + h * v, w) - objective(s - h * v, w)) / (2 * h)
        want = (dx.double() * v.double()).sum()
        # the third derivative of y along v is of the order of |v|^3 / |s|^3: about h^2 of the value
        size = (dx.double() * v.double()).abs().sum() + (y.double() * d.double()).abs().sum()
        assert abs(num - want) <= float(size) * (8 * h * h + 2.0 ** -18 / h), (float(num), float(want))
        num = (objective(s, w + h * u) - objective(s, w - h * u)) / (2 * h)
        want = (dw.double() * u.double()).sum()
        assert abs(num - want) <= float(size) * (2.0 ** -18 / h), (float(num), float(want))


def test_offsets_past_32_bits(ddp):
    """Three rows, 2**31 + 8 elements apart."""
    width, far = 1500, (1 << 31) + 8
    buf = torch.empty(2 * far + width + 16, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((3, width), (far, 1), 3)
    x.copy_(_rand(0, 3, width, "bf16"))
    y = torch.empty(2 * far + width + 16, dtype=torch.int8, device="cuda").as_strided((3, width), (far, 1), 1)
    sc = torch.empty(3, device="cuda")
    ddp.rms_norm([x], None, [y], scale=[sc], eps=EPS)
    check_norm(y, x, None, EPS, sc)
    d = _rand(1, 3, width, "bf16").cuda()
    s = x.clone()
    dw = torch.empty(width, device="cuda")
    ddp.rms_norm_grad([x], None, [d], [x], dweight=[dw], eps=EPS)
    check_norm_grad(x, dw, s, None, d, None, EPS)


def test_captured_and_replayed(ddp):
    """Forward and backward in one graph, accumulating onto a flat gradient; new values between
    the replays, each replay against the eager calls, bit for bit."""
    rows, width = [65, 30], 2051
    x = [torch.empty(n, width, dtype=torch.bfloat16, device="cuda") for n in rows]
    d = [torch.empty_like(t) for t in x]
    y, dx, kept = ([torch.empty_like(t) for t in x] for _ in range(3))
    w = _weight(0, width, "bf16")
    flat = [torch.zeros(width + 5, device="cuda") for _ in rows]
    dw = [f[3:3 + width] for f in flat]
    ws = torch.empty(ddp.rms_norm_grad_workspace(rows, width), dtype=torch.uint8, device="cuda")

    def step():
        ddp.rms_norm(x, w, y, residual=d, sum_out=kept, eps=EPS)
        ddp.rms_norm_grad(kept, w, y, dx, dsum=d, dweight=dw, accumulate=True, eps=EPS, workspace=ws)

    def fill(seed):
        for r, n in enumerate(rows):
            x[r].copy_(_rand(seed + r, n, width, "bf16"))
            d[r].copy_(_rand(seed + 50 + r, n, width, "bf16"))
            flat[r].fill_(0.25)

    fill(0)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        step()
    torch.cuda.synchronize()
    for rep in range(4):
        fill(100 * rep)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in y + dx + kept + flat]
        fill(100 * rep)
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, y + dx + kept + flat):
            assert torch.equal(a, b), rep


def test_two_streams_at_once(ddp):
    rows, width = 2000, 4096
    xs = [_rand(k, rows, width, "bf16").cuda() for k in range(2)]
    ds = [_rand(9 + k, rows, width, "bf16").cuda() for k in range(2)]
    want = []
    for k in range(2):
        dx, dw = torch.empty_like(xs[k]), torch.empty(width, device="cuda")
        ddp.rms_norm_grad([xs[k]], None, [ds[k]], [dx], dweight=[dw], eps=EPS)
        want.append((dx, dw))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [(torch.empty_like(xs[k]), torch.empty(width, device="cuda")) for k in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for k, st in enumerate(streams):      # each call's workspace is its stream's own
            ddp.rms_norm_grad([xs[k]], None, [ds[k]], [outs[k][0]], dweight=[outs[k][1]], eps=EPS, stream=st)
    torch.cuda.synchronize()
    for k in range(2):
        assert torch.equal(outs[k][0], want[k][0]) and torch.equal(outs[k][1], want[k][1])


def test_shapes_with_more_dimensions(ddp):
    x = _rand(0, 12, 96, "f32").cuda().view(3, 4, 96)
    y = torch.empty_like(x)
    ddp.rms_norm([x], None, [y], eps=EPS)
    check_norm(y.view(12, 96), x.view(12, 96), None, EPS)
    one = torch.empty(96, device="cuda")
    ddp.rms_norm([x[0, 0]], None, [one], eps=EPS)
    assert torch.equal(one, y[0, 0])
    none = torch.empty(0, 96, device="cuda")
    ddp.rms_norm([none], None, [torch.empty(0, 96, device="cuda")], eps=EPS)
    dw = torch.full((96,), 7.0, device="cuda")
    ddp.rms_norm_grad([none], None, [none], [none], dweight=[dw], accumulate=True, eps=EPS)
    assert (dw == 7).all()
    ddp.rms_norm_grad([none], None, [none], [none], dweight=[dw], eps=EPS)
    assert (dw == 0).all()


def test_python_refusals(ddp):
    x = torch.zeros(4, 8, device="cuda")
    y = torch.zeros(4, 8, device="cuda")
    with pytest.raises(ValueError):
        ddp.rms_norm([x.cpu()], None, [y])
    with pytest.raises(ValueError):
        ddp.rms_norm([], None, [])
    with pytest.raises(ValueError):
        ddp.rms_norm([x], None, [y, y])
    with pytest.raises(ValueError):
        ddp.rms_norm([x], None, [y[:3]])
    with pytest.raises(ValueError):
        ddp.rms_norm([x], None, [torch.zeros(8, 4, device="cuda").t()])
    with pytest.raises(ValueError):
        ddp.rms_norm([x], torch.ones(7, device="cuda"), [y])
    with pytest.raises(TypeError):
        ddp.rms_norm([x.half()], None, [y])
    with pytest.raises(ValueError):
        ddp.rms_norm([x], None, [y], residual=[x.bfloat16()])
    with pytest.raises(ValueError):     # a broadcast row
        ddp.rms_norm([x[:1].expand(4, 8).unflatten(0, (2, 2))[:, 0]], None, [y])
    with pytest.raises(ddp.DDPError):
        ddp.rms_norm([x[:1].expand(4, 8)], None, [y])
    with pytest.raises(ddp.DDPError):   # 8 bits without scales
        ddp.rms_norm([x], None, [torch.zeros(4, 8, device="cuda", dtype=torch.int8)])
    with pytest.raises(ValueError):     # scales of another length
        ddp.rms_norm([x], None, [torch.zeros(4, 8, device="cuda", dtype=torch.int8)],
                     scale=[torch.zeros(3, device="cuda")])
    with pytest.raises(ValueError):     # strides that differ between ranks
        ddp.rms_norm([x, torch.zeros(4, 9, device="cuda")[:, :8]], None, [y, torch.zeros_like(y)])
    with pytest.raises(ValueError):     # rows not one distance apart
        ddp.rms_norm([torch.zeros(3, 3, 8, device="cuda")[:, :2]], None, [torch.zeros(6, 8, device="cuda")])
    with pytest.raises(ddp.DDPError):
        ddp.rms_norm_grad([x], None, [x], [y], dweight=[torch.zeros(8, device="cuda")],
                          workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        ddp.rms_norm_grad([x], None, [x], [y.bfloat16()])
