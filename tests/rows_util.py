"""Shared by the tests of the operators over rows of tokens: matrices with
gaps at any alignment, the definitions in 64 bits, and the error bounds the
tests hold the kernels to.

Bounds.  U = 2**-24 is half a step of f32, HALF[t] half a step of an output
type.  A sum of n terms of one sign in f32 is off by at most (its longest chain
of additions) * U relative; with at least 64 threads to a row that chain is at
most n / 64 + 24 (a thread's own terms, then trees over the lanes, the waves
and the partial sums).  Each further product, quotient or root adds U or two.
"""
import math

import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133}   # half the least step, and more


def chain(n):
    return n / 64 + 24


def matrix(t, pad=0, shift=0, device="cuda:0"):
    """A [rows, width] copy of t on the device, its rows `pad` elements apart and its first
    element `shift` elements into a buffer whose other bytes hold a pattern."""
    rows, width = t.shape
    size = t.element_size()
    buf = torch.full(((shift + rows * (width + pad) + 8) * size,), 0x5A, dtype=torch.uint8, device=device)
    flat = buf.view(t.dtype)
    m = flat[shift:shift + rows * (width + pad)].view(rows, width + pad)[:, :width]
    m.copy_(t)
    return m


def gaps_untouched(m):
    """Whether the bytes around and between a matrix()'s rows still hold the pattern."""
    base = m._base if m._base is not None else m
    rows, width = m.shape
    size = m.element_size()
    raw = base.view(torch.uint8).clone()
    off = m.storage_offset()
    pitch = m.stride(0) if rows > 1 else width
    for r in range(rows):
        raw[(off + r * pitch) * size:(off + r * pitch + width) * size] = 0x5A
    return bool((raw == 0x5A).all())


# ---------------------------------------------------------------- norm

def norm_sum(x, residual):
    """The kept sum: added in f32, rounded to the dtype (exact for both steps' order)."""
    return x if residual is None else (x.float() + residual.float()).to(x.dtype)


def norm_64(s, weight, eps):
    h = s.double()
    rho = 1.0 / torch.sqrt(h.square().mean(1, keepdim=True) + eps)
    y = h * rho
    return (y if weight is None else y * weight.double()), rho


def norm_rel(width):
    """Relative error of y before its last rounding: half that of the sum of squares, and
    the root, quotient, mean and two products."""
    return (chain(width) / 2 + 8) * U


def check_norm(got, s, weight, eps, scale=None, what=""):
    want, _ = norm_64(s, weight, eps)
    got64 = got.double()
    rel = norm_rel(s.shape[1])
    if scale is None:
        tol = want.abs() * (rel + HALF[got.dtype]) * (1 + 2 ** -7) + TINY[got.dtype]
        bad = ((got64 - want).abs() > tol).nonzero()
        assert bad.numel() == 0, (what, bad[:4], got64[tuple(bad[0])], want[tuple(bad[0])])
        return
    top = 127.0 if got.dtype == torch.int8 else 448.0
    most = want.abs().amax(1)
    step = (most / top)
    assert ((scale.double() - step).abs() <= step * (rel + 2 * U) + 2.0 ** -149).all(), what
    value = got64 * scale.double()[:, None]
    # y / scale in f32 is off by its own relative error and three products, then half a step
    code = (want / torch.where(step > 0, step, torch.ones_like(step))[:, None]).abs()
    half = torch.full_like(code, 0.5)
    if got.dtype != torch.int8:   # 3 bits of mantissa, exponents from -6
        half = torch.maximum(code * 2.0 ** -4, torch.full_like(code, 2.0 ** -10))
    off = (half + code * (2 * rel + 8 * U)) * step[:, None] * (1 + 1e-6)
    # a scale below the least normal float has steps of 2**-149
    off = off + got64.abs() * 2.0 ** -149
    bad = ((value - want).abs() > off).nonzero()
    assert bad.numel() == 0, (what, bad[:4], value[tuple(bad[0])], want[tuple(bad[0])], step[bad[0][0]])


def norm_grad_64(s, weight, dy, dsum, eps):
    h, d = s.double(), dy.double()
    rho = 1.0 / torch.sqrt(h.square().mean(1, keepdim=True) + eps)
    g = d if weight is None else d * weight.double()
    dx = rho * (g - h * rho * rho * (g * h).mean(1, keepdim=True))
    if dsum is not None:
        dx = dx + dsum.double()
    return dx, (d * h * rho).sum(0)


def check_norm_grad(dx, dw, s, weight, dy, dsum, eps, old=None, what=""):
    """dw None: not asked for; old: what dw held before, for an accumulating call."""
    want, wdw = norm_grad_64(s, weight, dy, dsum, eps)
    width, rows = s.shape[1], s.shape[0]
    h, d = s.double(), dy.double()
    rho = 1.0 / torch.sqrt(h.square().mean(1, keepdim=True) + eps)
    g = d if weight is None else d * weight.double()
    rel = norm_rel(width)
    # rho has the relative error `rel`; the mean of g s that of its chain over |g s|
    big = rho * (g.abs() + h.abs() * rho * rho * (g * h).abs().mean(1, keepdim=True))
    tol = big * (4 * rel + (chain(width) + 12) * U)
    if dsum is not None:
        tol = tol + dsum.double().abs() * 2 * U
    tol = tol + (want.abs() + tol) * HALF[dx.dtype] + TINY[dx.dtype]
    bad = ((dx.double() - want).abs() > tol).nonzero()
    assert bad.numel() == 0, (what, bad[:4], dx[tuple(bad[0])], want[tuple(bad[0])])
    if dw is None:
        return
    # a column's sum: any order over the rows is at most `rows` additions
    tol = (d * h * rho).abs().sum(0) * (rel + (rows + 4) * U)
    if old is not None:
        wdw = wdw + old.double()
        tol = tol + (wdw.abs() + tol) * U
    tol = tol + (wdw.abs() + tol) * HALF[dw.dtype] + TINY[dw.dtype]
    bad = ((dw.double() - wdw).abs() > tol).nonzero()
    assert bad.numel() == 0, (what, "dweight", bad[:4], dw[bad[0]], wdw[bad[0]])


# ---------------------------------------------------------------- distillation

def distill_64(logits, teacher, index, weight, tau, grad_scale=1.0):
    """Lists over the ranks, all on the CPU or all on the GPU: loss, row losses, gradients, and
    for each what their errors are measured against: (losses' magnitudes, q, p scaled)."""
    n = len(logits)
    rows, parts, total = [], [], 0.0
    for r in range(n):
        z = logits[r].double() / tau
        vocab = z.shape[1]
        idx = index[r].long()
        t = teacher[r].double()
        ok = (idx >= 0) & (idx < vocab) & (t > -math.inf)
        w = torch.ones(z.shape[0], dtype=torch.float64, device=z.device) if weight is None \
            else weight[r].double()
        live = ok.any(1) & (w > 0)
        w = torch.where(live, w, torch.zeros_like(w))
        t = torch.where(ok & live[:, None], t / tau, torch.full_like(t, -math.inf))
        t = torch.where(live[:, None], t, torch.zeros_like(t))
        logp = torch.log_softmax(t, 1)
        p = torch.where(ok & live[:, None], logp.exp(), torch.zeros_like(t))
        z = torch.where(live[:, None], z, torch.zeros_like(z))
        logq = torch.log_softmax(z, 1)
        at = torch.where(ok, idx, torch.zeros_like(idx))
        lq = logq.gather(1, at)
        kl = torch.where(p > 0, p * (logp - lq), torch.zeros_like(p)).sum(1)
        mag = torch.where(p > 0, p * (logp.abs() + lq.abs() + 1), torch.zeros_like(p)).sum(1)
        row = torch.where(live, tau * tau * kl, torch.zeros_like(kl))
        sure = torch.where(live, tau * tau * mag, torch.zeros_like(kl))
        dense = torch.zeros_like(z).scatter_add_(1, at, p)
        q = logq.exp()
        rows.append((row, sure, w))
        parts.append((q, dense, live))
        total = total + w.sum()
    den = total if total > 0 else torch.ones_like(total)
    loss = sum((row * w).sum() for row, _, w in rows) / den
    loss_mag = sum((sure * w).sum() for _, sure, w in rows) / den
    grads, mags = [], []
    for (q, dense, live), (_, _, w) in zip(parts, rows):
        c = (grad_scale * n * tau) * (w / den)[:, None]
        zero = torch.zeros_like(q)
        grads.append(torch.where(live[:, None], c * (q - dense), zero))
        mags.append(torch.where(live[:, None], abs(c) * (q + dense), zero))
    return loss, [r[0] for r in rows], grads, loss_mag, [r[1] for r in rows], mags


def distill_rel(logits, tau):
    """Error of a logarithm of q or p, so also the relative error of q and p: the sum's chain
    over the vocabulary, and the exponents' own rounding, two steps of the farthest logit
    that still counts (one more than 104 below the largest has exp = 0 in f32)."""
    vocab = logits[0].shape[1]
    return (chain(max(vocab, 1024)) + 3 * 104 + 16) * U


def check_distill(loss, row_loss, dlogits, logits, teacher, index, weight, tau, grad_scale=1.0, what=""):
    w_loss, w_rows, w_grads, m_loss, m_rows, m_grads = distill_64(logits, teacher, index, weight, tau,
                                                                   grad_scale)
    tokens = sum(z.shape[0] for z in logits)
    rel = distill_rel(logits, tau)
    for r, (got, want, mag) in enumerate(zip(row_loss or [], w_rows, m_rows)):
        got = got.double()
        assert torch.equal(torch.isnan(got), torch.isnan(want)), (what, r)
        assert torch.equal(torch.isinf(got), torch.isinf(want)), (what, r)
        fine = torch.isfinite(want)
        bad = ((got - want).abs()[fine] > mag[fine] * 3 * rel + 1e-37).nonzero()
        assert bad.numel() == 0, (what, "row_loss", r, bad[:4], got[fine][bad[0]], want[fine][bad[0]])
    if math.isfinite(float(w_loss)):
        # two sums over the tokens, each in a chain of at most tokens / 64 + 24
        tol = float(m_loss) * (3 * rel + 2 * (chain(tokens) + 4) * U) + 1e-37
        assert abs(float(loss) - float(w_loss)) <= tol, (what, float(loss), float(w_loss), tol)
    else:
        assert math.isnan(float(loss)) == math.isnan(float(w_loss)) and not math.isfinite(float(loss))
    for r, (got, want, mag) in enumerate(zip(dlogits or [], w_grads, m_grads)):
        got64 = got.double()
        assert torch.equal(torch.isnan(got64), torch.isnan(want)), (what, r)
        tol = mag * (3 * rel + (chain(tokens) + 12) * U)
        tol = tol + (want.abs() + tol) * HALF[got.dtype] + TINY[got.dtype]
        bad = ((got64 - want).abs() > tol).nonzero()
        assert bad.numel() == 0, (what, "dlogits", r, bad[:4], got64[tuple(bad[0])], want[tuple(bad[0])],
                                  tol[tuple(bad[0])])
