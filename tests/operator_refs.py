"""Plain 64-bit forms of the operators around the scan, token by token, with
the error bounds their float32 kernels are held to (test code only).

Every bound counts roundings, in units of 2^-24 (half a float32 step), from
the operations a kernel does; a store in bfloat16 adds half a step of that
type, 2^-8 of the value.  Where errors travel along the recurrence the bound
travels with it (a running error bound).
"""
import math

import torch

U = 2.0 ** -24
F = torch.float64


def half_step(dtype):
    """Half a step of a type, relative to the value: what one rounding moves."""
    return torch.finfo(dtype).eps / 2


def check(got, ref, bound, what):
    """|got - ref| <= half a step of got's type (+ its smallest normal number)
    + bound, elementwise; NaN and infinities at the same places."""
    g = got.detach().cpu().to(F)
    ref = torch.as_tensor(ref, dtype=F)
    assert g.shape == ref.shape, "%s: shape %s, not %s" % (what, tuple(g.shape), tuple(ref.shape))
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isnan(g), torch.isnan(ref)), "%s: NaN elsewhere" % what
    assert torch.equal(torch.isfinite(g), fine), "%s: infinities elsewhere" % what
    room = half_step(got.dtype) * (ref.abs() + bound) + bound + torch.finfo(got.dtype).tiny
    off = (g - ref).abs() - room
    off = off[fine]
    assert off.numel() == 0 or off.max().item() <= 0, "%s: %d of %d values off, worst by %.3g over a room of %.3g" % (
        what, int((off > 0).sum()), off.numel(), off.max().item(), room[fine][off.argmax()].item())


# ---- gated recurrence


def starts(seq_idx, b, L):
    first = torch.zeros(b, L, dtype=torch.bool)
    if seq_idx is not None:
        first[:, 1:] = seq_idx[:, 1:] != seq_idx[:, :-1]
    return first


def gated(x, r_raw, g_raw, lam, init=None, seq_idx=None, c=8.0):
    """(h, bound of |error of h|, parts) in 64 bits; parts feed gated_bwd."""
    x, r_raw, g_raw, lam = (t.detach().cpu().to(F) for t in (x, r_raw, g_raw, lam))
    b, L, D = x.shape
    first = starts(None if seq_idx is None else seq_idx.cpu(), b, L)
    r, g = torch.sigmoid(r_raw), torch.sigmoid(g_raw)
    u = c * torch.nn.functional.softplus(lam, threshold=1e9) * r
    om, a = -torch.expm1(-u), torch.exp(-u)
    beta = torch.sqrt(-torch.expm1(-2 * u))
    inp = beta * g * x
    h = torch.zeros(b, D, dtype=F) if init is None else init.detach().cpu().to(F)
    size, err = h.abs(), torch.zeros(b, D, dtype=F)
    hs, before, errs, errs_before = [], [], [], []
    for t in range(L):
        at = first[:, t, None]
        h, size, err = (torch.where(at, torch.zeros_like(v), v) for v in (h, size, err))
        before.append(h)
        errs_before.append(err)
        # a product of sigmoids, square root and x: 60 roundings; 1 - a: 60;
        # the update and the products over spans that join segments: 4
        new = a[:, t] * size + inp[:, t].abs()
        err = a[:, t] * err + U * (4 * new + 60 * inp[:, t].abs() + 60 * om[:, t] * size)
        size = new
        h = a[:, t] * h + inp[:, t]
        hs.append(h)
        errs.append(err)
    if L == 0:
        return x, torch.zeros_like(x), None
    stack = lambda v: torch.stack(v, 1)  # noqa: E731
    return stack(hs), stack(errs), dict(x=x, r=r, g=g, u=u, a=a, om=om, beta=beta, first=first, before=stack(before),
                                        err_before=stack(errs_before), lam=lam)


def gated_bwd(parts, dy, dfinal=None):
    """Gradients and bounds, each {name: (value, bound)}."""
    x, r, g, u, decay, om, beta, first, before, eb, lam = (
        parts[k] for k in ("x", "r", "g", "u", "a", "om", "beta", "first", "before", "err_before", "lam"))
    b, L, D = x.shape
    dy = dy.detach().cpu().to(F)
    carry = torch.zeros(b, D, dtype=F) if dfinal is None else dfinal.detach().cpu().to(F)
    csize, cerr = carry.abs(), torch.zeros(b, D, dtype=F)
    dhs, sizes, errs = [None] * L, [None] * L, [None] * L
    for t in range(L - 1, -1, -1):
        dh = dy[:, t] + carry
        size = dy[:, t].abs() + csize
        err = cerr + U * 4 * size
        dhs[t], sizes[t], errs[t] = dh, size, err
        keep = ~first[:, t, None]
        a = decay[:, t]
        carry = torch.where(keep, a * dh, torch.zeros_like(dh))
        csize = torch.where(keep, a * size, torch.zeros_like(dh))
        cerr = torch.where(keep, a * err + U * 60 * om[:, t] * size, torch.zeros_like(dh))
    dh, size, err = torch.stack(dhs, 1), torch.stack(sizes, 1), torch.stack(errs, 1)
    a = decay
    w = torch.where(beta > 0, u * a * a / beta.clamp_min(1e-300), torch.zeros_like(u))
    p = dh * (u * a * before - w * g * x)
    each = (u * a * before).abs() + (w * g * x).abs()
    # u is off by 50 roundings of itself, so a = e^-u by 50 u of them relative
    # to a, and a^2 by 100 u; the other factors by 120
    perr = err * each + size * (u * a * eb + U * (120 + 100 * u) * each)
    lead = torch.sigmoid(lam) / torch.nn.functional.softplus(lam, threshold=1e9)
    dlam = -lead * p.sum((0, 1))
    # float32 sums over 64 tokens, wider ones above
    dlam_err = lead * (perr + 64 * U * p.abs()).sum((0, 1)) + 8 * U * dlam.abs()
    out = {"x": (dh * beta * g, err * beta * g + 60 * U * size * beta * g),
           "g_raw": (dh * beta * x * g * (1 - g), (err + 90 * U * size) * (beta * x * g).abs()),
           "r_raw": (-(1 - r) * p, (1 - r) * perr + 40 * U * p.abs()),
           "lam": (dlam, dlam_err), "init_state": (carry, cerr)}
    return out


# ---- norm and rotation of B and C


def _turned(v, pos, inv_freq, interleaved, sign=1.0):
    R = 2 * inv_freq.numel()
    if R == 0:
        return v, v.abs()
    ang = sign * pos.to(F)[..., None, None] * inv_freq.to(F)
    c, s = torch.cos(ang), torch.sin(ang)
    j = torch.arange(R // 2)
    e0, e1 = (2 * j, 2 * j + 1) if interleaved else (j, j + R // 2)
    out, size = v.clone(), v.abs()
    p, q = v[..., e0], v[..., e1]
    out[..., e0], out[..., e1] = p * c - q * s, q * c + p * s
    size[..., e0] = size[..., e1] = p.abs() + q.abs()
    return out, size


def norm_rotate(v, w, inv_freq, pos, eps, interleaved):
    """(out, bound): the sum of N squares moves the scale by N/2 roundings, a
    cosine or sine by 16 (its reduced angle and the function), the rest 10."""
    v, w = v.detach().cpu().to(F), w.detach().cpu().to(F)
    N = v.shape[-1]
    n = v / torch.sqrt(v.square().mean(-1, keepdim=True) + eps) * w
    out, size = _turned(n, pos.cpu(), inv_freq.detach().cpu(), interleaved)
    return out, U * (N / 2 + 26) * size


def norm_rotate_bwd(v, w, inv_freq, pos, eps, interleaved, d):
    v, w, d = (t.detach().cpu().to(F) for t in (v, w, d))
    N = v.shape[-1]
    rs = 1 / torch.sqrt(v.square().mean(-1, keepdim=True) + eps)
    dn, size = _turned(d, pos.cpu(), inv_freq.detach().cpu(), interleaved, -1.0)
    n = v * rs
    m, msize = (dn * w * n).mean(-1, keepdim=True), (size * w.abs() * n.abs()).mean(-1, keepdim=True)
    dv = rs * (dn * w - n * m)
    dv_err = U * rs * ((N / 2 + 30) * size * w.abs() + (2 * N + 60) * n.abs() * msize)
    dw = (dn * n).sum((0, 1, 2))
    # float32 running sums of at most 64 rows, wider ones above
    dw_err = U * (64 + N / 2 + 30) * (size * n.abs()).sum((0, 1, 2))
    return (dv, dv_err), (dw, dw_err)


# ---- projections


def act(z, name):
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2.0))
    return z


def act_slope(z, name):
    if name == "silu":
        q = torch.sigmoid(z)
        return q * (1 + z * (1 - q))
    if name == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def linear(x, w, bias=None, residual=None, activation="none"):
    """(out, bound, z, bound of z).  A sum of K exact or once-rounded products:
    2 K roundings (an adder may truncate).  An activation's slope is at most
    1.13; its own evaluation 40 roundings of |z| (the exponential of an
    argument of 16 is off by about 20)."""
    x, w = x.detach().cpu().to(F), w.detach().cpu().to(F)
    K = x.shape[-1]
    z, size = x @ w.T, x.abs() @ w.abs().T
    if bias is not None:
        z, size = z + bias.detach().cpu().to(F), size + bias.detach().cpu().to(F).abs()
    zerr = U * (2 * K + 4) * size
    out, err = act(z, activation), 1.13 * zerr + (0 if activation == "none" else 40 * U) * z.abs()
    if residual is not None:
        out = out + residual.detach().cpu().to(F)
        err = err + 2 * U * out.abs()
    return out, err, z, zerr


def linear_bwd(x, w, dy, z=None, activation="none"):
    """{name: (value, bound)}; a bfloat16 dz enters its products rounded, by
    half a step, unless it is dy itself."""
    t = x.dtype
    x, w, dy = (v.detach().cpu().to(F) for v in (x, w, dy))
    dz = dy if activation == "none" else dy * act_slope(z.detach().cpu().to(F), activation)
    derr = torch.zeros_like(dz) if activation == "none" else 60 * U * dy.abs()
    perr = derr if activation == "none" or t == torch.float32 else derr + half_step(t) * dz.abs()
    M, N = dz.shape
    return {"x": (dz @ w, perr @ w.abs() + 2 * N * U * (dz.abs() @ w.abs())),
            "weight": (dz.T @ x, perr.T @ x.abs() + 2 * M * U * (dz.abs().T @ x.abs())),
            "bias": (dz.sum(0), derr.sum(0) + 66 * U * dz.abs().sum(0))}
