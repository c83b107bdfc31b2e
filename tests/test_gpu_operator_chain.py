"""The operators around the scan in the order a layer calls them, each stage
against the form of its operator on the GPU's own inputs to it."""
import math

import pytest
import torch

import operator_refs as refs
import oracle
from gpu_helpers import TOL_BF16, compare
from state_space_sequence_scan_b200 import ssd

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32


def _weights(g, n, k, dtype):
    return (torch.randn(n, k, generator=g) / math.sqrt(k)).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [FP, BF])
def test_gated_block_forward_and_backward(dtype):
    """projections -> gated recurrence over packed rows -> projection into the
    residual stream, and back."""
    b, L, M, D = 2, 300, 72, 136
    g = torch.Generator().manual_seed(1)
    x = torch.randn(b, L, M, generator=g).to(dtype).cuda()
    wu, wg, wo = _weights(g, D, M, dtype), _weights(g, 2 * D, M, dtype), _weights(g, M, D, dtype)
    bg = (0.1 * torch.randn(2 * D, generator=g)).cuda()
    lam = (-5 + torch.randn(D, generator=g)).cuda()
    ids = torch.cumsum(torch.rand(b, L, generator=g) < 0.02, 1).to(torch.int32).cuda()
    dout = torch.randn(b, L, M, generator=g).to(dtype).cuda()

    u, zu = ssd.linear_fwd_preact(x, wu, activation="gelu")
    gates = ssd.linear_fwd(x, wg, bias=bg)
    r, i = gates[..., :D], gates[..., D:]
    y, fin, st = ssd.gated_scan_fwd_states(u, r, i, lam, seq_idx=ids)
    out = ssd.linear_fwd(y, wo, residual=x)

    dl = ssd.linear_bwd(y, wo, dout, want_dbias=False)
    dgates = torch.empty_like(gates)
    dg = ssd.gated_scan_bwd(u, r, i, lam, st, dl["x"], seq_idx=ids, out={"r_raw": dgates[..., :D], "g_raw": dgates[..., D:]})
    dgl = ssd.linear_bwd(x, wg, dgates)
    dul = ssd.linear_bwd(x, wu, dg["x"], preact=zu, activation="gelu", want_dbias=False)

    flat = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
    for got, (ref, err, _, _), what in ((flat(u), refs.linear(flat(x), wu, None, None, "gelu"), "u"),
                                        (flat(gates), refs.linear(flat(x), wg, bg), "gates"),
                                        (flat(out), refs.linear(flat(y), wo, None, flat(x)), "out")):
        refs.check(got, ref, err, what)
    h, err, parts = refs.gated(u, r, i, lam, None, ids)
    refs.check(y, h, err, "y")
    ref = refs.linear_bwd(flat(y), wo, flat(dout))
    refs.check(flat(dl["x"]), *ref["x"], "dy")
    refs.check(dl["weight"], *ref["weight"], "dwo")
    for k, (v, e) in refs.gated_bwd(parts, dl["x"]).items():
        refs.check(dg[k], v, e, "d" + k)
    ref = refs.linear_bwd(flat(x), wg, flat(dgates))
    for k in ("x", "weight", "bias"):
        refs.check(flat(dgl[k]) if k == "x" else dgl[k], *ref[k], "gates' d" + k)
    ref = refs.linear_bwd(flat(x), wu, flat(dg["x"]), flat(zu), "gelu")
    refs.check(flat(dul["x"]), *ref["x"], "dx")
    refs.check(dul["weight"], *ref["weight"], "dwu")


def test_gated_block_gradient_is_its_difference():
    """The whole block in float32: the gradient along a direction of x and of
    lam against the central difference of the block's own 64-bit form.  The
    form is smooth, so the difference at 1e-6 is exact to about 1e-9; the
    kernels' gradient is a float32 one (relative 1e-4 leaves room for the sums
    over a few hundred tokens and four products)."""
    b, L, M, D = 1, 150, 24, 40
    g = torch.Generator().manual_seed(2)
    x = torch.randn(b, L, M, generator=g).cuda()
    wu, wg, wo = _weights(g, D, M, FP), _weights(g, 2 * D, M, FP), _weights(g, M, D, FP)
    lam = (-5 + torch.randn(D, generator=g)).cuda()
    dout = torch.randn(b, L, M, generator=g).cuda()
    u = ssd.linear_fwd(x, wu)
    gates = ssd.linear_fwd(x, wg)
    y, _, st = ssd.gated_scan_fwd_states(u, gates[..., :D], gates[..., D:], lam)
    dl = ssd.linear_bwd(y, wo, dout)
    dg = ssd.gated_scan_bwd(u, gates[..., :D], gates[..., D:], lam, st, dl["x"])
    dx = (dout + ssd.linear_bwd(x, wu, dg["x"])["x"]
          + ssd.linear_bwd(x, wg, torch.cat([dg["r_raw"], dg["g_raw"]], -1))["x"])
    c = lambda t: t.double().cpu()  # noqa: E731

    def loss(xx, ll):
        ga = xx @ c(wg).T
        h, _, _ = refs.gated(xx @ c(wu).T, ga[..., :D], ga[..., D:], ll)
        return float((c(dout) * (xx + h @ c(wo).T)).sum())

    vx, vl, eps = torch.randn(x.shape, generator=g).double(), torch.randn(D, generator=g).double(), 1e-6
    for got, want in ((float((c(dx) * vx).sum()), (loss(c(x) + eps * vx, c(lam)) - loss(c(x) - eps * vx, c(lam))) / (2 * eps)),
                      (float((c(dg["lam"]) * vl).sum()), (loss(c(x), c(lam) + eps * vl) - loss(c(x), c(lam) - eps * vl)) / (2 * eps))):
        assert got == pytest.approx(want, rel=1e-4, abs=1e-3)


def test_scan_layer_with_projections_and_rotated_keys():
    """in-projection -> conv -> norm and rotation of B and C -> scan -> gated
    norm -> out-projection with the residual."""
    b, L, M, H, P, G, N = 2, 200, 128, 4, 64, 2, 128
    g = torch.Generator().manual_seed(3)
    HP, Cd = H * P, H * P + 2 * G * N
    x = torch.randn(b, L, M, generator=g).to(BF).cuda()
    w_in, w_out = _weights(g, HP + Cd + H, M, BF), _weights(g, M, HP, BF)
    cw, cb = (torch.randn(Cd, 4, generator=g) / 2).cuda(), (0.1 * torch.randn(Cd, generator=g)).cuda()
    wB, wC = (1 + 0.1 * torch.randn(N, generator=g)).cuda(), (1 + 0.1 * torch.randn(N, generator=g)).cuda()
    inv = (10000.0 ** (-torch.arange(N // 2) / (N / 2))).cuda()
    dt_bias = torch.full((H,), -3.0).cuda()
    A = -torch.exp(torch.rand(H, generator=g)).cuda()
    D, wn = torch.ones(H).cuda(), torch.ones(HP).cuda()

    both = ssd.linear_fwd(x, w_in)
    refs.check(both.view(-1, both.shape[-1]), *refs.linear(x.view(-1, M), w_in)[:2], "in-projection")
    z, xbc = both[..., :HP].contiguous(), both[..., HP:HP + Cd].contiguous()
    dt_raw = both[..., HP + Cd:].float().contiguous()
    xs, B, C = ssd.conv1d_silu_split(xbc, cw, cb, H, P, G, N)
    B, C = B * 0.25, C * 0.25
    Bn, Cn = ssd.bc_norm_rotate_fwd(B, C, wB, wC, inv)
    p = torch.arange(L).repeat(b, 1)
    refs.check(Bn, *refs.norm_rotate(B, wB, inv, p, 1e-5, False), "B")
    refs.check(Cn, *refs.norm_rotate(C, wC, inv, p, 1e-5, False), "C")
    y, _ = ssd.chunk_scan_fwd(xs, dt_raw, dt_bias, A, Bn, Cn, D, chunk_size=128)
    c = lambda t: t.float().cpu().numpy()  # noqa: E731
    yr, _ = oracle.scan(c(xs), c(dt_raw), c(dt_bias), c(A), c(Bn), c(Cn), c(D))
    compare(y.cpu().double().numpy(), yr, TOL_BF16, "scan on rotated keys")
    v = ssd.gated_rmsnorm(y.view(b * L, HP), z.view(b * L, HP), wn, P).to(BF)
    out = ssd.linear_fwd(v, w_out, residual=x.view(b * L, M))
    refs.check(out, *refs.linear(v, w_out, None, x.view(b * L, M))[:2], "out-projection")


def test_rotation_depends_on_distance_only():
    """The scan of rotated keys and queries reads C_i . B_j at the distance
    i - j: moving every position by the same amount leaves y but for the
    roundings of B and C to bf16.  Each value of either is off by half a step,
    2^-8 of its size, in either run, so a product by 4 * 2^-8 of the product
    of the sizes, and y by that much of the scan of all sizes, where an
    element's size is that of its rotated pair; the scan's own fp16 operands
    add less than another 2^-8 of it."""
    b, L, H, P, G, N = 1, 200, 4, 64, 1, 128
    g = torch.Generator().manual_seed(4)
    xs = torch.randn(b, L, H, P, generator=g).to(BF).cuda()
    B, C = (torch.randn(b, L, G, N, generator=g).to(BF).cuda() for _ in range(2))
    one, inv = torch.ones(N).cuda(), (10000.0 ** (-torch.arange(N // 2) / (N / 2))).cuda()
    dt_raw, A = torch.randn(b, L, H, generator=g).cuda(), -torch.ones(H).cuda()
    bias, D = torch.full((H,), -3.0).cuda(), torch.zeros(H).cuda()
    ys = []
    for first in (0, 777777):
        pos = (first + torch.arange(L, dtype=torch.int32))[None].cuda()
        Bn, Cn = ssd.bc_norm_rotate_fwd(B, C, one, one, inv, positions=pos)
        ys.append(ssd.chunk_scan_fwd(xs, dt_raw, bias, A, Bn, Cn, D)[0].cpu().double())
    pair = lambda t: torch.hypot(t[..., :64].float(), t[..., 64:].float()).repeat(1, 1, 1, 2)  # noqa: E731
    size = ssd.chunk_scan_fwd(xs.float().abs(), dt_raw, bias, A, pair(Bn), pair(Cn), D)[0].cpu().double()
    assert ((ys[0] - ys[1]).abs() <= 5 * 2.0 ** -8 * size).all()
    assert (ys[0] - ys[1]).abs().max() > 0 and ys[0].abs().max() > 1


def test_operators_on_streams_of_their_own_at_once():
    """Projections of both types (tensor memory, pairs of CTAs, early-started
    launches), the gated recurrence (tiles that wait for others), the norm
    and the scan, each on its stream with its own workspace, over and over: the bits of calls alone."""
    g = torch.Generator().manual_seed(17)
    randn = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    bf = torch.bfloat16
    xs, ws, dys = randn(700, 1100), randn(900, 1100), randn(700, 900)
    xb, wb, dyb = randn(2000, 768).to(bf), randn(1536, 768).to(bf), randn(2000, 1536).to(bf)
    v, gates, lam = randn(1, 5000, 256).to(bf), randn(1, 5000, 512).to(bf), torch.full((256,), -4.0).cuda()
    B, C, dB, dC = (randn(2, 500, 4, 128).to(bf) for _ in range(4))
    w, inv = torch.ones(128).cuda(), torch.rand(64, generator=g).cuda()

    def gated():
        y, fin, st = ssd.gated_scan_fwd_states(v, gates[..., :256], gates[..., 256:], lam)
        d = ssd.gated_scan_bwd(v, gates[..., :256], gates[..., 256:], lam, st, v)
        return [y, fin] + [d[k] for k in ("x", "r_raw", "g_raw", "lam")]

    def norm():
        d = ssd.bc_norm_rotate_bwd(B, C, w, w, inv, dB, dC)
        return list(ssd.bc_norm_rotate_fwd(B, C, w, w, inv)) + [d[k] for k in sorted(d)]

    def scan():
        x = v[..., :128].reshape(1, 5000, 2, 64).contiguous()
        b = torch.tanh(B[0].float()).to(bf).reshape(1, 500, 4, 128)[:, :, :1].repeat(1, 10, 1, 1).contiguous()
        dt, bias, a, d = torch.zeros(1, 5000, 2).cuda(), torch.full((2,), -3.0).cuda(), torch.full((2,), -1.0).cuda(), torch.ones(2).cuda()
        return list(ssd.chunk_scan_fwd(x, dt, bias, a, b, b, d, chunk_size=128))

    calls = [gated, norm, scan,
             lambda: [ssd.linear_fwd(xs, ws, activation="gelu")] + list(ssd.linear_bwd(xs, ws, dys).values()),
             lambda: [ssd.linear_fwd(xb, wb, activation="silu"), ssd.linear_fwd(xb, wb, out_dtype=torch.float32)] +
             list(ssd.linear_bwd(xb, wb, dyb, preact=dyb, activation="silu", wide_dz=True).values())]
    want = [f() for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        got = []
        for f, s in zip(calls, streams):
            with torch.cuda.stream(s):
                got.append(f())
        torch.cuda.synchronize()
        for p, q in zip(want, got):
            assert all(torch.equal(a, b) for a, b in zip(p, q))
