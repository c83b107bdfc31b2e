"""GPU parity of the norm and rotation of B and C with its 64-bit form."""
import math

import pytest
import torch

import operator_refs as refs
from state_space_sequence_scan_b200 import ssd

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32


def make(b, L, G, N, R, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    B, C, dB, dC = (torch.randn(b, L, G, N, generator=g).to(dtype).cuda() for _ in range(4))
    wB, wC = (1 + 0.1 * torch.randn(N, generator=g)).cuda(), (1 + 0.1 * torch.randn(N, generator=g)).cuda()
    j = torch.arange(R // 2, dtype=torch.float64)
    inv = (10000.0 ** (-2 * j / max(R, 1))).float().cuda() if R else None
    return B, C, dB, dC, wB, wC, inv


def run_all(shape, R, dtype, il, pos, seed=1, eps=1e-5, what=""):
    b, L, G, N = shape
    B, C, dB, dC, wB, wC, inv = make(b, L, G, N, R, dtype, seed)
    p = torch.arange(L).repeat(b, 1) if pos is None else pos
    gp = None if pos is None else pos.to(torch.int32).cuda()
    f = torch.zeros(0) if inv is None else inv
    Bo, Co = ssd.bc_norm_rotate_fwd(B, C, wB, wC, inv, positions=gp, eps=eps, interleaved=il)
    d = ssd.bc_norm_rotate_bwd(B, C, wB, wC, inv, dB, dC, positions=gp, eps=eps, interleaved=il)
    for v, w, o, g, k in ((B, wB, Bo, dB, "B"), (C, wC, Co, dC, "C")):
        ref, err = refs.norm_rotate(v, w, f, p, eps, il)
        refs.check(o, ref, err, what + k)
        (dv, dv_err), (dw, dw_err) = refs.norm_rotate_bwd(v, w, f, p, eps, il, g)
        refs.check(d[k], dv, dv_err, what + "d" + k)
        refs.check(d["weight_" + k], dw, dw_err, what + "dw" + k)


# widths: powers of two, other multiples of 16, odd multiples, odd, tiny and large
CASES = [(1, 1, 1, 128, 128), (2, 5, 1, 64, 64), (2, 3, 8, 128, 64), (1, 33, 3, 16, 16), (2, 7, 2, 256, 256),
         (1, 9, 2, 512, 128), (3, 4, 2, 96, 96), (2, 5, 3, 80, 40), (1, 6, 1, 112, 112), (2, 3, 2, 100, 50), (1, 5, 2, 7, 6),
         (1, 4, 1, 1, 0), (1, 3, 2, 2, 2), (1, 2, 1, 1000, 998), (2, 4, 2, 128, 0), (1, 4, 2, 48, 32), (1, 2, 1, 8192, 4096),
         (2, 300, 1, 128, 128), (2, 4, 5, 128, 128)]


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("il", [False, True], ids=["halves", "interleaved"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "b%d_L%d_G%d_N%d_R%d" % c)
def test_norm_rotate_parity(case, il, dtype):
    b, L, G, N, R = case
    g = torch.Generator().manual_seed(N + L)
    pos = torch.randint(0, 1 << 20, (b, L), generator=g) if L % 2 else None
    run_all((b, L, G, N), R, dtype, il, pos, seed=N, what="%s " % (case,))


@pytest.mark.parametrize("il", [False, True])
def test_far_and_negative_positions(il):
    """Every 32-bit position: the reduced angle is as exact at 2^31 - 1 as at
    0.  The form multiplies in 64 bits, where an angle of 2^31 is off by 2^-22;
    the kernel's turn, rounded to 2^-53 of itself, by as much: 4 units each of
    2^-24, on top of the 16 of the bound, that far out."""
    pos = torch.tensor([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, -(2 ** 30), 1000003]])
    b, L, G, N, R = 1, 8, 2, 128, 128
    B, C, dB, dC, wB, wC, inv = make(b, L, G, N, R, FP, 3)
    Bo, Co = ssd.bc_norm_rotate_fwd(B, C, wB, wC, inv, positions=pos.to(torch.int32).cuda(), interleaved=il)
    for v, w, o in ((B, wB, Bo), (C, wC, Co)):
        ref, err = refs.norm_rotate(v, w, inv, pos, 1e-5, il)
        refs.check(o, ref, err * (N / 2 + 26 + 8) / (N / 2 + 26), "far")


def test_frequencies_of_more_than_a_turn():
    """inv_freq is any number of radians per position, negative ones and whole
    turns among them."""
    B, C, dB, dC, wB, wC, _ = make(1, 6, 1, 16, 16, FP, 4)
    inv = torch.tensor([7.0, -1.0, 100.0, 2 * math.pi, math.pi, 0.0, -50.25, 1e-8]).cuda()
    Bo, _ = ssd.bc_norm_rotate_fwd(B, C, wB, wC, inv)
    ref, err = refs.norm_rotate(B, wB, inv, torch.arange(6)[None], 1e-5, False)
    refs.check(Bo, ref, err, "frequencies")


@pytest.mark.parametrize("dtype", [FP, BF])
def test_zero_rows_and_eps(dtype):
    """A row of zeros is normed to zeros; eps keeps its gradient finite."""
    B, C, dB, dC, wB, wC, inv = make(2, 3, 2, 64, 64, dtype, 5)
    B[:, 1] = 0
    for eps in (1e-5, 1e-12, 1.0):
        Bo, Co = ssd.bc_norm_rotate_fwd(B, C, wB, wC, inv, eps=eps)
        d = ssd.bc_norm_rotate_bwd(B, C, wB, wC, inv, dB, dC, eps=eps)
        assert Bo[:, 1].abs().max() == 0 and torch.isfinite(d["B"]).all()
        e32 = float(torch.tensor(eps, dtype=torch.float32))
        (dv, dv_err), _ = refs.norm_rotate_bwd(B, wB, inv, torch.arange(3).repeat(2, 1), e32, False, dB)
        refs.check(d["B"], dv, dv_err, "zero rows")


def test_bad_rows_stay_alone():
    B, C, dB, dC, wB, wC, inv = make(2, 40, 3, 128, 128, FP, 6)
    want = ssd.bc_norm_rotate_fwd(B, C, wB, wC, inv) + tuple(
        ssd.bc_norm_rotate_bwd(B, C, wB, wC, inv, dB, dC)[k] for k in "BC")
    B[1, 7, 1] = math.nan
    C[0, 3, 0, 5] = math.inf
    got = ssd.bc_norm_rotate_fwd(B, C, wB, wC, inv) + tuple(
        ssd.bc_norm_rotate_bwd(B, C, wB, wC, inv, dB, dC)[k] for k in "BC")
    for k, (p, q) in enumerate(zip(want, got)):
        keep = torch.ones(2, 40, 3, dtype=torch.bool)
        keep[(1, 7, 1) if k % 2 == 0 else (0, 3, 0)] = False
        assert torch.equal(p.cpu()[keep], q.cpu()[keep]), k


def test_many_rows_sum_in_order():
    """More rows than a launch has warps: the weights' gradients against the
    form (float32 running sums of a few rows each), the same bits twice."""
    run_all((3, 4001, 2, 32), 32, BF, False, None, seed=7, what="many rows ")
    B, C, dB, dC, wB, wC, inv = make(3, 4001, 2, 32, 32, BF, 8)
    p, q = (ssd.bc_norm_rotate_bwd(B, C, wB, wC, inv, dB, dC) for _ in range(2))
    assert all(torch.equal(p[k], q[k]) for k in p)


def test_empty_stream_graph_and_workspace():
    B, C, dB, dC, wB, wC, inv = make(2, 0, 2, 64, 64, FP, 9)
    Bo, Co = ssd.bc_norm_rotate_fwd(B, C, wB, wC, inv)
    assert Bo.shape == B.shape and ssd.bc_norm_rotate_bwd(B, C, wB, wC, inv, dB, dC)["weight_B"].abs().max() == 0
    B, C, dB, dC, wB, wC, inv = make(2, 50, 2, 64, 64, BF, 9)
    n = ssd.bc_norm_rotate_bwd_workspace_size(2, 50, 2, 64)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")

    def both():
        d = ssd.bc_norm_rotate_bwd(B, C, wB, wC, inv, dB, dC, workspace=ws)
        return list(ssd.bc_norm_rotate_fwd(B, C, wB, wC, inv)) + [d[k] for k in sorted(d)]

    want = both()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = both()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = both()
    B.mul_(0.5)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(out, both()))
    with pytest.raises(ssd.SSDError):
        ssd.bc_norm_rotate_bwd(B, C, wB, wC, inv, dB, dC, workspace=ws[:n - 1])


def test_norm_rotate_refuses():
    B, C, dB, dC, wB, wC, inv = make(2, 4, 2, 64, 64, FP, 10)
    for k, f in enumerate([
            lambda: ssd.bc_norm_rotate_fwd(B, C[:1], wB, wC, inv), lambda: ssd.bc_norm_rotate_fwd(B, C.bfloat16(), wB, wC, inv),
            lambda: ssd.bc_norm_rotate_fwd(B, C, wB[:5], wC, inv), lambda: ssd.bc_norm_rotate_fwd(B, C, wB, wC, torch.cat([inv, inv])),
            lambda: ssd.bc_norm_rotate_fwd(B, C, wB, wC, inv.double()), lambda: ssd.bc_norm_rotate_fwd(B, C, wB, wC, inv.cpu()),
            lambda: ssd.bc_norm_rotate_fwd(B.transpose(1, 2), C.transpose(1, 2), wB, wC, inv),
            lambda: ssd.bc_norm_rotate_fwd(B, C, wB, wC, inv, positions=torch.zeros(2, 4, dtype=torch.int64, device="cuda")),
            lambda: ssd.bc_norm_rotate_fwd(B.half(), C.half(), wB, wC, inv), lambda: ssd.bc_norm_rotate_bwd(B, C, wB, wC, inv, dB, dC[:1])]):
        with pytest.raises(ValueError):
            f()
            pytest.fail("call %d was taken" % k)
    with pytest.raises(ssd.SSDError):
        ssd.bc_norm_rotate_fwd(B, C, wB, wC, inv, eps=-1.0)


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("case", [(2, 9001, 1, 128, 128), (1, 5000, 3, 64, 32), (1, 1500, 2, 512, 512), (1, 40, 37, 256, 256),
                                  (1, 3000, 1, 248, 240)], ids=lambda c: "b%d_L%d_G%d_N%d_R%d" % c)
def test_norm_rotate_many_tokens(case, dtype):
    """More tokens than lane groups of a launch, so that each goes round; and
    many groups of few tokens, which are split."""
    b, L, G, N, R = case
    run_all((b, L, G, N), R, dtype, L % 3 == 0, None, seed=N + G, what="%s " % (case,))


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("case", [(1, 1, 1, 128, 128), (1, 1, 3, 64, 64), (2, 37, 5, 64, 32), (1, 3, 33, 256, 256), (1, 9, 3, 512, 128),
                                  (2, 4095, 2, 128, 64), (1, 5, 2, 100, 50)], ids=lambda c: "b%d_L%d_G%d_N%d_R%d" % c)
def test_no_eps_and_places_without_a_row(case, dtype):
    """eps 0 with no row of zeros: every value is finite, at sizes where lanes
    of a block's tail, of an item's last groups and of a last turn have no row."""
    b, L, G, N, R = case
    run_all((b, L, G, N), R, dtype, N % 3 == 0, None, seed=N + L, eps=0.0, what="eps 0 %s " % (case,))


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("il", [False, True], ids=["halves", "interleaved"])
@pytest.mark.parametrize("N,R", [(128, 64), (128, 0), (512, 128), (100, 50)])
def test_infinities_past_the_rotated_part_stay_alone(N, R, il, dtype):
    """Elements from rot_dim on have no partner: an infinite element, weight or
    gradient there shows in its own place (and, through the mean, as the
    formulas have it) and in no neighbour's."""
    b, L, G = 1, 5, 2
    last = N - 20
    for what in ("element", "weight", "gradient"):
        B, C, dB, dC, wB, wC, inv = make(b, L, G, N, R, dtype, 23)
        if what == "element":
            B[0, 2, 1, last] = math.inf
            C[0, 4, 0, last + 3] = -math.inf
        elif what == "weight":
            wB[last] = wC[last + 5] = math.inf
        else:
            dB[0, 1, 1, last] = math.inf
            dC[0, 3, 0, last + 3] = -math.inf
        p, f = torch.arange(L)[None], torch.zeros(0) if inv is None else inv
        Bo, Co = ssd.bc_norm_rotate_fwd(B, C, wB, wC, inv, interleaved=il)
        d = ssd.bc_norm_rotate_bwd(B, C, wB, wC, inv, dB, dC, interleaved=il)
        for v, w, o, g, k in ((B, wB, Bo, dB, "B"), (C, wC, Co, dC, "C")):
            ref, err = refs.norm_rotate(v, w, f, p, 1e-5, il)
            refs.check(o, ref, err, "%s %s" % (what, k))
            (dv, dv_err), (dw, dw_err) = refs.norm_rotate_bwd(v, w, f, p, 1e-5, il, g)
            refs.check(d["weight_" + k], dw, dw_err, "%s dw%s" % (what, k))
            if what != "weight":     # (an infinite weight makes a whole row's mean infinite)
                refs.check(d[k], dv, dv_err, "%s d%s" % (what, k))


# 1 / (2 pi) = floor(2^240 / (2 pi)) / 2^240, from 80 digits of pi
PI_80 = 31415926535897932384626433832795028841971693993751058209749445923078164062862089
INV_2PI = (10 ** 79 << 240) // (2 * PI_80)


def angles_reduced_exactly(pos, inv_freq):
    """position * inv_freq modulo a turn, in radians: the product and its
    reduction in whole numbers (the frequency as the fraction that it is),
    rounded to 64 bits at the end."""
    out = torch.empty(pos.numel(), inv_freq.numel(), dtype=torch.float64)
    for i, p in enumerate(pos.flatten().tolist()):
        for j, f in enumerate(inv_freq.tolist()):
            n, d = f.as_integer_ratio()
            t = (p * n * INV_2PI // d) % (1 << 240)
            out[i, j] = 2 * math.pi * (t if t < 1 << 239 else t - (1 << 240)) / float(1 << 240)
    return out.view(*pos.shape, -1)


@pytest.mark.parametrize("case", [(128, 24), (20, 20)], ids=["units", "other"])
@pytest.mark.parametrize("il", [False, True], ids=["halves", "interleaved"])
def test_large_frequencies_at_far_positions(il, case):
    """The reduced angle is right to 2^-32 of a turn (4 units of 2^-24 of a
    radian are 160 times that) for every position and frequencies up to 2^40
    radians per position: the bound is the one of near positions."""
    N, R = case
    inv = torch.tensor([1.0, -0.1, 7.0, 100.0, -1e4, 12345.678, 3e8, 1e12, 1e-8, -1e-5, 2 * math.pi, 0.7071][:R // 2]).cuda()
    pos = torch.tensor([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, -(2 ** 30) - 1, 1000003, 2147480011]])
    L = pos.shape[1]
    B, C, dB, dC, wB, wC, _ = make(1, L, 2, N, 0, FP, 31)
    p = pos.to(torch.int32).cuda()
    Bo, _ = ssd.bc_norm_rotate_fwd(B, C, wB, wC, inv, positions=p, interleaved=il)
    d = ssd.bc_norm_rotate_bwd(B, C, wB, wC, inv, dB, dC, positions=p, interleaved=il)
    ang = angles_reduced_exactly(pos, inv)[:, :, None]
    j = torch.arange(inv.numel())
    e0, e1 = (2 * j, 2 * j + 1) if il else (j, j + inv.numel())

    def turned(v, sign):
        c, s, out, size = torch.cos(ang), sign * torch.sin(ang), v.clone(), v.abs()
        out[..., e0], out[..., e1] = v[..., e0] * c - v[..., e1] * s, v[..., e1] * c + v[..., e0] * s
        size[..., e0] = size[..., e1] = v[..., e0].abs() + v[..., e1].abs()
        return out, size

    v, w, g = B.cpu().double(), wB.cpu().double(), dB.cpu().double()
    rs = 1 / torch.sqrt(v.square().mean(-1, keepdim=True) + float(torch.tensor(1e-5)))
    ref, size = turned(v * rs * w, 1)
    refs.check(Bo, ref, refs.U * (N / 2 + 26) * size, "far, large")
    dn, size = turned(g, -1)
    n = v * rs
    m, msize = (dn * w * n).mean(-1, keepdim=True), (size * w.abs() * n.abs()).mean(-1, keepdim=True)
    refs.check(d["B"], rs * (dn * w - n * m), refs.U * rs * ((N / 2 + 30) * size * w.abs() + (2 * N + 60) * n.abs() * msize), "far, large dB")
