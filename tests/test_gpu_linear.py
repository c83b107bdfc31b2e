"""GPU parity of the projections with their 64-bit form."""
import math

import pytest
import torch

import operator_refs as refs
from state_space_sequence_scan_b200 import ssd

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32


def make(M, N, K, dtype, seed, bias=True, residual=True, out=None):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g).to(dtype).cuda()
    w = (torch.randn(N, K, generator=g) / math.sqrt(K)).to(dtype).cuda()
    b = torch.randn(N, generator=g).cuda() if bias else None
    r = torch.randn(M, N, generator=g).to(out or dtype).cuda() if residual else None
    dy = torch.randn(M, N, generator=g).to(dtype).cuda()
    return x, w, b, r, dy


def run_all(M, N, K, dtype, act, bias=True, residual=True, out=None, seed=1):
    what = "linear %s " % ((M, N, K, dtype, act),)
    x, w, b, r, dy = make(M, N, K, dtype, seed, bias, residual, out)
    y, z = ssd.linear_fwd_preact(x, w, bias=b, residual=r, activation=act, out_dtype=out)
    ref, err, zr, zerr = refs.linear(x, w, b, r, act)
    refs.check(y, ref, err, what + "out")
    refs.check(z, zr, zerr, what + "preact")
    assert torch.equal(y, ssd.linear_fwd(x, w, bias=b, residual=r, activation=act, out_dtype=out))
    d = ssd.linear_bwd(x, w, dy, preact=z, activation=act)
    for k, (v, e) in refs.linear_bwd(x, w, dy, z, act).items():
        refs.check(d[k], v, e, what + "d" + k)


# one row to several tiles of rows; widths and depths off and on every tile edge
CASES = [(1, 8, 8), (1, 1, 1), (1, 2560, 512), (3, 24, 40), (4, 130, 264), (7, 129, 127), (16, 768, 1536), (17, 256, 64), (31, 33, 65),
         (64, 512, 256), (65, 100, 72), (127, 128, 128), (128, 129, 200), (129, 264, 333), (200, 1001, 771), (256, 512, 512),
         (257, 513, 520), (300, 3352, 96), (512, 96, 2048), (1000, 72, 1000), (1023, 768, 24)]


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "M%d_N%d_K%d" % c)
def test_linear_parity(case, dtype):
    M, N, K = case
    act = ("none", "silu", "gelu")[(M + N + K) % 3]
    run_all(M, N, K, dtype, act, seed=M + N + K)


@pytest.mark.parametrize("dtype,out", [(FP, None), (BF, None), (BF, FP)])
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("M", [5, 150])
def test_linear_epilogues(M, bias, residual, act, dtype, out):
    run_all(M, 136, 200, dtype, act, bias, residual, out, seed=M)


@pytest.mark.parametrize("dtype", [FP, BF])
def test_linear_activation_over_its_range(dtype):
    """An identity product makes the output the activation of its input, from
    -100 to 100; infinities go through as the formulas have them."""
    v = torch.linspace(-100, 100, 128 * 60).reshape(60, 128).to(dtype).cuda()
    eye = torch.eye(128).to(dtype).cuda()
    for act in ("silu", "gelu"):
        y = ssd.linear_fwd(v, eye, activation=act)
        ref, err, _, _ = refs.linear(v, eye, None, None, act)
        refs.check(y, ref, err + 1e-36, act)
        d = ssd.linear_bwd(v, eye, torch.ones_like(v), preact=v, activation=act, want_dweight=False)
        want = refs.linear_bwd(v, eye, torch.ones_like(v), v, act)["x"]
        refs.check(d["x"], want[0], want[1] + 1e-36, act + " slope")
        assert d["weight"] is None


@pytest.mark.parametrize("dtype", [FP, BF])
def test_linear_bad_rows_stay_alone(dtype):
    """NaN in a row of x reaches its own row of the output only, also where
    tiles are padded; a NaN channel of the weight its own column."""
    x, w, b, r, dy = make(130, 200, 100, dtype, 3)
    want = ssd.linear_fwd(x, w, bias=b, residual=r, activation="silu")
    x[77] = math.nan
    got = ssd.linear_fwd(x, w, bias=b, residual=r, activation="silu")
    keep = torch.arange(130) != 77
    assert torch.isnan(got[77]).all() and torch.equal(want.cpu()[keep], got.cpu()[keep])
    x[77] = 0
    want = ssd.linear_fwd(x, w, bias=b, residual=r)
    w[199] = math.inf
    got = ssd.linear_fwd(x, w, bias=b, residual=r)
    assert torch.equal(want[:, :199], got[:, :199]) and not torch.isfinite(got[:, 199]).any()


@pytest.mark.parametrize("dtype", [FP, BF])
def test_linear_leading_axes_and_in_place_residual(dtype):
    x, w, b, r, dy = make(60, 72, 64, dtype, 4)
    want = ssd.linear_fwd(x, w, bias=b, residual=r, activation="gelu")
    got = ssd.linear_fwd(x.view(3, 4, 5, 64), w, bias=b, residual=r.view(3, 4, 5, 72), activation="gelu")
    assert torch.equal(got.view(60, 72), want)
    d, e = ssd.linear_bwd(x, w, dy), ssd.linear_bwd(x.view(3, 20, 64), w, dy.view(3, 20, 72))
    assert torch.equal(d["x"], e["x"].view(60, 64)) and torch.equal(d["weight"], e["weight"])
    assert ssd.linear_fwd(x[0], w, bias=b).shape == (72,)
    # out may be the residual's own memory
    lib = ssd.load_library()
    ws = torch.empty(ssd.linear_workspace_size(60, 72, 64, dtype), dtype=torch.uint8, device="cuda")
    c = r.clone()
    st = lib.ssd_linear_fwd(x.data_ptr(), w.data_ptr(), b.data_ptr(), c.data_ptr(), c.data_ptr(), None, 60, 72, 64, 2,
                            ssd.DTYPES[dtype], ssd.DTYPES[dtype], ws.data_ptr(), ws.numel(),
                            torch.cuda.current_stream().cuda_stream)
    assert st == 0 and torch.equal(c, want)


@pytest.mark.parametrize("dtype", [FP, BF])
def test_linear_no_rows(dtype):
    x, w, b, r, dy = make(0, 24, 40, dtype, 5)
    assert ssd.linear_fwd(x, w, bias=b).shape == (0, 24)
    d = ssd.linear_bwd(x, w, dy)
    assert d["x"].shape == (0, 40) and d["weight"].abs().max() == 0 and d["bias"].abs().max() == 0


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("shape", [(5, 264, 520), (300, 520, 264), (257, 129, 65)])
def test_linear_same_bits_stream_graph_workspace(shape, dtype):
    M, N, K = shape
    x, w, b, r, dy = make(M, N, K, dtype, 6)
    n, nb = ssd.linear_workspace_size(M, N, K, dtype), ssd.linear_workspace_size(M, N, K, dtype, backward=True)
    wf = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    wb = torch.full((nb,), 255, dtype=torch.uint8, device="cuda")

    def both(own=True):
        y, z = ssd.linear_fwd_preact(x, w, bias=b, residual=r, activation="silu", workspace=wf if own else None)
        d = ssd.linear_bwd(x, w, dy, preact=z, activation="silu", workspace=wb if own else None)
        return [y, z] + [d[k] for k in ("x", "weight", "bias")]

    want = both()
    assert ssd.read_device_status(wf) == 0 and ssd.read_device_status(wb) == 0
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = both(own=False)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = both()
    x.mul_(0.5)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(out, both()))
    with pytest.raises(ssd.SSDError):
        ssd.linear_fwd(x, w, workspace=wf[:n - 1])
    with pytest.raises(ssd.SSDError):
        ssd.linear_bwd(x, w, dy, workspace=wb[:nb - 1])


def test_linear_wanted_gradients_alone():
    x, w, b, r, dy = make(200, 136, 72, BF, 7)
    z = ssd.linear_fwd_preact(x, w, bias=b, activation="gelu")[1]
    full = ssd.linear_bwd(x, w, dy, preact=z, activation="gelu")
    for k in ("x", "weight", "bias"):
        d = ssd.linear_bwd(x, w, dy, preact=z, activation="gelu", want_dx=k == "x", want_dweight=k == "weight",
                           want_dbias=k == "bias")
        assert torch.equal(d[k], full[k]) and sum(v is not None for v in d.values()) == 1
    assert all(v is None for v in ssd.linear_bwd(x, w, dy, want_dx=False, want_dweight=False, want_dbias=False).values())


def test_linear_refuses():
    x, w, b, r, dy = make(4, 24, 40, BF, 8)
    for k, f in enumerate([
            lambda: ssd.linear_fwd(x[:, :32], w), lambda: ssd.linear_fwd(x, w.float()), lambda: ssd.linear_fwd(x, w, bias=b.bfloat16()),
            lambda: ssd.linear_fwd(x, w, residual=r[:2]), lambda: ssd.linear_fwd(x, w, residual=r, out_dtype=FP),
            lambda: ssd.linear_fwd(x, w, activation="tanh"), lambda: ssd.linear_fwd(x, w, out_dtype=torch.float16),
            lambda: ssd.linear_fwd(x.half(), w.half()), lambda: ssd.linear_fwd(x.t(), w[:, :4]),
            lambda: ssd.linear_fwd(x, w.cpu()), lambda: ssd.linear_bwd(x, w, dy, activation="silu"),
            lambda: ssd.linear_bwd(x, w, dy.float()), lambda: ssd.linear_bwd(x, w, dy[:2])]):
        with pytest.raises(ValueError):
            f()
            pytest.fail("call %d was taken" % k)
    with pytest.raises(ssd.SSDError):                       # an offset of one element: rows not 16-byte aligned
        ssd.linear_fwd(torch.zeros(4 * 40 + 1, dtype=BF, device="cuda")[1:].view(4, 40), w)
    with pytest.raises(ssd.SSDError):
        ssd.linear_fwd(x.float(), w.float(), out_dtype=BF)


# few rows (up to 8, 16, 32 and one more), long and short depths, rows that start on 16 bytes, on pairs and on single elements
@pytest.mark.parametrize("M", [1, 8, 9, 16, 32, 33])
@pytest.mark.parametrize("N,K", [(48, 4096), (40, 5118), (33, 4099), (257, 514), (1001, 31)])
def test_linear_few_rows(M, N, K):
    run_all(M, N, K, BF, ("none", "silu", "gelu")[M % 3], bias=M % 2 == 0, residual=N % 2 == 0, seed=M + N)


# fp32 products of both tile sizes, in one and in several parts of k
@pytest.mark.parametrize("M,N,K", [(640, 1300, 200), (65, 63, 1500), (1100, 1200, 130)])
def test_linear_f32_tiles(M, N, K):
    run_all(M, N, K, FP, "silu", seed=K)


# fp32 products large enough for the tensor cores (three bf16 parts an operand): depths within, at and beyond a segment of 512 and
# a stage of 64, odd sizes
@pytest.mark.parametrize("M,N,K", [(700, 1100, 1500), (513, 1025, 512), (1000, 777, 1027), (2000, 520, 65), (257, 4000, 600)])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_linear_f32_in_parts(M, N, K, act):
    run_all(M, N, K, FP, act, bias=act == "gelu", residual=act == "gelu", seed=K)


def test_linear_f32_in_parts_keeps_every_value():
    """Values at the ends of float32's range and special ones: an infinity or
    NaN shows where a chain of fp32 fma would show it, and nowhere else; the
    largest float does not become an infinity; small ones keep their bits."""
    M, N, K = 900, 1000, 1100
    x, w, _, _, dy = make(M, N, K, FP, 77)
    w = torch.where(w.abs() < 1e-3, torch.full_like(w, 1e-3), w)
    x[3, 5], x[10, 700], x[11, 9], x[12, 1] = math.inf, -math.inf, math.nan, torch.finfo(FP).max
    w[7, 8], w[9, 30] = math.inf, math.nan
    x[20] *= 1e-30
    w[21] = 2.0 ** torch.arange(K).remainder(24).sub(12).float()   # sums that need more than 8 bits of each value
    x[22] = 1 + 2.0 ** -23
    ref, err, _, _ = refs.linear(x, w)
    refs.check(ssd.linear_fwd(x, w), ref, err, "special values")
    fine = torch.isfinite(dy)
    assert fine.all()
    d = ssd.linear_bwd(x, w, dy, want_dbias=False)
    for k, (v, e) in refs.linear_bwd(x, w, dy).items():
        if k != "bias":
            # the largest float times |dy| > 1 lies beyond float32: its rounding is an infinity, whatever computes it
            refs.check(d[k], v.to(FP), e, "special values d" + k)


@pytest.mark.parametrize("M,N,K,dtype", [(700, 1100, 1500, FP), (128, 640, 4096, BF), (40, 200, 333, BF)])
def test_linear_chains_captured_back_to_back(M, N, K, dtype):
    """Launches that start under the end of the one before, several calls in a
    row on one workspace, captured and replayed on new inputs, and on a stream
    of their own: the bits of separate calls."""
    sets = [make(M, N, K, dtype, seed=200 + k) for k in range(2)]
    one = [t.clone() for t in sets[0]]
    ws = torch.full((max(ssd.linear_workspace_size(M, N, K, dtype), ssd.linear_workspace_size(M, N, K, dtype, True)),), 255,
                    dtype=torch.uint8, device="cuda")

    def go(x, w, b, r, dy, workspace=None):
        y, z = ssd.linear_fwd_preact(x, w, bias=b, residual=r, activation="silu", workspace=workspace)
        d = ssd.linear_bwd(x, w, dy, preact=z, activation="silu", workspace=workspace)
        y2 = ssd.linear_fwd(x, w, residual=y, workspace=workspace)
        return [y, z, d["x"], d["weight"], d["bias"], y2]

    want = [go(*s) for s in sets]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        go(*one, workspace=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got = go(*one, workspace=ws)
    torch.cuda.synchronize()
    for k in (1, 0, 1):
        for t, v in zip(one, sets[k]):
            t.copy_(v)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want[k])), k
    assert ssd.read_device_status(ws) == 0


@pytest.mark.parametrize("M", [60, 700], ids=["cores", "parts"])
def test_linear_f32_activations_to_their_last_bits(M):
    """float32 results hold the activation to a few roundings of itself over
    its whole range, not of its argument.  The counts, in units of 2^-24 of
    the result: the exponential 4 (two units in the last place), 1 + e, the
    quotient and the product one each, the argument -z^2/2 two roundings of
    itself, erf 4; then half a step of what each is added to."""
    z = torch.linspace(-80, 80, 640).repeat(M, 1).cuda()
    eye = torch.eye(640).cuda()
    y = ssd.linear_fwd(z, eye, activation="silu")
    f = z.cpu().double()
    s, t = torch.sigmoid(f), torch.sigmoid(-f)
    refs.check(y, f * s, refs.U * 8 * (f * s).abs(), "silu")
    ones = torch.ones_like(z)
    d = ssd.linear_bwd(z, eye, ones, preact=z, activation="silu", want_dweight=False)["x"]
    refs.check(d, s * (1 + f * t), refs.U * 8 * s * (1 + 2 * f.abs() * t), "silu slope")
    d = ssd.linear_bwd(z, eye, ones, preact=z, activation="gelu", want_dweight=False)["x"]
    want = refs.act_slope(f, "gelu")
    bell = f.abs() * torch.exp(-f * f / 2) / math.sqrt(2 * math.pi)
    refs.check(d, want, refs.U * (4 + bell * (f * f + 10)), "gelu slope")


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("M,N,K", [(4194240 + 77, 8, 8), (4200000, 3, 9), (9, 4194240 + 130, 8)])
def test_linear_millions_of_rows_and_outputs(M, N, K, dtype):
    """More rows or outputs than 65535 tiles of 64, both directions."""
    run_all(M, N, K, dtype, "silu", seed=3)


def takes_parts(M, N, K, backward=False):
    """Whether fp32 products of this size run in bf16 parts: those need their room."""
    return ssd.linear_workspace_size(M, N, K, FP, backward) >= 8 * (M * K + N * K)


def some_floats(M, K, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(M, K, generator=g) * 2.0 ** torch.randint(-60, 60, (M, K), generator=g)).cuda()


@pytest.mark.parametrize("M,N,K", [(1024, 1024, 1024), (900, 1100, 1100), (1500, 1030, 1030)])
def test_linear_f32_in_parts_products_with_one(M, N, K):
    """An identity on either side gives the other operand back, bit for bit:
    all three parts of a value arrive, in the forward and in both products of
    the backward."""
    assert takes_parts(M, N, K) and takes_parts(N, M, M) and takes_parts(K, K, K, True)
    x, eye = some_floats(M, K, 1), torch.eye(N, K).cuda()
    assert torch.equal(ssd.linear_fwd(x, eye), torch.nn.functional.pad(x, (0, N - K)))
    w, eye = some_floats(N, M, 2), torch.eye(M).cuda()
    assert torch.equal(ssd.linear_fwd(eye, w), w.t())
    v, eye = some_floats(K, K, 3), torch.eye(K).cuda()
    assert torch.equal(ssd.linear_bwd(v, eye, v, want_dweight=False)["x"], v)
    assert torch.equal(ssd.linear_bwd(eye, v, eye, want_dweight=False)["x"], v)
    assert torch.equal(ssd.linear_bwd(v, eye, eye, want_dx=False)["weight"], v)
    assert torch.equal(ssd.linear_bwd(eye, eye, v, want_dx=False)["weight"], v.t())


@pytest.mark.parametrize("M,N,K", [(1024, 1024, 1024), (1100, 900, 1027)])
def test_linear_f32_in_parts_single_products(M, N, K):
    """One product a sum: of its nine partial products the three left out are
    at most 2^-24 of it, and the tensor cores cut its last addition by less
    than 2^-23, so 2^-22 holds.  (hi mid is up to 2^-8 of it, mid mid and hi lo
    about 2^-18: none can be missing.)"""
    assert takes_parts(M, N, K)
    g = torch.Generator().manual_seed(5)
    at = torch.randint(0, K, (M,), generator=g)
    v = torch.randn(M, generator=g)
    v[::7] = 1.0038986                    # of all values the one whose parts leave most out
    x, w = torch.zeros(M, K), torch.randn(N, K, generator=g)
    w[::5] = 1.0038986
    x[torch.arange(M), at] = v
    ref = v.double()[:, None] * w.t().double()[at]
    got = ssd.linear_fwd(x.cuda(), w.cuda()).cpu().double()
    assert ((got - ref).abs() <= 2.0 ** -22 * ref.abs()).all()
    got = ssd.linear_bwd(torch.zeros(M, N).cuda(), w.t().contiguous().cuda(), x.cuda(), want_dweight=False)["x"].cpu().double()
    assert takes_parts(M, K, N, True) and ((got - ref).abs() <= 2.0 ** -22 * ref.abs()).all()
    got = ssd.linear_bwd(w.t().contiguous().cuda(), torch.zeros(M, N).cuda(), x.t().contiguous().cuda(), want_dx=False)["weight"].cpu().double()
    assert takes_parts(K, M, N, True) and ((got - ref).abs() <= 2.0 ** -22 * ref.abs()).all()


def test_linear_f32_in_parts_long_sums():
    """Random sums of 6144.  The tensor cores cut a sum at every step of 16 k,
    by half of 2^-23 of it on average: 32 steps at full size a segment of 512,
    its size two thirds of the end's on average over them, are 1.3e-6; 12
    segments are added with 2^-24 each, the partial products left out are
    2^-24 at most.  So 2e-6 in the mean square; sums of all k in one would be
    12 times as far off in their bias."""
    M, N, K = 1024, 1024, 6144
    assert takes_parts(M, N, K)
    g = torch.Generator().manual_seed(9)
    x, w = torch.randn(M, K, generator=g), torch.randn(N, K, generator=g)
    ref = x.double() @ w.double().t()
    off = ssd.linear_fwd(x.cuda(), w.cuda()).cpu().double() - ref
    assert float(off.square().mean().sqrt() / ref.square().mean().sqrt()) <= 2e-6
    d = ssd.linear_bwd(x.t().contiguous().cuda(), torch.zeros(M, M).cuda(), w.t().contiguous().cuda(), want_dx=False)["weight"]
    off = d.cpu().double() - ref.t()
    assert float(off.square().mean().sqrt() / ref.square().mean().sqrt()) <= 2e-6


# both sides of the rule that gives few rows 16 warps: up to 8 rows on 16 bytes, k from 1024 (and outputs up to 6400) or from 4096
@pytest.mark.parametrize("M", [8, 9])
@pytest.mark.parametrize("N,K", [(40, 1016), (40, 1024), (40, 1026), (6400, 1024), (6416, 1024), (6416, 4096), (6416, 4088)])
@pytest.mark.parametrize("out", [None, FP])
def test_linear_few_rows_of_either_warp_count(M, N, K, out):
    run_all(M, N, K, BF, "silu", out=out, seed=M + K)


def wide_bwd(x, w, dy, z, activation):
    """{name: (value, bound)} with dz in two bfloat16 parts: the first leaves at
    most 2^-8 of a value, the second 2^-8 of that; and two products an element."""
    out = refs.linear_bwd(x, w, dy, z, activation)
    f = torch.float64
    x, w, dy = (v.cpu().to(f) for v in (x, w, dy))
    dz = dy * refs.act_slope(z.cpu().to(f), activation)
    perr = 60 * refs.U * dy.abs() + 2.0 ** -16 * dz.abs()
    M, N = dz.shape
    out["x"] = (out["x"][0], perr @ w.abs() + 2 * N * refs.U * 2 * (dz.abs() @ w.abs()))
    out["weight"] = (out["weight"][0], perr.T @ x.abs() + 2 * M * refs.U * 2 * (dz.abs().T @ x.abs()))
    return out


# one tile and several, one and several parts of k, both widths, rows that are padded, rows that end inside a stage
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,N,K", [(1, 8, 8), (5, 264, 520), (65, 100, 72), (127, 129, 65), (300, 520, 264), (1000, 768, 1536), (2049, 1001, 771)])
def test_linear_wide_dz(M, N, K, act):
    x, w, b, r, dy = make(M, N, K, BF, M + K)
    z = ssd.linear_fwd_preact(x, w, bias=b, activation=act)[1]
    n = ssd.linear_workspace_size(M, N, K, BF, backward=True, wide_dz=True)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")     # (bf16 NaN where nothing is written)
    d = ssd.linear_bwd(x, w, dy, preact=z, activation=act, wide_dz=True, workspace=ws)
    assert ssd.read_device_status(ws) == 0
    for k, (v, e) in wide_bwd(x, w, dy, z, act).items():
        refs.check(d[k], v, e, "wide d" + k)
    again = ssd.linear_bwd(x, w, dy, preact=z, activation=act, wide_dz=True)
    narrow = ssd.linear_bwd(x, w, dy, preact=z, activation=act)
    assert all(torch.equal(d[k], again[k]) for k in d) and torch.equal(d["bias"], narrow["bias"])
    for k in ("x", "weight", "bias"):
        one = ssd.linear_bwd(x, w, dy, preact=z, activation=act, wide_dz=True, want_dx=k == "x", want_dweight=k == "weight",
                             want_dbias=k == "bias")
        assert torch.equal(one[k], d[k])
    if n > 256:
        with pytest.raises(ssd.SSDError):
            ssd.linear_bwd(x, w, dy, preact=z, activation=act, wide_dz=True, workspace=ws[:n - 1])


def test_linear_wide_dz_is_nearer():
    """Against 64 bits: with dz whole only the stores' roundings are left (2^-8
    at most, 0.0017 in the mean square of random values); rounded, dz adds as much again."""
    x, w, b, r, dy = make(1500, 1000, 800, BF, 9)
    z = ssd.linear_fwd_preact(x, w, bias=b, activation="silu")[1]
    ref = refs.linear_bwd(x, w, dy, z, "silu")
    off = {}
    for wide in (False, True):
        d = ssd.linear_bwd(x, w, dy, preact=z, activation="silu", wide_dz=wide)
        off[wide] = [float((d[k].cpu().double() - ref[k][0]).square().mean().sqrt() / ref[k][0].square().mean().sqrt()) for k in ("x", "weight")]
    stored = [float((ref[k][0].bfloat16().double() - ref[k][0]).square().mean().sqrt() / ref[k][0].square().mean().sqrt()) for k in ("x", "weight")]
    assert all(o <= 1.01 * s for o, s in zip(off[True], stored)) and all(o >= 1.2 * s for o, s in zip(off[False], stored))


@pytest.mark.parametrize("dtype,act", [(FP, "silu"), (FP, "none"), (BF, "none")])
@pytest.mark.parametrize("shape", [(40, 72, 64), (700, 1100, 1500), (130, 129, 200)])
def test_linear_wide_dz_where_dz_is_whole(shape, dtype, act):
    """The flag changes nothing there."""
    x, w, b, r, dy = make(*shape, dtype, 11)
    z = ssd.linear_fwd_preact(x, w, bias=b, activation=act)[1]
    p, q = (ssd.linear_bwd(x, w, dy, preact=z, activation=act, wide_dz=wide) for wide in (False, True))
    assert all(torch.equal(p[k], q[k]) for k in p)


def test_linear_wide_dz_bad_values_and_graph():
    """A NaN or an infinity in a row of dy reaches that row of dx only; captured and replayed on new inputs."""
    x, w, b, r, dy = make(300, 200, 136, BF, 12)
    z = ssd.linear_fwd_preact(x, w, bias=b, activation="silu")[1]
    go = lambda: ssd.linear_bwd(x, w, dy, preact=z, activation="silu", wide_dz=True)  # noqa: E731
    want = go()
    dy[77, 3], dy[78, 5] = math.nan, math.inf
    got = go()
    keep = torch.ones(300, dtype=torch.bool)
    keep[77] = keep[78] = False
    assert torch.equal(got["x"].cpu()[keep], want["x"].cpu()[keep]) and not torch.isfinite(got["x"][77:79]).any()
    cols = torch.ones(200, dtype=torch.bool)
    cols[3] = cols[5] = False
    assert torch.equal(got["weight"].cpu()[cols], want["weight"].cpu()[cols])
    dy[77, 3] = dy[78, 5] = 1.0
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = go()
    dy.mul_(0.75)
    x.add_(0.5)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[k], v) for k, v in go().items())


def off_by(got, ref):
    return float((got.double() - ref).square().mean().sqrt() / ref.square().mean().sqrt())


@pytest.mark.parametrize("M,N,K", [(300, 520, 8192), (40, 200, 8000), (1024, 2560, 4096), (8, 2560, 8192), (20, 513, 32767)])
@pytest.mark.parametrize("positive", [False, True])
def test_linear_bf16_long_sums_in_float32(M, N, K, positive):
    """bf16 products are exact, and a float32 result holds their sum to a few
    of its own roundings.  The tensor cores cut a sum at each step of 16 k, by
    half of 2^-23 of it on average: 64 steps a segment of up to 1024, the sum
    at half (positive values) or two thirds of its end on average, are 2.5e-6
    at most; the segments are added with 2^-24 each, at random.  (Few rows: 32
    steps.)"""
    g = torch.Generator().manual_seed(K + M)
    x, w = torch.randn(M, K, generator=g).bfloat16().cuda(), torch.randn(N, K, generator=g).bfloat16().cuda()
    if positive:
        x, w = x.abs(), w.abs()
    ref = x.double() @ w.double().t()
    assert off_by(ssd.linear_fwd(x, w, out_dtype=FP), ref) <= 2.6e-6
    y = torch.randn(M, N, generator=g).cuda()
    z = ssd.linear_fwd(x, w, residual=y, bias=y[0], out_dtype=FP)
    assert off_by(z, ref + y.double() + y[0].double()) <= 2.6e-6


def test_linear_bf16_gradient_over_many_rows():
    """A weight's gradient over 160 000 rows of positive values: within 2 percent of what the store's rounding leaves."""
    M, N, K = 160001, 2560, 2560
    g = torch.Generator(device="cuda").manual_seed(3)
    x, dy = (torch.rand(M, n, generator=g, device="cuda").bfloat16() for n in (K, N))
    ref = dy[:, :128].double().t() @ x.double()
    w = torch.zeros(N, K, dtype=BF, device="cuda")
    d = ssd.linear_bwd(x, w, dy, want_dx=False, want_dbias=False)["weight"][:128]
    assert off_by(d, ref) <= 1.02 * off_by(ref.bfloat16(), ref)
    z = torch.full((M, N), 20.0, dtype=BF, device="cuda")       # silu's slope is 1 there
    e = ssd.linear_bwd(x, w, dy, preact=z, activation="silu", want_dx=False, want_dbias=False, wide_dz=True)["weight"][:128]
    assert off_by(e, ref) <= 1.02 * off_by(ref.bfloat16(), ref)


def test_linear_f32_in_parts_down_to_their_last_bit():
    """Three parts hold all bits of values from 2^-110 on; below, the last
    part's smallest number is 2^-133, so a value is off by 2^-134 at most."""
    assert takes_parts(1024, 1024, 1024)
    g, eye = torch.Generator().manual_seed(4), torch.eye(1024).cuda()
    for e in (-100, -109, -110, -111, -120, -126):
        x = ((1 + torch.rand(1024, 1024, generator=g)) * 2.0 ** e).cuda()
        off = max((ssd.linear_fwd(x, eye) - x).abs().max().item(), (ssd.linear_fwd(eye, x).t() - x).abs().max().item())
        assert off <= (0 if e >= -110 else 2.0 ** -134), e
