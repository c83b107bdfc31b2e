"""GPU parity of the gated recurrence (scan, backward, step) with its 64-bit
form, within the bounds derived there, and what must hold exactly."""
import math

import pytest
import torch

import operator_refs as refs
from state_space_sequence_scan_b200 import ssd

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32


def make(b, L, D, dtype, seed, halves=True, decay=(0.9, 0.999)):
    """x, r_raw, g_raw (halves of one tensor, or apart), lam with a in `decay`
    at an open gate, init; on the GPU."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(b, L, D, generator=g).to(dtype)
    gates = torch.randn(b, L, 2 * D, generator=g).to(dtype).cuda()
    r, i = gates[..., :D], gates[..., D:]
    if not halves:
        r, i = r.contiguous(), i.contiguous()
    a = decay[0] + (decay[1] - decay[0]) * torch.rand(D, generator=g, dtype=torch.float64)
    lam = torch.log(torch.expm1(-torch.log(a) / 8.0)).float()
    return x.cuda(), r, i, lam.cuda(), torch.randn(b, D, generator=g).cuda()


def ids_of(b, L, seed, chance=0.05):
    g = torch.Generator().manual_seed(seed)
    return torch.cumsum(torch.rand(b, L, generator=g) < chance, 1).to(torch.int32)


def grads_in(b, L, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(b, L, D, generator=g).to(dtype).cuda(), torch.randn(b, D, generator=g).cuda()


def run_all(x, r, i, lam, init, ids, dy, dfin, what, **kw):
    """Forward with states and backward against the form."""
    b, L, D = x.shape
    y, fin, states = ssd.gated_scan_fwd_states(x, r, i, lam, init_state=init, seq_idx=ids, **kw)
    d = ssd.gated_scan_bwd(x, r, i, lam, states, dy, dfinal_state=dfin, init_state=init, seq_idx=ids, **kw)
    h, err, parts = refs.gated(x, r, i, lam, init, ids, kw.get("decay_scale", 8.0))
    refs.check(y, h, err, what + " y")
    refs.check(fin, h[:, -1], err[:, -1], what + " final")
    at = [min(64 * (c + 1), L) - 1 for c in range(states.shape[1])]
    refs.check(states, h[:, at], err[:, at], what + " states")
    for k, (v, e) in refs.gated_bwd(parts, dy, dfin).items():
        refs.check(d[k], v, e, "%s d%s" % (what, k))


# lengths around the 64-token chunks, the segments inside them and spans of many chunks; odd and one-channel widths
CASES = [(1, 1, 1), (2, 1, 70), (1, 2, 64), (3, 7, 5), (2, 8, 66), (1, 63, 128), (2, 64, 64), (1, 65, 63), (2, 127, 33),
         (1, 128, 130), (3, 129, 65), (2, 200, 257), (1, 1023, 64), (1, 2049, 65), (2, 2500, 34), (1, 4200, 70)]


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("shape", CASES, ids=lambda s: "b%d_L%d_D%d" % s)
def test_gated_parity(shape, dtype):
    b, L, D = shape
    x, r, i, lam, init = make(b, L, D, dtype, seed=L + D)
    dy, dfin = grads_in(b, L, D, dtype, seed=L)
    run_all(x, r, i, lam, init, None, dy, dfin, "gated %s" % (shape,))


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("shape", [(2, 1, 9), (2, 64, 40), (3, 131, 67), (2, 777, 64), (1, 2300, 66)],
                         ids=lambda s: "b%d_L%d_D%d" % s)
def test_gated_packed_rows(shape, dtype):
    b, L, D = shape
    x, r, i, lam, init = make(b, L, D, dtype, seed=L, halves=False)
    ids = ids_of(b, L, seed=L).cuda()
    dy, dfin = grads_in(b, L, D, dtype, seed=L)
    run_all(x, r, i, lam, init, ids, dy, dfin, "packed %s" % (shape,))
    run_all(x, r, i, lam, None, ids, dy, None, "packed, no states %s" % (shape,))


def test_gated_every_token_its_own_document():
    b, L, D = 2, 300, 70
    x, r, i, lam, init = make(b, L, D, FP, seed=5)
    ids = torch.arange(L, dtype=torch.int32).flip(0).repeat(b, 1).contiguous().cuda()
    dy, dfin = grads_in(b, L, D, FP, seed=6)
    run_all(x, r, i, lam, init, ids, dy, dfin, "one-token documents")


@pytest.mark.parametrize("decay", [(1 - 2e-6, 1 - 1e-7), (0.5, 0.9), (1e-6, 0.01), (1e-30, 1e-20)])
def test_gated_short_and_long_memories(decay):
    """From states that hardly decay (1 - a is then what carries the bits) to
    ones gone after a token, where products over a chunk underflow."""
    x, r, i, lam, init = make(2, 700, 66, FP, seed=11, decay=decay)
    dy, dfin = grads_in(2, 700, 66, FP, seed=12)
    run_all(x, r, i, lam, init, None, dy, dfin, "decay %s" % (decay,))


@pytest.mark.parametrize("scale", [0.5, 8.0, 100.0])
def test_gated_decay_scale(scale):
    x, r, i, lam, init = make(2, 150, 40, FP, seed=13)
    dy, dfin = grads_in(2, 150, 40, FP, seed=14)
    run_all(x, r, i, lam, init, None, dy, dfin, "scale", decay_scale=scale)


@pytest.mark.parametrize("dtype", [FP, BF])
def test_gated_shut_and_open_gates(dtype):
    """Gates far out on both sides.  Where the recurrence gate is shut (r
    underflows), a = 1, the input's factor is 0 and every gradient is finite:
    the state passes through."""
    b, L, D = 2, 130, 64
    x, r, i, lam, init = make(b, L, D, dtype, seed=15, halves=False)
    r[:, :, ::3] = -200.0
    r[:, :, 1::3] = 200.0
    i[:, ::2] = -200.0
    dy, dfin = grads_in(b, L, D, dtype, seed=16)
    y, fin, states = ssd.gated_scan_fwd_states(x, r, i, lam, init_state=init)
    assert torch.equal(fin[:, ::3], init[:, ::3])
    d = ssd.gated_scan_bwd(x, r, i, lam, states, dy, dfinal_state=dfin, init_state=init)
    for k, v in d.items():
        assert torch.isfinite(v).all(), k
    assert d["r_raw"][:, :, ::3].abs().max() == 0 and d["x"][:, :, ::3].abs().max() == 0
    h, err, parts = refs.gated(x, r, i, lam, init)
    # a shut gate's own factor is below float32's range: off by less than its smallest normal number's root
    refs.check(y, h, err + 1.1e-19 * 200, "y")
    refs.check(d["init_state"], refs.gated_bwd(parts, dy, dfin)["init_state"][0],
               refs.gated_bwd(parts, dy, dfin)["init_state"][1] + 1e-18, "dinit")


def test_gated_lam_far_out():
    """lam where softplus vanishes: no decay, no input, no gradient of lam."""
    x, r, i, lam, init = make(2, 90, 8, FP, seed=17)
    lam[:4] = -1000.0
    lam[4] = -math.inf
    y, fin, states = ssd.gated_scan_fwd_states(x, r, i, lam, init_state=init)
    assert torch.equal(fin[:, :5], init[:, :5])
    dy, _ = grads_in(2, 90, 8, FP, seed=18)
    d = ssd.gated_scan_bwd(x, r, i, lam, states, dy, init_state=init)
    assert d["lam"][:5].abs().max() == 0
    assert all(torch.isfinite(v).all() for v in d.values())


def test_gated_bad_values_stay_in_their_document():
    """NaN and infinities in one document leave the others' outputs, gradients
    and the final state as they are."""
    b, L, D = 2, 400, 66
    x, r, i, lam, init = make(b, L, D, FP, seed=19, halves=False)
    ids = torch.zeros(b, L, dtype=torch.int32)
    ids[:, 100:] = 1
    ids[:, 250:] = 2
    ids = ids.cuda()
    dy, dfin = grads_in(b, L, D, FP, seed=20)

    def both():
        y, fin, st = ssd.gated_scan_fwd_states(x, r, i, lam, init_state=init, seq_idx=ids)
        d = ssd.gated_scan_bwd(x, r, i, lam, st, dy, dfinal_state=dfin, init_state=init, seq_idx=ids)
        return y, fin, d

    y0, fin0, d0 = both()
    x[:, 120] = math.nan
    x[:, 130] = math.inf
    y1, fin1, d1 = both()
    assert torch.isnan(y1[:, 140]).any()
    out = torch.cat([torch.arange(100), torch.arange(250, L)])
    assert torch.equal(y0[:, out], y1[:, out]) and torch.equal(fin0, fin1)
    for k in ("x", "r_raw", "g_raw"):
        assert torch.equal(d0[k][:, out], d1[k][:, out]), k
    assert torch.equal(d0["init_state"], d1["init_state"])
    # a NaN gradient in the middle document stays there too
    x[:, 120] = x[:, 130] = 0.5
    dy[:, 200] = math.nan
    y2, fin2, d2 = both()
    for k in ("x", "r_raw", "g_raw"):
        assert torch.equal(d0[k][:, 250:], d2[k][:, 250:]) and torch.equal(d0[k][:, :100], d2[k][:, :100]), k
    assert torch.equal(d0["init_state"], d2["init_state"])


def test_gated_no_tokens_and_no_rows():
    x, r, i, lam, init = make(2, 0, 10, FP, seed=21)
    y, fin, st = ssd.gated_scan_fwd_states(x, r, i, lam, init_state=init)
    assert y.shape == (2, 0, 10) and torch.equal(fin, init) and st.shape == (2, 0, 10)
    _, fin = ssd.gated_scan_fwd(x, r, i, lam)
    assert fin.abs().max() == 0
    d = ssd.gated_scan_bwd(x, r, i, lam, st, x, dfinal_state=init)
    assert torch.equal(d["init_state"], init) and d["lam"].abs().max() == 0
    x, r, i, lam, init = make(0, 5, 10, FP, seed=21)
    y, fin, st = ssd.gated_scan_fwd_states(x, r, i, lam, init_state=init)
    assert y.shape == (0, 5, 10) and ssd.gated_scan_bwd(x, r, i, lam, st, x)["lam"].abs().max() == 0


@pytest.mark.parametrize("dtype", [FP, BF])
def test_gated_in_pieces(dtype):
    """A sequence run in two calls, the state handed over, is the sequence run
    in one: the same per-token arithmetic, so only the joining of segments
    differs (the bound of the form)."""
    b, L, D, cut = 2, 500, 66, 203
    x, r, i, lam, init = make(b, L, D, dtype, seed=22, halves=False)
    y, fin = ssd.gated_scan_fwd(x, r, i, lam, init_state=init)
    first = [t[:, :cut].contiguous() for t in (x, r, i)]
    rest = [t[:, cut:].contiguous() for t in (x, r, i)]
    y1, mid = ssd.gated_scan_fwd(*first, lam, init_state=init)
    y2, end = ssd.gated_scan_fwd(*rest, lam, init_state=mid)
    h, err, _ = refs.gated(x, r, i, lam, init)
    refs.check(torch.cat([y1, y2], 1), h, err, "pieces")
    refs.check(end, h[:, -1], err[:, -1], "pieces' end")


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("shape", [(1, 1), (1, 2560), (3, 67), (5, 1001), (256, 130), (300, 64)], ids=lambda s: "b%d_D%d" % s)
def test_gated_step_parity(shape, dtype):
    b, D = shape
    x, r, i, lam, state = make(b, 1, D, dtype, seed=b + D)
    x, r, i = x[:, 0], r[:, 0], i[:, 0]
    h, err, _ = refs.gated(x[:, None], r[:, None], i[:, None], lam, state)
    y = ssd.gated_step(x, r, i, lam, state)
    refs.check(y, h[:, 0], err[:, 0], "step y")
    refs.check(state, h[:, 0], err[:, 0], "step state")


def test_gated_steps_follow_the_scan():
    b, L, D = 3, 40, 130
    x, r, i, lam, state = make(b, L, D, BF, seed=30)
    h, err, _ = refs.gated(x, r, i, lam, state)
    for t in range(L):
        y = ssd.gated_step(x[:, t], r[:, t], i[:, t], lam, state)
        refs.check(y, h[:, t], err[:, t], "step %d" % t)


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("D", [66, 65])
def test_gated_strides_and_unaligned_rows(D, dtype):
    """Rows of one wide tensor at odd element offsets give the bits of
    contiguous ones, and gradients land in the halves of one tensor."""
    b, L = 2, 300
    g = torch.Generator().manual_seed(40)
    wide = torch.randn(b, L, 3 * D + 5, generator=g).to(dtype).cuda()
    x, r, i = wide[..., 1:D + 1], wide[..., D + 2:2 * D + 2], wide[..., 2 * D + 3:3 * D + 3]
    lam = torch.full((D,), -4.0, device="cuda")
    dy, dfin = grads_in(b, L, D, dtype, seed=41)
    a = ssd.gated_scan_fwd_states(x, r, i, lam)
    c = ssd.gated_scan_fwd_states(x.contiguous(), r.contiguous(), i.contiguous(), lam)
    assert all(torch.equal(p, q) for p, q in zip(a, c))
    both = torch.full((b, L, 2 * D + 3), 7.0, dtype=dtype, device="cuda")
    da = ssd.gated_scan_bwd(x, r, i, lam, a[2], dy, dfinal_state=dfin,
                            out={"r_raw": both[..., 1:D + 1], "g_raw": both[..., D + 2:2 * D + 2]})
    dc = ssd.gated_scan_bwd(x.contiguous(), r.contiguous(), i.contiguous(), lam, a[2], dy, dfinal_state=dfin)
    assert all(torch.equal(da[k], dc[k]) for k in dc)
    assert (both[..., 0] == 7).all() and (both[..., D + 1] == 7).all() and (both[..., 2 * D + 2] == 7).all()


def test_gated_same_bits_every_time_and_within_bounds_of_memory():
    """Repeated calls give the same bits, on another stream too, with guard
    values around the outputs left alone (they are rows of larger buffers in
    a caching allocator: the neighbours are what would be hit)."""
    b, L, D = 2, 3000, 130
    x, r, i, lam, init = make(b, L, D, BF, seed=50)
    ids = ids_of(b, L, seed=51, chance=0.002).cuda()
    dy, dfin = grads_in(b, L, D, BF, seed=52)

    def both():
        y, fin, st = ssd.gated_scan_fwd_states(x, r, i, lam, init_state=init, seq_idx=ids)
        d = ssd.gated_scan_bwd(x, r, i, lam, st, dy, dfinal_state=dfin, init_state=init, seq_idx=ids)
        return [y, fin, st] + [d[k] for k in ("x", "r_raw", "g_raw", "lam", "init_state")]

    want = both()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for n in range(6):
        with torch.cuda.stream(s if n % 2 else torch.cuda.current_stream()):
            got = both()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want, got)), n


def test_gated_workspace_status_and_reuse():
    """A caller's workspace, dirty from other use, is enough at its size; the
    status word reads OK; one byte less is refused."""
    b, L, D = 2, 2200, 66
    x, r, i, lam, init = make(b, L, D, FP, seed=60)
    dy, dfin = grads_in(b, L, D, FP, seed=61)
    n = ssd.gated_scan_workspace_size(b, L, D, FP)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    y, fin, st = ssd.gated_scan_fwd_states(x, r, i, lam, init_state=init, workspace=ws)
    assert ssd.read_device_status(ws) == 0
    h, err, _ = refs.gated(x, r, i, lam, init)
    refs.check(y, h, err, "dirty workspace")
    nb = ssd.gated_scan_workspace_size(b, L, D, FP, backward=True)
    wb = torch.full((nb,), 255, dtype=torch.uint8, device="cuda")
    d = ssd.gated_scan_bwd(x, r, i, lam, st, dy, dfinal_state=dfin, init_state=init, workspace=wb)
    assert ssd.read_device_status(wb) == 0
    e = ssd.gated_scan_bwd(x, r, i, lam, st, dy, dfinal_state=dfin, init_state=init)
    assert all(torch.equal(d[k], e[k]) for k in d)
    with pytest.raises(ssd.SSDError):
        ssd.gated_scan_fwd(x, r, i, lam, workspace=ws[:n - 1])
    with pytest.raises(ssd.SSDError):
        ssd.gated_scan_bwd(x, r, i, lam, st, dy, workspace=wb[:nb - 1])


def test_gated_captured_and_replayed():
    """Forward, backward and a step in one graph, replayed on new inputs."""
    b, L, D = 1, 2100, 66
    x, r, i, lam, init = make(b, L, D, BF, seed=70, halves=False)
    dy, dfin = grads_in(b, L, D, BF, seed=71)

    def both():
        y, fin, st = ssd.gated_scan_fwd_states(x, r, i, lam, init_state=init)
        d = ssd.gated_scan_bwd(x, r, i, lam, st, dy, dfinal_state=dfin, init_state=init)
        z = ssd.gated_step(x[:, 0], r[:, 0], i[:, 0], lam, fin)
        return [y, fin, st, z] + [d[k] for k in ("x", "r_raw", "g_raw", "lam", "init_state")]

    both()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = both()
    for seed in (72, 73):
        for t, n in zip((x, r, i, init), make(b, L, D, BF, seed=seed, halves=False)[:3] + (init * 0.5,)):
            t.copy_(n)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, both()))


def test_gated_refuses():
    x, r, i, lam, init = make(2, 70, 10, FP, seed=80)
    dy, dfin = grads_in(2, 70, 10, FP, seed=81)
    y, fin, st = ssd.gated_scan_fwd_states(x, r, i, lam)
    bad = [lambda: ssd.gated_scan_fwd(x, r[:, :60], i, lam), lambda: ssd.gated_scan_fwd(x, r.contiguous(), i, lam),
           lambda: ssd.gated_scan_fwd(x, r, i, lam.double()), lambda: ssd.gated_scan_fwd(x, r, i, lam.cpu()),
           lambda: ssd.gated_scan_fwd(x.half(), r, i, lam), lambda: ssd.gated_scan_fwd(x.bfloat16(), r, i, lam),
           lambda: ssd.gated_scan_fwd(x, r, i, lam, init_state=init[:1]),
           lambda: ssd.gated_scan_fwd(x, r, i, lam, seq_idx=torch.zeros(2, 70, dtype=torch.int64, device="cuda")),
           lambda: ssd.gated_scan_fwd(x[0], r[0], i[0], lam),
           lambda: ssd.gated_scan_bwd(x, r, i, lam, st[:, :1], dy), lambda: ssd.gated_scan_bwd(x, r, i, lam, st, dy[:1]),
           lambda: ssd.gated_scan_bwd(x, r, i, lam, st, dy, out={"r_raw": dy, "g_raw": dy}),
           lambda: ssd.gated_step(x, r, i, lam, init), lambda: ssd.gated_step(x[:, 0], r[:, 0], i[:, 0], lam, init.half())]
    for k, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail("call %d was taken" % k)
    for scale in (0.0, -1.0, math.inf, math.nan):
        with pytest.raises(ssd.SSDError):
            ssd.gated_scan_fwd(x, r, i, lam, decay_scale=scale)
    with pytest.raises(ssd.SSDError):
        ssd.gated_scan_bwd(x, r, i, lam, None, dy)


# more tiles than CTAs: each CTA goes round several times.  Widths whose rows start on 16 bytes, on pairs, on single elements.
@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("packed", [False, True], ids=["rows", "packed"])
@pytest.mark.parametrize("D", [4096, 4098, 4099])
def test_gated_many_tiles(D, packed, dtype):
    b, L = 2, 530
    x, r, i, lam, init = make(b, L, D, dtype, seed=D, halves=D != 4099)
    ids = ids_of(b, L, seed=D, chance=0.02).cuda() if packed else None
    dy, dfin = grads_in(b, L, D, dtype, seed=D + 1)
    run_all(x, r, i, lam, init, ids, dy, dfin, "many tiles %d" % D)


@pytest.mark.parametrize("dtype", [FP, BF])
def test_gated_a_few_gates_shut_among_open_ones(dtype):
    """Warps whose gates are all open take another path than ones that hold a
    shut gate or a decay gone within a token; tiles here hold both."""
    b, L, D = 2, 400, 192
    x, r, i, lam, init = make(b, L, D, dtype, seed=81, halves=False)
    g = torch.Generator().manual_seed(82)
    for v in (r, i):
        far = (torch.rand(b, L, D, generator=g) < 0.0005).cuda()
        v[far] = torch.where(torch.rand(b, L, D, generator=g).cuda() < 0.5, -45.0, 45.0)[far].to(dtype)
    lam[5], lam[100] = 3.0, 30.0
    ids = ids_of(b, L, seed=83, chance=0.02).cuda()
    dy, dfin = grads_in(b, L, D, dtype, seed=84)
    run_all(x, r, i, lam, init, None, dy, dfin, "a few shut")
    run_all(x, r, i, lam, init, ids, dy, dfin, "a few shut, packed")


def test_gated_two_streams_at_once():
    """Two calls in flight at the same time, each with tiles that wait for
    others of its own."""
    b, L, D = 1, 6000, 320
    sets = [make(b, L, D, BF, seed=90 + k) for k in range(2)]
    dys = [grads_in(b, L, D, BF, seed=92 + k) for k in range(2)]

    def go(k):
        x, r, i, lam, init = sets[k]
        y, fin, st = ssd.gated_scan_fwd_states(x, r, i, lam, init_state=init)
        d = ssd.gated_scan_bwd(x, r, i, lam, st, dys[k][0], dfinal_state=dys[k][1], init_state=init)
        return [y, fin] + [d[n] for n in ("x", "r_raw", "g_raw", "lam", "init_state")]

    want = [go(k) for k in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append(go(k))
        torch.cuda.synchronize()
        for k in range(2):
            assert all(torch.equal(p, q) for p, q in zip(want[k], got[k]))


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("packed", [False, True], ids=["rows", "packed"])
@pytest.mark.parametrize("D", [64, 66, 65])
def test_gated_nan_gates_reach_what_they_enter(D, packed, dtype):
    """A NaN input gate is in its own token's input, so in the states after it
    and in its own gradients; the gradient that runs back to earlier tokens
    does not hold it.  One of the recurrence gate or of x likewise by the form."""
    b, L = 2, 300
    for what in ("g", "r", "x"):
        x, r, i, lam, init = make(b, L, D, dtype, seed=95, halves=False)
        {"g": i, "r": r, "x": x}[what][0, 170, 7] = math.nan
        {"g": i, "r": r, "x": x}[what][1, 64, D - 1] = math.nan
        ids = ids_of(b, L, seed=96, chance=0.01).cuda() if packed else None
        dy, dfin = grads_in(b, L, D, dtype, seed=97)
        run_all(x, r, i, lam, init, ids, dy, dfin, "NaN in %s" % what)
        if what == "g":
            _, _, st = ssd.gated_scan_fwd_states(x, r, i, lam, init_state=init, seq_idx=ids)
            d = ssd.gated_scan_bwd(x, r, i, lam, st, dy, dfinal_state=dfin, init_state=init, seq_idx=ids)
            assert torch.isnan(d["x"]).sum() == 2 and torch.isfinite(d["init_state"]).all()


def test_gated_gradients_that_overlap_are_refused():
    """out's two gradients may be columns of one tensor, but not share an
    element of it."""
    b, L, D = 2, 70, 10
    x, r, i, lam, init = make(b, L, D, FP, seed=80)
    dy, dfin = grads_in(b, L, D, FP, seed=81)
    st = ssd.gated_scan_fwd_states(x, r, i, lam)[2]
    want = ssd.gated_scan_bwd(x, r, i, lam, st, dy)
    flat = torch.zeros(b * L * 25 + 40, device="cuda")
    at = lambda s: torch.as_strided(flat, (b, L, D), (25 * L, 25, 1), s)  # noqa: E731
    for s in (0, 1, 9, 16, 24, 30):
        for pair in ((0, s), (s, 0)):
            with pytest.raises(ValueError):
                ssd.gated_scan_bwd(x, r, i, lam, st, dy, out={"r_raw": at(pair[0]), "g_raw": at(pair[1])})
    for s in (10, 15, 35):
        d = ssd.gated_scan_bwd(x, r, i, lam, st, dy, out={"r_raw": at(0), "g_raw": at(s)})
        assert torch.equal(d["r_raw"], want["r_raw"]) and torch.equal(d["g_raw"], want["g_raw"])
