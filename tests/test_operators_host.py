"""The operators around the scan, host side: the 64-bit forms the GPU tests
compare with against differences, and what the entry points refuse (no GPU)."""
import ctypes
import math

import pytest
import torch

import operator_refs as refs
from state_space_sequence_scan_b200 import ssd

F = torch.float64


@pytest.fixture(scope="module")
def lib():
    from state_space_sequence_scan_b200 import build
    build.build_library()
    return ssd.load_library()


def _rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=F)


def _difference(f, inputs, k, direction, eps=1e-5):
    """Central difference of f along a direction of inputs[k]."""
    lo, hi = list(inputs), list(inputs)
    lo[k], hi[k] = inputs[k] - eps * direction, inputs[k] + eps * direction
    return (f(*hi) - f(*lo)) / (2 * eps)


@pytest.mark.parametrize("packed", [False, True])
def test_gated_form_gradients_are_its_differences(packed):
    b, L, D = 2, 9, 3
    ins = [_rand(1, b, L, D), _rand(2, b, L, D), _rand(3, b, L, D), _rand(4, D) - 3, _rand(5, b, D)]
    dy, dfin = _rand(6, b, L, D), _rand(7, b, D)
    ids = torch.tensor([[0, 0, 0, 1, 1, 1, 1, 2, 2], [5, 5, 4, 4, 4, 4, 4, 4, 4]], dtype=torch.int32) if packed else None

    def loss(x, r, g, lam, init):
        h, _, _ = refs.gated(x, r, g, lam, init, ids)
        return float((dy * h).sum() + (dfin * h[:, -1]).sum())

    _, _, parts = refs.gated(*ins, ids)
    grads = refs.gated_bwd(parts, dy, dfin)
    for k, name in enumerate(("x", "r_raw", "g_raw", "lam", "init_state")):
        v = _rand(10 + k, *ins[k].shape)
        want = _difference(loss, ins, k, v)
        assert float((grads[name][0] * v).sum()) == pytest.approx(want, rel=1e-6, abs=1e-8), name


def test_gated_form_is_the_recurrence_of_its_definition():
    """a and the input's factor written as in the definition, one channel."""
    x, r, g, lam = _rand(1, 1, 5, 1), _rand(2, 1, 5, 1), _rand(3, 1, 5, 1), torch.tensor([-2.0], dtype=F)
    h, want = 0.7, []
    for t in range(5):
        s = lambda v: 1 / (1 + math.exp(-v))  # noqa: E731
        a = math.exp(-8.0 * math.log(1 + math.exp(-2.0)) * s(r[0, t, 0]))
        h = a * h + math.sqrt(1 - a * a) * s(g[0, t, 0]) * float(x[0, t, 0])
        want.append(h)
    got, _, _ = refs.gated(x, r, g, lam, torch.tensor([[0.7]], dtype=F))
    assert got[0, :, 0].tolist() == pytest.approx(want, rel=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rotate_form_gradients_are_its_differences(interleaved):
    b, L, G, N = 2, 3, 2, 10
    ins = [_rand(1, b, L, G, N), 1 + 0.1 * _rand(2, N)]
    inv = torch.tensor([1.0, 0.3, 0.01], dtype=F)
    pos, d = torch.tensor([[0, 5, 1000], [7, -3, 2]]), _rand(3, b, L, G, N)

    def loss(v, w):
        return float((d * refs.norm_rotate(v, w, inv, pos, 1e-5, interleaved)[0]).sum())

    grads = refs.norm_rotate_bwd(ins[0], ins[1], inv, pos, 1e-5, interleaved, d)
    for k in range(2):
        v = _rand(10 + k, *ins[k].shape)
        assert float((grads[k][0] * v).sum()) == pytest.approx(_difference(loss, ins, k, v), rel=1e-6, abs=1e-8)


@pytest.mark.parametrize("activation", ["none", "silu", "gelu"])
def test_linear_form_gradients_are_its_differences(activation):
    ins, dy = [_rand(1, 4, 5), _rand(2, 3, 5), _rand(3, 3)], _rand(4, 4, 3)

    def loss(x, w, bias):
        return float((dy * refs.linear(x, w, bias, None, activation)[0]).sum())

    z = refs.linear(*ins)[2]
    grads = refs.linear_bwd(ins[0], ins[1], dy, z, activation)
    for k, name in enumerate(("x", "weight", "bias")):
        v = _rand(10 + k, *ins[k].shape)
        assert float((grads[name][0] * v).sum()) == pytest.approx(_difference(loss, ins, k, v), rel=1e-6, abs=1e-8)


FAKE = 0x10000     # aligned stand-in, never dereferenced: the calls fail validation first


def _ws(lib, fn, *args):
    n = ctypes.c_size_t(0)
    return getattr(lib, fn)(*args, ctypes.byref(n)), n.value


def test_gated_refuses_on_host(lib):
    def fwd(p=FAKE, y=FAKE, lam=FAKE, b=2, L=100, D=10, ldx=10, ldg=20, c=8.0, dtype=1, ws=FAKE, wsb=1 << 40, ids=None):
        return lib.ssd_gated_scan_fwd(p, p, p, lam, None, ids, y, None, None, b, L, D, ldx, ldg, c, dtype, ws, wsb, None)

    assert fwd(p=None) == 1 and fwd(y=None) == 1 and fwd(lam=None) == 1
    assert fwd(D=0) == 1 and fwd(b=-1) == 1 and fwd(L=-1) == 1
    assert fwd(ldx=9) == 1 and fwd(ldg=9) == 1
    for c in (0.0, -1.0, math.inf, math.nan):
        assert fwd(c=c) == 1
    assert fwd(dtype=2) == 2 and fwd(b=1 << 20) == 2 and fwd(L=1 << 31) == 2 and fwd(D=1 << 31, ldx=1 << 31, ldg=1 << 31) == 2
    assert fwd(p=FAKE + 1) == 3 and fwd(dtype=0, p=FAKE + 2) == 3 and fwd(lam=FAKE + 2) == 3 and fwd(ids=FAKE + 2) == 3
    assert fwd(ws=None) == 4 and fwd(wsb=255) == 4 and fwd(ws=FAKE + 128) == 3

    def bwd(p=FAKE, st=FAKE, dlam=FAKE, dx=FAKE, L=100, ldd=20, ws=FAKE, wsb=1 << 40):
        return lib.ssd_gated_scan_bwd(p, p, p, FAKE, None, None, st, p, None, dx, FAKE, FAKE, dlam, None, 2, L, 10, 10, 20,
                                      ldd, 8.0, 1, ws, wsb, None)

    assert bwd(p=None) == 1 and bwd(dx=None) == 1 and bwd(dlam=None) == 1
    assert bwd(st=None) == 1                        # more than one chunk needs the states
    assert bwd(ldd=9) == 1
    assert bwd(st=FAKE + 2) == 3 and bwd(dx=FAKE + 1) == 3
    assert bwd(ws=None) == 4 and bwd(wsb=300) == 4

    def step(p=FAKE, state=FAKE, b=2, D=10, ldx=10, ldg=10, c=8.0, dtype=1):
        return lib.ssd_gated_step(p, p, p, FAKE, state, FAKE, b, D, ldx, ldg, c, dtype, None)

    assert step(b=0) == 0
    assert step(p=None) == 1 and step(state=None) == 1 and step(D=0) == 1 and step(ldg=5) == 1 and step(c=0.0) == 1
    assert step(dtype=9) == 2 and step(b=70000) == 2
    assert step(p=FAKE + 1) == 3 and step(state=FAKE + 2) == 3
    assert _ws(lib, "ssd_gated_scan_workspace_size", 1, 100, 10, 1, 0)[0] == 0
    assert _ws(lib, "ssd_gated_scan_workspace_size", 1, 100, 10, 1, 2)[0] == 1
    assert _ws(lib, "ssd_gated_scan_workspace_size", 1, 100, 0, 1, 0)[0] == 1
    assert lib.ssd_gated_scan_workspace_size(1, 100, 10, 1, 0, None) == 1


def test_norm_rotate_refuses_on_host(lib):
    def fwd(p=FAKE, o=FAKE, w=FAKE, f=FAKE, pos=None, b=1, L=3, G=2, N=16, R=16, eps=1e-5, il=0, dtype=1):
        return lib.ssd_bc_norm_rotate_fwd(p, p, w, w, f, pos, o, o, b, L, G, N, R, eps, il, dtype, None)

    assert fwd(b=0) == 0 and fwd(L=0) == 0
    assert fwd(p=None) == 1 and fwd(o=None) == 1 and fwd(w=None) == 1 and fwd(f=None) == 1
    assert fwd(G=0) == 1 and fwd(N=0) == 1 and fwd(R=18) == 1 and fwd(R=3) == 1 and fwd(R=-2) == 1
    assert fwd(eps=-1.0) == 1 and fwd(eps=math.nan) == 1 and fwd(il=2) == 1
    assert fwd(dtype=5) == 2 and fwd(N=8200) == 2 and fwd(b=1 << 31) == 2
    assert fwd(p=FAKE + 8) == 3 and fwd(o=FAKE + 2) == 3 and fwd(w=FAKE + 4) == 3 and fwd(f=FAKE + 2) == 3
    assert fwd(pos=FAKE + 1) == 3

    def bwd(p=FAKE, dw=FAKE, ws=FAKE, wsb=1 << 40):
        return lib.ssd_bc_norm_rotate_bwd(p, p, FAKE, FAKE, FAKE, None, p, p, p, p, dw, dw, 1, 3, 2, 16, 16, 1e-5, 0, 1, ws,
                                          wsb, None)

    assert bwd(p=None) == 1 and bwd(dw=None) == 1 and bwd(p=FAKE + 8) == 3 and bwd(dw=FAKE + 4) == 3
    assert bwd(ws=None) == 4 and bwd(wsb=16) == 4 and bwd(ws=FAKE + 16) == 3
    assert _ws(lib, "ssd_bc_norm_rotate_bwd_workspace_size", 1, 3, 0, 16)[0] == 1


def test_linear_refuses_on_host(lib):
    def fwd(p=FAKE, w=FAKE, o=FAKE, bias=None, res=None, M=4, N=8, K=16, act=0, it=1, ot=1, ws=FAKE, wsb=1 << 40):
        return lib.ssd_linear_fwd(p, w, bias, res, o, None, M, N, K, act, it, ot, ws, wsb, None)

    assert fwd(p=None) == 1 and fwd(w=None) == 1 and fwd(o=None) == 1
    assert fwd(M=-1) == 1 and fwd(N=0) == 1 and fwd(K=0) == 1 and fwd(act=3) == 1
    assert fwd(it=2) == 2 and fwd(it=0, ot=1) == 2 and fwd(it=1, ot=3) == 2 and fwd(M=1 << 31) == 2
    assert fwd(p=FAKE + 8) == 3 and fwd(o=FAKE + 8) == 3 and fwd(bias=FAKE + 4) == 3 and fwd(res=FAKE + 2) == 3
    assert fwd(ws=None) == 4 and fwd(wsb=100) == 4 and fwd(ws=FAKE + 64) == 3

    def bwd(x=FAKE, w=FAKE, dy=FAKE, z=None, dx=FAKE, dw=FAKE, act=0, ws=FAKE, wsb=1 << 40):
        return lib.ssd_linear_bwd(x, w, dy, z, dx, dw, FAKE, 4, 8, 16, act, 1, ws, wsb, None)

    assert bwd(dy=None) == 1 and bwd(w=None) == 1 and bwd(x=None) == 1 and bwd(act=9) == 1
    assert bwd(act=1) == 1                          # an activation needs the pre-activation
    assert bwd(dx=FAKE + 8) == 3 and bwd(z=FAKE + 2, act=1) == 3
    assert bwd(ws=None) == 4 and bwd(wsb=256) == 4
    assert _ws(lib, "ssd_linear_workspace_size", 4, 8, 16, 1, 3)[0] == 1


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(1, 4, 8)
    lam = torch.zeros(8)
    with pytest.raises(ValueError):
        ssd.gated_scan_fwd(x, x, x, lam)
    with pytest.raises(ValueError):
        ssd.gated_step(x[:, 0], x[:, 0], x[:, 0], lam, torch.zeros(1, 8))
    with pytest.raises(ValueError):
        ssd.bc_norm_rotate_fwd(x[None], x[None], lam, lam, None)
    with pytest.raises(ValueError):
        ssd.linear_fwd(x, torch.zeros(3, 8))
    with pytest.raises(ValueError):
        ssd.linear_bwd(x, torch.zeros(3, 8), torch.zeros(1, 4, 3))


def test_row_spacing_check():
    """Evenly spaced rows pass with their spacing, anything else is refused."""
    dev, t = torch.device("cpu"), torch.float32
    both = torch.zeros(2, 3, 20)
    assert ssd._rows("x", both[..., 10:], (2, 3, 10), t, dev) == (both.data_ptr() + 40, 20)
    assert ssd._rows("x", both[:, :1, 5:10], (2, 1, 5), t, dev)[1] == 60
    assert ssd._rows("x", both[:1, :1, :4], (1, 1, 4), t, dev)[1] == 4
    for bad in (both[:, :2, :10], both.transpose(0, 1)[..., :10], torch.zeros(3, 10).expand(2, 3, 10),
                torch.zeros(2, 10, 3).transpose(1, 2), both[..., ::2]):
        with pytest.raises(ValueError):
            ssd._rows("x", bad, tuple(bad.shape), t, dev)


def test_sizes_on_both_sides_of_the_limits(lib):
    """What the header allows is taken, one more is not."""
    def gated(b, L, D, dtype=1, back=0):
        return _ws(lib, "ssd_gated_scan_workspace_size", b, L, D, dtype, back)[0]

    assert gated(65535, 1, 1) == 0 and gated(65536, 1, 1) == 2
    assert gated(1, (1 << 31) - 1, 64) == 0 and gated(1, 1 << 31, 64) == 2
    assert gated(1, 1, (1 << 31) - 1) == 0 and gated(1, 1, 1 << 31) == 2
    assert gated(32768, 65535, 4096) == 2 and gated(32768, 64 * 1023, 4096) == 0 and gated(32768, 64 * 1024, 4096) == 2

    def norm(b, L, G, N):
        return _ws(lib, "ssd_bc_norm_rotate_bwd_workspace_size", b, L, G, N)[0]

    assert norm(1, 1, 65535, 8192) == 0 and norm(1, 1, 65536, 8192) == 2 and norm(1, 1, 1, 8193) == 2
    assert norm(1 << 10, 1 << 22, 1, 8) == 0 and norm(1 << 10, (1 << 23) - 1, 1, 8) == 0 and norm(1 << 10, 1 << 23, 1, 8) == 2
    assert norm(1 << 10, 1 << 20, 8, 8) == 2 and norm(1 << 10, (1 << 20) - 1, 8, 8) == 0

    def linear(M, N, K, dtype=1, back=0):
        return _ws(lib, "ssd_linear_workspace_size", M, N, K, dtype, back)[0]

    most = (1 << 31) - 513
    for dtype in (0, 1):
        for back in (0, 1):
            assert linear(most, 8, 8, dtype, back) == 0 and linear(most + 1, 8, 8, dtype, back) == 2
            assert linear(8, most, 8, dtype, back) == 0 and linear(8, most + 1, 8, dtype, back) == 2
            assert linear(8, 8, most, dtype, back) == 0 and linear(8, 8, most + 1, dtype, back) == 2
            assert linear(1 << 20, 8, (1 << 18) - 1, dtype, back) == 0 and linear(1 << 20, 8, 1 << 18, dtype, back) == 2


def test_rows_that_share_elements():
    """_rows_share against the sets of their elements' addresses."""
    g = torch.Generator().manual_seed(1)
    pick = lambda lo, hi: int(torch.randint(lo, hi + 1, (), generator=g))  # noqa: E731
    for _ in range(3000):
        rows, width, size = pick(0, 5), pick(1, 6), (2, 4)[pick(0, 1)]
        ld, p, q = width + pick(0, 8), pick(0, 60), pick(0, 60)
        one, two = ({size * (at + r * ld + e) for r in range(rows) for e in range(width)} for at in (p, q))
        assert ssd._rows_share(size * p, size * q, rows, width, ld, size) == bool(one & two)


def test_linear_wide_dz_on_host(lib):
    """The flag goes with every activation of the backward, and with none of the forward's."""
    def bwd(act, wsb, z=FAKE, M=4):
        return lib.ssd_linear_bwd(FAKE, FAKE, FAKE, z, FAKE, FAKE, FAKE, M, 8, 16, act, 1, FAKE, wsb, None)

    n = _ws(lib, "ssd_linear_workspace_size", 4, 8, 16, 1, 2)
    assert n[0] == 0 and n[1] > _ws(lib, "ssd_linear_workspace_size", 4, 8, 16, 1, 1)[1]
    assert bwd(0x101, n[1] - 1) == 4 and bwd(0x102, n[1] - 1) == 4 and bwd(0x100, n[1] - 1) == 4
    assert bwd(0x103, 1 << 40) == 1 and bwd(0x201, 1 << 40) == 1 and bwd(-1, 1 << 40) == 1 and bwd(0x101, 1 << 40, z=None) == 1
    assert lib.ssd_linear_fwd(FAKE, FAKE, None, None, FAKE, None, 4, 8, 16, 0x101, 1, 1, FAKE, 1 << 40, None) == 1
    most = (1 << 30) - 513
    assert _ws(lib, "ssd_linear_workspace_size", most, 8, 8, 1, 2)[0] == 0 and _ws(lib, "ssd_linear_workspace_size", most + 1, 8, 8, 1, 2)[0] == 2
