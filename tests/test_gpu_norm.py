"""moe_rmsnorm, moe_rmsnorm_backward and moe_combine_backward against their
formulas in float64.

Tolerances, fixed before the first run.  u = 2^-24 is half a float32 step.  An
output of type t is rounded once: r = finfo(t).eps / 2 of its value.  Float32
sums: a row of H elements goes through at most 16 sequential terms per thread,
6 lane exchanges and 16 wave sums, so with the products each sum is off by at
most N = 48 steps u of the sum of its terms' magnitudes; a statistic built
from it (division, root, product) by a few more, taken as 64 u.  Elements of
an e4m3 block are off by at most 2^-4 of their value, or half the smallest
step, 2^-10 of the block's scale.
"""
import pytest
import torch

import mixture_experts_layer_amd as M

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
STAT = 64 * U
TYPES = [torch.bfloat16, torch.float32]


def _rand(shape, seed, scale=1.0, dtype=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def _close(got, ref, rel, extra=0.0):
    """|got - ref| <= rel * |ref| + extra everywhere."""
    bad = (got.double() - ref).abs() > rel * ref.abs() + extra
    assert not bad.any(), (int(bad.sum()), bad.numel(),
                           float(((got.double() - ref).abs() / ref.abs().clamp_min(1e-30)).max()))


def _step(dt):
    return torch.finfo(dt).eps / 2


def _norm(x, res, w, eps=1e-6, sum=True, y=True, y8=True, rstd=True):
    T, H = x.shape
    o = dict(sum=torch.empty_like(x) if sum else None, y=torch.empty_like(x) if y else None,
             y8=torch.empty(T, H, device=DEV, dtype=torch.float8_e4m3fn) if y8 else None,
             scale=torch.full((T, M.mx_pitch(H)), 77, device=DEV, dtype=torch.uint8) if y8 else None,
             rstd=torch.empty(T, device=DEV) if rstd else None)
    M.moe_rmsnorm(x, res, w, eps, T, H, M.dtype_code(x), o["sum"], o["y"], o["y8"], o["scale"], o["rstd"])
    return o


def _reference(x, res, w, eps=1e-6):
    s = x if res is None else (x.float() + res.float()).to(x.dtype)    # one float32 addition: exact
    rstd = 1 / torch.sqrt(s.double().square().mean(1) + eps)
    return s, rstd, s.double() * rstd[:, None] * w.double()


def check_mx(q, scale, ref, rel):
    """An MXFP8 tensor against real rows known to `rel`: the scale is the least
    that holds the block's largest element, and every element the nearest."""
    T, H = ref.shape
    assert not scale[:, H // 32:].any()
    b = scale[:, :H // 32].double()
    top = ref.reshape(T, H // 32, 32).abs().amax(-1)
    f = torch.exp2(b - 127)
    assert (top * (1 - rel) <= 448 * f).all()
    assert ((top * (1 + rel) >= 224 * f) | (b == 0)).all()
    val = q.double() * f.repeat_interleave(32, dim=1)
    _close(val, ref, 2.0 ** -4 + rel, (2.0 ** -10 * f).repeat_interleave(32, dim=1) * (1 + rel))


SHAPES = [(1, 32), (3, 96), (64, 256), (2, 480), (515, 544), (7, 4096), (33, 7168), (5, 8192), (2, 8224),
          (3, 16384)]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("residual", [True, False])
def test_norm(T, H, dt, residual):
    x, w = _rand((T, H), 1, 2.0, dt), _rand((H,), 2, 1.0, dt)
    x[0] *= 1e-3
    res = _rand((T, H), 3, 1.0, dt) if residual else None
    o = _norm(x, res, w)
    s, rstd, y = _reference(x, res, w)
    assert torch.equal(o["sum"], s)
    _close(o["rstd"], rstd, STAT)
    _close(o["y"], y, _step(dt) + STAT + 3 * U)
    check_mx(o["y8"], o["scale"], y, STAT + 3 * U)


@pytest.mark.parametrize("dt", TYPES)
def test_norm_rounds_once_to_8_bits(dt):
    """Every element of 2^24 is the e4m3 value nearest to the formula's float64
    value: both are within 2^-51 of the real one, so that an element lies between
    them and a border 2^-4 apart in about one case of 2^46."""
    T, H, eps = 4096, 4096, 2.0 ** -20
    x, res, w = _rand((T, H), 51, 1.5, dt), _rand((T, H), 52, 1.0, dt), (1 + _rand((H,), 53, 0.1)).to(dt)
    o = _norm(x, res, w, eps=eps)
    ref = _reference(x, res, w, eps)[2].reshape(T, H // 32, 32)
    k = torch.exp2(o["scale"].double() - 127)[:, :, None]
    a = (ref / k).abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -6))) - 3)       # 3 mantissa bits, least step 2^-9
    want = torch.round(a / step) * step * torch.sign(ref)
    assert (a.amax(-1) <= 448).all() and (a.amax(-1) > 224).all()
    assert torch.equal(o["y8"].double().reshape(want.shape), want)


@pytest.mark.parametrize("want", ["sum", "y", "y8", "rstd"])
def test_norm_outputs_alone_equal_those_together(want):
    x, res, w = _rand((9, 4096), 4, 1.0, torch.bfloat16), _rand((9, 4096), 5, 1.0, torch.bfloat16), _rand((4096,), 6, 1.0, torch.bfloat16)
    a, none = _norm(x, res, w), dict(sum=False, y=False, y8=False, rstd=False)
    b = _norm(x, res, w, **dict(none, **{want: True}))
    keys = ("y8", "scale") if want == "y8" else (want,)
    for k in keys:
        assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8))


def test_norm_extremes_and_blocks_at_the_scale_border():
    H = 256
    x = torch.zeros(6, H, device=DEV)
    x[1] = 1e-38                       # a row of tiny values: the scale stays at its least
    x[2] = 3e18                        # squares near the top of float32
    x[3, :32] = torch.linspace(-1, 1, 32)
    x[4, 0] = 448.0
    x[5, 40] = 450.0
    w = torch.ones(H, device=DEV)
    o = _norm(x, None, w, eps=1.0)
    s, rstd, y = _reference(x, None, w, eps=1.0)
    _close(o["y"], y, 2 * U + STAT, 1e-44)
    check_mx(o["y8"], o["scale"], y, STAT + 3 * U)
    assert not o["y8"].view(torch.uint8)[0].any() and not o["scale"][0].any()
    # an eps of zero leaves a row of zeros undefined, and only that row
    o = _norm(x, None, w, eps=0.0)
    assert torch.isfinite(o["y"][2:]).all()


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("rows,weight,eps", [(2.0 ** 126, 4.0, 1e-6), (2.0 ** -100, 2.0 ** -45, 0.0), (2.0 ** -120, 2.0 ** -20, 0.0),
                                             (2.0 ** 100, 2.0 ** 100, 1e-6)])
def test_norm_products_outside_float32(dt, rows, weight, eps):
    """s * weight may leave float32's range where s * rstd * weight does not."""
    x, w = _rand((70, 544), 61, 0.3, dt).clamp(-1.9, 1.9) * rows, _rand((544,), 62, 1.0, dt) * weight
    x[0], w[:32] = rows * 1.5, weight
    assert torch.isfinite(x).all() and torch.isfinite(w).all()
    o = _norm(x, None, w, eps=eps)
    _, _, y = _reference(x, None, w, eps=eps)
    _close(o["y"], y, _step(dt) + 2.0 ** -40)
    check_mx(o["y8"], o["scale"], y, 2.0 ** -40)


def test_norm_nan_stays_in_its_row():
    x, w = _rand((5, 512), 7, 1.0, torch.bfloat16), _rand((512,), 8, 1.0, torch.bfloat16)
    good = _norm(x, None, w)
    x[2, 17] = float("nan")
    o = _norm(x, None, w)
    assert torch.isnan(o["y"][2]).all() and torch.isnan(o["rstd"][2])
    keep = [0, 1, 3, 4]
    for k in ("y", "scale", "rstd"):
        assert torch.equal(o[k][keep], good[k][keep])


@pytest.mark.parametrize("which", ["x", "residual"])
def test_norm_sum_in_place(which):
    x, res, w = (_rand(s, i, 1.0, torch.bfloat16) for i, s in enumerate([(70, 4096), (70, 4096), (4096,)]))
    ref = _norm(x, res, w)
    a, b = x.clone(), res.clone()
    y = torch.empty_like(x)
    M.moe_rmsnorm(a, b, w, 1e-6, 70, 4096, 1, a if which == "x" else b, y, None, None, None)
    assert torch.equal(a if which == "x" else b, ref["sum"]) and torch.equal(y, ref["y"])


def test_norm_rows_past_2_31_elements():
    H, T = 4096, 2 ** 31 // 4096 + 5
    x = torch.zeros(T, H, device=DEV, dtype=torch.bfloat16)
    tail = _rand((4, H), 9, 1.0, torch.bfloat16)
    x[-4:] = tail
    w = _rand((H,), 10, 1.0, torch.bfloat16)
    y8 = torch.empty(T, H, device=DEV, dtype=torch.float8_e4m3fn)
    sc = torch.empty(T, H // 32, device=DEV, dtype=torch.uint8)
    M.moe_rmsnorm(x, None, w, 1e-6, T, H, 1, None, x, y8, sc, None)      # y over x
    ref = _norm(tail, None, w)
    assert torch.equal(x[-4:], ref["y"]) and torch.equal(sc[-4:], ref["scale"])
    assert torch.equal(y8[-4:].view(torch.uint8), ref["y8"].view(torch.uint8))


def _backward(dy, dsum, s, w, rstd, dx=None):
    T, H = s.shape
    dt = M.dtype_code(s)
    dx = torch.empty_like(s) if dx is None else dx
    dw = torch.empty(H, device=DEV)
    ws = torch.empty(M.moe_rmsnorm_backward_workspace_size(T, H, dt), device=DEV, dtype=torch.uint8)
    M.moe_rmsnorm_backward(dy, dsum, s, w, rstd, T, H, dt, dx, dw, ws, ws.numel())
    return dx, dw


def _backward_reference(dy, dsum, s, w, rstd):
    r, s, dy, w = rstd.double()[:, None], s.double(), dy.double(), w.double()
    xh, g = s * r, dy * w
    m = (g * xh).mean(1, keepdim=True)
    dx = r * (g - xh * m)
    # magnitudes of the terms that the float32 sums and differences round
    size = r * (g.abs() + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    if dsum is not None:
        dx, size = dx + dsum.double(), size + dsum.double().abs()
    return dx, size, (dy * xh).sum(0), (dy * xh).abs().sum(0)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,H", SHAPES + [(1025, 256), (2051, 96)])
@pytest.mark.parametrize("residual", [True, False])
def test_norm_backward(T, H, dt, residual):
    s, w, dy = _rand((T, H), 11, 2.0, dt), _rand((H,), 12, 1.0, dt), _rand((T, H), 13, 0.1, dt)
    dsum = _rand((T, H), 14, 0.1, dt) if residual else None
    rstd = (1 / torch.sqrt(s.double().square().mean(1) + 1e-6)).float()
    dx, dw = _backward(dy, dsum, s, w, rstd)
    rx, size, rw, wsize = _backward_reference(dy, dsum, s, w, rstd)
    _close(dx, rx, _step(dt), size * STAT)
    # a column's sum: at most 5 rows per block, 16 blocks' sums, 32 partial sums
    _close(dw, rw, U, wsize * 64 * U)


def test_norm_backward_against_differences():
    T, H = 3, 64
    x, res, w = _rand((T, H), 15), _rand((T, H), 16), _rand((H,), 17)
    dy, dsum = _rand((T, H), 18), _rand((T, H), 19)
    o = _norm(x, res, w, eps=1e-3)
    dx, dw = _backward(dy, dsum, o["sum"], w, o["rstd"])

    def loss(x, w):
        s = x + res.double()
        y = s / torch.sqrt(s.square().mean(1, keepdim=True) + 1e-3) * w
        return float((y * dy.double()).sum() + (s * dsum.double()).sum())
    h = 1e-5
    for t, c in ((0, 0), (1, 33), (2, 63)):
        d = torch.zeros(T, H, device=DEV, dtype=torch.float64)
        d[t, c] = h
        num = (loss(x.double() + d, w.double()) - loss(x.double() - d, w.double())) / (2 * h)
        assert abs(num - float(dx[t, c])) <= 1e-4 * max(1, abs(num))    # s is rounded to float32
        e = d[t]
        num = (loss(x.double(), w.double() + e) - loss(x.double(), w.double() - e)) / (2 * h)
        assert abs(num - float(dw[c])) <= 1e-4 * max(1, abs(num))


@pytest.mark.parametrize("over", ["dy", "dsum", "s"])
def test_norm_backward_in_place_and_repeatable(over):
    T, H, dt = 700, 4096, torch.bfloat16
    a = dict(dy=_rand((T, H), 20, 0.1, dt), dsum=_rand((T, H), 21, 0.1, dt), s=_rand((T, H), 22, 1.0, dt))
    w, rstd = _rand((H,), 23, 1.0, dt), torch.ones(T, device=DEV)
    dx, dw = _backward(a["dy"], a["dsum"], a["s"], w, rstd)
    dx2, dw2 = _backward(a["dy"], a["dsum"], a["s"], w, rstd, dx=a[over])
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_norm_backward_without_rows():
    dw = torch.ones(64, device=DEV)
    M.moe_rmsnorm_backward(None, None, None, None, None, 0, 64, 1, None, dw, None, 0)
    assert not dw.any()


def _dst(T, k, rows, seed, drop=0.0):
    """dst_row as a permutation writes it: distinct rows, -1 where dropped."""
    g = torch.Generator().manual_seed(seed)
    d = torch.randperm(rows, generator=g)[:T * k].reshape(T, k).to(torch.int32)
    d[torch.rand(T, k, generator=g) < drop] = -1
    return d.to(DEV)


@pytest.mark.parametrize("dt,ydt", [(a, b) for a in TYPES for b in TYPES])
@pytest.mark.parametrize("T,k,H", [(1, 1, 32), (33, 8, 7168), (5, 9, 96), (3, 32, 256), (130, 2, 4096), (2, 3, 16384)])
@pytest.mark.parametrize("drop", [0.0, 0.4])
def test_combine_backward(T, k, H, dt, ydt, drop):
    rows = T * k + 3
    dst, w = _dst(T, k, rows, 24, drop), _rand((T, k), 25).abs()
    dy, yp = _rand((T, H), 26, 0.1, dt), _rand((rows, H), 27, 1.0, ydt)
    dyp, dw = torch.full((rows, H), 7.0, device=DEV, dtype=ydt), torch.full((T, k), 7.0, device=DEV)
    M.moe_combine_backward(dy, M.dtype_code(dt), yp, M.dtype_code(ydt), dst, w, T, k, H, dyp, dw)
    ref = torch.full((rows, H), 7.0, device=DEV, dtype=ydt)
    keep = dst.reshape(-1) >= 0
    at = dst.reshape(-1).long()[keep]
    ref[at] = (w.reshape(-1, 1) * dy.float().repeat_interleave(k, 0)).to(ydt)[keep]    # one rounding each: exact
    assert torch.equal(dyp, ref)
    prod = dy.double().repeat_interleave(k, 0)[keep] * yp.double()[at]
    want, size = torch.zeros(T * k, device=DEV, dtype=torch.float64), torch.zeros(T * k, device=DEV, dtype=torch.float64)
    want[keep], size[keep] = prod.sum(1), prod.abs().sum(1)
    _close(dw.reshape(-1), want, U, size * STAT)
    M.moe_combine_backward(dy, M.dtype_code(dt), yp, M.dtype_code(ydt), dst, w, T, k, H, yp, dw)   # over y_perm
    assert torch.equal(yp[at], ref[at])


def test_calls_on_another_stream_and_in_a_graph():
    T, H, dt = 300, 4096, torch.bfloat16
    x, res, w, dy = _rand((T, H), 30, 1.0, dt), _rand((T, H), 31, 1.0, dt), _rand((H,), 32, 1.0, dt), _rand((T, H), 33, 0.1, dt)
    s, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(T, device=DEV)
    dx, dw = torch.empty_like(x), torch.empty(H, device=DEV)
    ws = torch.empty(M.moe_rmsnorm_backward_workspace_size(T, H, 1), device=DEV, dtype=torch.uint8)

    def step():
        M.moe_rmsnorm(x, res, w, 1e-6, T, H, 1, s, y, None, None, rstd)
        M.moe_rmsnorm_backward(dy, None, s, w, rstd, T, H, 1, dx, dw, ws, ws.numel())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        x.copy_(_rand((T, H), 40 + i, 1.0, dt))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (s, y, rstd, dx, dw)]
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (s, y, rstd, dx, dw)):
            assert torch.equal(a, b)
