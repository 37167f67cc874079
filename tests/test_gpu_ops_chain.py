"""The operators around the layer, run one after another as a program runs
them: a serving step (norm with residual -> router -> permutation -> MXFP8
experts -> combine) and a training step (the same through the float32 training
experts, then every backward pass), against the formulas in float64.

The serving step's tolerance: the experts' part is within 2^-7 of the formula
in 2-norm (tests/test_gpu_mxfp8.py); combine adds bfloat16 roundings of the
expert rows and of the sum, 2^-8 each at most: 2^-7 + 2^-8 + 2^-8 = 2^-6.  The
training step is float32 throughout; its longest chain is 7 products and sums
of at most 512 terms, each off by 512 u of its magnitudes with errors of
random sign: 1e-5 of a gradient's 2-norm, as for one block, times 7.
"""
import pytest
import torch

import mixture_experts_layer_amd as M
from test_gpu_mxfp8 import quantize, value

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-6


def _rand(shape, seed, scale=1.0, dtype=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def _e(*shape, dtype=torch.float32):
    return torch.empty(shape, device=DEV, dtype=dtype)


def _route_and_permute(y, w_r, T, H, E, k, mode, dt):
    logits, ids, w = _e(T, E), _e(T, k, dtype=torch.int32), _e(T, k)
    M.moe_route(y, w_r, dt, T, H, E, k, mode, None, None, logits, ids, w)
    counts, off = _e(E, dtype=torch.int32), _e(E + 1, dtype=torch.int32)
    src, dst = _e(T * k, dtype=torch.int32), _e(T, k, dtype=torch.int32)
    n = M.moe_permute_workspace_size(T, k, E)
    ws = torch.empty(max(n, 16), device=DEV, dtype=torch.uint8)
    M.moe_permute(ids, T, k, E, 0, E, None, 0, dt, counts, off, src, dst, None, ws, n)
    return logits, ids, w, off, src, dst


@pytest.mark.parametrize("T", [1, 37, 700])
def test_serving_step(T):
    H, I, E, k = 512, 192, 16, 4
    bf = torch.bfloat16
    x, res, nw = _rand((T, H), 1, 1.0, bf), _rand((T, H), 2, 1.0, bf), _rand((H,), 3, 0.1, bf) + 1
    w_r = _rand((E, H), 4, H ** -0.5, bf)
    (w13, s13), (w2, s2) = quantize(_rand((E, 2 * I, H), 5, H ** -0.5)), quantize(_rand((E, H, I), 6, I ** -0.5))
    stream, y, y8 = _e(T, H, dtype=bf), _e(T, H, dtype=bf), _e(T, H, dtype=torch.float8_e4m3fn)
    ys, out, yp = _e(T, M.mx_pitch(H), dtype=torch.uint8), _e(T, H, dtype=bf), _e(T * k, H, dtype=bf)
    ws = torch.empty(M.moe_grouped_ffn_mxfp8_workspace_size(T * k, E, H, I), device=DEV, dtype=torch.uint8)
    M.moe_rmsnorm(x, res, nw, EPS, T, H, 1, stream, y, y8, ys, None)
    _, ids, w, off, src, dst = _route_and_permute(y, w_r, T, H, E, k, 0, 1)
    M.moe_grouped_ffn_mxfp8(y8, ys, src, off, E, T * k, H, I, w13, s13, w2, s2, yp, 1, ws, ws.numel())
    M.moe_combine(yp, 1, dst, w, T, k, H, None, out, 1)
    # the formula on the same ids and weights
    s = (x.float() + res.float()).to(bf)
    assert torch.equal(stream, s)
    n = s.double() / torch.sqrt(s.double().square().mean(1, keepdim=True) + EPS) * nw.double()
    a, d13, d2 = value(*quantize(n)), value(w13, s13), value(w2, s2)
    want = torch.zeros(T, H, device=DEV, dtype=torch.float64)
    for j in range(k):
        for e in range(E):
            t = (ids[:, j] == e).nonzero().reshape(-1)
            if t.numel():
                z = a[t] @ d13[e].t()
                h = torch.nn.functional.silu(z[:, :I]) * z[:, I:]
                want[t] += w[t, j:j + 1].double() * (value(*quantize(h)) @ d2[e].t())
    assert float((out.double() - want).norm()) <= 2.0 ** -6 * float(want.norm())


@pytest.mark.parametrize("T,k", [(48, 2), (5, 3)])
def test_training_step(T, k):
    """Loss <out, G> + <stream, G2>; the router's own gradient by torch on the
    library's ids."""
    H, I, E, dt = 128, 96, 8, 0
    x, res, nw, w_r = _rand((T, H), 11), _rand((T, H), 12), _rand((H,), 13, 0.2) + 1, _rand((E, H), 14, H ** -0.5)
    w13, w2 = _rand((E, 2 * I, H), 15, H ** -0.5), _rand((E, H, I), 16, I ** -0.5)
    G, G2 = _rand((T, H), 17), _rand((T, H), 18)
    R = T * k
    stream, y, rstd = _e(T, H), _e(T, H), _e(T)
    M.moe_rmsnorm(x, res, nw, EPS, T, H, dt, stream, y, None, None, rstd)
    logits, ids, w, off, src, dst = _route_and_permute(y, w_r, T, H, E, k, 0, dt)
    gu, yp, out = _e(R, 2 * I), _e(R, H), _e(T, H)
    n = max(M.moe_grouped_ffn_train_workspace_size(R, E, H, I, dt), M.moe_grouped_ffn_backward_workspace_size(R, E, H, I, dt))
    ws = torch.empty(n, device=DEV, dtype=torch.uint8)
    M.moe_grouped_ffn_train(None, y, src, off, E, R, H, I, w13, w2, dt, gu, yp, ws, n)
    M.moe_combine(yp, 0, dst, w, T, k, H, None, out, 0)
    # backward
    dyp, dw = _e(R, H), _e(T, k)
    M.moe_combine_backward(G, 0, yp, 0, dst, w, T, k, H, dyp, dw)
    dxp, d13, d2 = _e(R, H), torch.empty_like(w13), torch.empty_like(w2)
    M.moe_grouped_ffn_backward(dyp, None, y, src, off, E, R, H, I, w13, w2, dt, gu, dxp, d13, d2, ws, n)
    dy = _e(T, H)
    M.moe_combine(dxp, 0, dst, torch.ones(T, k, device=DEV), T, k, H, None, dy, 0)     # the copies' sum
    dl = torch.zeros(T, E, device=DEV).scatter_(1, ids.long(), w * (dw - (w * dw).sum(1, keepdim=True)))
    dy += dl @ w_r
    dx, dnw = _e(T, H), _e(H)
    wsn = torch.empty(M.moe_rmsnorm_backward_workspace_size(T, H, dt), device=DEV, dtype=torch.uint8)
    M.moe_rmsnorm_backward(dy, G2, stream, nw, rstd, T, H, dt, dx, dnw, wsn, wsn.numel())
    # the same by autograd in float64
    p = [t.double().requires_grad_() for t in (x, nw, w13, w2, w_r)]
    s = p[0] + res.double()
    yy = s / torch.sqrt(s.square().mean(1, keepdim=True) + EPS) * p[1]
    ww = torch.softmax((yy @ p[4].t()).gather(1, ids.long()), 1)
    o = torch.zeros(T, H, device=DEV, dtype=torch.float64)
    for j in range(k):
        for t in range(T):
            e = int(ids[t, j])
            z = p[2][e] @ yy[t]
            o[t] = o[t] + ww[t, j] * (p[3][e] @ (torch.nn.functional.silu(z[:I]) * z[I:]))
    ((o * G.double()).sum() + (s * G2.double()).sum()).backward()
    tol = 7e-5
    assert float((out.double() - o.detach()).norm()) <= tol * float(o.detach().norm())
    for got, ref in ((dx, p[0]), (dnw, p[1]), (d13, p[2]), (d2, p[3]), (dl.t() @ y, p[4])):
        assert float((got.double() - ref.grad).norm()) <= tol * float(ref.grad.norm())


# (19 rows: every expert full and pairs dropped; 122: none dropped, blank rows in
# every expert; 26 lies between)
@pytest.mark.parametrize("C", [19, 26, 122])
@pytest.mark.parametrize("dt", [0, 1])
def test_padded_and_dropped_tokens(dt, C):
    """With a capacity, the padded layout gives the packed layout's outputs and
    gradients (sums in another order: each within 1e-5 or, in bfloat16, 2^-7 of
    the formula in 2-norm), dropped pairs get zero gradients, and the blank rows
    add nothing."""
    T, H, I, E, k = 61, 96, 64, 5, 2
    d = [torch.float32, torch.bfloat16][dt]
    x, w_r, G = _rand((T, H), 41, 1.0, d), _rand((E, H), 42, H ** -0.5, d), _rand((T, H), 43, 1.0, d)
    w13, w2 = _rand((E, 2 * I, H), 44, H ** -0.5, d), _rand((E, H, I), 45, I ** -0.5, d)
    _, ids, w, _, _, _ = _route_and_permute(x, w_r, T, H, E, k, 0, dt)

    def run(padded):
        rows = E * C if padded else T * k
        i32 = torch.int32
        cnt, off, src, dst, drop = _e(E, dtype=i32), _e(E + 1, dtype=i32), _e(rows, dtype=i32), _e(T, k, dtype=i32), _e(1, dtype=i32)
        xp = _e(rows, H, dtype=d)
        wsp = torch.empty(max(M.moe_permute_workspace_size(T, k, E), 16), device=DEV, dtype=torch.uint8)
        M.moe_permute_capacity(ids, T, k, E, 0, E, C, padded, x, H, dt, cnt, off, src, dst, xp, drop, wsp, wsp.numel())
        n = max(M.moe_grouped_ffn_train_workspace_size(rows, E, H, I, dt), M.moe_grouped_ffn_backward_workspace_size(rows, E, H, I, dt))
        ws = torch.empty(n, device=DEV, dtype=torch.uint8)
        gu, yp, out = _e(rows, 2 * I), _e(rows, H, dtype=d), _e(T, H, dtype=d)
        M.moe_grouped_ffn_train(xp, None, None, off, E, rows, H, I, w13, w2, dt, gu, yp, ws, n)
        M.moe_combine(yp, dt, dst, w, T, k, H, None, out, dt)
        dyp, dw = torch.zeros(rows, H, device=DEV, dtype=d), _e(T, k)
        M.moe_combine_backward(G, dt, yp, dt, dst, w, T, k, H, dyp, dw)
        dxp, d13, d2 = _e(rows, H, dtype=d), torch.empty_like(w13), torch.empty_like(w2)
        M.moe_grouped_ffn_backward(dyp, xp, None, None, off, E, rows, H, I, w13, w2, dt, gu, dxp, d13, d2, ws, n)
        dx = _e(T, H, dtype=d)
        M.moe_combine(dxp, dt, dst, torch.ones(T, k, device=DEV), T, k, H, None, dx, dt)
        if padded:
            blank = src < 0
            assert not yp[blank].any() and not dxp[blank].any()
            assert int(blank.sum()) == rows - int(cnt.sum()) and (C < 122 or blank.any())
        assert not dw[dst < 0].any() and int((dst < 0).sum()) == int(drop) and (C > 19 or int(drop) > 0)
        return out, dw, dx, d13, d2
    for p, q in zip(run(0), run(1)):
        p, q = p.double(), q.double()
        assert float((p - q).norm()) <= 2 * (2.0 ** -7 if dt else 1e-5) * float(p.norm())


def test_rows_past_2_31_elements():
    """Expert rows and their gradients beyond 32-bit element offsets: the last
    rows equal those of a small call."""
    H, I, E = 4096, 32, 2
    R = 2 ** 31 // H + 700
    bf = torch.bfloat16
    x, w13, w2 = _rand((300, H), 21, 1.0, bf), _rand((E, 2 * I, H), 22, H ** -0.5, bf), _rand((E, H, I), 23, 0.2, bf)
    src = (torch.arange(R, device=DEV) % 300).int()
    off = torch.tensor([0, R - 500, R], dtype=torch.int32, device=DEV)
    tail_off = torch.tensor([0, 0, 500], dtype=torch.int32, device=DEV)
    tail_src = src[-500:].clone()
    dy_tail = _rand((500, H), 24, 0.1, bf)
    dy = torch.zeros(R, H, device=DEV, dtype=bf)
    dy[-500:] = dy_tail

    def train(rows, o, s, d):
        gu, y, dx = _e(rows, 2 * I), _e(rows, H, dtype=bf), _e(rows, H, dtype=bf)
        d13, d2 = torch.empty_like(w13), torch.empty_like(w2)
        n = max(M.moe_grouped_ffn_train_workspace_size(rows, E, H, I, 1), M.moe_grouped_ffn_backward_workspace_size(rows, E, H, I, 1))
        ws = torch.empty(n, device=DEV, dtype=torch.uint8)
        M.moe_grouped_ffn_train(None, x, s, o, E, rows, H, I, w13, w2, 1, gu, y, ws, n)
        M.moe_grouped_ffn_backward(d, None, x, s, o, E, rows, H, I, w13, w2, 1, gu, dx, d13, d2, ws, n)
        return y[-500:].clone(), dx[-500:].clone(), d13[1].clone(), d2[1].clone()
    for a, b in zip(train(R, off, src, dy), train(500, tail_off, tail_src, dy_tail)):
        assert torch.equal(a, b)
    del dy
    torch.cuda.empty_cache()
    (x8, xs), (q13, s13), (q2, s2) = quantize(x.float()), quantize(w13.float()), quantize(w2.float())

    def mx(rows, o, s):
        y = _e(rows, H, dtype=bf)
        n = M.moe_grouped_ffn_mxfp8_workspace_size(rows, E, H, I)
        ws = torch.empty(n, device=DEV, dtype=torch.uint8)
        M.moe_grouped_ffn_mxfp8(x8, xs, s, o, E, rows, H, I, q13, s13, q2, s2, y, 1, ws, n)
        return y[-500:].clone()
    # (the small call takes 16-row kernels, so the sums' order may differ: both
    # within 2^-7 of the formula)
    big, small = mx(R, off, src).double(), mx(500, tail_off, tail_src).double()
    assert float((big - small).norm()) <= 2.0 ** -6 * float(small.norm())
    torch.cuda.empty_cache()
