"""moe_grouped_ffn_train and moe_grouped_ffn_backward against their formulas
in float64.

Tolerances, fixed before the first run.  r = finfo(t).eps / 2 is the rounding
of a value to the block's type, u = 2^-24 that of a float32 step.  A product
over n terms accumulated in float32 is off by at most n u of the sum of its
terms' magnitudes.  An operand that was itself rounded (h, dg, du) or carries
an error adds that error times the other operand's magnitude, and the output
is rounded once.  `check` applies that bound to every element, and, since a
wrong term could hide below a sum of worst cases, bounds the whole output: the
roundings of a product's terms are independent, each of root mean square
r / sqrt(3) at most, so with the two or three roundings that an output passes
its error's 2-norm stays below 2 r of the output's (float32: below 1e-5).
"""
import pytest
import torch

import mixture_experts_layer_amd as M

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


def _rand(shape, seed, scale=1.0, dtype=F32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


class Block:
    """Experts of the given row counts, in rows of their own or gathered."""

    def __init__(self, counts, H, I, dt, gather=True, spare=0, tokens=None, seed=0):
        self.E, self.H, self.I, self.dt = len(counts), H, I, dt
        self.R = sum(counts)
        self.max_rows = self.R + spare
        self.offsets = torch.tensor([0] + counts).cumsum(0).to(torch.int32).to(DEV)
        T = tokens or max(1, self.R // 2)
        self.x = _rand((T if gather else self.max_rows, H), seed + 1, 1.0, dt)
        g = torch.Generator().manual_seed(seed)
        self.src = torch.randint(0, T, (max(self.max_rows, 1),), generator=g).to(torch.int32).to(DEV) if gather else None
        s = H ** -0.5
        self.w13, self.w2 = _rand((self.E, 2 * I, H), seed + 2, s, dt), _rand((self.E, H, I), seed + 3, s, dt)
        self.dy = _rand((self.max_rows, H), seed + 4, 0.1, dt)

    def _x(self):
        return (None, self.x, self.src) if self.src is not None else (self.x, None, None)

    def forward(self):
        c = M.dtype_code(self.dt)
        gu = torch.full((self.max_rows, 2 * self.I), 7.0, device=DEV)
        y = torch.full((self.max_rows, self.H), 7.0, device=DEV, dtype=self.dt)
        ws = torch.full((M.moe_grouped_ffn_train_workspace_size(self.max_rows, self.E, self.H, self.I, c),), 255,
                        device=DEV, dtype=torch.uint8)
        M.moe_grouped_ffn_train(*self._x(), self.offsets, self.E, self.max_rows, self.H, self.I, self.w13, self.w2, c,
                                gu, y, ws, ws.numel())
        return gu, y

    def backward(self, gu, dx=True, dw=True):
        c = M.dtype_code(self.dt)
        dx = torch.full((self.max_rows, self.H), 7.0, device=DEV, dtype=self.dt) if dx else None
        dw13 = torch.full_like(self.w13, 7.0) if dw else None
        dw2 = torch.full_like(self.w2, 7.0) if dw else None
        ws = torch.full((M.moe_grouped_ffn_backward_workspace_size(self.max_rows, self.E, self.H, self.I, c),), 255,
                        device=DEV, dtype=torch.uint8)
        M.moe_grouped_ffn_backward(self.dy, *self._x(), self.offsets, self.E, self.max_rows, self.H, self.I, self.w13,
                                   self.w2, c, gu, dx, dw13, dw2, ws, ws.numel())
        return dx, dw13, dw2

    def rows(self, e):
        a, b = int(self.offsets[e]), int(self.offsets[e + 1])
        x = self.x[self.src[a:b].long()] if self.src is not None else self.x[a:b]
        return a, b, x.double()


def check(got, ref, size, dt):
    """got against ref: elements within r |ref| + size, the whole within 2 r."""
    r = torch.finfo(dt).eps / 2
    err = (got.double() - ref).abs()
    bad = err > r * ref.abs() * (1 + 1e-6) + size
    assert not bad.any(), (int(bad.sum()), bad.numel(), float((err / (r * ref.abs() + size)).max()))
    norm = float(ref.norm())
    assert float(err.norm()) <= (2 * r if dt == BF16 else 1e-5) * norm + 1e-30, float(err.norm()) / norm


def verify(b, gu, y, dx, dw13, dw2):
    r = torch.finfo(b.dt).eps / 2
    I, H = b.I, b.H
    for e in range(b.E):
        lo, hi, x = b.rows(e)
        w13, w2, dy = b.w13[e].double(), b.w2[e].double(), b.dy[lo:hi].double()
        if hi == lo:
            assert dw13 is None or not (dw13[e].any() or dw2[e].any())
            continue
        # forward
        z, zsize = x @ w13.t(), (x.abs() @ w13.abs().t()) * (H * U)
        check(gu[lo:hi], z, zsize, F32)
        g, u, gs, us = z[:, :I], z[:, I:], zsize[:, :I], zsize[:, I:]
        s = torch.sigmoid(g)
        h = g * s * u
        hs = r * h.abs() + 1.1 * gs * (u.abs() + us) + (g * s).abs() * us + 8 * U * h.abs()
        check(y[lo:hi], h @ w2.t(), (hs @ w2.abs().t()) + (h.abs() @ w2.abs().t()) * (I * U), b.dt)
        if dx is None and dw2 is None:
            continue
        # backward, from the saved g and u
        g, u = gu[lo:hi, :I].double(), gu[lo:hi, I:].double()
        s = torch.sigmoid(g)
        h, ds = g * s * u, s * (1 + g * (1 - s))
        dh, dhs = dy @ w2, (dy.abs() @ w2.abs()) * (H * U)
        d = torch.cat([dh * u * ds, dh * g * s], 1)
        dsize = torch.cat([dhs * (u * ds).abs() + dh.abs() * u.abs() * 16 * U, dhs * (g * s).abs()], 1) + (r + 8 * U) * d.abs()
        n = hi - lo
        if dx is not None:
            check(dx[lo:hi], d @ w13, dsize @ w13.abs() + (d.abs() @ w13.abs()) * (2 * I * U), b.dt)
        if dw2 is not None:
            hs = (r + 8 * U) * h.abs()
            check(dw2[e], dy.t() @ h, dy.abs().t() @ (hs + n * U * h.abs()), b.dt)
            check(dw13[e], d.t() @ x, (dsize + n * U * d.abs()).t() @ x.abs(), b.dt)


# counts: empty experts first, last and between; one row; around the tiles of
# 128 and 256 rows and the chunks of 64 and 16
COUNTS = [[1], [0, 1, 0], [63, 0, 65, 16], [129, 127, 1, 0, 17], [0, 256, 257, 33]]
SIZES = [(32, 32), (96, 160), (256, 512), (288, 352), (1056, 64), (64, 1056)]


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("H,I", SIZES)
def test_forward_and_backward(counts, H, I, dt):
    b = Block(counts, H, I, dt, gather=(H + I) % 128 != 0, spare=3, seed=len(counts))
    gu, y = b.forward()
    dx, dw13, dw2 = b.backward(gu)
    torch.cuda.synchronize()
    verify(b, gu, y, dx, dw13, dw2)
    for t in (gu, y, dx):                      # rows behind the last expert's
        assert (t[b.R:] == 7.0).all()


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("counts,H,I", [([0, 1000, 513, 300], 512, 256), ([1031, 511], 288, 544), ([2049], 1024, 416)])
def test_large_tiles(counts, H, I, gather):
    b = Block(counts, H, I, BF16, gather=gather, seed=9)
    gu, y = b.forward()
    verify(b, gu, y, *b.backward(gu))


def test_many_experts_with_few_rows():
    g = torch.Generator().manual_seed(5)
    counts = torch.randint(0, 9, (300,), generator=g).tolist()
    b = Block(counts, 128, 96, BF16, seed=11)
    gu, y = b.forward()
    verify(b, gu, y, *b.backward(gu))


@pytest.mark.parametrize("dt", [BF16, F32])
def test_parts_of_the_backward_alone(dt):
    b = Block([70, 0, 130], 256, 96, dt, seed=12)
    gu, _ = b.forward()
    dx, dw13, dw2 = b.backward(gu)
    a, none13, none2 = b.backward(gu, dw=False)
    assert none13 is None and torch.equal(a, dx)
    none, c, d = b.backward(gu, dx=False)
    assert none is None and torch.equal(c, dw13) and torch.equal(d, dw2)


def test_matches_the_inference_path():
    """The training forward is moe_grouped_ffn on the same rows."""
    b = Block([300, 0, 129, 4], 512, 256, BF16, seed=13)
    _, y = b.forward()
    ws = torch.empty(M.moe_grouped_ffn_workspace_size(b.R, b.E, b.H, b.I, 1), device=DEV, dtype=torch.uint8)
    want = torch.empty(b.R, b.H, device=DEV, dtype=BF16)
    M.moe_grouped_ffn(None, b.x, b.src, b.offsets, b.E, b.R, b.H, b.I, b.w13, b.w2, 1, want, 1, ws, ws.numel())
    # each is within its own roundings of the formula: twice those apart
    assert float((y[:b.R].double() - want.double()).norm()) <= 4 * 2.0 ** -8 * float(want.double().norm())


@pytest.mark.parametrize("dt", [BF16, F32])
def test_no_rows_gives_zero_gradients(dt):
    b = Block([0, 0, 0], 96, 64, dt, seed=14)
    dw13, dw2 = torch.ones_like(b.w13), torch.ones_like(b.w2)
    M.moe_grouped_ffn_backward(None, None, None, None, None, 3, 0, 96, 64, None, None, M.dtype_code(dt), None, None,
                               dw13, dw2, None, 0)
    assert not dw13.any() and not dw2.any()
    b.max_rows = 5                      # rows there are, but none of them an expert's
    b.dy, b.src = _rand((5, 96), 1, 1.0, dt), torch.zeros(5, device=DEV, dtype=torch.int32)
    gu, y = b.forward()
    dx, dw13, dw2 = b.backward(gu)
    assert (gu == 7).all() and (y == 7).all() and (dx == 7).all() and not dw13.any() and not dw2.any()


@pytest.mark.parametrize("dt", [BF16, F32])
def test_offsets_outside_the_rows_are_experts_without_rows(dt):
    b = Block([40, 30, 20, 10], 64, 96, dt, seed=15)
    gu, y = b.forward()
    good = b.backward(gu)
    b.offsets = torch.tensor([0, 40, 70, 90, 2 ** 31 - 1], dtype=torch.int32, device=DEV)   # the last one runs out
    gu2, y2 = b.forward()
    dx, dw13, dw2 = b.backward(gu)
    assert torch.equal(gu2[:90], gu[:90]) and torch.equal(y2[:90], y[:90]) and (gu2[90:] == 7).all() and (y2[90:] == 7).all()
    assert torch.equal(dx[:90], good[0][:90]) and (dx[90:] == 7).all()
    assert torch.equal(dw13[:3], good[1][:3]) and torch.equal(dw2[:3], good[2][:3]) and not dw13[3].any() and not dw2[3].any()
    b.offsets = torch.tensor([0, 40, 10, -5, 200], dtype=torch.int32, device=DEV)           # backwards, negative
    dx, dw13, dw2 = b.backward(gu)
    assert torch.equal(dw2[0], good[2][0]) and not dw2[1:].any() and not dw13[1:].any() and (dx[40:] == 7).all()


def test_nan_stays_with_its_expert():
    b = Block([70, 37, 130], 96, 160, BF16, gather=False, seed=16)
    gu, y = b.forward()
    good = b.backward(gu)
    b.x[70:107] = float("nan")
    b.dy[70:107] = float("inf")
    gu2, y2 = b.forward()
    dx, dw13, dw2 = b.backward(gu2)
    keep = list(range(70)) + list(range(107, 237))
    assert torch.isnan(y2[70:107]).all() and torch.isnan(dw13[1]).all()
    assert torch.equal(y2[keep], y[keep]) and torch.equal(dx[keep], good[0][keep])
    assert torch.equal(dw13[[0, 2]], good[1][[0, 2]]) and torch.equal(dw2[[0, 2]], good[2][[0, 2]])


def test_gradients_against_differences():
    b = Block([3, 0, 5], 32, 64, F32, seed=17)
    gu, _ = b.forward()
    dx, dw13, dw2 = b.backward(gu)

    def loss(x, w13, w2):
        total = 0.0
        for e in range(b.E):
            lo, hi = int(b.offsets[e]), int(b.offsets[e + 1])
            z = x[lo:hi] @ w13[e].t()
            h = torch.nn.functional.silu(z[:, :b.I]) * z[:, b.I:]
            total += float(((h @ w2[e].t()) * b.dy[lo:hi].double()).sum())
        return total
    args = [b.x[b.src.long()].double(), b.w13.double(), b.w2.double()]
    for i, grad in ((0, dx), (1, dw13), (2, dw2)):
        for at in ((0, 1), (4, 30)) if i == 0 else ((0, 5, 3), (2, 20, 31), (1, 0, 0)):
            d = torch.zeros_like(args[i])
            d[at] = 1e-6
            plus, minus = list(args), list(args)
            plus[i], minus[i] = args[i] + d, args[i] - d
            num = (loss(*plus) - loss(*minus)) / 2e-6
            assert abs(num - float(grad[at])) <= 1e-5 * max(1.0, abs(num))


def test_repeatable_on_other_streams_and_in_a_graph():
    b = Block([300, 5, 0, 411], 512, 160, BF16, seed=18)
    c = 1
    gu, y = torch.empty(b.R, 2 * b.I, device=DEV), torch.empty(b.R, b.H, device=DEV, dtype=BF16)
    dx, dw13, dw2 = torch.empty_like(y), torch.empty_like(b.w13), torch.empty_like(b.w2)
    n = max(M.moe_grouped_ffn_train_workspace_size(b.R, b.E, b.H, b.I, c),
            M.moe_grouped_ffn_backward_workspace_size(b.R, b.E, b.H, b.I, c))
    ws = torch.empty(n, device=DEV, dtype=torch.uint8)

    def step():
        M.moe_grouped_ffn_train(None, b.x, b.src, b.offsets, b.E, b.R, b.H, b.I, b.w13, b.w2, c, gu, y, ws, n)
        M.moe_grouped_ffn_backward(b.dy, None, b.x, b.src, b.offsets, b.E, b.R, b.H, b.I, b.w13, b.w2, c, gu, dx, dw13,
                                   dw2, ws, n)
    outs = (gu, y, dx, dw13, dw2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    first = [t.clone() for t in outs]
    step()
    torch.cuda.synchronize()
    for p, q in zip(first, outs):
        assert torch.equal(p, q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        b.x.copy_(_rand(tuple(b.x.shape), 30 + i, 1.0, BF16))
        b.offsets.copy_(torch.tensor([0, 300 - 10 * i, 300, 310 + i, b.R], dtype=torch.int32))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        step()
        torch.cuda.synchronize()
        for p, q in zip(got, outs):
            assert torch.equal(p, q)
    verify(b, *outs)
