"""moe_grouped_ffn_train and moe_grouped_ffn_backward with gu in bfloat16.

What is saved is the float32 form's gu rounded once, so the two forms are
compared bit for bit, and the gradients with the formula in float64 from the
rows themselves.  Tolerance of an element, fixed before the first run: as in
test_gpu_train.py, with g and u off by r = 2^-8 of themselves beside the
product's own error.  SiLU' is at most 1.1 and its slope at most 1/2 (at 0).
The whole: a gradient passes the roundings of g, u, of the operand made from
them and its own, four of root mean square r / sqrt(3) each (g's times a slope
of about 1), together 1.2 r: below 2 r of its 2-norm, as `check` has it.
"""
import pytest
import torch

import mixture_experts_layer_amd as M
from test_gpu_train import BF16, COUNTS, DEV, SIZES, U, Block, _rand, check

pytestmark = pytest.mark.gpu
R = 2.0 ** -8


def forward(b, dt):
    gu = torch.full((b.max_rows, 2 * b.I), 7.0, device=DEV, dtype=dt)
    y = torch.full((b.max_rows, b.H), 7.0, device=DEV, dtype=BF16)
    n = M.moe_grouped_ffn_train_workspace_size(b.max_rows, b.E, b.H, b.I, 1)
    ws = torch.full((n,), 255, device=DEV, dtype=torch.uint8)
    M.moe_grouped_ffn_train(*b._x(), b.offsets, b.E, b.max_rows, b.H, b.I, b.w13, b.w2, 1, gu, y, ws, n)
    return gu, y


def verify(b, dx, dw13, dw2):
    for e in range(b.E):
        lo, hi, x = b.rows(e)
        if lo == hi:
            assert not (dw13[e].any() or dw2[e].any())
            continue
        w13, w2, dy, I, n = b.w13[e].double(), b.w2[e].double(), b.dy[lo:hi].double(), b.I, hi - lo
        z, zs = x @ w13.t(), (x.abs() @ w13.abs().t()) * (b.H * U)
        zs = zs + R * (z.abs() + zs)
        g, u, gs, us = z[:, :I], z[:, I:], zs[:, :I], zs[:, I:]
        s = torch.sigmoid(g)
        silu, ds = g * s, s * (1 + g * (1 - s))
        dh, dhs = dy @ w2, (dy.abs() @ w2.abs()) * (b.H * U)
        h, hs = silu * u, 1.1 * gs * (u.abs() + us) + silu.abs() * us
        slope, slopes = u * ds, 0.5 * gs * (u.abs() + us) + ds.abs() * us
        d = torch.cat([dh * slope, dh * silu], 1)
        dsize = torch.cat([(dh.abs() + dhs) * slopes + dhs * slope.abs(), (dh.abs() + dhs) * 1.1 * gs + dhs * silu.abs()], 1)
        dsize = dsize + (R + 16 * U) * (d.abs() + dsize)
        hs = hs + (R + 16 * U) * (h.abs() + hs)
        check(dx[lo:hi], d @ w13, dsize @ w13.abs() * (1 + R) + (d.abs() @ w13.abs()) * (2 * I * U), BF16)
        check(dw2[e], dy.t() @ h, dy.abs().t() @ (hs * (1 + R) + n * U * h.abs()), BF16)
        check(dw13[e], d.t() @ x, (dsize * (1 + R) + n * U * d.abs()).t() @ x.abs(), BF16)


def run(b):
    wide, y = forward(b, torch.float32)
    gu, y2 = forward(b, BF16)
    assert torch.equal(y, y2) and torch.equal(gu, wide.to(BF16))
    assert (gu[b.R:] == 7).all()
    got = b.backward(gu)
    for p, q in zip(got, b.backward(gu.float())):
        assert torch.equal(p, q)
    assert (got[0][b.R:] == 7).all()
    verify(b, *got)


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("H,I", SIZES)
def test_forward_and_backward(counts, H, I):
    run(Block(counts, H, I, BF16, gather=(H + I) % 128 != 0, spare=3, seed=len(counts)))


@pytest.mark.parametrize("counts,H,I", [([0, 1000, 513, 300], 512, 256), ([1031, 511], 288, 544), ([2049], 1024, 416)])
def test_large_tiles(counts, H, I):
    run(Block(counts, H, I, BF16, seed=9))


def test_graph_replays():
    b = Block([300, 5, 0, 411], 512, 160, BF16, seed=18)
    gu, y = torch.empty(b.R, 2 * b.I, device=DEV, dtype=BF16), torch.empty(b.R, b.H, device=DEV, dtype=BF16)
    dx, dw13, dw2 = torch.empty_like(y), torch.empty_like(b.w13), torch.empty_like(b.w2)
    n = max(M.moe_grouped_ffn_train_workspace_size(b.R, b.E, b.H, b.I, 1),
            M.moe_grouped_ffn_backward_workspace_size(b.R, b.E, b.H, b.I, 1))
    ws = torch.empty(n, device=DEV, dtype=torch.uint8)

    def step():
        M.moe_grouped_ffn_train(None, b.x, b.src, b.offsets, b.E, b.R, b.H, b.I, b.w13, b.w2, 1, gu, y, ws, n)
        M.moe_grouped_ffn_backward(b.dy, None, b.x, b.src, b.offsets, b.E, b.R, b.H, b.I, b.w13, b.w2, 1, gu, dx, dw13,
                                   dw2, ws, n)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        b.x.copy_(_rand(tuple(b.x.shape), 30 + i, 1.0, BF16))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (gu, y, dx, dw13, dw2)]
        step()
        torch.cuda.synchronize()
        for p, q in zip(got, (gu, y, dx, dw13, dw2)):
            assert torch.equal(p, q)
    verify(b, dx, dw13, dw2)
