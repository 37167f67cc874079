"""moe_grouped_ffn_train and moe_grouped_ffn_backward with gu of 16 bits per
value.

What is saved is read back by a decoder written from the form's definition and
held against the float32 form's gu: off by at most 2^-11 of the value plus
2^-17 of the largest of its four.  The gradients are compared bit for bit with
those of a float32 gu that holds the decoded values, and with the formula in
float64 from the rows themselves.  Tolerance of an element, fixed before the
first run: as in test_gpu_train.py, with g and u off by the above beside the
product's own error.  SiLU' is at most 1.1 and its slope at most 1/2 (at 0).
The whole: a gradient passes the rounding of the operand made from g and u and
its own, r / sqrt(3) each at most in root mean square (r = 2^-8), together
0.82 r, and those of g and u, an eighth of that each: 0.84 r of its 2-norm; with
many elements it is held to 0.85 r, with few to the 2 r of `check`.
"""
import pytest
import torch

import mixture_experts_layer_amd as M
from test_gpu_train import BF16, COUNTS, DEV, SIZES, U, Block, _rand, check

pytestmark = pytest.mark.gpu
R = 2.0 ** -8


def decode(gu):
    """The values of a 16-bit gu, in float32 (exactly: 11 significant bits)."""
    v = gu.view(torch.int16).int() & 0xffff
    e = ((v >> 13) & 3).reshape(v.shape[0], -1, 4)
    e = e[..., 0] | e[..., 1] << 2 | e[..., 2] << 4 | e[..., 3] << 6
    sign, field, low = v >> 15, (v >> 10) & 7, v & 1023
    half = torch.where(field > 0, (1024 + low).double() * torch.exp2((field - 25).double()), low.double() * 2.0 ** -24)
    scale = torch.exp2((e - 119).double()).repeat_interleave(4, 1)
    return (torch.where(sign > 0, -half, half) * scale).float()


def largest_of_four(v):
    return v.abs().reshape(v.shape[0], -1, 4).amax(-1).repeat_interleave(4, 1)


def gu_size(v):
    return 2.0 ** -11 * v.abs() + 2.0 ** -17 * largest_of_four(v)


def forward(b, dt):
    gu = torch.full((b.max_rows, 2 * b.I), 7.0, device=DEV, dtype=dt)
    y = torch.full((b.max_rows, b.H), 7.0, device=DEV, dtype=BF16)
    n = M.moe_grouped_ffn_train_workspace_size(b.max_rows, b.E, b.H, b.I, 1)
    ws = torch.full((n,), 255, device=DEV, dtype=torch.uint8)
    M.moe_grouped_ffn_train(*b._x(), b.offsets, b.E, b.max_rows, b.H, b.I, b.w13, b.w2, 1, gu, y, ws, n)
    return gu, y


def verify(b, dx, dw13, dw2, whole=2 * R):
    for e in range(b.E):
        lo, hi, x = b.rows(e)
        if lo == hi:
            assert not (dw13[e].any() or dw2[e].any())
            continue
        w13, w2, dy, I, n = b.w13[e].double(), b.w2[e].double(), b.dy[lo:hi].double(), b.I, hi - lo
        z, zs = x @ w13.t(), (x.abs() @ w13.abs().t()) * (b.H * U)
        zs = zs + gu_size(z.abs() + zs)
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
        for got, ref, size in (
                (dx[lo:hi], d @ w13, dsize @ w13.abs() * (1 + R) + (d.abs() @ w13.abs()) * (2 * I * U)),
                (dw2[e], dy.t() @ h, dy.abs().t() @ (hs * (1 + R) + n * U * h.abs())),
                (dw13[e], d.t() @ x, (dsize * (1 + R) + n * U * d.abs()).t() @ x.abs())):
            check(got, ref, size, BF16)
            assert float((got.double() - ref).norm()) <= whole * float(ref.norm())


def run(b, whole=2 * R):
    wide, y = forward(b, torch.float32)
    gu, y2 = forward(b, BF16)
    assert torch.equal(y, y2) and (gu[b.R:] == 7).all()
    held, want = decode(gu[:b.R]), wide[:b.R].double()
    assert ((held.double() - want).abs() <= gu_size(want)).all()
    got = b.backward(gu)
    for p, q in zip(got, b.backward(torch.cat([held, torch.full_like(wide[b.R:], 7.0)]))):
        assert torch.equal(p, q)
    assert (got[0][b.R:] == 7).all()
    verify(b, *got, whole=whole)


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("H,I", SIZES)
def test_forward_and_backward(counts, H, I):
    run(Block(counts, H, I, BF16, gather=(H + I) % 128 != 0, spare=3, seed=len(counts)))


@pytest.mark.parametrize("counts,H,I", [([0, 1000, 513, 300], 512, 256), ([1031, 511], 288, 544), ([2049], 1024, 416)])
def test_large_tiles(counts, H, I):
    run(Block(counts, H, I, BF16, seed=9), whole=0.85 * R)


def test_saved_values_of_every_size():
    """Rows from 2^-120 to 2^90, rows of zeros, columns of very different sizes
    side by side, the largest codes, and values that are not finite."""
    H, I = 64, 96
    b = Block([150, 0, 170], H, I, BF16, gather=False, seed=31)
    b.x *= torch.exp2(torch.linspace(-120, 90, b.R, device=DEV).round())[:, None].to(BF16)
    b.x[5:9] = 0
    b.w13 *= torch.exp2(-torch.arange(2 * I, device=DEV) % 13)[:, None].to(BF16)
    b.w13[0, :4], b.x[10] = 0.125, 1.0       # one group of the same value
    b.w13[2, 17, 3] = float("inf")          # g of column 17 alone, in the last expert's rows
    b.x[150:, 3] = b.x[150:, 3].abs() + 2.0 ** -126
    wide, _ = forward(b, torch.float32)
    gu, _ = forward(b, BF16)
    held, want = decode(gu), wide.double()
    group = torch.zeros(2 * I, dtype=torch.bool, device=DEV)
    group[16:20] = True
    keep = ~group
    assert ((held[:150].double() - want[:150]).abs() <= gu_size(want[:150]) + 2.0 ** -149).all()
    assert ((held[150:, keep].double() - want[150:, keep]).abs() <= gu_size(want[150:])[:, keep] + 2.0 ** -149).all()
    assert not torch.isfinite(want[150:, 17]).any() and not torch.isfinite(held[150:, 17]).any()
    assert not held[5:9].any()


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
            assert torch.equal(p.view(torch.int16), q.view(torch.int16))     # (gu holds no numbers)
    verify(b, dx, dw13, dw2)
