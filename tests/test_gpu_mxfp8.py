"""moe_grouped_ffn_mxfp8 against its formula in float64 on the values that the
MXFP8 elements and scales stand for.

Tolerances, fixed before the first run.  The scaled matrix instruction adds a
block of products with 16 significant bits at least: a product over n terms is
off by at most m = 2^-13 of the sum of the terms' magnitudes (blocks of 64 or
128, each off by a few units of its largest term's 2^-16, and float32 between
them).  h then is brought to e4m3: an element moves by at most 2^-4 of itself
(2^-10 of the block's scale below the normal range) from where the formula has
it, and where its own error carries it over a rounding border or its block's
scale over a power of two, by a whole step, 2^-3.  So an output is off by at
most sum |w2| (2^-3 |h| + |dh|) from W2 h with h unrounded; the sharper check
feeds the formula's own rounding of h and bounds the whole output: an element
next to a border (a share of about 2^-9, from errors of 2^-13 in steps of
2^-4) moves by 2^-3 of itself, so the 2-norm's error stays below
2^-3 sqrt(2^-9) = 2^-7.5 of the norm, taken with the output's own rounding as
2^-7.
"""
import pytest
import torch

import mixture_experts_layer_amd as M

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
MFMA = 2.0 ** -13


def _rand(shape, seed, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV) * scale


def quantize(v):
    """MXFP8 of v: elements, padded scale bytes."""
    K = v.shape[-1]
    b = v.double().reshape(v.shape[:-1] + (K // 32, 32))
    top = b.abs().amax(-1)
    e = torch.ceil(torch.log2(top.clamp_min(2.0 ** -140) / 448)).clamp(min=-127)
    e = torch.where((e > -127) & (top <= 448 * torch.exp2(e - 1)), e - 1, e)
    e = torch.where(top > 448 * torch.exp2(e), e + 1, e)
    q = (b * torch.exp2(-e)[..., None]).float().to(torch.float8_e4m3fn).reshape(v.shape)
    s = torch.zeros(v.shape[:-1] + (M.mx_pitch(K),), device=DEV, dtype=torch.uint8)
    s[..., :K // 32] = (e + 127).to(torch.uint8)
    return q, s


def value(q, s):
    K = q.shape[-1]
    f = torch.exp2(s[..., :K // 32].double() - 127)
    return q.double() * f.repeat_interleave(32, dim=-1)


class Block:
    def __init__(self, counts, H, I, gather=True, spare=0, seed=0, spread=False):
        self.E, self.H, self.I, self.R = len(counts), H, I, sum(counts)
        self.max_rows = self.R + spare
        self.offsets = torch.tensor([0] + counts).cumsum(0).to(torch.int32).to(DEV)
        T = max(1, self.R // 2) if gather else max(1, self.max_rows)
        g = torch.Generator().manual_seed(seed)
        self.src = torch.randint(0, T, (max(self.max_rows, 1),), generator=g).to(torch.int32).to(DEV) if gather else None
        x, s = _rand((T, H), seed + 1), H ** -0.5
        w13, w2 = _rand((self.E, 2 * I, H), seed + 2, s), _rand((self.E, H, I), seed + 3, s)
        if spread:          # blocks of very different scales
            x = x * torch.exp2(torch.randint(-6, 7, (T, H // 32), generator=g).to(DEV)).repeat_interleave(32, -1)
            w13 = w13 * torch.exp2(torch.randint(-4, 3, (self.E, 2 * I, H // 32), generator=g).to(DEV)).repeat_interleave(32, -1)
        (self.x8, self.xs), (self.w13, self.w13s), (self.w2, self.w2s) = quantize(x), quantize(w13), quantize(w2)

    def run(self, y_dt=BF16):
        y = torch.full((max(self.max_rows, 1), self.H), 7.0, device=DEV, dtype=y_dt)
        n = M.moe_grouped_ffn_mxfp8_workspace_size(self.max_rows, self.E, self.H, self.I)
        ws = torch.full((n,), 255, device=DEV, dtype=torch.uint8)
        M.moe_grouped_ffn_mxfp8(self.x8, self.xs, self.src, self.offsets, self.E, self.max_rows, self.H, self.I, self.w13,
                                self.w13s, self.w2, self.w2s, y, M.dtype_code(y_dt), ws, n)
        return y

    def verify(self, y):
        r = torch.finfo(y.dtype).eps / 2
        x = value(self.x8, self.xs)
        err2 = ref2 = 0.0
        for e in range(self.E):
            a, b = int(self.offsets[e]), int(self.offsets[e + 1])
            if a == b:
                continue
            xe = x[self.src[a:b].long()] if self.src is not None else x[a:b]
            w13, w2, I = value(self.w13[e], self.w13s[e]), value(self.w2[e], self.w2s[e]), self.I
            z, zs = xe @ w13.t(), (xe.abs() @ w13.abs().t()) * MFMA
            s = torch.sigmoid(z[:, :I])
            h = z[:, :I] * s * z[:, I:]
            dh = 1.1 * zs[:, :I] * (z[:, I:].abs() + zs[:, I:]) + (z[:, :I] * s).abs() * zs[:, I:]
            top = h.abs().reshape(b - a, -1, 32).amax(-1).repeat_interleave(32, -1)
            size = (2.0 ** -3 * h.abs() + dh + 2.0 ** -17 * top) @ w2.abs().t() + (h.abs() @ w2.abs().t()) * MFMA * 1.2
            got, ref = y[a:b].double(), h @ w2.t()
            bad = (got - ref).abs() > r * ref.abs() + size
            assert not bad.any(), (e, int(bad.sum()), bad.numel())
            ref = value(*quantize(h)) @ w2.t()
            err2, ref2 = err2 + float((got - ref).square().sum()), ref2 + float(ref.square().sum())
        assert err2 <= 2.0 ** -14 * ref2 + 1e-30, (err2 / ref2) ** 0.5


# few rows per expert: the direct kernel; about 100: 128-row tiles; over 384:
# 256-row tiles.  Contractions of 32, 64 and 96 past a multiple of 128.
FEW = [[1], [0, 2, 0, 17], [8] * 9, [0, 0, 0, 33, 1, 0, 0, 0]]
MANY = [[0, 100, 129], [256, 0, 9], [1000, 0, 513]]
SIZES = [(32, 32), (96, 160), (256, 192), (544, 1056), (1152, 64)]


@pytest.mark.parametrize("H,I", SIZES)
@pytest.mark.parametrize("counts", FEW + MANY, ids=lambda c: "-".join(map(str, c)))
def test_block(counts, H, I):
    b = Block(counts, H, I, gather=(H + I) % 128 != 0, spare=2, seed=len(counts), spread=(H > 32))
    for y_dt in (BF16, F32):
        y = b.run(y_dt)
        b.verify(y)
        assert (y[b.R:] == 7).all()


def test_full_width():
    b = Block([3, 0, 1, 4], 4096, 1536, seed=20)
    b.verify(b.run())


def test_many_experts():
    g = torch.Generator().manual_seed(3)
    b = Block(torch.randint(0, 5, (1024,), generator=g).tolist(), 64, 32, seed=21)
    b.verify(b.run())


def test_paths_agree_on_the_same_rows():
    """A row's output depends on its expert and itself alone, whichever kernel
    takes it: the same rows, few (direct) and repeated among many (tiles)."""
    b = Block([5, 7], 512, 256, gather=False, seed=22)
    few = b.run(F32)
    for times in (20, 90):
        m = Block([5 * times, 7 * times], 512, 256, gather=True, seed=22)
        m.x8, m.xs, m.w13, m.w13s, m.w2, m.w2s = b.x8, b.xs, b.w13, b.w13s, b.w2, b.w2s
        m.src = torch.cat([torch.arange(5).repeat(times), 5 + torch.arange(7).repeat(times)]).to(torch.int32).to(DEV)
        y = m.run(F32)
        m.verify(y)
        want = few[m.src.long()].double()
        assert float((y.double() - want).norm()) <= 2.0 ** -7 * float(want.norm())
        # every copy of a row the same bits
        assert torch.equal(y[:5], y[5:10]) and torch.equal(y[5 * times:5 * times + 7], y[-7:])


def test_scale_bytes_behind_the_blocks_do_not_matter():
    for counts in ([3, 5], [100, 30]):
        b = Block(counts, 160, 96, seed=23)
        want = b.run(F32)
        for s, K in ((b.xs, 160), (b.w13s, 160), (b.w2s, 96)):
            s[..., K // 32:] = 255
        assert torch.equal(b.run(F32), want)


def test_zero_rows_zero_blocks_and_extreme_scales():
    for counts in ([9, 4], [150, 40]):
        b = Block(counts, 256, 128, gather=False, seed=24)
        b.x8.view(torch.uint8)[0] = 0                  # a row of zeros: y = 0
        b.x8.view(torch.uint8)[1, 32:64] = 0x80        # a block of negative zeros
        b.xs[2] = torch.where(b.xs[2] > 0, b.xs[2] - 60, b.xs[2])
        b.w2s[1] = torch.where(b.w2s[1] > 0, b.w2s[1] + 30, b.w2s[1])
        y = b.run(F32)
        assert not y[0].any() and torch.isfinite(y).all()
        b.verify(y)


def test_bad_offsets_are_experts_without_rows():
    for counts in ([9, 4, 6], [150, 40, 60]):
        b = Block(counts, 96, 64, gather=False, seed=25)
        good = b.run(F32)
        a = counts[0]
        b.offsets = torch.tensor([0, a, a - 1, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
        y = b.run(F32)
        assert torch.equal(y[:a], good[:a]) and (y[a:] == 7).all()


def test_graph_replays():
    b = Block([30, 0, 11, 200], 512, 192, seed=26)
    n = M.moe_grouped_ffn_mxfp8_workspace_size(b.R, b.E, b.H, b.I)
    ws, y = torch.empty(n, device=DEV, dtype=torch.uint8), torch.empty(b.R, b.H, device=DEV, dtype=BF16)

    def step():
        M.moe_grouped_ffn_mxfp8(b.x8, b.xs, b.src, b.offsets, b.E, b.R, b.H, b.I, b.w13, b.w13s, b.w2, b.w2s, y, 1, ws, n)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        b.x8.copy_(quantize(_rand((b.x8.shape[0], b.H), 50 + i))[0])
        b.offsets.copy_(torch.tensor([0, 30 + i, 30 + i, 41, b.R], dtype=torch.int32))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = y.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, y)
    b.verify(y)


# one case for each pair of kernels that the two products may take: wide h
# (columns in groups of 32, contraction split over 2 and 4 waves), h in float32
# from groups of 8 and 16 columns, direct up with tiled down, tiled up with
# direct down
# more than 64 rows per expert, and few outputs: 16-row blocks all the same
@pytest.mark.parametrize("counts,H,I", [([300, 0, 129], 1376, 32), ([1030], 96, 64), ([65], 4096, 192), ([300], 160, 480)])
def test_many_rows_and_few_columns(counts, H, I):
    b = Block(counts, H, I, seed=28, spread=True)
    for y_dt in (BF16, F32):
        b.verify(b.run(y_dt))


@pytest.mark.parametrize("counts,H,I", [
    ([1, 0, 3], 64, 2080), ([2, 1], 96, 6240), ([8] * 9, 256, 1056), ([1, 2], 4096, 192),
    ([1, 2, 0, 1] * 18, 1376, 288), ([2, 1, 3] * 32, 160, 224), ([70], 256, 128), ([33, 50], 288, 2112)])
def test_each_choice_of_kernels(counts, H, I):
    b = Block(counts, H, I, seed=27)
    for y_dt in (BF16, F32):
        b.verify(b.run(y_dt))
