"""The C ABI of the operators around the layer (include/moe_ops.h) on the
host: declared, exported and bound alike, and bad arguments are rejected
before anything reaches a GPU.  No call here gets to a kernel launch."""
import ctypes
import inspect
import os
import re
import subprocess

import pytest
import torch

import mixture_experts_layer_amd as M
from conftest import ROOT

HEADER = os.path.join(ROOT, "include", "moe_ops.h")
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
P, MIS = 1 << 20, (1 << 20) + 4        # stand-ins for device addresses


def _header():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_declared_exported_and_bound_alike():
    names = sorted(set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", _header())))
    assert names == sorted(M.OPS_SYMBOLS)
    out = subprocess.run(["nm", "-D", "--defined-only", M.lib_path()], capture_output=True,
                         text=True, check=True).stdout
    assert set(names) <= set(re.findall(r"\sT\s(moe_\w+)", out))
    for n in names:
        assert n in M.__all__
        args = re.search(n + r"\s*\(([^)]*)\)", _header()).group(1)
        want = [a.split()[-1].lstrip("*") for a in args.split(",")]
        got = list(inspect.signature(getattr(M, n)).parameters)
        assert got == want, n
        assert len(want) == len(getattr(M.get_lib(), n).argtypes)


def test_mx_pitch():
    macro = re.search(r"#define MOE_MX_PITCH\(K\) (.*)", open(HEADER).read()).group(1)
    for K in (32, 96, 128, 160, 4096, 7168):
        want = eval(macro.replace("(K)", str(K)).replace("/", "//"))
        assert M.mx_pitch(K) == want >= K // 32 and want % 4 == 0


def _st(fn, *args):
    return getattr(M.lib, fn)(*args)


NORM = dict(x=P, residual=P, weight=P, eps=1e-6, T=4, H=256, dt=1, sum=P, y=P, y8=P, y8_scale=P,
            rstd=P, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(dt=2), INVALID), (dict(dt=-1), INVALID),
    (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(H=0), INVALID), (dict(H=-32), INVALID), (dict(H=100), UNSUPPORTED),
    (dict(H=16416), UNSUPPORTED), (dict(x=None), INVALID), (dict(weight=None), INVALID),
    (dict(y8=None), INVALID), (dict(y8_scale=None), INVALID),
    (dict(sum=None, y=None, y8=None, y8_scale=None, rstd=None), INVALID),
] + [({n: MIS}, INVALID) for n in ("x", "residual", "weight", "sum", "y", "y8", "y8_scale", "rstd")])
def test_rmsnorm_rejects(kw, status):
    a = dict(NORM, **kw)
    assert _st("moe_rmsnorm", *a.values()) == status


def test_rmsnorm_without_rows_is_a_no_op():
    assert _st("moe_rmsnorm", *dict(NORM, T=0).values()) == 0
    assert _st("moe_rmsnorm", *dict(NORM, T=0, x=None, weight=None).values()) == 0


NORM_BWD = dict(dy=P, dsum=P, s=P, weight=P, rstd=P, T=4, H=256, dt=1, dx=P, dweight=P, ws=P,
                ws_bytes=1 << 20, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(dt=2), INVALID), (dict(H=0), INVALID), (dict(H=48), UNSUPPORTED),
    (dict(H=16416), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(ws_bytes=4 * 256 * 4 - 1), WORKSPACE),
    (dict(T=0, dweight=None), INVALID),
] + [({n: None}, INVALID) for n in ("dy", "s", "weight", "rstd", "dx", "dweight")]
  + [({n: MIS}, INVALID) for n in ("dy", "dsum", "s", "weight", "rstd", "dx", "dweight", "ws")])
def test_rmsnorm_backward_rejects(kw, status):
    assert _st("moe_rmsnorm_backward", *dict(NORM_BWD, **kw).values()) == status


def test_rmsnorm_backward_workspace():
    q = M.moe_rmsnorm_backward_workspace_size
    assert q(1, 256, 1) >= 256 * 4 and q(8192, 7168, 1) >= 7168 * 4
    assert q(10 ** 9, 16384, 0) <= 1 << 30          # bounded however many rows
    for bad in ((-1, 256, 1), (4, 100, 1), (4, 256, 2), (4, 16416, 1)):
        assert q(*bad) == 0


COMBINE = dict(dy=P, dt=1, y_perm=P, y_perm_dt=1, dst_row=P, topk_w=P, T=4, k=2, H=256, dy_perm=P,
               dtopk_w=P, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(k=33), UNSUPPORTED), (dict(dt=5), INVALID),
    (dict(y_perm_dt=-1), INVALID), (dict(H=0), INVALID), (dict(H=33), UNSUPPORTED),
    (dict(H=16416), UNSUPPORTED), (dict(T=2 ** 30, k=2), UNSUPPORTED),
] + [({n: None}, INVALID) for n in ("dy", "y_perm", "dst_row", "topk_w", "dy_perm", "dtopk_w")]
  + [({n: MIS}, INVALID) for n in ("dy", "y_perm", "dst_row", "topk_w", "dy_perm", "dtopk_w")])
def test_combine_backward_rejects(kw, status):
    assert _st("moe_combine_backward", *dict(COMBINE, **kw).values()) == status


def test_the_binding_refuses_what_an_address_would_not_show():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    w = torch.zeros(256, dtype=torch.bfloat16)
    args = lambda **kw: [dict(x=x, residual=None, weight=w, eps=1e-6, T=4, H=256, dt=1, sum=None,  # noqa: E731
                              y=x, y8=None, y8_scale=None, rstd=None, **{})[n] if n not in kw else kw[n]
                         for n in list(NORM)[:-1]]
    with pytest.raises(ValueError, match="not a GPU"):
        M.moe_rmsnorm(*args())
    with pytest.raises(TypeError, match="x is torch.float32"):
        M.moe_rmsnorm(*args(x=x.float()))
    with pytest.raises(ValueError, match="not contiguous"):
        M.moe_rmsnorm(*args(x=torch.zeros(4, 512, dtype=torch.bfloat16)[:, ::2]))
    with pytest.raises(ValueError, match="fewer than"):
        M.moe_rmsnorm(*args(x=x[:3]))


TRAIN = dict(x_perm=None, x=P, src_token=P, offsets=P, E_loc=4, max_rows=16, H=256, I_loc=128, w13=P, w2=P, dt=1,
             gu=P, y_perm=P, ws=P, ws_bytes=1 << 20, stream=0)
BACKWARD = dict(dy_perm=P, x_perm=None, x=P, src_token=P, offsets=P, E_loc=4, max_rows=16, H=256, I_loc=128, w13=P,
                w2=P, dt=1, gu=P, dx_perm=P, dw13=P, dw2=P, ws=P, ws_bytes=1 << 20, stream=0)
BLOCK_SHAPES = [
    (dict(E_loc=0), INVALID), (dict(max_rows=-1), INVALID), (dict(H=0), INVALID), (dict(I_loc=0), INVALID),
    (dict(E_loc=1025), UNSUPPORTED), (dict(H=40), UNSUPPORTED), (dict(I_loc=48), UNSUPPORTED),
    (dict(H=65568), UNSUPPORTED), (dict(I_loc=65568), UNSUPPORTED), (dict(H=65536, I_loc=32768), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", BLOCK_SHAPES + [
    (dict(dt=2), INVALID), (dict(ws=None), WORKSPACE), (dict(ws_bytes=16 * 128 * 2 - 1), WORKSPACE),
    (dict(x=None), INVALID), (dict(src_token=None), INVALID),
] + [({n: None}, INVALID) for n in ("offsets", "w13", "w2", "gu", "y_perm")]
  + [({n: MIS}, INVALID) for n in ("x_perm", "x", "src_token", "offsets", "w13", "w2", "gu", "y_perm", "ws")])
def test_grouped_ffn_train_rejects(kw, status):
    assert _st("moe_grouped_ffn_train", *dict(TRAIN, **kw).values()) == status


@pytest.mark.parametrize("kw,status", BLOCK_SHAPES + [
    (dict(dt=2), INVALID), (dict(ws=None), WORKSPACE), (dict(ws_bytes=3 * 16 * 128 * 2 - 1), WORKSPACE),
    (dict(x=None), INVALID), (dict(src_token=None), INVALID), (dict(dw2=None), INVALID), (dict(dw13=None), INVALID),
    (dict(dx_perm=None, dw13=None, dw2=None), INVALID), (dict(max_rows=0, dw13=None), INVALID),
] + [({n: None}, INVALID) for n in ("dy_perm", "offsets", "w13", "w2", "gu")]
  + [({n: MIS}, INVALID) for n in ("dy_perm", "x_perm", "x", "src_token", "offsets", "w13", "w2", "gu", "dx_perm",
                                   "dw13", "dw2", "ws")])
def test_grouped_ffn_backward_rejects(kw, status):
    assert _st("moe_grouped_ffn_backward", *dict(BACKWARD, **kw).values()) == status


def test_training_without_rows_needs_nothing_but_the_gradients():
    none = dict(x=None, src_token=None, offsets=None, w13=None, w2=None, gu=None, ws=None, ws_bytes=0, max_rows=0)
    assert _st("moe_grouped_ffn_train", *dict(TRAIN, y_perm=None, **none).values()) == 0
    assert _st("moe_grouped_ffn_backward", *dict(BACKWARD, dy_perm=None, dw13=None, dw2=None, **none).values()) == 0


def test_training_workspaces():
    f, b = M.moe_grouped_ffn_train_workspace_size, M.moe_grouped_ffn_backward_workspace_size
    assert f(65536, 128, 4096, 1536, 1) >= 65536 * 1536 * 2 and b(65536, 128, 4096, 1536, 1) >= 3 * 65536 * 1536 * 2
    assert f(2 ** 22, 8, 4096, 14336, 1) == 2 ** 23 * 14336         # sizes beyond 32 bits
    for q in (f, b):
        for bad in ((-1, 4, 256, 128, 1), (4, 0, 256, 128, 1), (4, 4, 256, 100, 1), (4, 4, 256, 128, 3)):
            assert q(*bad) == 0


MX = dict(x8=P, x_scale=P, src_token=P, offsets=P, E_loc=4, max_rows=16, H=256, I_loc=128, w13=P, w13_scale=P, w2=P,
          w2_scale=P, y_perm=P, y_dt=1, ws=P, ws_bytes=1 << 20, stream=0)


@pytest.mark.parametrize("kw,status", BLOCK_SHAPES + [
    (dict(y_dt=2), INVALID), (dict(ws=None), WORKSPACE), (dict(ws_bytes=16 * 128), WORKSPACE),
] + [({n: None}, INVALID) for n in ("x8", "x_scale", "offsets", "w13", "w13_scale", "w2", "w2_scale", "y_perm")]
  + [({n: MIS}, INVALID) for n in ("x8", "x_scale", "src_token", "offsets", "w13", "w13_scale", "w2", "w2_scale",
                                   "y_perm", "ws")])
def test_grouped_ffn_mxfp8_rejects(kw, status):
    assert _st("moe_grouped_ffn_mxfp8", *dict(MX, **kw).values()) == status


def test_mxfp8_workspace_and_no_rows():
    q = M.moe_grouped_ffn_mxfp8_workspace_size
    assert q(65536, 128, 4096, 1536) >= 65536 * (1536 + 48)
    for bad in ((-1, 4, 256, 128), (4, 0, 256, 128), (4, 4, 256, 100), (4, 4, 65568, 32)):
        assert q(*bad) == 0
    none = {n: None for n in ("x8", "x_scale", "offsets", "w13", "w13_scale", "w2", "w2_scale", "y_perm", "ws")}
    assert _st("moe_grouped_ffn_mxfp8", *dict(MX, max_rows=0, **none).values()) == 0


def test_more_rows_than_a_launch_holds_are_refused():
    assert _st("moe_rmsnorm", *dict(NORM, T=2 ** 22, H=8192).values()) == UNSUPPORTED
    assert _st("moe_combine_backward", *dict(COMBINE, T=2 ** 22, H=8192, k=1).values()) == UNSUPPORTED


def test_a_workspace_for_the_largest_batch_serves_all():
    import random
    rng = random.Random(7)
    for q, tail in ((M.moe_grouped_ffn_mxfp8_workspace_size, ()), (M.moe_grouped_ffn_train_workspace_size, (1,)),
                    (M.moe_grouped_ffn_backward_workspace_size, (1,))):
        for _ in range(400):
            E, H, I = rng.choice([1, 8, 60, 128, 1024]), 32 * rng.randint(1, 256), 32 * rng.randint(1, 256)
            a, b = sorted(int(2 ** rng.uniform(0, 20)) for _ in range(2))
            assert 0 < q(a, E, H, I, *tail) <= q(b, E, H, I, *tail), (a, b, E, H, I)
    sizes = [M.moe_rmsnorm_backward_workspace_size(T, 4096, 1) for T in range(1, 2000, 7)]
    assert sizes == sorted(sizes)


class _OnDevice(torch.Tensor):
    """A CPU tensor that says it lives on a GPU, for the binding's own logic."""

    @staticmethod
    def __new__(cls, t, device):
        self = torch.Tensor._make_subclass(cls, t)
        self.where = device
        return self

    def get_device(self):
        return self.where


def test_the_binding_runs_on_the_tensors_device(monkeypatch):
    """Tensors of another GPU than the current one: the call is made with that
    GPU current and on its current stream; tensors of two GPUs are refused."""
    from contextlib import contextmanager
    from types import SimpleNamespace

    from mixture_experts_layer_amd import ops
    current, seen = [0], []

    @contextmanager
    def device(d):
        old, current[0] = current[0], d
        yield
        current[0] = old
    stub = SimpleNamespace(Tensor=torch.Tensor, cuda=SimpleNamespace(current_device=lambda: current[0], device=device),
                           _C=SimpleNamespace(_cuda_getCurrentRawStream=lambda d: 1000 + d))
    monkeypatch.setattr(ops, "_TORCH", stub)
    monkeypatch.setattr(ops, "_TYPES", {"f": (torch.float32,)})
    monkeypatch.setattr(ops, "_LIB", SimpleNamespace(f=lambda *a: seen.append((current[0], a[-1])) or 0))
    t0, t1 = _OnDevice(torch.zeros(4), 0), _OnDevice(torch.zeros(4), 1)
    ops._call("f", (("a", t0, "f", 4),), (t0,), None)
    ops._call("f", (("a", t1, "f", 4),), (t1,), None)
    ops._call("f", (("a", t1, "f", 4),), (t1,), 77)
    assert seen == [(0, 1000), (1, 1001), (1, 77)] and current[0] == 0
    with pytest.raises(ValueError, match="not cuda:0"):
        ops._call("f", (("a", t0, "f", 4), ("b", t1, "f", 4)), (t0, t1), None)


@pytest.mark.parametrize("fn,dt,shapes", [
    # (max_rows, E_loc, H, I_loc, accepted): the rows' own limit; float32 rows of
    # outputs; a float32 gradient; the gather of 2^28 rows in bfloat16
    ("train", 0, [(2 ** 28, 1, 32, 32, True), (2 ** 30 + 1, 1, 32, 32, False), (2 ** 29, 1, 32, 32, False),
                  (2 ** 26, 1, 32, 256, False), (64, 64, 4096, 16384, True), (64, 128, 4096, 16384, False)]),
    ("train", 1, [(2 ** 28 - 16, 1, 32, 32, True), (2 ** 28, 1, 32, 32, False), (64, 128, 4096, 16384, True)]),
    ("mxfp8", None, [(2 ** 30, 1, 32, 32, True), (2 ** 30 + 1, 1, 32, 32, False), (2 ** 30, 1, 32, 2048, False)])])
def test_shapes_past_a_launch_are_refused(fn, dt, shapes):
    tail = () if dt is None else (dt,)
    for rows, E, H, I, good in shapes:
        assert (getattr(M, f"moe_grouped_ffn_{fn}_workspace_size")(rows, E, H, I, *tail) > 0) == good
        # with a workspace of one byte an accepted shape stops there, a refused one before
        want = WORKSPACE if good else UNSUPPORTED
        if fn == "train":
            assert (M.moe_grouped_ffn_backward_workspace_size(rows, E, H, I, dt) > 0) == good
            assert _st("moe_grouped_ffn_train", P, P, P, P, E, rows, H, I, P, P, dt, P, P, P, 1, 0) == want
            assert _st("moe_grouped_ffn_backward", P, P, P, P, P, E, rows, H, I, P, P, dt, P, P, P, P, P, 1, 0) == want
        else:
            assert _st("moe_grouped_ffn_mxfp8", P, P, P, P, E, rows, H, I, P, P, P, P, P, 1, P, 1, 0) == want


@pytest.fixture
def calls(monkeypatch):
    """The binding's calls with tensors that say they live on GPU 0: [(function,
    arguments as the library would get them)]."""
    from contextlib import nullcontext
    from types import SimpleNamespace

    from mixture_experts_layer_amd import ops
    seen = []
    ops._setup()
    monkeypatch.setattr(ops, "_TORCH", SimpleNamespace(Tensor=torch.Tensor, cuda=SimpleNamespace(
        current_device=lambda: 0, device=lambda d: nullcontext())))
    monkeypatch.setattr(ops, "_launch", lambda fn, argv, dev, stream: seen.append((fn, argv)) or 0)
    return seen


def _gpu(*shape, dt=torch.bfloat16):
    return _OnDevice(torch.zeros(shape, dtype=dt), 0)


def test_the_saved_projections_may_be_of_the_rows_type(calls):
    """gu of a bfloat16 block is float32 or a bfloat16 tensor for the 16-bit form,
    as the caller has it; the C entries read which from dt, and the binding from
    the tensor."""
    b, f, i = torch.bfloat16, torch.float32, torch.int32
    z = _gpu

    def train(t, gu, dt):
        M.moe_grouped_ffn_train(None, z(4, 64, dt=t), z(4, dt=i), z(3, dt=i), 2, 4, 64, 32, z(2, 64, 64, dt=t),
                                z(2, 64, 32, dt=t), dt, gu, z(4, 64, dt=t), z(64, dt=torch.uint8), 64)

    def backward(t, gu, dt):
        M.moe_grouped_ffn_backward(z(4, 64, dt=t), None, z(4, 64, dt=t), z(4, dt=i), z(3, dt=i), 2, 4, 64, 32,
                                   z(2, 64, 64, dt=t), z(2, 64, 32, dt=t), dt, gu, z(4, 64, dt=t), None, None,
                                   z(64, dt=torch.uint8), 64)
    flag = int(re.search(r"#define MOE_GU_16 (\w+)", open(HEADER).read()).group(1), 0)
    for call, at in ((train, 10), (backward, 11)):
        for t, gu, dt, want in ((b, z(4, 64), 1, 1 | flag), (b, z(4, 64, dt=f), 1, 1), (f, z(4, 64, dt=f), 0, 0)):
            call(t, gu, dt)
            assert calls.pop()[1][at] == want
        for t, gu, dt in ((f, z(4, 64), 0), (b, z(4, 64, dt=torch.float16), 1)):
            with pytest.raises(TypeError, match="gu is"):
                call(t, gu, dt)
        with pytest.raises(ValueError, match="gu holds 192 elements"):
            call(b, z(3, 64), 1)
    for fn, a in (("moe_grouped_ffn_train", TRAIN), ("moe_grouped_ffn_backward", BACKWARD)):
        assert _st(fn, *dict(a, dt=1 | flag, ws_bytes=1).values()) == WORKSPACE
        assert _st(fn, *dict(a, dt=0 | flag).values()) == INVALID
        assert _st(fn, *dict(a, dt=2 | flag).values()) == INVALID
        q = getattr(M, fn + "_workspace_size")
        assert q(16, 4, 256, 128, 1 | flag) == q(16, 4, 256, 128, 1) > 0 == q(16, 4, 256, 128, flag)


def test_experts_of_2_32_bytes_are_refused_in_bfloat16_training():
    """The gate/up product addresses an expert's W13 by 32-bit offsets and a
    buffer of at most 2^32 - 1 bytes: 4 H I in bfloat16."""
    for H, I in ((32768, 32768), (65536, 16384), (16384, 65536)):
        for fn, a in (("moe_grouped_ffn_train", TRAIN), ("moe_grouped_ffn_backward", BACKWARD)):
            q = getattr(M, fn + "_workspace_size")
            assert q(16, 1, H, I, 1) == 0 < q(16, 1, H, I - 32, 1)
            assert q(16, 1, H, I, 0) > 0                # float32 is read by 64-bit addresses
            for size, want in ((I, UNSUPPORTED), (I - 32, WORKSPACE)):
                assert _st(fn, *dict(a, E_loc=1, H=H, I_loc=size, ws_bytes=1).values()) == want
        assert M.moe_grouped_ffn_mxfp8_workspace_size(16, 1, H, I) > 0      # 2^31 bytes


def test_the_documented_limit_of_rows_is_the_one_that_holds():
    limit = re.search(r"T \* (min\(64 \* ceil\(H / 512\), 1024\))\s*(?:\*\s*)?below 2\^32", open(HEADER).read()).group(1)
    for H in (32, 512, 544, 4096, 8192, 16384):
        threads = eval(limit, {"min": min, "ceil": lambda v: int(-(-v // 1)), "H": H})
        most = (2 ** 32 - 1) // threads
        for T, want in ((most, INVALID), (most + 1, UNSUPPORTED)):
            if T < 2 ** 31:
                assert _st("moe_rmsnorm", *dict(NORM, T=T, H=H, x=None).values()) == want
                assert _st("moe_combine_backward", *dict(COMBINE, T=T, H=H, k=1, dy=None).values()) == want


def test_the_combine_gradient_refuses_rows_shorter_than_those_it_reads(calls):
    """Every row that dst_row names is read in y_perm and written in dy_perm."""
    f, i = torch.float32, torch.int32

    def call(y_perm, dy_perm):
        M.moe_combine_backward(_gpu(4, 64), 1, y_perm, 1, _gpu(4, 2, dt=i), _gpu(4, 2, dt=f), 4, 2, 64, dy_perm,
                               _gpu(4, 2, dt=f))
    for rows in (8, 11):
        call(_gpu(8, 64), _gpu(rows, 64))
    assert len(calls) == 2
    for y, dy in ((8, 7), (11, 8)):
        with pytest.raises(ValueError, match="dy_perm holds .* fewer than"):
            call(_gpu(y, 64), _gpu(dy, 64))
    both = _gpu(8, 64)
    call(both, both)
    assert len(calls) == 3
