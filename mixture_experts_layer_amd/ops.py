"""Python binding of the operators around the layer (include/moe_ops.h), with
the names and argument orders of the C entry points.

Arguments are contiguous torch tensors on one GPU (or None for NULL).  Unlike
the raw C entry points, which see only addresses, a call here refuses a tensor
whose type, layout, size or device is not what the entry point will read; it
runs on that GPU's current stream unless `stream` names another of its
streams.  What lies in the tensors is not looked at: that src_token names rows
of x or x8, and dst_row rows of y_perm, is the caller's to hold.
"""
from __future__ import annotations

from ._abi import MOE_BF16, MOE_F32, MOE_GU_16


def mx_pitch(K: int) -> int:
    """Scale bytes of an MXFP8 row of K elements (MOE_MX_PITCH)."""
    return (K + 127) // 128 * 4


_TORCH = _LIB = _TYPES = None


def _setup():
    global _TORCH, _LIB, _TYPES
    import torch

    from . import get_lib
    _TORCH = torch
    _TYPES = {MOE_F32: (torch.float32,), MOE_BF16: (torch.bfloat16,), "f": (torch.float32,),
              "i": (torch.int32,), "b": (torch.uint8,), "8": (torch.float8_e4m3fn, torch.uint8)}
    _LIB = get_lib()


def _call(fn, tensors, args, stream):
    """Check `tensors` ((name, tensor or None, type, least elements) each) and
    call the library's `fn` with `args`, in which a tensor stands for its
    address, and the stream appended."""
    if _LIB is None:
        _setup()
    dev = None
    for name, t, kind, least in tensors:
        if t is None:
            continue
        want = _TYPES.get(kind)
        if want is not None and t.dtype not in want:
            raise TypeError(f"{fn}: {name} is {t.dtype}, not {want[0]}")
        if not t.is_contiguous():
            raise ValueError(f"{fn}: {name} is not contiguous")
        if t.numel() < least:
            raise ValueError(f"{fn}: {name} holds {t.numel()} elements, fewer than {least}")
        d = t.get_device()
        if d != dev:
            if d < 0 or dev is not None:
                raise ValueError(f"{fn}: {name} is on {t.device}, not " +
                                 ("a GPU" if dev is None else f"cuda:{dev}"))
            dev = d
    tensor = _TORCH.Tensor
    argv = [a.data_ptr() if isinstance(a, tensor) else a for a in args]
    here = _TORCH.cuda.current_device()
    if dev is None or dev == here:
        status = _launch(fn, argv, here, stream)
    else:
        with _TORCH.cuda.device(dev):
            status = _launch(fn, argv, dev, stream)
    if status != 0:
        from . import MoEError
        raise MoEError(fn, status)


def _launch(fn, argv, dev, stream):
    if stream is None:
        # the handle of torch.cuda.current_stream(dev), without the stream object
        stream = _TORCH._C._cuda_getCurrentRawStream(dev)
    return getattr(_LIB, fn)(*argv, stream)


def _gu(gu, dt):
    """dt of a training block's rows, its gu's type for _call, and dt as the
    library takes it: with bfloat16 rows a gu of that type is the 16-bit form."""
    dt &= ~MOE_GU_16
    if _LIB is None:
        _setup()
    if dt == MOE_BF16 and gu is not None and gu.dtype == _TYPES[MOE_BF16][0]:
        return dt, MOE_BF16, dt | MOE_GU_16
    return dt, "f", dt


def moe_rmsnorm(x, residual, weight, eps, T, H, dt, sum, y, y8, y8_scale, rstd, stream=None):
    n = T * H
    _call("moe_rmsnorm",
          (("x", x, dt, n), ("residual", residual, dt, n), ("weight", weight, dt, H),
           ("sum", sum, dt, n), ("y", y, dt, n), ("y8", y8, "8", n),
           ("y8_scale", y8_scale, "b", T * mx_pitch(H)), ("rstd", rstd, "f", T)),
          (x, residual, weight, eps, T, H, dt, sum, y, y8, y8_scale, rstd), stream)


def moe_rmsnorm_backward_workspace_size(T, H, dt) -> int:
    from . import lib
    return lib.moe_rmsnorm_backward_workspace_size(T, H, dt)


def moe_rmsnorm_backward(dy, dsum, s, weight, rstd, T, H, dt, dx, dweight, ws, ws_bytes,
                         stream=None):
    n = T * H
    _call("moe_rmsnorm_backward",
          (("dy", dy, dt, n), ("dsum", dsum, dt, n), ("s", s, dt, n), ("weight", weight, dt, H),
           ("rstd", rstd, "f", T), ("dx", dx, dt, n), ("dweight", dweight, "f", H),
           ("ws", ws, "b", ws_bytes)),
          (dy, dsum, s, weight, rstd, T, H, dt, dx, dweight, ws, ws_bytes), stream)


def moe_combine_backward(dy, dt, y_perm, y_perm_dt, dst_row, topk_w, T, k, H, dy_perm, dtopk_w,
                         stream=None):
    _call("moe_combine_backward",
          (("dy", dy, dt, T * H), ("y_perm", y_perm, y_perm_dt, 0),
           ("dst_row", dst_row, "i", T * k), ("topk_w", topk_w, "f", T * k),
           ("dy_perm", dy_perm, y_perm_dt, 0 if y_perm is None else y_perm.numel()),
           ("dtopk_w", dtopk_w, "f", T * k)),
          (dy, dt, y_perm, y_perm_dt, dst_row, topk_w, T, k, H, dy_perm, dtopk_w), stream)


def moe_grouped_ffn_train_workspace_size(max_rows, E_loc, H, I_loc, dt) -> int:
    from . import lib
    return lib.moe_grouped_ffn_train_workspace_size(max_rows, E_loc, H, I_loc, dt)


def moe_grouped_ffn_train(x_perm, x, src_token, offsets, E_loc, max_rows, H, I_loc, w13, w2, dt, gu,
                          y_perm, ws, ws_bytes, stream=None):
    n = max_rows * H
    dt, kind, flagged = _gu(gu, dt)
    _call("moe_grouped_ffn_train",
          (("x_perm", x_perm, dt, n), ("x", x, dt, 0),
           ("src_token", src_token, "i", 0 if x_perm is not None else max_rows),
           ("offsets", offsets, "i", E_loc + 1), ("w13", w13, dt, 2 * E_loc * I_loc * H),
           ("w2", w2, dt, E_loc * I_loc * H), ("gu", gu, kind, 2 * max_rows * I_loc),
           ("y_perm", y_perm, dt, n), ("ws", ws, "b", ws_bytes)),
          (x_perm, x, src_token, offsets, E_loc, max_rows, H, I_loc, w13, w2, flagged, gu, y_perm,
           ws, ws_bytes), stream)


def moe_grouped_ffn_backward_workspace_size(max_rows, E_loc, H, I_loc, dt) -> int:
    from . import lib
    return lib.moe_grouped_ffn_backward_workspace_size(max_rows, E_loc, H, I_loc, dt)


def moe_grouped_ffn_backward(dy_perm, x_perm, x, src_token, offsets, E_loc, max_rows, H, I_loc, w13,
                             w2, dt, gu, dx_perm, dw13, dw2, ws, ws_bytes, stream=None):
    n, weights = max_rows * H, E_loc * I_loc * H
    dt, kind, flagged = _gu(gu, dt)
    _call("moe_grouped_ffn_backward",
          (("dy_perm", dy_perm, dt, n), ("x_perm", x_perm, dt, n), ("x", x, dt, 0),
           ("src_token", src_token, "i", 0 if x_perm is not None else max_rows),
           ("offsets", offsets, "i", E_loc + 1), ("w13", w13, dt, 2 * weights),
           ("w2", w2, dt, weights), ("gu", gu, kind, 2 * max_rows * I_loc),
           ("dx_perm", dx_perm, dt, n), ("dw13", dw13, dt, 2 * weights),
           ("dw2", dw2, dt, weights), ("ws", ws, "b", ws_bytes)),
          (dy_perm, x_perm, x, src_token, offsets, E_loc, max_rows, H, I_loc, w13, w2, flagged,
           gu, dx_perm, dw13, dw2, ws, ws_bytes), stream)


def moe_grouped_ffn_mxfp8_workspace_size(max_rows, E_loc, H, I_loc) -> int:
    from . import lib
    return lib.moe_grouped_ffn_mxfp8_workspace_size(max_rows, E_loc, H, I_loc)


def moe_grouped_ffn_mxfp8(x8, x_scale, src_token, offsets, E_loc, max_rows, H, I_loc, w13,
                          w13_scale, w2, w2_scale, y_perm, y_dt, ws, ws_bytes, stream=None):
    rows, weights = 0 if src_token is not None else max_rows, E_loc * I_loc * H
    _call("moe_grouped_ffn_mxfp8",
          (("x8", x8, "8", rows * H), ("x_scale", x_scale, "b", rows * mx_pitch(H)),
           ("src_token", src_token, "i", max_rows), ("offsets", offsets, "i", E_loc + 1),
           ("w13", w13, "8", 2 * weights), ("w13_scale", w13_scale, "b", 2 * E_loc * I_loc * mx_pitch(H)),
           ("w2", w2, "8", weights), ("w2_scale", w2_scale, "b", E_loc * H * mx_pitch(I_loc)),
           ("y_perm", y_perm, y_dt, max_rows * H), ("ws", ws, "b", ws_bytes)),
          (x8, x_scale, src_token, offsets, E_loc, max_rows, H, I_loc, w13, w13_scale, w2, w2_scale,
           y_perm, y_dt, ws, ws_bytes), stream)
