"""Cases, plain forms and calls of the operators around the MoE layer: the RMS
norm in front of it (with the residual's addition and an 8-bit output), expert
blocks in MXFP8, and the backward passes of the norm, of the grouped SwiGLU
experts and of the combine.

Sizes are those of the workloads (workloads/__init__.py): Mixtral-8x7B,
Qwen3-235B-A22B (all experts, and its tensor-parallel share with I/P = 192),
DeepSeek-V3 and the toy float32 layer.

MXFP8 is the OCP microscaling format: e4m3 elements and one E8M0 scale 2^e per
32 consecutive elements along the contraction; a row of K elements has
4 * ceil(K / 128) scale bytes, of which the first K / 32 are used.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        import mixture_experts_layer_amd
        _LIB = mixture_experts_layer_amd
    return _LIB


def listed():
    """Three operators are met at one token (decode), in a serving batch and
    in prefill or a training step; the backward passes in training steps."""
    return [
        # one decoded token of the Qwen3 shape entering the layer: pure latency
        dict(name="norm_token", op="norm", T=1, H=4096, dtype="bf16", residual=True, y=True, y8=True),
        # a prefill batch of the Qwen3 shape: both the router's and the experts' rows are written
        dict(name="norm_prefill", op="norm", T=8192, H=4096, dtype="bf16", residual=True, y=True, y8=True),
        # an odd micro-batch of the toy float32 layer
        dict(name="norm_bwd_f32", op="norm_bwd", T=77, H=256, dtype="f32", residual=False),
        # a training micro-batch of the DeepSeek-V3 width, the residual's gradient joining
        dict(name="norm_bwd_train", op="norm_bwd", T=8191, H=7168, dtype="bf16", residual=True),
        # one decoded token of the Qwen3 tensor-parallel share: 8 rows for 8 experts
        dict(name="mxfp8_token", op="mxfp8", T=1, H=4096, I=192, E=128, k=8, beta=0.15),
        # a serving batch of the Qwen3 shape, four rows per expert: the weights are the traffic
        dict(name="mxfp8_serve", op="mxfp8", T=64, H=4096, I=1536, E=128, k=8, beta=0.15),
        # a prefill batch of the Qwen3 shape: matrix-core bound
        dict(name="mxfp8_prefill", op="mxfp8", T=8192, H=4096, I=1536, E=128, k=8, beta=0.15),
        # a step of the toy float32 layer
        dict(name="train_f32", op="train", T=64, H=256, I=512, E=8, k=2, dtype="f32", beta=0.0),
        # a small micro-batch of the Qwen3 shape, ragged and few rows per expert: weights and their gradients are the traffic
        dict(name="train_ragged", op="train", T=509, H=4096, I=1536, E=128, k=8, dtype="bf16", beta=0.15),
        # a full step of the Mixtral shape: matrix-core bound
        dict(name="train_step", op="train", T=4096, H=4096, I=14336, E=8, k=2, dtype="bf16", beta=0.0),
        # gradients of the combine for an odd, short batch of the DeepSeek-V3 width
        dict(name="combine_bwd_odd", op="combine_bwd", T=33, H=7168, E=256, k=8, dtype="bf16"),
        # gradients of the combine for a full step of the Qwen3 shape
        dict(name="combine_bwd_step", op="combine_bwd", T=8192, H=4096, E=128, k=8, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return w["bytes"] / 5e12 + w["flops"] / 1e15


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["norm", "norm_bwd", "mxfp8", "train", "combine_bwd"])
        H = 32 * _log_int(rng, 4, 224)
        dtype = "f32" if rng.random() < 0.2 else "bf16"
        if op == "norm":
            y8 = rng.random() < 0.7
            c = dict(op=op, T=_log_int(rng, 1, 8192), H=H, dtype=dtype, residual=rng.random() < 0.7,
                     y=not y8 or rng.random() < 0.6, y8=y8)
        elif op == "norm_bwd":
            c = dict(op=op, T=_log_int(rng, 1, 8192), H=H, dtype=dtype, residual=rng.random() < 0.6)
        elif op == "combine_bwd":
            c = dict(op=op, T=_log_int(rng, 1, 8192), H=H, E=rng.choice([8, 60, 128, 256]), k=rng.randint(1, 8),
                     dtype=dtype)
        else:
            E = rng.choice([1, 4, 8, 20, 64, 128])
            I = 32 * _log_int(rng, 1, 64)
            c = dict(op=op, T=_log_int(rng, 1, 8192), H=H, I=I, E=E, k=rng.randint(1, min(8, E)),
                     beta=rng.choice([0.0, 0.15, 0.3]))
            if op == "train":
                c["dtype"] = dtype
                if dtype == "f32":      # the float32 layer is small
                    c.update(T=min(c["T"], 512), H=min(H, 1024), I=min(I, 512), E=min(E, 8),
                             k=min(c["k"], min(E, 8)))
        if _cost(c) <= most:
            return c


# ---------------------------------------------------------------- inputs

def _dt(case):
    return torch.float32 if case.get("dtype") == "f32" else torch.bfloat16


def _randn(g, shape, scale=1.0, dtype=torch.float32):
    t = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)
    return (t if scale == 1.0 else t.mul_(scale)).to(dtype)


def _experts(g, E, shape, scale, dtype):
    out = torch.empty((E,) + shape, device=DEV, dtype=dtype)
    for e in range(E):
        out[e] = _randn(g, shape, scale, dtype)
    return out


def _pitch(K):
    return 4 * ((K + 127) // 128)


def _mx(v):
    """MXFP8 of v along its last axis, held in v's type: the elements' values
    and the scale bytes, unpadded.  The scale of a block of 32 is the smallest
    2^e with max|v| / 2^e <= 448 = 0.875 * 2^9, e >= -127."""
    b = v.reshape(v.shape[:-1] + (v.shape[-1] // 32, 32))
    m, ex = torch.frexp(b.abs().amax(-1))
    e = torch.where(m == 0, torch.full_like(ex, -127), ex - 9 + (m > 0.875).to(ex.dtype)).clamp_min(-127)
    q = torch.ldexp(b, -e.unsqueeze(-1)).to(torch.float8_e4m3fn)
    return q.reshape(v.shape), (e + 127).to(torch.uint8)


def _padded(s, K):
    out = torch.zeros(s.shape[:-1] + (_pitch(K),), device=s.device, dtype=torch.uint8)
    out[..., :K // 32] = s
    return out


def _mx_experts(g, E, shape, scale):
    q = torch.empty((E,) + shape, device=DEV, dtype=torch.float8_e4m3fn)
    s = torch.zeros((E, shape[0], _pitch(shape[1])), device=DEV, dtype=torch.uint8)
    for e in range(E):
        qe, se = _mx(_randn(g, shape, scale))
        q[e] = qe
        s[e, :, :shape[1] // 32] = se
    return q, s


def _routing(g, T, E, k, beta):
    """Top-k ids of Zipf-skewed random logits, and the permutation by expert
    that the layer's dispatch makes: offsets, source tokens, rows of (t, j)."""
    logits = _randn(g, (T, E))
    if beta:
        rank = torch.randperm(E, generator=g, device=DEV).float() + 1
        logits -= beta * rank.log()
    top, ids = logits.topk(k, dim=1)
    flat = ids.reshape(-1)
    order = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, device=DEV, dtype=torch.int32)
    offsets[1:] = counts.cumsum(0)
    src = (order // k).to(torch.int32)
    dst = torch.empty_like(flat, dtype=torch.int32)
    dst[order] = torch.arange(T * k, device=DEV, dtype=torch.int32)
    return offsets, counts, src, dst.reshape(T, k), torch.softmax(top, 1).contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    T, H, dt = case["T"], case["H"], _dt(case)
    s = {"case": case, "T": T, "H": H, "dt": dt}
    e = lambda *shape, dtype=dt: torch.empty(shape, device=DEV, dtype=dtype)  # noqa: E731
    if case["op"] in ("norm", "norm_bwd"):
        s["x"] = _randn(g, (T, H), 1.5, dt)
        s["w"] = (1 + _randn(g, (H,), 0.1)).to(dt)
        s["res"] = _randn(g, (T, H), 1.0, dt) if case["residual"] else None
        if case["op"] == "norm":
            s.update(sum=e(T, H) if case["residual"] else None, y=e(T, H) if case["y"] else None, rstd=e(T, dtype=torch.float32))
            if case["y8"]:
                s.update(y8=e(T, H, dtype=torch.float8_e4m3fn),
                         y8_scale=torch.zeros((T, _pitch(H)), device=DEV, dtype=torch.uint8))
        else:       # x is the summed stream that the forward normed, res its own gradient
            s["dy"] = _randn(g, (T, H), 0.02, dt)
            s["rstd"] = torch.rsqrt(s["x"].double().square().mean(1) + EPS).float()
            s.update(dx=e(T, H), dw=e(H, dtype=torch.float32))
        return s
    E, k = case["E"], case["k"]
    offsets, counts, src, dst, w = _routing(g, T, E, k, case.get("beta", 0.0))
    R = T * k
    if case["op"] == "combine_bwd":
        s.update(dy=_randn(g, (T, H), 0.02, dt), y_perm=_randn(g, (R, H), 1.0, dt), dst=dst, topk_w=w,
                 dy_perm=e(R, H), dw=e(T, k, dtype=torch.float32))
        return s
    I = case["I"]
    # the plan that a program with these rows keeps: the experts that have any, and the largest count
    active = counts.nonzero().reshape(-1)
    s.update(I=I, E=E, R=R, offsets=offsets, src=src, active=active, cap=int(counts.max()), start=offsets[:-1].long()[active],
             count=counts[active], every=active.numel() == E, scale=1.0 / math.sqrt(H))
    if case["op"] == "mxfp8":
        x8, xs = _mx(_randn(g, (T, H)))
        s.update(x8=x8, xs=_padded(xs, H), y=e(R, H, dtype=torch.bfloat16))
        s["w13"], s["w13s"] = _mx_experts(g, E, (2 * I, H), s["scale"])
        s["w2"], s["w2s"] = _mx_experts(g, E, (H, I), s["scale"])
        return s
    s.update(x=_randn(g, (T, H), 1.0, dt), dy=_randn(g, (R, H), 0.02, dt),
             w13=_experts(g, E, (2 * I, H), s["scale"], dt), w2=_experts(g, E, (H, I), s["scale"], dt),
             gu=e(R, 2 * I), y=e(R, H), dx=e(R, H), dw13=e(E, 2 * I, H), dw2=e(E, H, I))
    return s


# ---------------------------------------------------------------- plain forms

def _unmx(q, s):
    """Values of an MXFP8 tensor in float32."""
    K = q.shape[-1]
    f = torch.ldexp(torch.ones((), device=q.device), s[..., :K // 32].to(torch.int32) - 127)
    return (q.float().reshape(q.shape[:-1] + (K // 32, 32)) * f.unsqueeze(-1)).reshape(q.shape)


def _blocks(s):
    """Row numbers [experts with rows][largest count], and which are rows."""
    c = torch.arange(s["cap"], device=DEV)
    live = c < s["count"].unsqueeze(1)
    return torch.where(live, s["start"].unsqueeze(1) + c, torch.zeros_like(c)), live


def _of(s, w):
    return w if s["every"] else w[s["active"]]


def _norm_plain(s):
    x = s["x"].float()
    out = {}
    if s["res"] is not None:
        out["sum"] = (x + s["res"].float()).to(s["dt"])
        x = out["sum"].float()
    rstd = torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
    y = x * rstd * s["w"].float()
    out["rstd"] = rstd.reshape(-1)
    if s["y"] is not None:
        out["y"] = y.to(s["dt"])
    if s["case"]["y8"]:
        out["y8"], scale = _mx(y)
        out["y8_scale"] = _padded(scale, s["H"]).view(torch.float8_e8m0fnu)
    return out


def _norm_bwd_plain(s):
    xh = s["x"].float() * s["rstd"].unsqueeze(1)
    dy = s["dy"].float()
    g = dy * s["w"].float()
    dx = s["rstd"].unsqueeze(1) * (g - xh * (g * xh).mean(1, keepdim=True))
    if s["res"] is not None:
        dx = dx + s["res"].float()
    return {"dx": dx.to(s["dt"]), "dw": (dy * xh).sum(0)}


def _mxfp8_plain(s):
    rows, live = _blocks(s)
    x = _unmx(s["x8"], s["xs"])[s["src"].long()[rows]]
    I = s["I"]
    gu = torch.bmm(x, _unmx(_of(s, s["w13"]), _of(s, s["w13s"])).transpose(1, 2))
    h = torch.nn.functional.silu(gu[..., :I]) * gu[..., I:]
    q, sc = _mx(h)
    y = torch.bmm(_unmx(q, sc), _unmx(_of(s, s["w2"]), _of(s, s["w2s"])).transpose(1, 2))
    return {"y": y[live].to(torch.bfloat16)}


def _train_plain(s):
    rows, live = _blocks(s)
    keep = live.unsqueeze(-1)
    I = s["I"]
    x = s["x"].float()[s["src"].long()[rows]] * keep
    dy = s["dy"].float()[rows] * keep
    w13, w2 = _of(s, s["w13"]).float(), _of(s, s["w2"]).float()
    gu = torch.bmm(x, w13.transpose(1, 2))
    g, u = gu[..., :I], gu[..., I:]
    sg = torch.sigmoid(g)
    h = g * sg * u
    y = torch.bmm(h, w2.transpose(1, 2))
    dh = torch.bmm(dy, w2)
    dgu = torch.cat([dh * u * sg * (1 + g * (1 - sg)), dh * g * sg], -1)
    dx = torch.bmm(dgu, w13)
    dw13, dw2 = torch.bmm(dgu.transpose(1, 2), x).to(s["dt"]), torch.bmm(dy.transpose(1, 2), h).to(s["dt"])
    if not s["every"]:
        dw13 = torch.zeros_like(s["w13"]).index_copy_(0, s["active"], dw13)
        dw2 = torch.zeros_like(s["w2"]).index_copy_(0, s["active"], dw2)
    return {"y": y[live].to(s["dt"]), "dx": dx[live].to(s["dt"]), "dw13": dw13, "dw2": dw2}


def _combine_bwd_plain(s):
    dy = s["dy"].float()
    dy_perm = torch.empty_like(s["dy_perm"])
    rows = s["dst"].long().reshape(-1)
    dy_perm[rows] = (s["topk_w"].unsqueeze(-1) * dy.unsqueeze(1)).to(s["dt"]).reshape(rows.numel(), -1)
    dw = (s["y_perm"][rows].reshape(s["T"], -1, s["H"]).float() * dy.unsqueeze(1)).sum(-1)
    return {"dy_perm": dy_perm, "dw": dw}


# ---------------------------------------------------------------- the framework's calls

def _ws(s, name, size):
    """The workspace that a program keeps beside its buffers."""
    if name not in s:
        s[name] = torch.empty(max(size(), 16), device=DEV, dtype=torch.uint8)
    return s[name]


def _own(s):
    M = _lib()
    op, T, H = s["case"]["op"], s["T"], s["H"]
    if op == "norm":
        y8, sc = s.get("y8"), s.get("y8_scale")
        M.moe_rmsnorm(s["x"], s["res"], s["w"], EPS, T, H, M.dtype_code(s["dt"]), s["sum"], s["y"], y8, sc, s["rstd"])
        out = {"rstd": s["rstd"]}
        if s["sum"] is not None:
            out["sum"] = s["sum"]
        if s["y"] is not None:
            out["y"] = s["y"]
        if y8 is not None:
            out.update(y8=y8, y8_scale=sc.view(torch.float8_e8m0fnu))
        return out
    dt = M.dtype_code(s["dt"])
    if op == "norm_bwd":
        ws = _ws(s, "ws", lambda: M.moe_rmsnorm_backward_workspace_size(T, H, dt))
        M.moe_rmsnorm_backward(s["dy"], s["res"], s["x"], s["w"], s["rstd"], T, H, dt, s["dx"], s["dw"], ws, ws.numel())
        return {"dx": s["dx"], "dw": s["dw"]}
    if op == "combine_bwd":
        M.moe_combine_backward(s["dy"], dt, s["y_perm"], dt, s["dst"], s["topk_w"], T, s["case"]["k"], H, s["dy_perm"], s["dw"])
        return {"dy_perm": s["dy_perm"], "dw": s["dw"]}
    E, R, I = s["E"], s["R"], s["I"]
    if op == "mxfp8":
        ws = _ws(s, "ws", lambda: M.moe_grouped_ffn_mxfp8_workspace_size(R, E, H, I))
        M.moe_grouped_ffn_mxfp8(s["x8"], s["xs"], s["src"], s["offsets"], E, R, H, I, s["w13"], s["w13s"], s["w2"],
                                s["w2s"], s["y"], M.MOE_BF16, ws, ws.numel())
        return {"y": s["y"]}
    ws = _ws(s, "ws", lambda: max(M.moe_grouped_ffn_train_workspace_size(R, E, H, I, dt),
                                  M.moe_grouped_ffn_backward_workspace_size(R, E, H, I, dt)))
    M.moe_grouped_ffn_train(None, s["x"], s["src"], s["offsets"], E, R, H, I, s["w13"], s["w2"], dt, s["gu"], s["y"],
                            ws, ws.numel())
    M.moe_grouped_ffn_backward(s["dy"], None, s["x"], s["src"], s["offsets"], E, R, H, I, s["w13"], s["w2"], dt, s["gu"],
                               s["dx"], s["dw13"], s["dw2"], ws, ws.numel())
    return {"y": s["y"], "dx": s["dx"], "dw13": s["dw13"], "dw2": s["dw2"]}


PLAIN = {"norm": _norm_plain, "norm_bwd": _norm_bwd_plain, "mxfp8": _mxfp8_plain, "train": _train_plain,
         "combine_bwd": _combine_bwd_plain}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    T, H, op = case["T"], case["H"], case["op"]
    b = 4 if case.get("dtype") == "f32" else 2
    if op == "norm":
        per = b * (1 + 2 * case["residual"] + case["y"]) + case["y8"] * (1 + 1 / 32)
        return {"bytes": int(T * H * per + H * b + 4 * T), "flops": T * H * (4 + case["residual"] + 2 * case["y8"])}
    if op == "norm_bwd":
        return {"bytes": T * H * b * (3 + case["residual"]) + H * (b + 4) + 4 * T, "flops": 9 * T * H}
    k, E = case["k"], case["E"]
    R = T * k
    if op == "combine_bwd":
        return {"bytes": (T + 2 * R) * H * b + 12 * R, "flops": 3 * R * H}
    I = case["I"]
    touched = E * (1 - (1 - k / E) ** T)      # experts with rows, were routing uniform
    if op == "mxfp8":
        per = 1 + 1 / 32
        return {"bytes": int(T * H * per + touched * 3 * H * I * per + R * H * 2 + 4 * (R + E)), "flops": 6 * R * H * I}
    return {"bytes": int(b * (T * H + 3 * R * H + (touched + E) * 3 * H * I)) + 4 * (R + E), "flops": 18 * R * H * I}


# ---------------------------------------------------------------- the definitions in 64 bits

def _blocks_of_32(v):
    """v / 2^e in e4m3 and 2^e, from the format's definition, in float64."""
    shape = v.shape
    v = v.reshape(-1, 32)
    top = v.abs().max(dim=1).values
    e = torch.ceil(torch.log2(top / 448)).clamp(min=-127)       # -inf where a block is all zeros
    e = torch.where(top > 448 * torch.exp2(e), e + 1, e)
    e = torch.where((top <= 448 * torch.exp2(e - 1)) & (e > -127), e - 1, e)
    a = (v / torch.exp2(e)[:, None]).abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)      # e4m3: 3 mantissa bits, least 2^-9
    q = torch.round(a / step) * step * torch.sign(v)
    return q.reshape(shape), torch.exp2(e).reshape(shape[:-1] + (shape[-1] // 32,))


def _value(q, s):
    q = q.double()
    f = torch.exp2(s[..., :q.shape[-1] // 32].double() - 127)
    return q * f.repeat_interleave(32, dim=-1)


def exact(case, seed):
    s = prepare(case, seed)
    op, T, H = case["op"], case["T"], case["H"]
    if op == "norm":
        x, out = s["x"].double(), {}
        if s["res"] is not None:
            out["sum"] = x + s["res"].double()
            x = out["sum"].to(s["dt"]).double()
        r = 1 / torch.sqrt((x * x).sum(1) / H + EPS)
        y = x * r[:, None] * s["w"].double()
        out["rstd"] = r
        if case["y"]:
            out["y"] = y
        if case["y8"]:
            q, sc = _blocks_of_32(y)
            pad = torch.full((T, _pitch(H)), 2.0 ** -127, device=DEV, dtype=torch.float64)
            pad[:, :H // 32] = sc
            out.update(y8=q, y8_scale=pad)
        return out
    if op == "norm_bwd":
        x, w, dy = s["x"].double(), s["w"].double(), s["dy"].double()
        r = s["rstd"].double()[:, None]
        dot = (dy * w * x).sum(1, keepdim=True) / H
        dx = r * dy * w - r ** 3 * x * dot
        return {"dx": dx if s["res"] is None else dx + s["res"].double(), "dw": torch.einsum("th,th->h", dy, x * r)}
    if op == "combine_bwd":
        out = {"dy_perm": torch.zeros(T * case["k"], H, device=DEV, dtype=torch.float64),
               "dw": torch.zeros(T, case["k"], device=DEV, dtype=torch.float64)}
        for j in range(case["k"]):
            at = s["dst"][:, j].long()
            out["dy_perm"][at] = s["topk_w"][:, j:j + 1].double() * s["dy"].double()
            out["dw"][:, j] = (s["dy"].double() * s["y_perm"][at].double()).sum(1)
        return out
    at, I, src = s["offsets"].tolist(), s["I"], s["src"].long()
    if op == "mxfp8":
        y = torch.zeros(s["R"], H, device=DEV, dtype=torch.float64)
        x = _value(s["x8"], s["xs"])
        for e in range(s["E"]):
            a, b = at[e], at[e + 1]
            if a < b:
                z = x[src[a:b]] @ _value(s["w13"][e], s["w13s"][e]).t()
                h, sc = _blocks_of_32(z[:, :I] / (1 + torch.exp(-z[:, :I])) * z[:, I:])
                y[a:b] = (h * sc.repeat_interleave(32, dim=-1)) @ _value(s["w2"][e], s["w2s"][e]).t()
        return {"y": y}
    out = {n: torch.zeros(s[n].shape, device=DEV, dtype=torch.float64) for n in ("y", "dx", "dw13", "dw2")}
    for e in range(s["E"]):
        a, b = at[e], at[e + 1]
        if a < b:
            x, dy, w13, w2 = s["x"][src[a:b]].double(), s["dy"][a:b].double(), s["w13"][e].double(), s["w2"][e].double()
            z = x @ w13.t()
            g, u = z[:, :I], z[:, I:]
            p = 1 / (1 + torch.exp(-g))
            dh = dy @ w2
            d = torch.cat([dh * u * (p + g * p * (1 - p)), dh * g * p], 1)
            out["y"][a:b] = (g * p * u) @ w2.t()
            out["dx"][a:b] = d @ w13
            out["dw13"][e] = d.t() @ x
            out["dw2"][e] = dy.t() @ (g * p * u)
    return out
