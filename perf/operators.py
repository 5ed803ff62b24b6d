"""The measured cases of the residual-path operators: layer norm, dropout with the residual add,
and the two in one pass, forward and backward.

Every operator works on channels-last activations [B][T][C] with per-item lengths: frames at or
beyond an item's length are not read and come out as zeros (gradients: are ignored).  Random
numbers are inputs: ``rng`` holds {seed, offset} of a Philox4x32-10 stream, element e (its flat
index in [B][T][C]) uses the 16 bits number e % 8 of the block with counter (e // 8, offset), and
is dropped when they are below p * 65536.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}

# The most a drawn case may cost: the bytes of the largest listed case, and for the cases with a
# mask the elements of the largest listed one of those.
MAX_ELEMS = 64 * 3000 * 1024
MAX_DROP_ELEMS = 32 * 1500 * 1024


def _case(name, op, B, T, C, dtype, min_len, p=0.0, alpha=1.0, train=True):
    return {"name": name, "op": op, "B": B, "T": T, "C": C, "dtype": dtype, "min_len": min_len, "p": p,
            "alpha": alpha, "train": train}


def listed():
    return [
        # streaming inference: one new frame of 64 streams through a norm
        _case("ln_fwd_stream_64x1x512_bf16", "ln_fwd", 64, 1, 512, "bf16", 1.0, train=False),
        # a conformer training batch, lengths between half and all of the frames
        _case("ln_fwd_16x1500x512_bf16", "ln_fwd", 16, 1500, 512, "bf16", 0.5),
        # a wide model on long audio with a large batch
        _case("ln_fwd_64x3000x1024_bf16", "ln_fwd", 64, 3000, 1024, "bf16", 0.5),
        # the same conformer batch, backward
        _case("ln_bwd_16x1500x512_bf16", "ln_bwd", 16, 1500, 512, "bf16", 0.5),
        # float32 training at a channel count with no 16-byte rows
        _case("ln_bwd_8x733x519_f32", "ln_bwd", 8, 733, 519, "f32", 0.5),
        # a module's exit: dropout and the residual add
        _case("drop_fwd_16x1500x512_bf16", "drop_fwd", 16, 1500, 512, "bf16", 0.5, p=0.1),
        # its gradient on the wide backward batch, half-step residual of a feed-forward module
        _case("drop_bwd_32x1500x1024_f16", "drop_bwd", 32, 1500, 1024, "f16", 0.5, p=0.15, alpha=0.5),
        # streaming inference: residual add and the next module's norm, no dropout, no statistics kept
        _case("dal_fwd_stream_64x1x1024_bf16", "dal_fwd", 64, 1, 1024, "bf16", 1.0, train=False),
        # a module's exit and the next one's entry on the conformer batch
        _case("dal_fwd_16x1500x512_bf16", "dal_fwd", 16, 1500, 512, "bf16", 0.5, p=0.1),
        # the same at odd sizes: no row but the first starts on 16 bytes
        _case("dal_fwd_16x1499x1023_f16", "dal_fwd", 16, 1499, 1023, "f16", 0.5, p=0.1, alpha=0.5),
        _case("dal_bwd_16x1500x512_bf16", "dal_bwd", 16, 1500, 512, "bf16", 0.5, p=0.1),
        # the wide backward batch
        _case("dal_bwd_32x1500x1024_bf16", "dal_bwd", 32, 1500, 1024, "bf16", 0.5, p=0.1),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["ln_fwd", "ln_bwd", "drop_fwd", "drop_bwd", "dal_fwd", "dal_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    B, T, C = log_int(1, 64), log_int(1, 3000), log_int(32, 4096)
    if rng.random() < 0.5:
        C = max(32, C // 8 * 8)
    cap = (MAX_ELEMS if op == "ln_fwd" else MAX_DROP_ELEMS) // (2 if dtype == "f32" else 1)
    while B * T * C > cap:
        B, T = (B // 2, T) if B > 1 else (B, T // 2)
    min_len = rng.choice([1.0, 0.5, 0.75, 0.0])
    p, alpha, train = 0.0, 1.0, True
    if not op.startswith("ln"):
        p = rng.choice([0.05, 0.1, 0.15, 0.2, 0.3])
        alpha = rng.choice([1.0, 0.5])
    if op in ("ln_fwd", "dal_fwd") and rng.random() < 0.25:
        p, train = 0.0, False
    return {"op": op, "B": B, "T": T, "C": C, "dtype": dtype, "min_len": min_len, "p": p, "alpha": alpha,
            "train": train}


def _lengths(case):
    """Evenly spread from min_len * T to T; None where every frame is valid."""
    B, T = case["B"], case["T"]
    if case["min_len"] >= 1.0:
        return None
    lo = int(T * case["min_len"])
    return [T - (T - lo) * i // max(1, B - 1) for i in range(B)]


def work(case):
    B, T, C = case["B"], case["T"], case["C"]
    s = 4 if case["dtype"] == "f32" else 2
    ln = _lengths(case)
    rows = B * T if ln is None else sum(ln)
    V, N = rows * C, B * T * C
    op = case["op"]
    stats = 8 * B * T if case["train"] else 0
    if op == "ln_fwd":
        return {"bytes": V * s + N * s + stats + 8 * C, "flops": 8 * V}
    if op == "ln_bwd":
        return {"bytes": 2 * V * s + N * s + 8 * rows + 12 * C, "flops": 14 * V}
    if op == "drop_fwd":
        return {"bytes": 2 * V * s + N * s, "flops": 2 * V}
    if op == "drop_bwd":
        return {"bytes": V * s + N * s, "flops": V}
    if op == "dal_fwd":
        return {"bytes": 2 * V * s + 2 * N * s + stats + 8 * C, "flops": 10 * V}
    return {"bytes": 3 * V * s + 2 * N * s + 8 * rows + 12 * C, "flops": 16 * V}


def _inputs(case, seed):
    """The tensors of one case, from the seed alone."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    B, T, C, dt = case["B"], case["T"], case["C"], DTYPES[case["dtype"]]
    op = case["op"]

    def normal(*shape):
        return torch.randn(*shape, device=dev, generator=g)

    def stream():  # residual-stream values: unit spread around a channel offset
        return (normal(B, T, C) + 0.5 * normal(C)).to(dt)

    st = {"case": case}
    ln = _lengths(case)
    st["lengths"] = None
    if ln is not None:
        order = torch.randperm(B, device=dev, generator=g)
        st["lengths"] = torch.tensor(ln, dtype=torch.int32, device=dev)[order].contiguous()
    st["rng"] = torch.randint(0, 2 ** 62, (2,), device=dev, generator=g, dtype=torch.int64) if case["p"] > 0 else None
    if not op.startswith("drop"):
        st["gamma"] = 1.0 + 0.1 * normal(C)
        st["beta"] = 0.1 * normal(C)
    if op == "ln_fwd":
        st["x"] = stream()
    elif op in ("drop_fwd", "dal_fwd"):
        st["x"] = normal(B, T, C).to(dt)
        st["residual"] = stream()
    elif op == "drop_bwd":
        st["dy"] = normal(B, T, C).to(dt)
    else:
        st["x"] = stream()
        st["dy"] = normal(B, T, C).to(dt)
        if op == "dal_bwd":
            st["dh"] = normal(B, T, C).to(dt)
        xf = st["x"].float()
        mean = xf.mean(-1)
        var = ((xf - mean[..., None]) ** 2).mean(-1)
        st["mean"], st["rstd"] = mean.contiguous(), torch.rsqrt(var + EPS).contiguous()
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        import speech_encoder_depthwise_b200 as dw
        B, T, C, dt = case["B"], case["T"], case["C"], DTYPES[case["dtype"]]
        op = case["op"]

        def act():
            return torch.empty(B, T, C, dtype=dt, device="cuda")

        def f32(*shape):
            return torch.empty(*shape, dtype=torch.float32, device="cuda")

        if op.endswith("fwd"):
            st["y"] = act()
            if op == "dal_fwd":
                st["h"] = act()
            keep = op != "drop_fwd" and case["train"]
            st["mean"], st["rstd"] = (f32(B, T), f32(B, T)) if keep else (None, None)
        else:
            st["dx"] = act()
            if op == "dal_bwd":
                st["dresidual"] = act()
            if op != "drop_bwd":
                st["dgamma"], st["dbeta"] = f32(C), f32(C)
                n = dw.dw_layernorm_bwd_workspace_size(B, T, C)
                st["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    return st


def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    import speech_encoder_depthwise_b200 as dw
    case = st["case"]
    op, p, alpha = case["op"], case["p"], case["alpha"]
    if op == "ln_fwd":
        dw.dw_layernorm_fwd(st["x"], st["gamma"], st["beta"], st["y"], st["mean"], st["rstd"], st["lengths"], EPS)
        return (st["y"], st["mean"], st["rstd"]) if case["train"] else (st["y"],)
    if op == "ln_bwd":
        dw.dw_layernorm_bwd(st["x"], st["dy"], st["gamma"], st["mean"], st["rstd"], st["dx"], st["dgamma"],
                            st["dbeta"], st["lengths"], st["workspace"])
        return st["dx"], st["dgamma"], st["dbeta"]
    if op == "drop_fwd":
        dw.dw_dropout_add_fwd(st["x"], st["residual"], st["y"], st["rng"], p, alpha, st["lengths"])
        return (st["y"],)
    if op == "drop_bwd":
        dw.dw_dropout_add_bwd(st["dy"], st["dx"], st["rng"], p, alpha, st["lengths"])
        return (st["dx"],)
    if op == "dal_fwd":
        dw.dw_dropout_add_layernorm_fwd(st["x"], st["residual"], st["rng"], p, alpha, st["gamma"], st["beta"],
                                        st["h"], st["y"], st["mean"], st["rstd"], st["lengths"], EPS)
        return (st["h"], st["y"], st["mean"], st["rstd"]) if case["train"] else (st["h"], st["y"])
    dw.dw_dropout_add_layernorm_bwd(st["dy"], st["dh"], st["x"], st["gamma"], st["mean"], st["rstd"], st["rng"], p,
                                    alpha, st["dx"], st["dresidual"], st["dgamma"], st["dbeta"], st["lengths"],
                                    st["workspace"])
    return st["dx"], st["dresidual"], st["dgamma"], st["dbeta"]


# ---- the plain form -----------------------------------------------------------------------------

_M32 = 0xFFFFFFFF


def _philox_bits(n, rng):
    """The 16-bit numbers of elements 0 .. n-1 (int64 tensor), Philox4x32-10."""
    g = torch.arange((n + 7) // 8, dtype=torch.int64, device=rng.device)
    seed, offset = rng[0], rng[1]
    c0, c1 = g & _M32, (g >> 32) & _M32
    c2, c3 = (offset & _M32).expand_as(g), ((offset >> 32) & _M32).expand_as(g)
    k0, k1 = seed & _M32, (seed >> 32) & _M32
    for _ in range(10):
        # 32 x 32 -> 64 bit products: int64 wraps, its bits are those of the unsigned product
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (((b >> 32) & _M32) ^ c1 ^ k0, b & _M32, ((a >> 32) & _M32) ^ c3 ^ k1, a & _M32)
        k0, k1 = (k0 + 0x9E3779B9) & _M32, (k1 + 0xBB67AE85) & _M32
    w = torch.stack([c0, c1, c2, c3], 1)
    return torch.stack([w & 0xFFFF, w >> 16], 2).reshape(-1)[:n]


def _threshold(p):
    return math.floor(p * 65536 + 0.5)


def _multiplier(p, alpha):
    thr = _threshold(p)
    return alpha * 65536 / (65536 - thr) if thr < 65536 else 0.0


def _dropped_times(x, rng, p, alpha):
    """[kept] m x in float32 (a dropped element is zero whatever x holds)."""
    v = x.float() * _multiplier(p, alpha)
    if _threshold(p) == 0:
        return v
    keep = _philox_bits(x.numel(), rng).view(x.shape) >= _threshold(p)
    return torch.where(keep, v, torch.zeros_like(v))


def _masked(v, valid):
    return v if valid is None else torch.where(valid, v, torch.zeros_like(v))


def _run_plain(st):
    case = st["case"]
    op, p, alpha = case["op"], case["p"], case["alpha"]
    dt, T, lengths = DTYPES[case["dtype"]], case["T"], st["lengths"]
    valid = None
    if lengths is not None:
        valid = (torch.arange(T, device=lengths.device) < lengths[:, None])[..., None]
    if op == "drop_fwd":
        return (_masked(st["residual"].float() + _dropped_times(st["x"], st["rng"], p, alpha), valid).to(dt),)
    if op == "drop_bwd":
        return (_masked(_dropped_times(st["dy"], st["rng"], p, alpha), valid).to(dt),)
    if op in ("ln_fwd", "dal_fwd"):
        out = []
        if op == "ln_fwd":
            h = _masked(st["x"].float(), valid)
        else:
            h = _masked(st["residual"].float() + _dropped_times(st["x"], st["rng"], p, alpha), valid)
            out.append(h.to(dt))
        mean = h.sum(-1, keepdim=True) / case["C"]
        d = h - mean
        rstd = _masked(1.0 / torch.sqrt((d * d).sum(-1, keepdim=True) / case["C"] + EPS), valid)
        out.append(_masked(d * rstd * st["gamma"] + st["beta"], valid).to(dt))
        if case["train"]:
            out += [mean[..., 0], rstd[..., 0]]
        return tuple(out)
    xh = _masked((st["x"].float() - st["mean"][..., None]) * st["rstd"][..., None], valid)
    dy = _masked(st["dy"].float(), valid)
    dgamma = (dy.double() * xh).sum((0, 1)).float()
    dbeta = dy.double().sum((0, 1)).float()
    g = dy * st["gamma"]
    c1 = g.sum(-1, keepdim=True) / case["C"]
    c2 = (g * xh).sum(-1, keepdim=True) / case["C"]
    t = _masked(st["rstd"][..., None] * (g - c1 - xh * c2), valid)
    if op == "ln_bwd":
        return t.to(dt), dgamma, dbeta
    t = t + _masked(st["dh"].float(), valid)
    return _dropped_times(t, st["rng"], p, alpha).to(dt), t.to(dt), dgamma, dbeta


# ---- the definition in 64 bits --------------------------------------------------------------------

def _kept64(shape, rng, p):
    """Truth values of the kept elements: Philox4x32-10 in numpy, 64-bit unsigned."""
    thr = int(p * 65536 + 0.5)
    n = int(np.prod(shape))
    if thr == 0:
        return torch.ones(shape, dtype=torch.bool, device="cuda")
    seed, offset = (int(v) for v in rng.cpu())
    low, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    blocks = np.arange((n + 7) // 8, dtype=np.uint64)
    c = [blocks & low, blocks >> sh, np.uint64(offset & 0xFFFFFFFF), np.uint64(offset >> 32)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        lo_hi = np.uint64(0xD2511F53) * c[0]
        lo_hi2 = np.uint64(0xCD9E8D57) * c[2]
        c = [(lo_hi2 >> sh) ^ c[1] ^ np.uint64(key[0]), lo_hi2 & low, (lo_hi >> sh) ^ c[3] ^ np.uint64(key[1]),
             lo_hi & low]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    u = np.stack(c, 1).astype("<u4").view("<u2").reshape(-1)[:n]
    return torch.from_numpy(u >= thr).cuda().view(shape)


def exact(case, seed):
    st = _inputs(case, seed)
    op, B, T, C = case["op"], case["B"], case["T"], case["C"]
    if st["lengths"] is None:
        rows = torch.ones(B, T, dtype=torch.bool, device="cuda")
    else:
        rows = torch.arange(T, device="cuda")[None, :] < st["lengths"][:, None].long()
    live = rows.unsqueeze(-1).expand(B, T, C)
    thr = int(case["p"] * 65536 + 0.5)
    m = case["alpha"] / (1.0 - thr / 65536.0)

    def f64(name):
        return st[name].double().masked_fill(~live, 0.0)

    if not op.startswith("ln"):
        scale = _kept64((B, T, C), st["rng"], case["p"]).double().mul_(m)
    if op == "drop_fwd":
        return (f64("residual") + scale * f64("x"),)
    if op == "drop_bwd":
        return (scale * f64("dy"),)
    if op in ("ln_fwd", "dal_fwd"):
        h = f64("x") if op == "ln_fwd" else f64("residual") + scale * f64("x")
        var, mean = torch.var_mean(h, dim=-1, correction=0)
        rstd = ((var + EPS) ** -0.5).masked_fill(~rows, 0.0)
        y = (h - mean.unsqueeze(-1)).mul_(rstd.unsqueeze(-1)).mul_(st["gamma"].double()).add_(st["beta"].double())
        out = [] if op == "ln_fwd" else [h]
        out.append(y.masked_fill_(~live, 0.0))
        return tuple(out + ([mean, rstd] if case["train"] else []))
    rstd = st["rstd"].double().masked_fill(~rows, 0.0).unsqueeze(-1)
    xh = (f64("x") - st["mean"].double().unsqueeze(-1)) * rstd
    dy = f64("dy")
    dgamma = torch.einsum("btc,btc->c", dy, xh)
    dbeta = dy.sum(0).sum(0)
    g = dy * st["gamma"].double()
    t = rstd * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    if op == "ln_bwd":
        return t, dgamma, dbeta
    t = t + f64("dh")
    return scale * t, t, dgamma, dbeta
