"""What the training operators of the feed-forward half of a block are measured on: layer norm, 8-bit activation
checkpoints and the gated feed-forward block, forward and backward.

``run`` computes an operator either in its plain form (elementary torch operations in 32 bits, rounded once at the end)
or, where ``own`` is true, through the package's entry points.  ``exact`` computes the same from the definitions in 64
bits.  Sizes are those of the package's layouts (512/1408, 1024/4096, 4096/12288) and odd ones beside them.
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
DTYPES = {"bf16": BF16, "f32": F32}
GROUP = 32  # elements of a row that share one scale of an 8-bit checkpoint
EPS = 1e-5


def listed():
    return [
        # One row through the norm of the 512-wide layout: the latency of a call.
        dict(name="norm_fwd_row", op="norm_fwd", rows=1, cols=512, dtype="bf16", keep="none"),
        # The norm in front of the widest layout's feed-forward block, its input kept in 8 bits by the same call.
        dict(name="norm_fwd_keep", op="norm_fwd", rows=16384, cols=4096, dtype="bf16", keep="act8"),
        # Its backward pass from the 8-bit checkpoint, with both parameter gradients.
        dict(name="norm_bwd_kept", op="norm_bwd", rows=16384, cols=4096, dtype="bf16", keep="act8"),
        # A width that no vector divides, on an FP32 residual stream.
        dict(name="norm_bwd_odd", op="norm_bwd", rows=4099, cols=1409, dtype="f32", keep="none"),
        # The gate activations of a wide block kept for the backward pass.
        dict(name="act8_store", op="act8_store", rows=8192, cols=12288, dtype="bf16", keep="act8"),
        # A ragged checkpoint read back in full precision.
        dict(name="act8_load_odd", op="act8_load", rows=4099, cols=1411, dtype="f32", keep="act8"),
        # One token through the widest block: the weights are read once.
        dict(name="ffn_fwd_token", op="ffn_fwd", rows=1, d=4096, f=12288, keep="none", act="silu"),
        # An ordinary forward pass that keeps gate and up in 8 bits.
        dict(name="ffn_fwd_keep", op="ffn_fwd", rows=8192, d=1024, f=4096, keep="act8", act="silu"),
        # The widest block over a long batch.
        dict(name="ffn_fwd_wide", op="ffn_fwd", rows=16384, d=4096, f=12288, keep="none", act="silu"),
        # The backward pass of the 512-wide block from gate and up kept in 8 bits.
        dict(name="ffn_bwd_kept", op="ffn_bwd", rows=8192, d=512, f=1408, keep="act8", act="silu"),
        # The widest block's backward pass with gate and up computed again.
        dict(name="ffn_bwd_wide", op="ffn_bwd", rows=8192, d=4096, f=12288, keep="none", act="silu"),
        # A whole training step at sizes no tile or vector divides, input, gate and up kept in 8 bits.
        dict(name="ffn_step_odd", op="ffn_step", rows=1001, d=515, f=1411, keep="act8", act="gelu"),
    ]


def _spread(rng, low, high):
    """A whole number from low to high, spread over its logarithm; half of them as they fall, half rounded to 32s."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if n >= 64 and rng.random() < 0.5:
        n = (n + 31) // 32 * 32
    return max(low, min(high, n))


def draw(rng):
    most = max(work(c)["flops"] for c in listed())
    wide = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(["norm_fwd", "norm_bwd", "act8_store", "act8_load", "ffn_fwd", "ffn_fwd", "ffn_bwd", "ffn_bwd",
                         "ffn_step"])
        if op.startswith("ffn"):
            keep = "act8" if op == "ffn_step" else rng.choice(["none", "act8", "bf16"])
            case = dict(op=op, rows=_spread(rng, 1, 16384), d=_spread(rng, 64, 4096), f=_spread(rng, 64, 12288),
                        keep=keep, act=rng.choice(["silu", "gelu"]))
        else:
            keep = rng.choice(["none", "act8"]) if op.startswith("norm") else "act8"
            case = dict(op=op, rows=_spread(rng, 1, 32768), cols=_spread(rng, 64, 12288),
                        dtype=rng.choice(["bf16", "f32"]), keep=keep)
        w = work(case)
        if w["flops"] <= most and w["bytes"] <= wide:
            return case


# ---------------------------------------------------------------------------
# 8-bit checkpoints: per group of 32 consecutive elements of a row, int8 codes
# and one byte s that stands for the scale 2^(s - 127); s = 255 marks a group
# that held a NaN or an infinity.  One buffer: codes [rows, 32 G], then s [rows, G].
# ---------------------------------------------------------------------------
def _groups(cols):
    return (cols + GROUP - 1) // GROUP


def _encode(x):
    """The checkpoint buffer of an FP32 matrix."""
    rows, cols = x.shape
    g = _groups(cols)
    x = torch.nn.functional.pad(x, (0, g * GROUP - cols)).view(rows, g, GROUP)
    bits = x.abs().amax(-1).view(torch.int32)
    fine = bits < 0x7F800000
    s = torch.where(fine, (((bits.clamp(max=0x7F7FFFFF) + 0x1FFFF) >> 23) - 6).clamp(min=1), 255)
    inverse = ((254 - s).clamp(min=1) << 23).view(F32)
    codes = torch.round(torch.where(fine[..., None], x * inverse[..., None], 0.0)).to(torch.int8)
    return torch.cat([codes.reshape(-1).view(torch.uint8), s.to(torch.uint8).reshape(-1)])


def _decode(buf, rows, cols):
    """The FP32 values that a checkpoint buffer stands for."""
    g = _groups(cols)
    codes = buf[:rows * g * GROUP].view(torch.int8).view(rows, g, GROUP)
    scale = (buf[rows * g * GROUP:].to(torch.int32) << 23).view(F32).view(rows, g, 1)
    return (codes.to(F32) * scale).view(rows, g * GROUP)[:, :cols]


def _normal(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=F32).mul_(std)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, rows = case["op"], case["rows"]
    s = {"case": dict(case)}
    if not op.startswith("ffn"):
        cols, dt = case["cols"], DTYPES[case["dtype"]]
        # A residual stream: channels of different size and offset, a few of them large.
        size = 0.5 + _normal(gen, cols).abs()
        size[:: 97] *= 8
        x = (_normal(gen, rows, cols) * size + 0.2 * _normal(gen, cols)).to(dt)
        if op == "act8_load":
            s["kept"] = _encode(x.float())
            return s
        if op == "act8_store":
            s["x"] = x
            return s
        s["weight"], s["bias"] = 1 + _normal(gen, cols, std=0.1), _normal(gen, cols, std=0.1)
        if op == "norm_fwd":
            s["x"] = x
            return s
        f = x.float()
        s["mean"] = f.mean(-1)
        s["rstd"] = (f - s["mean"][:, None]).square().mean(-1).add(EPS).rsqrt()
        s["dy"] = _normal(gen, rows, cols, std=0.01).to(dt)
        if case["keep"] == "act8":
            s["kept"] = _encode(f)
        else:
            s["x"] = x
        return s
    d, f = case["d"], case["f"]
    s["x"] = _normal(gen, rows, d).to(BF16)
    s["w_gate"], s["w_up"] = (_normal(gen, f, d, std=d ** -0.5).to(BF16) for _ in range(2))
    if op != "ffn_fwd":
        s["dh"] = _normal(gen, rows, f, std=0.01).to(BF16)
    if op == "ffn_bwd" and case["keep"] != "none":
        gate, up = s["x"] @ s["w_gate"].T, s["x"] @ s["w_up"].T
        s["gate"], s["up"] = (_encode(t.float()) if case["keep"] == "act8" else t for t in (gate, up))
    return s


# ---------------------------------------------------------------------------
# The operators
# ---------------------------------------------------------------------------
def run(state):
    return (_run_own if own else _run_plain)(state, state["case"])


def _run_own(s, c):
    from fsdp2_gradient_packing_gb300 import fsdp_pack as fp
    op, rows = c["op"], c["rows"]
    if not op.startswith("ffn"):
        cols, dt = c["cols"], DTYPES[c["dtype"]]
        if op == "act8_store":
            kept = fp.Act8(rows, cols)
            fp.fsdp_act8_store(s["x"], kept)
            y = torch.empty(rows, cols, dtype=dt, device="cuda")
            fp.fsdp_act8_load(kept, y)
            return y
        if op == "act8_load":
            y = torch.empty(rows, cols, dtype=dt, device="cuda")
            fp.fsdp_act8_load(fp.Act8(rows, cols, s["kept"]), y)
            return y
        if op == "norm_fwd":
            y = torch.empty_like(s["x"])
            mean, rstd = (torch.empty(rows, dtype=F32, device="cuda") for _ in range(2))
            kept = fp.Act8(rows, cols) if c["keep"] == "act8" else None
            fp.fsdp_layer_norm_forward(s["x"], s["weight"], s["bias"], y, mean, rstd, eps=EPS, keep=kept)
            if kept is None:
                return y, mean, rstd
            back = torch.empty_like(y)
            fp.fsdp_act8_load(kept, back)
            return y, mean, rstd, back
        x = fp.Act8(rows, cols, s["kept"]) if c["keep"] == "act8" else s["x"]
        dx = torch.empty_like(s["dy"])
        dw, db = torch.empty_like(s["weight"]), torch.empty_like(s["weight"])
        fp.fsdp_layer_norm_backward(s["dy"], x, s["weight"], s["mean"], s["rstd"], dx, dw, db)
        return dx, dw, db
    d, f = c["d"], c["f"]
    act = fp.FSDP_ACT_SILU if c["act"] == "silu" else fp.FSDP_ACT_GELU
    x, wg, wu = s["x"], s["w_gate"], s["w_up"]
    gate = up = None
    out = []
    if op != "ffn_bwd":
        h = torch.empty(rows, f, dtype=BF16, device="cuda")
        if c["keep"] == "act8":
            gate, up = fp.Act8(rows, f), fp.Act8(rows, f)
        elif c["keep"] == "bf16":
            gate, up = torch.empty_like(h), torch.empty_like(h)
        fp.fsdp_gated_ffn_forward(x, wg, wu, h, gate=gate, up=up, activation=act)
        out.append(h)
        if op == "ffn_fwd":
            if c["keep"] == "act8":
                back = [torch.empty_like(h) for _ in range(2)]
                fp.fsdp_act8_load(gate, back[0])
                fp.fsdp_act8_load(up, back[1])
                out += back
            elif c["keep"] == "bf16":
                out += [gate, up]
            return out
        kept = fp.Act8(rows, d)
        fp.fsdp_act8_store(x, kept)
        x = kept
    elif c["keep"] == "act8":
        gate, up = fp.Act8(rows, f, s["gate"]), fp.Act8(rows, f, s["up"])
    elif c["keep"] == "bf16":
        gate, up = s["gate"], s["up"]
    dx = torch.empty(rows, d, dtype=BF16, device="cuda")
    dwg, dwu = torch.empty_like(wg), torch.empty_like(wu)
    fp.fsdp_gated_ffn_backward(s["dh"], x, wg, wu, dx, dwg, dwu, gate=gate, up=up, activation=act)
    return out + [dx, dwg, dwu]


def _act_and_slope(g, act):
    if act == "silu":
        t = torch.sigmoid(g)
        return g * t, t * (1 + g * (1 - t))
    t = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
    return g * t, t + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))


def _run_plain(s, c):
    op, rows = c["op"], c["rows"]
    if not op.startswith("ffn"):
        cols, dt = c["cols"], DTYPES[c["dtype"]]
        if op == "act8_store":
            return _decode(_encode(s["x"].float()), rows, cols).to(dt)
        if op == "act8_load":
            return _decode(s["kept"], rows, cols).to(dt)
        if op == "norm_fwd":
            x = s["x"].float()
            mean = x.mean(-1)
            centred = x - mean[:, None]
            rstd = (centred.square().mean(-1) + EPS).rsqrt()
            y = (centred * rstd[:, None] * s["weight"] + s["bias"]).to(dt)
            return (y, mean, rstd) if c["keep"] == "none" else (y, mean, rstd, _decode(_encode(x), rows, cols).to(dt))
        x = _decode(s["kept"], rows, cols) if c["keep"] == "act8" else s["x"].float()
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xh = (x - s["mean"][:, None]) * rstd
        g = dy * s["weight"]
        dx = rstd * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
        return dx.to(dt), (dy * xh).sum(0), dy.sum(0)
    x, wg, wu = s["x"].float(), s["w_gate"].float(), s["w_up"].float()
    out = []
    if op == "ffn_bwd" and c["keep"] != "none":
        g, u = (_decode(s[k], rows, c["f"]) if c["keep"] == "act8" else s[k].float() for k in ("gate", "up"))
    else:
        g, u = x @ wg.T, x @ wu.T
    if op != "ffn_bwd":
        out.append((_act_and_slope(g, c["act"])[0] * u).to(BF16))
        if c["keep"] == "act8":
            g, u = (_decode(_encode(t), rows, c["f"]) for t in (g, u))
        if op == "ffn_fwd":
            return out + ([g.to(BF16), u.to(BF16)] if c["keep"] != "none" else [])
        x = _decode(_encode(x), rows, c["d"])
    dh = s["dh"].float()
    a, slope = _act_and_slope(g, c["act"])
    dg, du = dh * u * slope, dh * a
    return out + [(dg @ wg + du @ wu).to(BF16), (dg.T @ x).to(BF16), (du.T @ x).to(BF16)]


def work(case):
    op, rows = case["op"], case["rows"]
    if not op.startswith("ffn"):
        cols, size = case["cols"], 2 if case["dtype"] == "bf16" else 4
        n, kept = rows * cols, rows * 33 * _groups(cols)
        if op in ("act8_store", "act8_load"):  # a store case reads its values back as well
            return {"bytes": (n * size + kept) * (2 if op == "act8_store" else 1), "flops": 2 * n}
        if op == "norm_fwd":
            back = kept * 2 + n * size if case["keep"] == "act8" else 0  # kept, and read back
            return {"bytes": 2 * n * size + back + 8 * rows + 8 * cols, "flops": 8 * n}
        return {"bytes": 2 * n * size + (kept if case["keep"] == "act8" else n * size) + 8 * rows + 12 * cols,
                "flops": 14 * n}
    d, f = case["d"], case["f"]
    product = 4 * rows * d * f
    kept = {"none": 0, "act8": 2 * rows * 33 * _groups(f), "bf16": 4 * rows * f}[case["keep"]]
    kept_x = rows * 33 * _groups(d)
    w, x, h = 4 * f * d, 2 * rows * d, 2 * rows * f
    if op == "ffn_fwd":
        back = kept + 4 * rows * f if case["keep"] == "act8" else 0
        return {"bytes": x + w + h + kept + back, "flops": product}
    if op == "ffn_bwd":
        return {"bytes": h + x + w + kept + x + w, "flops": (2 + (case["keep"] == "none")) * product}
    return {"bytes": 2 * x + 2 * w + 2 * h + 2 * kept + 2 * kept_x, "flops": 3 * product}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _power_of_two(e):
    """2^e in 64 bits, exactly (a power function may be an ulp off, which turns ties)."""
    return ((e.to(torch.int64) + 1023) << 52).view(F64)


def _kept_exact(x):
    """The values that the 8-bit checkpoint of x stands for: the least power of two 2^e (e >= -126) with max|x| <= 127 2^e
    over 32 consecutive elements, and the nearest whole multiple of it (ties to even)."""
    rows, cols = x.shape
    out = torch.zeros(rows, _groups(cols) * GROUP, dtype=F64, device=x.device)
    out[:, :cols] = x
    out = out.reshape(-1, GROUP)
    top = out.abs().max(dim=1, keepdim=True).values
    part, e = torch.frexp(top / 127)  # top / 127 = part 2^e with part in [0.5, 1)
    e = torch.where(part == 0.5, e - 1, e).clamp(min=-126)
    return (torch.round(out * _power_of_two(-e)) * _power_of_two(e)).reshape(rows, -1)[:, :cols]


def _read_exact(buf, rows, cols):
    g = _groups(cols)
    n = rows * g * GROUP
    e = buf[n:].to(torch.int64).repeat_interleave(GROUP) - 127
    return (buf[:n].view(torch.int8).to(F64) * _power_of_two(e)).reshape(rows, g * GROUP)[:, :cols]


def exact(case, seed):
    s, op, rows = prepare(case, seed), case["op"], case["rows"]
    if not op.startswith("ffn"):
        cols = case["cols"]
        if op == "act8_store":
            return _kept_exact(s["x"].to(F64))
        if op == "act8_load":
            return _read_exact(s["kept"], rows, cols)
        w, b = s["weight"].to(F64), s["bias"].to(F64)
        if op == "norm_fwd":
            x = s["x"].to(F64)
            var, mean = torch.var_mean(x, dim=1, correction=0)
            rstd = 1 / torch.sqrt(var + EPS)
            y = torch.addcmul(b, (x - mean.unsqueeze(1)) * rstd.unsqueeze(1), w)
            return (y, mean, rstd, _kept_exact(x)) if case["keep"] == "act8" else (y, mean, rstd)
        x = _read_exact(s["kept"], rows, cols) if case["keep"] == "act8" else s["x"].to(F64)
        dy, r = s["dy"].to(F64), s["rstd"].to(F64)
        xh = torch.einsum("ij,i->ij", x - s["mean"].to(F64).unsqueeze(1), r)
        c1 = torch.einsum("ij,ij,j->i", dy, xh, w) / cols
        c2 = torch.mv(dy, w) / cols
        dx = torch.einsum("ij,i->ij", dy * w - torch.outer(c2, torch.ones_like(w)) - torch.einsum("ij,i->ij", xh, c1), r)
        return dx, torch.einsum("ij,ij->j", dy, xh), torch.einsum("ij->j", dy)
    x, wg, wu = s["x"].to(F64), s["w_gate"].to(F64), s["w_up"].to(F64)

    def gated(g, u):
        return torch.nn.functional.silu(g) * u if case["act"] == "silu" else torch.nn.functional.gelu(g) * u

    if op == "ffn_bwd" and case["keep"] == "act8":
        g, u = _read_exact(s["gate"], rows, case["f"]), _read_exact(s["up"], rows, case["f"])
    elif op == "ffn_bwd" and case["keep"] == "bf16":
        g, u = s["gate"].to(F64), s["up"].to(F64)
    else:
        g, u = torch.einsum("td,fd->tf", x, wg), torch.einsum("td,fd->tf", x, wu)
    out = []
    if op != "ffn_bwd":
        out.append(gated(g, u))
        if case["keep"] == "act8":
            g, u = _kept_exact(g), _kept_exact(u)
        if op == "ffn_fwd":
            return out + ([g, u] if case["keep"] != "none" else [])
        x = _kept_exact(x)
    g, u = g.requires_grad_(), u.requires_grad_()
    dg, du = torch.autograd.grad(gated(g, u), (g, u), s["dh"].to(F64))
    dx = torch.einsum("tf,fd->td", dg, wg) + torch.einsum("tf,fd->td", du, wu)
    return out + [dx, torch.einsum("tf,td->fd", dg, x), torch.einsum("tf,td->fd", du, x)]
