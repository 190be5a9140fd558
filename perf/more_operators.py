"""What the operators at the two ends of a training step and in its recurrent layers are measured on: embedding lookup and
its gradient, the gated linear recurrence, distillation from a teacher's top logits and the clipped policy loss.

``run`` computes an operator either in its plain form (elementary torch operations in 32 bits, rounded once at the end)
or, where ``own`` is true, through the package's entry points.  ``exact`` computes the same from the definitions in 64
bits.  Widths are those of the package's layouts (512, 1024, 4096) and odd ones beside them; vocabularies are generic.
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
DTYPES = {"bf16": BF16, "f32": F32}
SCALE = 32.0        # of embedded rows
CLIP = (0.2, 0.28)  # below and above a probability ratio of 1
KL = 0.05


def listed():
    return [
        # The next tokens of a few sequences: the latency of a lookup.
        dict(name="embed_fwd_few", op="embed_fwd", rows=8, vocab=32768, d=1024, dtype="bf16"),
        # The embedding's gradient of a long batch, written whole in BF16 for the group that packs it.
        dict(name="embed_bwd", op="embed_bwd", rows=16384, vocab=32768, d=4096, dtype="bf16", add=False),
        # Lookup and gradient at sizes that no vector divides, added in FP32 to a tied output layer's gradient.
        dict(name="embed_step_odd", op="embed_step", rows=4099, vocab=5003, d=515, dtype="f32", add=True),
        # One token of each of 64 sequences, states read and written: a step of serving.
        dict(name="scan_fwd_token", op="scan_fwd", seqs=64, length=1, d=4096, dtype="bf16", packed=False),
        # One long sequence of a narrow model: work only along time.
        dict(name="scan_fwd_long", op="scan_fwd", seqs=1, length=65536, d=1024, dtype="bf16", packed=False),
        # A training pass of the widest layout, forward and backward.
        dict(name="scan_step", op="scan_step", seqs=4, length=8192, d=4096, dtype="bf16", packed=False),
        # Sequences of every length packed into one batch, an odd width, in FP32.
        dict(name="scan_step_packed", op="scan_step", seqs=23, length=435, d=1409, dtype="f32", packed=True),
        # The loss alone of a few rows over a large vocabulary: few rows to share among many SMs.
        dict(name="distill_fwd_few", op="distill_fwd", rows=16, vocab=131072, top=64, dtype="bf16", temperature=1.0),
        # Loss and gradient of a batch over a large vocabulary.
        dict(name="distill_step", op="distill_step", rows=4096, vocab=131072, top=64, dtype="bf16", temperature=1.0),
        # The gradient alone, in FP32, a vocabulary that no vector divides, softened by a temperature.
        dict(name="distill_bwd_odd", op="distill_bwd", rows=1001, vocab=50021, top=17, dtype="f32", temperature=2.0),
        # The loss and log-probabilities of a short batch, as for a metric.
        dict(name="policy_fwd", op="policy_fwd", rows=512, vocab=32768, dtype="bf16", temperature=1.0),
        # Loss and gradient of a batch of sampled sequences.
        dict(name="policy_step", op="policy_step", rows=8192, vocab=32768, dtype="bf16", temperature=0.7),
    ]


def _spread(rng, low, high):
    """A whole number from low to high, spread over its logarithm; half of them as they fall, half rounded to 32s."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if n >= 64 and rng.random() < 0.5:
        n = (n + 31) // 32 * 32
    return max(low, min(high, n))


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(["embed_fwd", "embed_bwd", "embed_step", "scan_fwd", "scan_step", "scan_step", "distill_fwd",
                         "distill_step", "distill_bwd", "policy_fwd", "policy_step", "policy_bwd"])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if op.startswith("embed"):
            case = dict(op=op, rows=_spread(rng, 1, 65536), vocab=_spread(rng, 256, 131072), d=_spread(rng, 64, 4096), dtype=dtype)
            if op != "embed_fwd":
                case["add"] = rng.random() < 0.5
        elif op.startswith("scan"):
            case = dict(op=op, seqs=_spread(rng, 1, 256), length=_spread(rng, 1, 65536), d=_spread(rng, 64, 4096), dtype=dtype,
                        packed=rng.random() < 0.5)
            if case["seqs"] * case["length"] > 131072 or case["packed"] and case["seqs"] * case["length"] > 16384:
                continue
        else:
            case = dict(op=op, rows=_spread(rng, 1, 8192), vocab=_spread(rng, 512, 262144), dtype=dtype,
                        temperature=rng.choice([0.7, 1.0, 2.0]))
            if op.startswith("distill"):
                case["top"] = _spread(rng, 1, 128)
        if work(case)["bytes"] <= most:
            return case


def _normal(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=F32).mul_(std)


def _uniform(gen, *shape):
    return torch.rand(*shape, generator=gen, device="cuda", dtype=F32)


def _active(rows):
    """Rows that count: the last 16 tokens of every 64 are padding or another's turn."""
    return rows // 64 * 48 + min(rows % 64, 48)


def _offsets(case, seed):
    """Where packed sequences of uneven lengths (some of them empty) begin and end."""
    gen = torch.Generator().manual_seed(seed)
    cuts = torch.sort(torch.randint(0, case["seqs"] * case["length"] + 1, (case["seqs"] - 1,), generator=gen)).values
    return torch.cat([torch.zeros(1, dtype=torch.int64), cuts, torch.tensor([case["seqs"] * case["length"]])])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    s = {"case": dict(case)}
    if op.startswith("embed"):
        rows, vocab, d = case["rows"], case["vocab"], case["d"]
        # Frequencies that fall as one over the rank, ranks in any order of ids, a few padding tokens among them.
        rank = (torch.exp(_uniform(gen, rows).double() * math.log(vocab + 1)) - 1).long().clamp(max=vocab - 1)
        tokens = torch.randperm(vocab, generator=gen, device="cuda")[rank]
        s["tokens"] = torch.where(_uniform(gen, rows) < 0.02, -1, tokens)
        if op != "embed_bwd":
            s["weight"] = _normal(gen, vocab, d, std=0.02).to(dt)
        if op != "embed_fwd":
            s["dout"] = _normal(gen, rows, d, std=0.01).to(BF16)
            if case["add"]:
                s["grad"] = _normal(gen, vocab, d, std=0.1).to(dt)
        return s
    if op.startswith("scan"):
        rows, d = case["seqs"] * case["length"], case["d"]
        s["x"] = _normal(gen, rows, d).to(dt)
        # Channels that forget at different rates, from a few tokens to thousands.
        s["bias"] = 1 + 7 * _uniform(gen, d)
        s["gate"] = _normal(gen, rows, d).to(dt)
        s["initial"] = _normal(gen, case["seqs"], d, std=0.3)
        if case["packed"]:
            s["offsets"] = _offsets(case, seed).to("cuda")
        if op == "scan_step":
            s["dh"] = _normal(gen, rows, d, std=0.01).to(dt)
            s["dfinal"] = _normal(gen, case["seqs"], d, std=0.01)
        return s
    rows, vocab = case["rows"], case["vocab"]
    logits = _normal(gen, rows, vocab, std=2.0)
    s["weight"] = torch.where(torch.arange(rows, device="cuda") % 64 < 48, 1 / _active(rows), 0.0)
    if op.startswith("distill"):
        top = min(case["top"], vocab)
        # Distinct tokens in every row, likely ones of the student too; some rows have fewer, a few rows none.
        first = torch.randint(0, vocab, (rows, 1), generator=gen, device="cuda")
        ids = (first + torch.arange(top, device="cuda") * (vocab // top)) % vocab
        falling = 8 - 1.5 * torch.log(torch.arange(1, top + 1, device="cuda", dtype=F32))
        s["teacher"] = (falling + _normal(gen, rows, top, std=0.5)).to(dt)
        logits.scatter_add_(1, ids, falling.expand(rows, top) + _normal(gen, rows, top))
        kept = torch.where(_uniform(gen, rows, 1) < 0.1, _uniform(gen, rows, 1) * top, float(top))
        s["ids"] = torch.where(torch.arange(top, device="cuda") < kept.floor(), ids, -1).to(torch.int32)
    else:
        s["ids"] = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
        logits.scatter_add_(1, s["ids"][:, None], 4 + 4 * _uniform(gen, rows, 1))
        s["advantage"] = _normal(gen, rows)
    s["logits"] = logits = logits.to(dt)
    scaled = [c.float() / case["temperature"] for c in logits.split(1024)]
    lse = torch.cat([c.logsumexp(-1) for c in scaled])
    if op.startswith("policy"):
        # Policies a few steps away; no ratio is at a border of the clipping, where the derivative jumps.
        logp = torch.cat([c.gather(1, i[:, None])[:, 0] for c, i in zip(scaled, s["ids"].split(1024))]) - lse
        drift = _normal(gen, rows, std=0.2)
        for border in (math.log(1 - CLIP[0]), math.log(1 + CLIP[1])):
            drift = torch.where((drift - border).abs() < 1e-3, border + 2e-3, drift)
        s["logp"] = logp
        s["old"], s["ref"] = logp - drift, logp - _normal(gen, rows, std=0.3)
    del scaled
    if op.endswith("bwd"):
        s["lse"] = lse
        s["dloss"] = 0.5 + _uniform(gen, rows)
    return s


# ---------------------------------------------------------------------------
# The operators
# ---------------------------------------------------------------------------
def run(state):
    return (_run_own if own else _run_plain)(state, state["case"])


def _run_own(s, c):
    from fsdp2_gradient_packing_gb300 import fsdp_pack as fp
    op, dt = c["op"], DTYPES[c["dtype"]]
    out = []
    if op.startswith("embed"):
        if op != "embed_bwd":
            out.append(torch.empty(c["rows"], c["d"], dtype=BF16, device="cuda"))
            fp.fsdp_embedding_forward(s["tokens"], s["weight"], out[0], scale=SCALE)
        if op != "embed_fwd":
            grad = s["grad"].clone() if c["add"] else torch.empty(c["vocab"], c["d"], dtype=dt, device="cuda")
            fp.fsdp_embedding_backward(s["tokens"], s["dout"], grad, scale=SCALE, accumulate=c["add"])
            out.append(grad)
        return out
    if op.startswith("scan"):
        x, gate, rows, d = s["x"], s["gate"], c["seqs"] * c["length"], c["d"]
        where = dict(offsets=s["offsets"]) if c["packed"] else dict(seq_len=c["length"])
        h, final = torch.empty_like(x), torch.empty_like(s["initial"])
        states = None
        if op == "scan_step":
            states = torch.empty(fp.fsdp_gated_scan_states(rows, d), d, dtype=F32, device="cuda")
        fp.fsdp_gated_scan_forward(x, gate, h, bias=s["bias"], initial=s["initial"], final=final, states=states, **where)
        if op == "scan_fwd":
            return h, final
        dx, dgate, dbias, dinitial = (torch.empty_like(t) for t in (x, gate, s["bias"], s["initial"]))
        fp.fsdp_gated_scan_backward(s["dh"], x, gate, states, dx, dgate, bias=s["bias"], dbias=dbias, initial=s["initial"],
                                    dinitial=dinitial, dfinal=s["dfinal"], **where)
        return h, final, dx, dgate, dbias, dinitial
    logits, rows = s["logits"], c["rows"]
    dlogits = None if op.endswith("fwd") else torch.empty_like(logits)
    if op == "distill_bwd":
        fp.fsdp_distill_loss_backward(logits, s["ids"], s["teacher"], s["lse"], dlogits, temperature=c["temperature"],
                                      weight=s["weight"], dloss=s["dloss"])
        return dlogits
    choice = dict(ref_logp=None if op.startswith("distill") else s["ref"], weight=s["weight"], temperature=c["temperature"],
                  clip_low=CLIP[0], clip_high=CLIP[1], kl=KL)
    if op == "policy_bwd":
        fp.fsdp_policy_loss_backward(logits, s["ids"], s["old"], s["advantage"], s["logp"], s["lse"], dlogits, dloss=s["dloss"],
                                     **choice)
        return dlogits
    loss, lse = torch.empty(rows, dtype=F32, device="cuda"), torch.empty(rows, dtype=F32, device="cuda")
    if op.startswith("distill"):
        fp.fsdp_distill_loss_forward(logits, s["ids"], s["teacher"], loss, lse, temperature=c["temperature"], weight=s["weight"],
                                     dlogits=dlogits)
        out = [loss, lse]
    else:
        logp = torch.empty(rows, dtype=F32, device="cuda")
        fp.fsdp_policy_loss_forward(logits, s["ids"], s["old"], s["advantage"], loss, logp, lse, dlogits=dlogits, **choice)
        out = [loss, logp, lse]
    return out if dlogits is None else out + [dlogits]


def _starts(s, c):
    """First row of every sequence with rows, and those sequences."""
    if not c["packed"]:
        return torch.arange(c["seqs"], device="cuda") * c["length"], torch.arange(c["seqs"], device="cuda")
    which = (s["offsets"][1:] > s["offsets"][:-1]).nonzero()[:, 0]
    return s["offsets"][which], which


def _linear_scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dimension 0, in log2(rows) doubling steps."""
    a, b, step = a.clone(), b.clone(), 1
    while step < a.shape[0]:
        b[step:] += a[step:] * b[:-step]  # the right side is whole before the left changes
        a[step:] = a[step:] * a[:-step]
        step *= 2
    return b


def _plain_scan(s, c):
    x, z = s["x"].float(), s["gate"].float() + s["bias"]
    a, keep = torch.sigmoid(z), torch.sigmoid(-z)
    first, which = _starts(s, c)
    b = keep * x
    b[first] += a[first] * s["initial"][which]
    cut = a.clone()
    cut[first] = 0.0
    h = _linear_scan(cut, b)
    last = torch.cat([first[1:], first.new_tensor([x.shape[0]])]) - 1
    final = s["initial"].clone()
    final[which] = h[last]
    if c["op"] == "scan_fwd":
        return h.to(s["x"].dtype), final
    before = torch.empty_like(h)
    before[1:] = h[:-1]
    before[first] = s["initial"][which]
    grad = s["dh"].float().clone()  # the conversion of an FP32 tensor is the tensor itself
    grad[last] += s["dfinal"][which]
    later = torch.zeros_like(cut)
    later[:-1] = cut[1:]
    total = _linear_scan(later.flip(0), grad.flip(0)).flip(0)
    dz = total * (before - x) * a * keep
    dinitial = s["dfinal"].clone()  # an empty sequence passes its state on
    dinitial[which] = (a * total)[first]
    dt = s["x"].dtype
    return h.to(dt), final, (keep * total).to(dt), dz.to(dt), dz.sum(0), dinitial


def _plain_teacher(s, c):
    """Probabilities and their logarithms over a row's top tokens (0 where there is none), and safe indices."""
    here = s["ids"] >= 0
    t = torch.where(here, s["teacher"].float() / c["temperature"], -math.inf)
    top = t.amax(-1, keepdim=True)
    e = torch.where(here, torch.exp(t - torch.where(top > -math.inf, top, 0.0)), 0.0)
    total = e.sum(-1, keepdim=True).clamp(min=1e-30)
    return e / total, torch.where(here, t - top - torch.log(total), 0.0), s["ids"].long().clamp(min=0)


def _run_plain(s, c):
    op, dt = c["op"], DTYPES[c["dtype"]]
    if op.startswith("embed"):
        tokens, out = s["tokens"], []
        here = tokens >= 0
        if op != "embed_bwd":
            rows = s["weight"][tokens.clamp(min=0)].float() * SCALE
            out.append(torch.where(here[:, None], rows, 0.0).to(BF16))
        if op != "embed_fwd":
            grad = torch.zeros(c["vocab"], c["d"], dtype=F32, device="cuda")
            grad.index_add_(0, tokens[here], s["dout"][here].float())
            grad *= SCALE
            if c["add"]:
                grad += s["grad"].float()
            out.append(grad.to(dt))
        return out
    if op.startswith("scan"):
        return _plain_scan(s, c)
    w, soft = s["weight"], c["temperature"]
    z = s["logits"].float() / soft
    if op.endswith("bwd"):
        lse = s["lse"]
    else:
        top = z.amax(-1, keepdim=True)
        lse = torch.log(torch.exp(z - top).sum(-1)) + top[:, 0]
    active = w != 0
    up = w * s["dloss"] if op.endswith("bwd") else w
    if op.startswith("distill"):
        q, log_q, ids = _plain_teacher(s, c)
        mass = q.sum(-1)
        out = [w * soft * soft * (q * (log_q - z.gather(1, ids) + lse[:, None])).sum(-1), torch.where(active, lse, 0.0)]
        if op == "distill_fwd":
            return out
        g = torch.exp(z - lse[:, None]) * mass[:, None]
        g.scatter_add_(1, ids, -q)
        g *= (up * soft)[:, None]
    else:
        logp = s["logp"] if op == "policy_bwd" else z.gather(1, s["ids"][:, None])[:, 0] - lse
        ratio, adv, rest = torch.exp(logp - s["old"]), s["advantage"], s["ref"] - logp
        clipped = ratio.clamp(1 - CLIP[0], 1 + CLIP[1])
        loss = -torch.minimum(ratio * adv, clipped * adv) + KL * (torch.exp(rest) - rest - 1)
        out = [w * loss] + [torch.where(active, t, 0.0) for t in (logp, lse)]
        if op == "policy_fwd":
            return out
        slope = torch.where(ratio * adv <= clipped * adv, -adv * ratio, 0.0) + KL * (1 - torch.exp(rest))
        g = torch.exp(z - lse[:, None]).neg_()
        g.scatter_add_(1, s["ids"][:, None], torch.ones_like(ratio)[:, None])
        g *= (up * slope / soft)[:, None]
    g = g.to(dt)
    return g if op.endswith("bwd") else out + [g]


def work(case):
    op, size = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op.startswith("embed"):
        rows, vocab, d = case["rows"], case["vocab"], case["d"]
        n = {"bytes": 0, "flops": 0}
        if op != "embed_bwd":  # each row of the table once, however often it is looked up
            n["bytes"] += 8 * rows + min(rows, vocab) * d * size + rows * d * 2
            n["flops"] += rows * d
        if op != "embed_fwd":
            n["bytes"] += 8 * rows + rows * d * 2 + vocab * d * size * (2 if case["add"] else 1)
            n["flops"] += 2 * rows * d
        return n
    if op.startswith("scan"):
        n, state = case["seqs"] * case["length"] * case["d"], 4 * case["seqs"] * case["d"]
        forward = 3 * n * size + 2 * state + 4 * case["d"]
        if op == "scan_fwd":
            return {"bytes": forward, "flops": 12 * n}
        return {"bytes": forward + 5 * n * size + 3 * state + 8 * case["d"], "flops": 36 * n}
    rows, active = case["rows"], _active(case["rows"])
    n = active * case["vocab"] * size + 16 * rows
    if op.startswith("distill"):
        n += active * min(case["top"], case["vocab"]) * (4 + size)
    else:
        n += 20 * rows
    flops = 4 * active * case["vocab"]
    if not op.endswith("fwd"):
        n, flops = n + rows * case["vocab"] * size, flops * 2
    return {"bytes": n, "flops": flops}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_scan(s, c):
    x, z = s["x"].to(F64), s["gate"].to(F64) + s["bias"].to(F64)
    a = 1 / (1 + torch.exp(-z))
    off = s["offsets"].tolist() if c["packed"] else [k * c["length"] for k in range(c["seqs"] + 1)]
    step = c["op"] == "scan_step"
    h, dx, dz = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    final, dinitial = s["initial"].to(F64), s["dfinal"].to(F64) if step else None

    def go(rows, state):
        """One or several sequences of one length; rows[t] picks their t-th rows."""
        h0 = state
        for t in rows:
            state = state + (1 - a[t]) * (x[t] - state)
            h[t] = state
        return h0, state

    def back(rows, h0, grad):
        for k in range(len(rows) - 1, -1, -1):
            t = rows[k]
            grad = grad + s["dh"][t].to(F64)
            dx[t] = grad / (1 + torch.exp(z[t]))
            dz[t] = grad * ((h[rows[k - 1]] if k else h0) - x[t]) * a[t] / (1 + torch.exp(z[t]))
            grad = grad * a[t]
        return grad

    if c["packed"]:
        groups = [(range(off[k], off[k + 1]), k) for k in range(c["seqs"])]
    else:
        groups = [([slice(t, None, c["length"]) for t in range(c["length"])], slice(None))]
    for rows, which in groups:
        if len(rows):
            h0, end = go(rows, final[which].clone())
            final[which] = end
            if step:
                dinitial[which] = back(rows, h0, dinitial[which].clone())
    return (h, final, dx, dz, torch.einsum("ij->j", dz), dinitial) if step else (h, final)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op.startswith("embed"):
        tokens, out = s["tokens"], []
        if op != "embed_bwd":
            table = torch.cat([s["weight"].to(F64) * SCALE, torch.zeros(1, case["d"], dtype=F64, device="cuda")])
            out.append(torch.index_select(table, 0, torch.where(tokens < 0, case["vocab"], tokens)))
        if op != "embed_fwd":
            # Rows in the order of their tokens, as differences of one running sum over each batch of columns.
            order = torch.argsort(tokens, stable=True)
            ends = torch.searchsorted(tokens[order], torch.arange(case["vocab"], device="cuda"), right=True)
            begins = torch.searchsorted(tokens[order], torch.arange(case["vocab"], device="cuda"))
            grad = torch.empty(case["vocab"], case["d"], dtype=F64, device="cuda")
            for at in range(0, case["d"], 256):
                part = s["dout"][:, at:at + 256].to(F64)[order]
                sums = torch.cat([torch.zeros_like(part[:1]), part.cumsum(0)])
                grad[:, at:at + 256] = (sums[ends] - sums[begins]) * SCALE
            out.append(grad + s["grad"].to(F64) if case["add"] else grad)
        return out
    if op.startswith("scan"):
        # The loop below costs some 60 us a row of time, and as much again backward.
        steps = case["seqs"] * case["length"] if case["packed"] else case["length"]
        return _exact_scan(s, case) if steps <= 70000 else None
    t, w = case["temperature"], s["weight"].to(F64)
    parts = []
    for at in range(0, case["rows"], 512):
        rows = slice(at, at + 512)
        z = s["logits"][rows].to(F64).requires_grad_()
        logits = torch.log_softmax(z / t, -1)
        lse = torch.logsumexp(z.detach() / t, -1)
        if op.startswith("distill"):
            ids = s["ids"][rows].long()
            teacher = (s["teacher"][rows].to(F64) / t).masked_fill(ids < 0, -math.inf)
            some = (ids >= 0).any(-1, keepdim=True)
            q = torch.where(some, torch.softmax(torch.where(some, teacher, 0.0), -1), 0.0)
            picked = torch.take_along_dim(logits, ids.clamp(min=0), 1)
            loss = t * t * (torch.special.xlogy(q, q) - q * picked).sum(-1)
            extra = []
        else:
            logp = torch.take_along_dim(logits, s["ids"][rows][:, None], 1)[:, 0]
            r, adv = torch.exp(logp - s["old"][rows].to(F64)), s["advantage"][rows].to(F64)
            held = torch.clip(r, 1 - CLIP[0], 1 + CLIP[1])
            gap = s["ref"][rows].to(F64) - logp
            loss = torch.maximum(-r * adv, -held * adv) + KL * (torch.expm1(gap) - gap)
            extra = [torch.where(w[rows] != 0, logp.detach(), 0.0)]
        loss = loss * w[rows]
        piece = [loss.detach()] + extra + [torch.where(w[rows] != 0, lse, 0.0)]
        if not op.endswith("fwd"):
            up = s["dloss"][rows].to(F64) if op.endswith("bwd") else torch.ones_like(loss)
            grad, = torch.autograd.grad(loss, z, up)
            piece = [grad] if op.endswith("bwd") else piece + [grad]
        parts.append(piece)
    out = [torch.cat(p) for p in zip(*parts)]
    return out[0] if op.endswith("bwd") else out
