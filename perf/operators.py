"""Cases, plain forms and calls of the gated delta rule and the norms around a block.

Four operators, as one layer of a gated-delta network uses them in turn:

  prefill     gated_delta_fwd: the chunked gated delta rule over whole prompts
  decode      gated_delta_update: the same recurrence, one token, state in place
  add_norm    add_rmsnorm_fwd / _bwd: residual + scale * x, then an RMS norm
  gated_norm  gated_rmsnorm_fwd / _bwd: an RMS norm per group with a silu gate

``run`` computes a case in plain torch operations, or with ``own`` set
through the framework's entry points; ``exact`` computes it in 64 bits from
the definition.
"""
import math
import random

import torch
import torch.nn.functional as F

own = False

CHUNK = 64  # steps of a chunk of the plain form
EPS = 1e-5
MOST_TOKEN_HEADS = 8 * 2048 * 32  # prefill: batch * length * heads of the largest case
MOST_FP32 = 2 * 1024 * 8          # the same for fp32 inputs
MOST_STATES = 192 * 32            # decode: batch * heads of the largest case
MOST_VALUES = 16384 * 4096        # norms: rows * width of the largest case


def listed():
    return [
        # one user's next token: all latency
        dict(name="decode-1", op="decode", dtype="bf16", batch=1, groups=16, heads=32,
             headdim=128, dstate=128),
        # a full server's next token: bound by the states
        dict(name="decode-192", op="decode", dtype="bf16", batch=192, groups=16, heads=32,
             headdim=128, dstate=128),
        # a small model in fp32 with sizes that no vector width divides evenly
        dict(name="decode-odd-f32", op="decode", dtype="f32", batch=33, groups=3, heads=9,
             headdim=77, dstate=70),
        # one long prompt: few sequences, a long chain
        dict(name="prompt-8192", op="prefill", dtype="bf16", batch=1, seqlen=8192, groups=16,
             heads=32, headdim=128, dstate=128, seqs=0, lens=0, h0=False),
        # a batch of prompts of the layers' usual length: the machine is full
        dict(name="prompts-8x2048", op="prefill", dtype="bf16", batch=8, seqlen=2048, groups=16,
             heads=32, headdim=128, dstate=128, seqs=0, lens=0, h0=False),
        # a server's batch: prompts of ragged lengths packed into one row, some
        # continued from a state, one empty and one of a single token
        dict(name="packed-24", op="prefill", dtype="bf16", batch=1, seqlen=9003, groups=16,
             heads=32, headdim=128, dstate=128, seqs=24, lens=7, h0=True),
        # a small fp32 model on a prompt of odd length
        dict(name="prompt-517-f32", op="prefill", dtype="f32", batch=2, seqlen=517, groups=2,
             heads=6, headdim=64, dstate=64, seqs=0, lens=0, h0=True),
        # the norm after the block: one decode step of a few users, per head
        dict(name="gated-norm-serve", op="gated_norm", dtype="bf16", rows=5, width=5120,
             group=64, shared=True, before=True, train=False),
        # a training step's norm after the block, forward and backward
        dict(name="gated-norm-train", op="gated_norm", dtype="bf16", rows=16384, width=4096,
             group=4096, shared=False, before=False, train=True),
        # odd groups in fp32, forward and backward
        dict(name="gated-norm-odd-f32", op="gated_norm", dtype="f32", rows=1003, width=1155,
             group=385, shared=False, before=False, train=True),
        # a training step's norm before the block, fp32 residual stream
        dict(name="add-norm-train", op="add_norm", dtype="bf16", residual="f32", rows=16384,
             width=2560, scaled=True, train=True),
        # the same in serving, residual kept in bf16
        dict(name="add-norm-serve", op="add_norm", dtype="bf16", residual="bf16", rows=64,
             width=2048, scaled=False, train=False),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "prefill", "prefill", "gated_norm", "add_norm"])
    if op in ("decode", "prefill"):
        dtype = rng.choice(["bf16", "bf16", "f32"])
        groups = rng.choice([1, 2, 3, 4, 8, 16])
        heads = groups * rng.choice([1, 2, 3, 4])
        headdim = rng.choice([64, 128, 128, 8 * rng.randint(4, 16), rng.randint(17, 128)])
        dstate = rng.choice([64, 128, 128, 8 * rng.randint(4, 16), rng.randint(17, 128)])
        c = dict(op=op, dtype=dtype, groups=groups, heads=heads, headdim=headdim, dstate=dstate)
        if op == "decode":
            return dict(c, batch=_log_uniform(rng, 1, min(256, MOST_STATES // heads)))
        most = (MOST_FP32 if dtype == "f32" else MOST_TOKEN_HEADS) // heads
        packed = rng.random() < 0.4
        batch = 1 if packed else rng.randint(1, 8)
        seqlen = _log_uniform(rng, 1 if not packed else 32, min(8192, most // batch))
        return dict(c, batch=batch, seqlen=seqlen, seqs=rng.randint(1, 24) if packed else 0,
                    lens=rng.randint(0, 10 ** 6) if packed else 0, h0=rng.random() < 0.5)
    dtype = rng.choice(["bf16", "f32"])
    train = rng.random() < 0.6
    if op == "gated_norm":
        group = rng.choice([64, 128, _log_uniform(rng, 16, 8192), _log_uniform(rng, 512, 8192)])
        ngroups = rng.choice([1, 1, 2, 3, 8, 40])
        ngroups = max(1, min(ngroups, 8192 // group))
        width = group * ngroups
        return dict(op=op, dtype=dtype, rows=_log_uniform(rng, 1, min(16384, MOST_VALUES // 2 // width)),
                    width=width, group=group, shared=rng.random() < 0.5,
                    before=rng.random() < 0.5, train=train)
    width = _log_uniform(rng, 64, 8192)
    return dict(op=op, dtype=dtype, residual=rng.choice(["f32", dtype]),
                rows=_log_uniform(rng, 1, min(16384, MOST_VALUES // 4 // width)), width=width,
                scaled=rng.random() < 0.5, train=train)


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _lengths(case):
    """Lengths of a packed case's sequences: random cuts, one empty sequence and one of a
    single token where there are enough, and a few rows behind the last one."""
    n, total = case["seqs"], case["seqlen"]
    r = random.Random(case["lens"])
    behind = min(3, total // 16)
    cuts = sorted(r.randint(0, total - behind) for _ in range(n - 1))
    if n >= 6:
        cuts[2] = cuts[1]
        cuts[4] = min(cuts[3] + 1, total - behind)
        cuts.sort()
    ends = cuts + [total - behind]
    return [b - a for a, b in zip([0] + ends[:-1], ends)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind = _type(case["dtype"])

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = dict(case=case)
    if case["op"] in ("decode", "prefill"):
        H, G, P, N = case["heads"], case["groups"], case["headdim"], case["dstate"]
        lead = (case["batch"],) if case["op"] == "decode" else (case["batch"], case["seqlen"])
        # queries and keys of a trained layer: behind a silu, so of one sign more
        # than of the other, and of length one
        s["q"] = F.normalize(F.silu(normal(*lead, G, N)), dim=-1).to(kind)
        s["k"] = F.normalize(F.silu(normal(*lead, G, N)), dim=-1).to(kind)
        s["v"] = normal(*lead, H, P).to(kind)
        s["dt"] = normal(*lead, H).to(kind)
        s["beta"] = normal(*lead, H).to(kind)
        s["A"] = -(1 + 15 * torch.rand(H, generator=g, device="cuda"))
        step = 1e-3 + (1e-1 - 1e-3) * torch.rand(H, generator=g, device="cuda")
        s["dt_bias"] = torch.log(torch.expm1(step))
        if case["op"] == "decode":
            s["state"] = 0.25 * normal(case["batch"], H, P, N)
            return s
        seqs = case["seqs"] or case["batch"]
        s["h0"] = 0.25 * normal(seqs, H, P, N) if case["h0"] else None
        s["cu_seqlens"] = None
        if case["seqs"]:
            lens = _lengths(case)
            starts = [0]
            for n in lens:
                starts.append(starts[-1] + n)
            s["lens"] = lens
            s["cu_seqlens"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
            s["y"] = torch.zeros(*lead, H, P, device="cuda", dtype=kind)
        return s
    rows, width = case["rows"], case["width"]
    s["x"] = normal(rows, width).to(kind)
    if case["op"] == "gated_norm":
        s["z"] = normal(rows, width).to(kind)
        s["weight"] = 1 + 0.1 * normal(case["group"] if case["shared"] else width)
    else:
        s["residual"] = (4 * normal(rows, width)).to(_type(case["residual"]))
        s["weight"] = 1 + 0.1 * normal(width)
        s["scale"] = 0.5 + 0.1 * normal(width) if case["scaled"] else None
    if case["train"]:
        s["dy"] = normal(rows, width).to(kind)
        if case["op"] == "add_norm":
            s["dres"] = normal(rows, width).to(_type(case["residual"]))
    return s


# ------------------------------------------------------------ plain forms


def _gates(s, kind=torch.float32):
    """Log decay per step and the writing strength."""
    dt = s["dt"].to(kind) + s["dt_bias"].to(kind)
    return torch.log1p(torch.exp(-dt.abs())).add(dt.clamp(min=0)) * s["A"].to(kind), \
        torch.sigmoid(s["beta"].to(kind))


def _decode_plain(s):
    c = s["case"]
    per = c["heads"] // c["groups"]
    q = s["q"].float().repeat_interleave(per, 1)
    k = s["k"].float().repeat_interleave(per, 1)
    g, beta = _gates(s)
    h = s["state"] * torch.exp(g)[..., None, None]
    u = beta[..., None] * (s["v"].float() - (h * k[:, :, None]).sum(-1))
    h += u[..., None] * k[:, :, None]
    s["state"].copy_(h)
    y = (h * q[:, :, None]).sum(-1) * c["dstate"] ** -0.5
    return y.to(s["q"].dtype), s["state"]


def _padded(s, t, length):
    """Rows of packed sequences as (sequences, length, ...), zeros behind each."""
    cu = s["cu_seqlens"].long()
    at = cu[:-1, None] + torch.arange(length, device="cuda")
    inside = at < cu[1:, None]
    got = t[0][at.clamp(max=t.shape[1] - 1)]
    return got.masked_fill(~inside.reshape(inside.shape + (1,) * (got.dim() - 2)), 0)


def _prefill_plain(s):
    c = s["case"]
    per, C = c["heads"] // c["groups"], CHUNK
    g, beta = _gates(s)
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    L = c["seqlen"]
    if s["cu_seqlens"] is not None:
        L = max(s["lens"])
        q, k, v, g, beta = (_padded(s, t, L) for t in (q, k, v, g, beta))
    n = -(-L // C)

    def chunks(t):  # (B, L, heads, ...) -> (B, heads, n, C, ...)
        t = F.pad(t.movedim(1, -1), (0, n * C - L)).movedim(-1, 1)
        t = t.reshape(t.shape[0], n, C, *t.shape[2:])
        return t.movedim(3, 1)

    q = chunks(q).repeat_interleave(per, 1) * c["dstate"] ** -0.5
    k = chunks(k).repeat_interleave(per, 1)
    v, g, beta = chunks(v), chunks(g), chunks(beta)
    cum = g.cumsum(-1)
    lower = torch.ones(C, C, dtype=torch.bool, device="cuda").tril()
    decay = torch.exp((cum[..., :, None] - cum[..., None, :]).masked_fill(~lower, -math.inf))
    kk = (k @ k.transpose(-1, -2)) * decay * beta[..., None]
    kk = kk.masked_fill(~lower.tril(-1), 0)
    inv = torch.eye(C, device="cuda").expand_as(kk).clone()
    for t in range(1, C):  # (I + kk)^-1, row by row
        inv[..., t, :] -= (kk[..., t, None, :t] @ inv[..., :t, :])[..., 0, :]
    u0 = inv @ (v * beta[..., None])
    w = inv @ (k * (beta * torch.exp(cum))[..., None])
    qk = (q @ k.transpose(-1, -2)) * decay
    qd = q * torch.exp(cum)[..., None]
    kd = k * torch.exp(cum[..., -1:] - cum)[..., None]
    last = torch.exp(cum[..., -1])
    P, N = c["headdim"], c["dstate"]
    h = torch.zeros(q.shape[0], c["heads"], N, P, device="cuda")
    if s["h0"] is not None:
        h += s["h0"].transpose(-1, -2)
    y = torch.empty_like(v)
    for i in range(n):
        u = u0[:, :, i] - w[:, :, i] @ h
        y[:, :, i] = qd[:, :, i] @ h + qk[:, :, i] @ u
        h = h * last[:, :, i, None, None] + kd[:, :, i].transpose(-1, -2) @ u
    y = y.movedim(1, 3).reshape(y.shape[0], n * C, c["heads"], P)[:, :L]
    h = h.transpose(-1, -2).contiguous()
    if s["cu_seqlens"] is None:
        return y.to(s["q"].dtype), h
    cu = s["cu_seqlens"].long()
    at = torch.arange(L, device="cuda")
    rows = cu[:-1, None] + at
    s["y"][0, rows[rows < cu[1:, None]]] = y[rows < cu[1:, None]].to(s["q"].dtype)
    return s["y"], h


def _gate(z):
    sig = torch.sigmoid(z)
    return z * sig, sig * (1 + z * (1 - sig))


def _gated_norm_plain(s):
    c = s["case"]
    rows, ng, gs = c["rows"], c["width"] // c["group"], c["group"]
    x, z = (s[n].float().view(rows, ng, gs) for n in ("x", "z"))
    w = s["weight"].view(-1, gs)
    gate, dgate = _gate(z)
    a = x if c["before"] else x * gate
    r = torch.rsqrt((a * a).mean(-1, keepdim=True) + EPS)
    n = a * r
    y = n * w * gate if c["before"] else n * w
    kind = s["x"].dtype
    out = {"y": y.view(rows, -1).to(kind)}
    if c["train"]:
        dy = s["dy"].float().view(rows, ng, gs)
        dz = dy * n * w * dgate if c["before"] else None
        dn = dy * gate if c["before"] else dy
        out["dweight"] = (dn * n).sum((0, 1) if c["shared"] else 0).view(-1)
        dn = dn * w
        da = r * (dn - n * (dn * n).mean(-1, keepdim=True))
        dx = da if c["before"] else da * gate
        dz = dz if c["before"] else da * x * dgate
        out.update(dx=dx.view(rows, -1).to(kind), dz=dz.view(rows, -1).to(kind))
    return out


def _add_norm_plain(s):
    c = s["case"]
    x = s["x"].float()
    if s["scale"] is not None:
        x = x * s["scale"]
    res = (s["residual"].float() + x).to(s["residual"].dtype)  # the stream that goes on
    h = res.float()
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    n = h * r
    out = {"y": (n * s["weight"]).to(s["x"].dtype), "residual": res}
    if c["train"]:
        dy = s["dy"].float()
        out["dweight"] = (dy * n).sum(0)
        dn = dy * s["weight"]
        dh = r * (dn - n * (dn * n).mean(-1, keepdim=True)) + s["dres"].float()
        out["dresidual"] = dh.to(s["residual"].dtype)
        if s["scale"] is not None:
            out["dscale"] = (dh * s["x"].float()).sum(0)
            dh = dh * s["scale"]
        out["dx"] = dh.to(s["x"].dtype)
    return out


# ------------------------------------------------------ the framework's calls


def _run_own(s):
    import selective_state_space_48_b200 as sss

    c = s["case"]
    if c["op"] == "decode":
        y = sss.gated_delta_update(s["state"], s["q"], s["k"], s["v"], s["dt"], s["A"], s["beta"],
                                   dt_bias=s["dt_bias"], out_dtype=s["q"].dtype)
        return y, s["state"]
    if c["op"] == "prefill":
        return sss.gated_delta_fwd(s["q"], s["k"], s["v"], s["dt"], s["A"], s["beta"],
                                   dt_bias=s["dt_bias"], h0=s["h0"], return_last_state=True,
                                   out_dtype=s["q"].dtype, y=s.get("y"),
                                   cu_seqlens=s["cu_seqlens"])
    if c["op"] == "gated_norm":
        kw = dict(eps=EPS, group_size=c["group"], norm_before_gate=c["before"])
        out = {"y": sss.gated_rmsnorm_fwd(s["x"], s["z"], s["weight"], **kw)}
        if c["train"]:
            out.update(sss.gated_rmsnorm_bwd(s["x"], s["z"], s["weight"], s["dy"], **kw))
        return out
    y, res = sss.add_rmsnorm_fwd(s["x"], s["residual"], s["weight"], scale=s["scale"], eps=EPS)
    out = {"y": y, "residual": res}
    if c["train"]:
        g = sss.add_rmsnorm_bwd(res, s["weight"], s["dy"], dresidual_out=s["dres"], x=s["x"],
                                scale=s["scale"], eps=EPS)
        out.update({n: t for n, t in g.items() if t is not None})
    return out


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "decode":
        return _decode_plain(state)
    if op == "prefill":
        return _prefill_plain(state)
    return _gated_norm_plain(state) if op == "gated_norm" else _add_norm_plain(state)


def work(case):
    """Bytes: each input once, each output once.  Flops of the delta rule: two readouts and
    one rank-one update of the state per token and head."""
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("decode", "prefill"):
        H, G, P, N = case["heads"], case["groups"], case["headdim"], case["dstate"]
        tokens = case["batch"] * case.get("seqlen", 1)
        nbytes = tokens * e * (2 * G * N + 2 * H * P + 2 * H) + 8 * H
        seqs = case.get("seqs") or case["batch"]
        reads = 1 if case["op"] == "decode" or case["h0"] else 0
        return {"bytes": nbytes + 4 * seqs * H * P * N * (1 + reads), "flops": 6 * tokens * H * P * N}
    n = case["rows"] * case["width"]
    if case["op"] == "gated_norm":
        moved = n * e * (6 if case["train"] else 3)
        wide = case["group"] if case["shared"] else case["width"]
        return {"bytes": moved + 4 * wide * (2 if case["train"] else 1),
                "flops": n * (30 if case["train"] else 10)}
    r = 4 if case["residual"] == "f32" else 2
    moved = n * (2 * e + 2 * r)
    if case["train"]:
        moved += n * (2 * e + 2 * r)
    cols = (2 if case["scaled"] else 1) * (2 if case["train"] else 1)
    return {"bytes": moved + 4 * case["width"] * cols, "flops": n * (18 if case["train"] else 7)}


# --------------------------------------------------------------- 64 bits


def _exact_delta(s):
    """The recurrence itself, token by token."""
    c = s["case"]
    f64 = torch.float64
    P, N, H = c["headdim"], c["dstate"], c["heads"]
    per = H // c["groups"]
    dt = s["dt"].to(f64) + s["dt_bias"].to(f64)
    a = torch.exp(s["A"].to(f64) * torch.logaddexp(dt, torch.zeros_like(dt)))
    b = 1 / (1 + torch.exp(-s["beta"].to(f64)))
    one = c["op"] == "decode"
    if one:
        spans = [(i, 0, 1) for i in range(c["batch"])]
    elif s["cu_seqlens"] is not None:
        cu = s["cu_seqlens"].tolist()
        spans = [(0, lo, hi) for lo, hi in zip(cu, cu[1:])]
    else:
        spans = [(i, 0, c["seqlen"]) for i in range(c["batch"])]
    lead = lambda t: t.to(f64)[:, None] if one else t.to(f64)  # noqa: E731
    q, k, v = lead(s["q"]), lead(s["k"]), lead(s["v"])
    a, b = (t[:, None] if one else t for t in (a, b))
    h = (s["state"] if one else s["h0"])
    h = h.to(f64).clone() if h is not None else torch.zeros(len(spans), H, P, N, dtype=f64, device="cuda")
    y = torch.zeros(v.shape, dtype=f64, device="cuda")
    rows = torch.tensor([r for r, _, _ in spans], device="cuda")
    first = torch.tensor([lo for _, lo, _ in spans], device="cuda")
    order = sorted(range(len(spans)), key=lambda i: spans[i][1] - spans[i][2])
    order_t = torch.tensor(order, device="cuda")
    rows, first, h = rows[order_t], first[order_t], h[order_t]
    lens = [spans[i][2] - spans[i][1] for i in order]  # longest first
    live = len(lens)
    for t in range(max(lens)):
        while lens[live - 1] <= t:
            live -= 1
        at = (rows[:live], first[:live] + t)
        kt, qt = (x[at].repeat_interleave(per, 1) for x in (k, q))
        ht = h[:live] * a[at][..., None, None]
        u = b[at][..., None] * (v[at] - (ht @ kt[..., None])[..., 0])
        ht += u[..., None] * kt[:, :, None]
        h[:live] = ht
        y[at] = (ht @ qt[..., None])[..., 0] / math.sqrt(N)
    back = torch.empty_like(h)
    back[order_t] = h
    return (y[:, 0] if one else y), back


def _exact_norm(s):
    """Through the derivatives of the formulas, by torch's differentiation in 64 bits."""
    c = s["case"]
    f64 = torch.float64
    leaf = lambda n: s[n].to(f64).requires_grad_(c["train"]) if s.get(n) is not None else None  # noqa: E731
    x, w = leaf("x"), leaf("weight")
    rows = c["rows"]
    if c["op"] == "gated_norm":
        z = leaf("z")
        gate = (z / (1 + torch.exp(-z)))
        a = x if c["before"] else x * gate
        a = a.reshape(rows, -1, c["group"])
        y = a / torch.sqrt(a.pow(2).sum(-1, keepdim=True) / c["group"] + EPS)
        y = (y * w.reshape(-1, c["group"])).reshape(rows, -1)
        y = y * gate if c["before"] else y
        out = {"y": y.detach()}
        if c["train"]:
            dx, dz, dw = torch.autograd.grad(y, (x, z, w), s["dy"].to(f64))
            out.update(dx=dx, dz=dz, dweight=dw)
        return out
    scale = leaf("scale")
    res = s["residual"].to(f64)
    total = res + (x if scale is None else x * scale)
    stored = total.detach().to(s["residual"].dtype).to(f64)
    h = stored.requires_grad_(c["train"])
    y = h / torch.sqrt(h.pow(2).sum(-1, keepdim=True) / c["width"] + EPS) * w
    out = {"y": y.detach(), "residual": stored.detach()}
    if c["train"]:
        dh, dw = torch.autograd.grad(y, (h, w), s["dy"].to(f64))
        dh = dh + s["dres"].to(f64)
        out.update(dresidual=dh, dweight=dw)
        out["dx"], *ds = torch.autograd.grad(total, [x] + ([scale] if scale is not None else []), dh)
        if ds:
            out["dscale"] = ds[0]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_delta(s) if case["op"] in ("decode", "prefill") else _exact_norm(s)
