"""The block around the MoE layer and its 8-bit activation checkpoints, as
measured cases.

Two operators of the training step (the first also of serving), each with its
gradient.  A case names one pass by "op" and "grad":

  norm     n = x rstd (offset + w): the norm before a block; its gradient
  block    the end of a block in one call: the norm after it, its gate, the
           residual scale and the residual, and the norm before the next block;
           their gradient
  keep     token rows kept in 8 bits and restored, sorted by expert, as the
           backward pass reads them
  experts  the experts' up products that keep g and u in 8 bits; the down
           product's gradient, which reads them in 8 bits
  combine  the combine's gradient, which reads the experts' results in 8 bits

8 bits: blocks of 32 columns of a row share a power of two, s = 2^(E - 127)
with E in a byte; a value is q s with a whole q of -127 .. 127.  With the
block's largest magnitude m 2^e, 1/2 <= m < 1, s is 2^(e - 7), or twice that
where the magnitude would round to 128.  Within a block, byte 4 (c % 8) + c / 8
holds column c.

`own` false: elementary torch operations in 32 bits, rounded once at the end.
`own` true: the calls of expert_routing_ffn_gb300.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
#: no call's workspace is larger (moe_train_workspace_size gives the exact size)
WORKSPACE_BYTES = 16 << 20
EPS = 1e-6
BLOCK = 32


def case_of(op, T, d, grad=False, N=8, k=1, I=64, type="bf16", zipf=0.0, drop=0.0, offset=0.0, scale=1.0, post=True, gate="none", next=True, y32=False, **more):
    return dict(op=op, grad=grad, T=T, d=d, N=N, k=k, I=I, type=type, zipf=zipf, drop=drop, offset=offset, scale=scale, post=post, gate=gate, next=next, y32=y32, **more)


def listed():
    return [
        # one token of a DeepSeek-V2-Lite-shaped layer: a call's latency
        case_of("norm", 1, 2048, name="norm-1tok-dsv2lite"),
        # the norm before a Granite-shaped layer, backwards, a long training batch, the residual's gradient added
        case_of("norm", 16384, 1536, grad=True, name="norm-grad-16384-granite"),
        # decode: 8 tokens behind a Mixtral-shaped layer, whose output is float32, and on to the next layer's norm
        case_of("block", 8, 4096, scale=0.22, y32=True, name="block-8-mixtral"),
        # a training batch behind a Qwen2-57B-shaped layer, backwards: a gate for each token
        case_of("block", 8192, 3584, grad=True, gate="token", name="block-grad-8192-qwen2"),
        # float32 rows of odd size, a gate for each value, weights that start from one
        case_of("block", 777, 1001, grad=True, gate="full", type="f32", offset=1.0, scale=0.5, name="block-grad-777-f32"),
        # 24 tokens of the tiny float32 layer: a call's latency
        case_of("keep", 24, 256, N=8, k=2, type="f32", name="keep-24-tiny-f32"),
        # a training batch of a Qwen2-57B-shaped layer, skewed load
        case_of("keep", 4096, 3584, N=64, k=8, zipf=1.1, name="keep-4096-qwen2"),
        # the tiny float32 layer's up products
        case_of("experts", 16, 256, N=8, k=2, I=512, type="f32", name="up-16-tiny-f32"),
        # the largest: up products of a Qwen2-57B-shaped layer's training batch, skewed load
        case_of("experts", 4096, 3584, N=64, k=8, I=2560, zipf=1.1, name="up-4096-qwen2"),
        # the down product's gradient in a DeepSeek-V2-Lite-shaped layer
        case_of("experts", 4096, 2048, grad=True, N=64, k=6, I=1408, name="down-grad-4096-dsv2lite"),
        # the combine's gradient of a batch of odd size, Granite shape, slots that no expert took
        case_of("combine", 1001, 1536, grad=True, N=40, k=8, drop=0.05, name="combine-grad-1001-granite"),
        # and of a training batch, Qwen2-57B shape
        case_of("combine", 4096, 3584, grad=True, N=64, k=8, zipf=1.1, name="combine-grad-4096-qwen2"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi, steps):
    """A size of the range, spread over its logarithm: a multiple of one of `steps`."""
    q = rng.choice(steps)
    return max(q, _log(rng, lo, hi) // q * q)


def draw(rng):
    op = rng.choice(("norm", "block", "block", "keep", "experts", "experts", "combine"))
    kind = rng.choice(("bf16", "bf16", "f32"))
    grad = op == "combine" or op != "keep" and rng.random() < 0.5
    if op in ("norm", "block"):
        while True:
            T, d = _log(rng, 1, 16384), _size(rng, 64, 8192, (1, 8, 64, 256))
            if T * d * (2 if kind == "bf16" else 4) <= 8192 * 3584 * 2:
                break
        c = dict(type=kind, offset=rng.choice((0.0, 1.0)))
        if op == "norm":
            return case_of(op, T, d, grad, **c)
        post = rng.random() < 0.7
        return case_of(op, T, d, grad, scale=rng.choice((1.0, 0.22, 0.5)), post=post, gate=rng.choice(("none", "token", "channel", "full")),
                       next=rng.random() < 0.7, y32=rng.random() < 0.3, **c)
    k, N = rng.choice((1, 2, 4, 6, 8)), rng.choice((8, 16, 40, 60, 64, 128))
    c = dict(zipf=rng.choice((0.0, 0.0, 1.1)), drop=rng.choice((0.0, 0.0, 0.1)))
    while True:
        if op != "experts":
            T, d = _log(rng, 1, 8192), _size(rng, 64, 4096, (1, 8, 64, 256))
            if T * k * d * (2 if kind == "bf16" else 4) <= 4096 * 8 * 3584 * 2:
                return case_of(op, T, d, grad, N, k, type=kind, **c)
        elif kind == "f32":
            return case_of(op, _log(rng, 1, 512), _size(rng, 64, 1024, (1, 8, 256)), grad, min(N, 16), k, _size(rng, 64, 1024, (1, 8, 64)), type="f32", **c)
        else:
            T, d, I = _log(rng, 1, 4096), _size(rng, 256, 4096, (8, 64, 256)), _size(rng, 64, 8192, (8, 64, 128))
            new = case_of(op, T, d, grad, N, k, I, **c)
            if work(new)["flops"] <= work(listed()[8])["flops"] and N * d * I <= 64 * 2560 * 3584:
                return new


# ---------------------------------------------------------------- inputs


def _by_expert(idx, N):
    """Slots sorted by expert, stable; those that no expert takes come last, with a row of zeros each."""
    key = torch.where(idx.reshape(-1) < 0, N, idx.reshape(-1)).long()
    order = torch.sort(key, stable=True).indices
    counts = torch.zeros(N + 1, dtype=torch.long, device=idx.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.cumsum(counts, 0) - counts
    pos = torch.empty_like(key)
    pos[order] = torch.arange(key.numel(), device=idx.device)
    inv = torch.where(key < N, pos, -2 - pos)
    perm = torch.where(key[order] < N, order, -1)
    return offsets.int(), perm.int(), inv.int().reshape(idx.shape)


def _to_8_bits(x):
    """x [rows, cols] -> q int8 [rows, blocks, 32] in column order and E uint8 [rows, blocks]."""
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    b = torch.zeros(rows, blocks * BLOCK, device=x.device)
    b[:, :cols] = x
    b = b.reshape(rows, blocks, BLOCK)
    big = b.abs().amax(2)
    m, e = torch.frexp(big)
    e = e.int() - 7 + (m * 128 >= 127.5)
    E = torch.where(big > 0, e + 127, 0).clamp(0, 254)
    q = torch.round(torch.ldexp(b, 127 - E[:, :, None]))
    return q.to(torch.int8), E.to(torch.uint8)


def _from_8_bits(q, E, cols):
    """The values that q and E stand for, in 32 bits (each of them exact)."""
    v = torch.ldexp(q.float(), E.int()[:, :, None] - 127)
    return v.reshape(q.shape[0], -1)[:, :cols]


def _as_kept(q):
    """Column order <-> the order of the bytes in a block."""
    return q.reshape(*q.shape[:2], 4, 8).transpose(2, 3).reshape(q.shape[0], -1).contiguous()


def _as_columns(q, E):
    return q.reshape(E.shape[0], E.shape[1], 8, 4).transpose(2, 3).reshape(E.shape[0], E.shape[1], BLOCK)


def prepare(case, seed):
    c = dict(case)
    T, d, N, k, I, op, grad = c["T"], c["d"], c["N"], c["k"], c["I"], c["op"], c["grad"]
    kind, rows, f32 = TYPES[c["type"]], T * k, torch.float32
    gen = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape, sd=1.0, mean=0.0, to=kind):
        return torch.empty(shape, dtype=to, device="cuda").normal_(mean, sd, generator=gen)

    def empty(*shape, to=kind):
        return torch.empty(shape, dtype=to, device="cuda")

    # what a program keeps between calls: the workspace and the outputs' buffers
    s = {"case": c, "ws": torch.zeros(WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")}
    if op in ("norm", "block"):

        def rstd(x):
            return torch.rsqrt(x.double().square().mean(1) + EPS).float()

        # a residual stream: a few channels are far larger than the rest
        loud = torch.where(torch.rand(d, generator=gen, device="cuda") < 0.003, 30.0, 1.0)
        stream = (normal(T, d, to=f32) * loud).to(kind)
        weight = normal(d, sd=0.1, mean=1.0 - c["offset"])
        if op == "norm":
            s.update(x=stream, w=weight, n=empty(T, d), rstd=empty(T, to=f32))
            if grad:
                s.update(rstd=rstd(stream), dn=normal(T, d, sd=0.1), add=normal(T, d, sd=0.1), dx=empty(T, d), dw=empty(d, to=f32))
            return s
        ykind = f32 if c["y32"] else kind
        s.update(y=normal(T, d, sd=0.5, to=ykind), gate=None, w_post=weight if c["post"] else None, w_next=normal(d, sd=0.1, mean=1.0 - c["offset"]) if c["next"] else None)
        if c["gate"] == "token":
            s["gate"] = torch.rand(T, generator=gen, device="cuda")
        elif c["gate"] != "none":
            s["gate"] = normal(d, sd=0.1, mean=0.5) if c["gate"] == "channel" else normal(T, d, sd=0.1, mean=0.5)
        if not grad:
            s.update(residual=stream, out=empty(T, d), next=empty(T, d) if c["next"] else None, rstd_post=empty(T, to=f32) if c["post"] else None,
                     rstd_next=empty(T, to=f32) if c["next"] else None)
            return s
        s.update(dout=normal(T, d, sd=0.1), dnext=normal(T, d, sd=0.1) if c["next"] else None, out=stream, rstd_post=rstd(s["y"]) if c["post"] else None,
                 rstd_next=rstd(stream) if c["next"] else None, dresidual=empty(T, d), dy=empty(T, d, to=ykind), dgate=None,
                 dw_post=empty(d, to=f32) if c["post"] else None, dw_next=empty(d, to=f32) if c["next"] else None)
        if c["gate"] != "none":
            s["dgate"] = empty(T, d) if c["gate"] == "full" else empty(d if c["gate"] == "channel" else T, to=f32)
        return s

    # the router's choice: softmax over N logits, skewed by a per-expert bias where the case says so
    logits = normal(T, N, to=f32)
    if c["zipf"]:
        logits = logits - c["zipf"] * torch.log(torch.argsort(torch.rand(N, generator=gen, device="cuda")).float() + 1.0)
    gate, idx = torch.topk(torch.softmax(logits, 1), k, dim=1)
    idx = idx.int()
    if c["drop"]:
        idx = torch.where(torch.rand(T, k, generator=gen, device="cuda") < c["drop"], -1, idx)
    s["offsets"], s["perm"], s["inv"] = _by_expert(idx, N)
    s["ends"] = s["offsets"].tolist()
    kept = s["ends"][-1]

    def expert_rows(t):
        t[kept:] = 0
        return t

    def room(n, cols):
        blocks = -(-cols // BLOCK)
        return empty(n, blocks * BLOCK, to=torch.int8), empty(n, blocks, to=torch.uint8)

    def in_8_bits(name, t):
        q, E = _to_8_bits(t.float())
        s[name], s[name + "_scale"] = _as_kept(q), E

    pre = 0.02 * math.sqrt(d)  # a pre-activation's deviation: unit inputs on weights of deviation 0.02
    if op == "keep":
        s["x_q"], s["x_scale"] = room(T, d)
        s.update(x=normal(T, d), x_perm=empty(rows, d))
    elif op == "combine":
        in_8_bits("y", expert_rows(normal(rows, d)))
        s.update(gate=gate.contiguous(), dout=normal(T, d), dy=empty(rows, d), dgate=empty(T, k, to=f32))
    elif not grad:
        s["g_q"], s["g_scale"] = room(rows, I)
        s["u_q"], s["u_scale"] = room(rows, I)
        s.update(x_perm=expert_rows(normal(rows, d)), wg=normal(N, I, d, sd=0.02), wu=normal(N, I, d, sd=0.02), h=empty(rows, I),
                 g=empty(rows, I, to=torch.bfloat16), u=empty(rows, I, to=torch.bfloat16))  # bf16 holds a value of 8 bits exactly
    else:
        in_8_bits("g", expert_rows(normal(rows, I, sd=pre)))
        in_8_bits("u", expert_rows(normal(rows, I, sd=pre)))
        s.update(dy=expert_rows(normal(rows, d)), wd=normal(N, I, d, sd=0.02), h=empty(rows, I), dg=empty(rows, I), du=empty(rows, I), dwd=empty(N, I, d))
    return s


# ---------------------------------------------------------------- one pass


def run(state):
    return (_own if own else _plain)(state)


def _there(**outputs):
    return {n: t for n, t in outputs.items() if t is not None}


def _own(s):
    import expert_routing_ffn_gb300 as moe

    c = s["case"]
    op, grad = c["op"], c["grad"]
    dims = moe.make_dims(c["T"], c["d"], c["N"], c["k"], c["I"], wtype=c["type"])
    if op == "norm":
        if not grad:
            moe.moe_norm_rows(dims, s["x"], s["w"], EPS, c["offset"], s["n"], s["rstd"])
            return {"n": s["n"], "rstd": s["rstd"]}
        moe.moe_norm_rows_grad(dims, s["dn"], s["x"], s["rstd"], s["w"], c["offset"], s["add"], s["dx"], s["dw"], False, s["ws"])
        return {"dx": s["dx"], "dw": s["dw"]}
    if op == "block":
        gate = {"none": moe.MOE_GATE_NONE, "token": moe.MOE_GATE_TOKEN, "channel": moe.MOE_GATE_CHANNEL, "full": moe.MOE_GATE_FULL}[c["gate"]]
        block = moe.make_block(eps=EPS, weight_offset=c["offset"], residual_scale=c["scale"], post_norm=c["post"], gate=gate)
        if not grad:
            moe.moe_block_out(dims, block, s["y"], s["residual"], s["gate"], s["w_post"], s["w_next"], s["out"], s["next"], s["rstd_post"], s["rstd_next"])
            return _there(out=s["out"], next=s["next"], rstd_post=s["rstd_post"], rstd_next=s["rstd_next"])
        moe.moe_block_out_grad(dims, block, s["dout"], s["dnext"], s["y"], s["out"], s["gate"], s["w_post"], s["w_next"], s["rstd_post"], s["rstd_next"],
                               s["dresidual"], s["dy"], s["dgate"], s["dw_post"], s["dw_next"], False, s["ws"])
        return _there(dresidual=s["dresidual"], dy=s["dy"], dgate=s["dgate"], dw_post=s["dw_post"], dw_next=s["dw_next"])
    if op == "keep":
        moe.moe_pack_rows(s["x"], s["x_q"], s["x_scale"])
        moe.moe_unpack_rows(s["x_q"], s["x_scale"], s["perm"], c["k"], s["x_perm"])
        return {"x_perm": s["x_perm"]}
    if op == "combine":
        moe.moe_combine_rows_grad_packed(dims, s["dout"], s["y"], s["y_scale"], s["gate"], s["inv"], s["dy"], s["dgate"])
        return {"dy": s["dy"], "dgate": s["dgate"]}
    if not grad:
        moe.moe_experts_up_packed(dims, s["x_perm"], s["offsets"], s["wg"], s["wu"], s["g_q"], s["g_scale"], s["u_q"], s["u_scale"], s["h"], s["ws"])
        # the kept values, so that they can be compared: a backward pass reads the 8 bits
        moe.moe_unpack_rows(s["g_q"], s["g_scale"], None, 1, s["g"])
        moe.moe_unpack_rows(s["u_q"], s["u_scale"], None, 1, s["u"])
        return {"h": s["h"], "g": s["g"], "u": s["u"]}
    moe.moe_experts_down_grad_packed(dims, s["dy"], s["g"], s["g_scale"], s["u"], s["u_scale"], s["offsets"], s["wd"], s["h"], s["dg"], s["du"], s["dwd"], False, s["ws"])
    return {"h": s["h"], "dg": s["dg"], "du": s["du"], "dwd": s["dwd"]}


def _experts(ends):
    """The experts that have rows, and their rows."""
    return ((e, slice(a, b)) for e, (a, b) in enumerate(zip(ends, ends[1:])) if b > a)


def _kept(s, name, cols):
    return _from_8_bits(_as_columns(s[name], s[name + "_scale"]), s[name + "_scale"], cols)


def _plain(s):
    c = s["case"]
    op, grad, d, I, k, kind = c["op"], c["grad"], c["d"], c["I"], c["k"], TYPES[c["type"]]
    if op == "norm":
        x, w = s["x"].float(), c["offset"] + s["w"].float()
        if not grad:
            rstd = 1.0 / torch.sqrt(x.square().mean(1) + EPS)
            return {"n": (x * rstd[:, None] * w).to(kind), "rstd": rstd}
        dx, dw = _norm_grad(s["dn"].float(), x, s["rstd"], w)
        return {"dx": (s["add"].float() + dx).to(kind), "dw": dw}
    if op == "block":
        return _plain_block_grad(s) if grad else _plain_block(s)
    if op == "keep":
        x = _from_8_bits(*_to_8_bits(s["x"].float()), d)
        return {"x_perm": torch.where((s["perm"] >= 0)[:, None], x[torch.clamp(s["perm"], min=0).long() // k], 0.0).to(kind)}
    if op == "combine":
        here, live = s["inv"] >= 0, s["perm"] >= 0
        dout, y = s["dout"].float(), _kept(s, "y", d)
        dgate = (torch.where(here[:, :, None], y[torch.clamp(s["inv"], min=0).long()], 0.0) * dout[:, None, :]).sum(2)
        slot = torch.clamp(s["perm"], min=0).long()
        return {"dy": torch.where(live[:, None], s["gate"].reshape(-1)[slot][:, None] * dout[slot // k], 0.0).to(kind), "dgate": dgate}
    if not grad:
        g, u = torch.zeros(s["h"].shape, device="cuda"), torch.zeros(s["h"].shape, device="cuda")
        for e, r in _experts(s["ends"]):  # one product per expert: its rows on its weights
            x = s["x_perm"][r].float()
            g[r], u[r] = x @ s["wg"][e].float().T, x @ s["wu"][e].float().T
        return {"h": (g * torch.sigmoid(g) * u).to(kind), "g": _from_8_bits(*_to_8_bits(g), I).bfloat16(), "u": _from_8_bits(*_to_8_bits(u), I).bfloat16()}
    g, u = _kept(s, "g", I), _kept(s, "u", I)
    sg = torch.sigmoid(g)
    h = g * sg * u
    dh, dwd = torch.zeros_like(g), torch.zeros_like(s["dwd"])
    for e, r in _experts(s["ends"]):
        dy = s["dy"][r].float()
        dh[r], dwd[e] = dy @ s["wd"][e].float().T, h[r].T @ dy
    return {"h": h.to(kind), "dg": (dh * u * sg * (1 + g * (1 - sg))).to(kind), "du": (dh * g * sg).to(kind), "dwd": dwd}


def _norm_grad(dn, x, rstd, w):
    n = x * rstd[:, None]
    g = dn * w
    return rstd[:, None] * (g - n * (g * n).mean(1, keepdim=True)), (dn * n).sum(0)


def _gate(s):
    g = s["gate"]
    return 1.0 if g is None else g.float()[:, None] if s["case"]["gate"] == "token" else g.float()


def _plain_block(s):
    c = s["case"]
    kind = TYPES[c["type"]]
    got, p = {}, s["y"].float()
    if c["post"]:
        got["rstd_post"] = 1.0 / torch.sqrt(p.square().mean(1) + EPS)
        p = p * got["rstd_post"][:, None] * (c["offset"] + s["w_post"].float())
    out = s["residual"].float() + c["scale"] * (_gate(s) * p)
    got["out"] = out.to(kind)
    if c["next"]:
        got["rstd_next"] = 1.0 / torch.sqrt(out.square().mean(1) + EPS)
        got["next"] = (out * got["rstd_next"][:, None] * (c["offset"] + s["w_next"].float())).to(kind)
    return got


def _plain_block_grad(s):
    c = s["case"]
    kind = TYPES[c["type"]]
    got, D, y = {}, s["dout"].float(), s["y"].float()
    if c["next"]:
        more, got["dw_next"] = _norm_grad(s["dnext"].float(), s["out"].float(), s["rstd_next"], c["offset"] + s["w_next"].float())
        D = D + more
    got["dresidual"] = D.to(kind)
    w = c["offset"] + s["w_post"].float() if c["post"] else 1.0
    p = y * s["rstd_post"][:, None] * w if c["post"] else y
    dq = c["scale"] * D
    if c["gate"] == "full":
        got["dgate"] = (dq * p).to(kind)
    elif c["gate"] != "none":
        got["dgate"] = (dq * p).sum(1 if c["gate"] == "token" else 0)
    dp = dq * _gate(s)
    if c["post"]:
        dp, got["dw_post"] = _norm_grad(dp, y, s["rstd_post"], w)
    got["dy"] = dp.to(s["y"].dtype)
    return got


# ---------------------------------------------------------------- the definition, in 64 bits


def _nearest_8_bits(x):
    """x rounded to 8 bits by blocks, on the host: the least power of two s for which no |x| / s rounds above 127."""
    rows, cols = x.shape
    b = np.zeros((rows, -(-cols // BLOCK) * BLOCK))
    b[:, :cols] = x
    b = b.reshape(rows, -1, BLOCK)
    big = np.abs(b).max(2)
    e = np.where(big > 0, np.ceil(np.log2(np.maximum(big, 2.0**-126))) - 8, -127)
    for _ in range(3):
        e = np.where((big > 0) & (np.rint(big * 2.0**-e) > 127), e + 1, e)
    s = 2.0 ** np.maximum(e, -127)[:, :, None]
    return (np.rint(b / s) * s).reshape(rows, -1)[:, :cols]


def exact(case, seed):
    op, grad = case["op"], case["grad"]
    s = prepare(case, seed)
    T, d, N, k, I, rows, o = case["T"], case["d"], case["N"], case["k"], case["I"], case["T"] * case["k"], case["offset"]
    f64 = dict(dtype=torch.float64, device="cuda")
    if op in ("norm", "block"):

        def leaf(name):
            t = s.get(name)
            return None if t is None else t.double().requires_grad_(grad)

        def normed(x, w):
            r = (torch.einsum("td,td->t", x, x) / d + EPS) ** -0.5
            return torch.einsum("td,t,d->td", x, r, o + w), r

        if op == "norm":
            x, w = leaf("x"), leaf("w")
            n, r = normed(x, w)
            if not grad:
                return {"n": n, "rstd": r}
            dx, dw = torch.autograd.grad(n, (x, w), s["dn"].double())
            return {"dx": s["add"].double() + dx, "dw": dw}
        y, gate, w_post, w_next = leaf("y"), leaf("gate"), leaf("w_post"), leaf("w_next")

        def branch():
            p, r = normed(y, w_post) if case["post"] else (y, None)
            if gate is not None:
                p = torch.einsum({"token": "td,t->td", "channel": "td,d->td", "full": "td,td->td"}[case["gate"]], p, gate)
            return case["scale"] * p, r

        if not grad:
            q, r = branch()
            out = s["residual"].double() + q
            n, rn = normed(out, w_next) if case["next"] else (None, None)
            return _there(out=out, next=n, rstd_post=r, rstd_next=rn)
        D, got = s["dout"].double(), {}
        if case["next"]:
            out = leaf("out")
            more, got["dw_next"] = torch.autograd.grad(normed(out, w_next)[0], (out, w_next), s["dnext"].double())
            D = D + more
        named = [(n, t) for n, t in (("dy", y), ("dgate", gate), ("dw_post", w_post)) if t is not None]
        got.update(zip([n for n, _ in named], torch.autograd.grad(branch()[0], [t for _, t in named], D)))
        return {"dresidual": D, **got}
    perm = s["perm"].long()
    live = perm >= 0
    slot = perm[live]
    if op == "keep":
        x_perm = torch.zeros(rows, d, **f64)
        x_perm[live] = torch.from_numpy(_nearest_8_bits(s["x"].double().cpu().numpy())).cuda()[slot // k]
        return {"x_perm": x_perm}

    def kept(name, cols):
        """A value at a time: the byte of column c is 4 (c % 8) + c / 8 of its block."""
        at = torch.arange(cols, device="cuda")
        byte = at // BLOCK * BLOCK + 4 * (at % 8) + at % BLOCK // 8
        return s[name][:, byte].double() * torch.exp2(s[name + "_scale"].double() - 127)[:, at // BLOCK]

    if op == "combine":
        dy, dgate = torch.zeros(rows, d, **f64), torch.zeros(rows, **f64)
        dout = s["dout"].double()[slot // k]
        dgate[slot] = torch.einsum("rd,rd->r", dout, kept("y", d)[live])
        dy[live] = dout * s["gate"].reshape(-1)[slot].double()[:, None]
        return {"dy": dy, "dgate": dgate.reshape(T, k)}
    expert = torch.repeat_interleave(torch.arange(N, device="cuda"), s["offsets"][1:].long() - s["offsets"][:-1].long())
    if not grad:
        # g and u in 8 bits have no value that 64 bits would settle: near the middle of two steps the sum's last bit decides
        got = {"h": torch.zeros(rows, I, **f64), "g": None, "u": None}
    else:
        g, u = kept("g", I), kept("u", I)
        sig = 1 / (1 + torch.exp(-g))
        h = g * sig * u
        got = {"h": h, "dg": torch.zeros_like(g), "du": torch.zeros_like(g), "dwd": torch.zeros(N, I, d, **f64)}
    for e in torch.unique(expert).tolist():
        at = torch.nonzero(expert == e)[:, 0]
        if not grad:
            x = s["x_perm"][at].double()
            a, b = torch.einsum("rd,id->ri", x, s["wg"][e].double()), torch.einsum("rd,id->ri", x, s["wu"][e].double())
            got["h"][at] = a / (1 + torch.exp(-a)) * b
        else:
            dy = s["dy"][at].double()
            dh = torch.einsum("rd,id->ri", dy, s["wd"][e].double())
            got["dg"][at], got["du"][at] = dh * u[at] * (sig[at] + g[at] * sig[at] * (1 - sig[at])), dh * g[at] * sig[at]
            got["dwd"][e] = torch.einsum("ri,rd->id", h[at], dy)
    return got


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    T, d, N, k, I, op, grad = (case[x] for x in ("T", "d", "N", "k", "I", "op", "grad"))
    size = 2 if case["type"] == "bf16" else 4
    row = T * d * size
    if op == "norm":
        return {"bytes": 4 * row + 4 * T + (size + 4) * d, "flops": 8 * T * d} if grad else {"bytes": 2 * row + 4 * T + size * d, "flops": 4 * T * d}
    if op == "block":
        y = T * d * (4 if case["y32"] else size)
        gate = {"none": 0, "token": 4 * T, "channel": size * d, "full": row}[case["gate"]]
        norms = case["post"] + case["next"]
        if not grad:
            return {"bytes": 2 * row + y + gate + case["next"] * row + norms * (4 * T + size * d), "flops": (3 + 4 * norms) * T * d}
        return {"bytes": 2 * row + 2 * y + 2 * gate + 2 * case["next"] * row + norms * (4 * T + (size + 4) * d), "flops": (3 + 8 * norms) * T * d}

    def kept(n, cols):
        return n * (-(-cols // BLOCK)) * (BLOCK + 1)

    slots = T * k * (1 - case["drop"])
    if op == "keep":
        return {"bytes": row + 2 * kept(T, d) + size * T * k * d + 4 * T * k, "flops": 3 * T * d + T * k * d}
    if op == "combine":
        return {"bytes": row + kept(slots, d) + size * T * k * d + 12 * T * k, "flops": 4 * slots * d}
    # experts that get a row, of T tokens that each take k of N alike; a skewed load leaves some of them out
    hit = N * (1 - (1 - k / N) ** T) if k < N else N
    if case["zipf"]:
        hit = min(hit, max(1.0, 0.75 * N))
    w, moved = size * hit * I * d, slots * size
    if not grad:
        return {"bytes": 2 * w + moved * d + moved * I + 4 * kept(slots, I) + 2 * moved * I, "flops": 4 * slots * I * d}
    return {"bytes": w + size * N * I * d + moved * d + 2 * kept(slots, I) + 3 * moved * I, "flops": 4 * slots * I * d}
