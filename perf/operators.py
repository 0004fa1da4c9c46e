"""The operators of the MoE layer's training step, as measured cases.

Five operators, each with its gradient: token rows sorted by expert
(moe_dispatch_rows), expert rows brought back to their tokens with the gates
applied (moe_combine_rows), the router's gradient from the gates
(moe_gate_grad), and the two grouped products of the experts' SwiGLU FFN
(moe_experts_up, moe_experts_down).

A case names one pass by "op":
  dispatch, dispatch_grad   x [T, d] -> rows grouped by expert, and back
  combine, combine_grad     rows [T k, d] -> sum over a token's slots of gate * row
  gate_grad                 dgate [T, k] -> dlogits [T, N], and the load-balance loss
  up, up_grad               g = x Wg^T, u = x Wu^T, h = SiLU(g) u per expert
  down, down_grad           y = h Wd per expert; its gradient goes through SwiGLU to dg, du
Layouts: weights are [N, I, d] (row i = intermediate channel i), rows are
row-major, expert indices int32 with -1 for a slot that no expert takes.

`own` false: elementary torch operations in 32 bits, rounded once at the end.
`own` true: the calls of expert_routing_ffn_gb300.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ROW_OPS = ("dispatch", "dispatch_grad", "combine", "combine_grad")
FFN_OPS = ("up", "up_grad", "down", "down_grad")
#: no call's workspace is larger (moe_train_workspace_size gives the exact size)
WORKSPACE_BYTES = 16 << 20


def case_of(op, T, d, N, k, I=64, type="bf16", zipf=0.0, drop=0.0, capacity=0, renorm=False, balance=0.0, **more):
    return dict(op=op, T=T, d=d, N=N, k=k, I=I, type=type, zipf=zipf, drop=drop, capacity=capacity, renorm=renorm, balance=balance, **more)


def listed():
    return [
        # one token of a DeepSeek-V2-Lite-shaped layer: a call's latency
        case_of("dispatch", 1, 2048, 64, 6, name="dispatch-1tok-dsv2lite"),
        # a training batch of a Qwen2-57B-shaped layer, skewed load
        case_of("dispatch", 4096, 3584, 64, 8, zipf=1.1, name="dispatch-4096-qwen2"),
        # fp32 rows of odd size with slots that no expert takes and a full expert's overflow dropped
        case_of("dispatch_grad", 777, 1000, 40, 8, type="f32", zipf=1.1, drop=0.1, capacity=200, name="dispatch-grad-777-f32"),
        # decode-size batch of a Mixtral-shaped layer
        case_of("combine", 8, 4096, 8, 2, name="combine-8-mixtral"),
        # the training batch on its way back, gates' gradient included
        case_of("combine_grad", 4096, 3584, 64, 8, zipf=1.1, name="combine-grad-4096-qwen2"),
        # router gradient of a decode-size batch, gates as the router's probabilities
        case_of("gate_grad", 32, 256, 64, 6, name="gate-grad-32-dsv2lite"),
        # router gradient of a long batch of a Granite-shaped layer: renormalised gates and the load-balance loss
        case_of("gate_grad", 16384, 256, 40, 8, zipf=1.1, renorm=True, balance=0.01, name="gate-grad-16384-granite"),
        # the tiny fp32 layer, 16 tokens
        case_of("up", 16, 256, 8, 2, 512, type="f32", name="up-16-tiny-f32"),
        # the largest: gate and up products of a Qwen2-57B-shaped layer's training batch, skewed load
        case_of("up", 4096, 3584, 64, 8, 2560, zipf=1.1, name="up-4096-qwen2"),
        # gradients of a DeepSeek-V2-Lite-shaped layer's up products: dx and both weights'
        case_of("up_grad", 4096, 2048, 64, 6, 1408, name="up-grad-4096-dsv2lite"),
        # 8 tokens of a Mixtral-shaped layer: every weight read for a row or two
        case_of("down", 8, 4096, 8, 2, 14336, name="down-8-mixtral"),
        # gradients of a Granite-shaped layer's down product, a batch of odd size
        case_of("down_grad", 1001, 1536, 40, 8, 512, drop=0.05, name="down-grad-1001-granite"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi, steps):
    """A size of the range, spread over its logarithm: a multiple of one of `steps`."""
    while True:
        q = rng.choice(steps)
        v = max(q, _log(rng, lo, hi) // q * q)
        if lo <= v <= hi and v != 3072:
            return v


def draw(rng):
    op = rng.choice(ROW_OPS + ("gate_grad",) + FFN_OPS)
    k = rng.choice((1, 2, 4, 6, 8))
    N = rng.choice((8, 16, 40, 60, 64, 128))
    c = dict(zipf=rng.choice((0.0, 0.0, 1.1)), drop=rng.choice((0.0, 0.0, 0.1)))
    most = max(work(x)["flops"] for x in listed())
    while True:
        if op in ROW_OPS:
            T, d = _log(rng, 1, 8192), _size(rng, 64, 4096, (1, 8, 64, 256))
            kind = rng.choice(("bf16", "bf16", "f32"))
            c["capacity"] = rng.choice((0, 0, max(1, 5 * T * k // (4 * N))))
            if T * k * d * (2 if kind == "bf16" else 4) <= 4096 * 8 * 3584 * 2:
                return case_of(op, T, d, N, k, type=kind, **c)
        elif op == "gate_grad":
            # renormalised gates of a token with one slot are constants: no gradient to compare
            renorm = k > 1 and rng.random() < 0.5
            return case_of(op, _log(rng, 1, 16384), 256, N, k, renorm=renorm, balance=rng.choice((0.0, 0.01)), **(dict(c, drop=0.0) if renorm else c))
        elif rng.random() < 0.25:
            T, d, I = _log(rng, 1, 512), _size(rng, 64, 1024, (1, 8, 256)), _size(rng, 64, 1024, (1, 8, 64))
            return case_of(op, T, d, min(N, 16), k, I, type="f32", **c)
        else:
            T, d, I = _log(rng, 1, 4096), _size(rng, 256, 4096, (8, 64, 256)), _size(rng, 64, 8192, (8, 64, 128))
            new = case_of(op, T, d, N, k, I, **c)
            if work(new)["flops"] <= most / 2 and N * d * I <= 64 * 2560 * 3584:
                return new


# ---------------------------------------------------------------- inputs


def _by_expert(idx, N, capacity):
    """Slots sorted by expert, stable; slots of no expert and those past an expert's capacity come last."""
    slots = idx.numel()
    key = idx.reshape(-1).long()
    key = torch.where((key < 0) | (key >= N), N, key)
    order = torch.sort(key, stable=True).indices
    if capacity > 0:
        counts = torch.zeros(N + 1, dtype=torch.long, device=idx.device).scatter_add_(0, key, torch.ones_like(key))
        first = torch.cumsum(counts, 0) - counts
        rank = torch.empty_like(key)
        rank[order] = torch.arange(slots, device=idx.device) - first[key[order]]
        key = torch.where(rank < capacity, key, N)
        order = torch.sort(key, stable=True).indices
    counts = torch.zeros(N + 1, dtype=torch.long, device=idx.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.cumsum(counts, 0) - counts
    pos = torch.empty_like(key)
    pos[order] = torch.arange(slots, device=idx.device)
    inv = torch.where(key < N, pos, -2 - pos)  # a slot without an expert: its zero row, below -1
    perm = torch.where(key[order] < N, order, -1)
    return offsets.int(), perm.int(), inv.int().reshape(idx.shape)


def prepare(case, seed):
    c = dict(case)
    T, d, N, k, I, op = c["T"], c["d"], c["N"], c["k"], c["I"], c["op"]
    kind, rows = TYPES[c["type"]], T * k
    gen = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape, sd=1.0, to=kind):
        return torch.empty(shape, dtype=to, device="cuda").normal_(0.0, sd, generator=gen)

    def empty(*shape, to=kind):
        return torch.empty(shape, dtype=to, device="cuda")

    # the router's choice: softmax over N logits, skewed by a per-expert bias where the case says so
    logits = normal(T, N, to=torch.float32)
    if c["zipf"]:
        place = torch.argsort(torch.rand(N, generator=gen, device="cuda")).float()
        logits = logits - c["zipf"] * torch.log(place + 1.0)
    prob = torch.softmax(logits, 1)
    gate, idx = torch.topk(prob, k, dim=1)
    idx = idx.int()
    if c["drop"]:
        idx = torch.where(torch.rand(T, k, generator=gen, device="cuda") < c["drop"], -1, idx)
    s = {"case": c, "idx": idx.contiguous(), "gate": gate.contiguous()}
    # what a program keeps between calls: the workspace and the outputs' buffers
    s["ws"] = torch.zeros(WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
    i32 = torch.int32
    if op == "dispatch":
        s.update(x=normal(T, d), x_perm=empty(rows, d), offsets=empty(N + 1, to=i32), perm=empty(rows, to=i32), inv=empty(T, k, to=i32))
        return s
    if op == "gate_grad":
        s.update(prob=prob, dgate=normal(T, k, sd=0.1, to=torch.float32), dlogits=empty(T, N, to=torch.float32), loss=empty(1, to=torch.float32))
        return s
    s["offsets"], s["perm"], s["inv"] = _by_expert(idx, N, c["capacity"])
    s["ends"] = s["offsets"].tolist()
    kept = s["ends"][-1]

    def expert_rows(t):
        t[kept:] = 0
        return t

    pre = 0.02 * math.sqrt(d)  # a pre-activation's deviation: unit inputs on weights of deviation 0.02
    if op == "dispatch_grad":
        s.update(dx_perm=expert_rows(normal(rows, d)), add=normal(T, d), dx=empty(T, d))
    elif op == "combine":
        s.update(y=expert_rows(normal(rows, d)), add=normal(T, d), out=empty(T, d))
    elif op == "combine_grad":
        s.update(y=expert_rows(normal(rows, d)), dout=normal(T, d), dy=empty(rows, d), dgate=empty(T, k, to=torch.float32))
    elif op == "up":
        s.update(x_perm=expert_rows(normal(rows, d)), wg=normal(N, I, d, sd=0.02), wu=normal(N, I, d, sd=0.02), g=empty(rows, I), u=empty(rows, I), h=empty(rows, I))
    elif op == "up_grad":
        s.update(x_perm=expert_rows(normal(rows, d)), dg=expert_rows(normal(rows, I)), du=expert_rows(normal(rows, I)), wg=normal(N, I, d, sd=0.02), wu=normal(N, I, d, sd=0.02),
                 dx_perm=empty(rows, d), dwg=empty(N, I, d), dwu=empty(N, I, d))
    else:
        g, u = expert_rows(normal(rows, I, sd=pre)), expert_rows(normal(rows, I, sd=pre))
        h = (torch.nn.functional.silu(g.float()) * u.float()).to(kind)
        s.update(g=g, u=u, h=h, wd=normal(N, I, d, sd=0.02))
        if op == "down":
            s.update(y=empty(rows, d))
        else:
            s.update(dy=expert_rows(normal(rows, d)), dg=empty(rows, I), du=empty(rows, I), dwd=empty(N, I, d))
    return s


# ---------------------------------------------------------------- one pass


def run(state):
    return (_own if own else _plain)(state)


def _own(s):
    import expert_routing_ffn_gb300 as moe

    c = s["case"]
    op = c["op"]
    dims = moe.make_dims(c["T"], c["d"], c["N"], c["k"], c["I"], wtype=c["type"], renorm_topk=int(c["renorm"]))
    if op == "dispatch":
        moe.moe_dispatch_rows(dims, s["x"], s["idx"], c["capacity"], s["x_perm"], s["offsets"], s["perm"], s["inv"], s["ws"])
        return {"x_perm": s["x_perm"], "offsets": s["offsets"], "perm": s["perm"], "inv": s["inv"]}
    if op == "dispatch_grad":
        moe.moe_dispatch_rows_grad(dims, s["dx_perm"], s["inv"], s["add"], s["dx"])
        return {"dx": s["dx"]}
    if op == "combine":
        moe.moe_combine_rows(dims, s["y"], s["gate"], s["inv"], s["add"], s["out"])
        return {"out": s["out"]}
    if op == "combine_grad":
        moe.moe_combine_rows_grad(dims, s["dout"], s["y"], s["gate"], s["inv"], s["dy"], s["dgate"])
        return {"dy": s["dy"], "dgate": s["dgate"]}
    if op == "gate_grad":
        moe.moe_gate_grad(dims, s["prob"], s["idx"], s["dgate"], c["balance"], s["dlogits"], s["loss"], s["ws"])
        return {"dlogits": s["dlogits"], "loss": s["loss"]}
    if op == "up":
        moe.moe_experts_up(dims, s["x_perm"], s["offsets"], s["wg"], s["wu"], s["g"], s["u"], s["h"], s["ws"])
        return {"g": s["g"], "u": s["u"], "h": s["h"]}
    if op == "up_grad":
        moe.moe_experts_up_grad(dims, s["dg"], s["du"], s["x_perm"], s["offsets"], s["wg"], s["wu"], s["dx_perm"], s["dwg"], s["dwu"], False, s["ws"])
        return {"dx": s["dx_perm"], "dwg": s["dwg"], "dwu": s["dwu"]}
    if op == "down":
        moe.moe_experts_down(dims, s["h"], s["offsets"], s["wd"], s["y"], s["ws"])
        return {"y": s["y"]}
    moe.moe_experts_down_grad(dims, s["dy"], s["h"], s["g"], s["u"], s["offsets"], s["wd"], s["dg"], s["du"], s["dwd"], False, s["ws"])
    return {"dg": s["dg"], "du": s["du"], "dwd": s["dwd"]}


def _experts(ends):
    """The experts that have rows, and their rows."""
    return ((e, slice(a, b)) for e, (a, b) in enumerate(zip(ends, ends[1:])) if b > a)


def _plain(s):
    c = s["case"]
    op, N, k, kind = c["op"], c["N"], c["k"], TYPES[c["type"]]
    if op == "dispatch":
        offsets, perm, inv = _by_expert(s["idx"], N, c["capacity"])
        rows = s["x"][torch.clamp(perm, min=0).long() // k]
        return {"x_perm": torch.where((perm >= 0)[:, None], rows, 0), "offsets": offsets, "perm": perm, "inv": inv}
    if op == "gate_grad":
        return _plain_gate_grad(s)
    if op in ROW_OPS:
        here = s["inv"] >= 0
        at = torch.clamp(s["inv"], min=0).long()
        if op == "combine_grad":
            gate = torch.where(here, s["gate"], 0.0)
            dout = s["dout"].float()
            rows = torch.where(here[:, :, None], s["y"][at].float(), 0.0)
            dgate = (rows * dout[:, None, :]).sum(2)
            token = torch.clamp(s["perm"], min=0).long()
            dy = torch.where((s["perm"] >= 0)[:, None], gate.reshape(-1)[token][:, None] * dout[token // k], 0.0)
            return {"dy": dy.to(kind), "dgate": dgate}
        rows = torch.where(here[:, :, None], s["y" if op == "combine" else "dx_perm"][at].float(), 0.0)
        if op == "combine":
            rows = rows * torch.where(here, s["gate"], 0.0)[:, :, None]
        return {"out" if op == "combine" else "dx": (s["add"].float() + rows.sum(1)).to(kind)}
    if op == "up":
        g, u, h = torch.zeros_like(s["g"]), torch.zeros_like(s["u"]), torch.zeros_like(s["h"])
    elif op == "up_grad":
        dx, dwg, dwu = torch.zeros_like(s["dx_perm"]), torch.zeros_like(s["dwg"]), torch.zeros_like(s["dwu"])
    elif op == "down":
        y = torch.zeros_like(s["y"])
    else:
        dg, du, dwd = torch.zeros_like(s["dg"]), torch.zeros_like(s["du"]), torch.zeros_like(s["dwd"])
    for e, r in _experts(s["ends"]):  # one product per expert: its rows on its weights
        if op == "up":
            x = s["x_perm"][r].float()
            ge, ue = x @ s["wg"][e].float().T, x @ s["wu"][e].float().T
            g[r], u[r], h[r] = ge, ue, ge * torch.sigmoid(ge) * ue
        elif op == "up_grad":
            x, a, b = s["x_perm"][r].float(), s["dg"][r].float(), s["du"][r].float()
            dx[r] = a @ s["wg"][e].float() + b @ s["wu"][e].float()
            dwg[e], dwu[e] = a.T @ x, b.T @ x
        elif op == "down":
            y[r] = s["h"][r].float() @ s["wd"][e].float()
        else:
            dy, ge, ue = s["dy"][r].float(), s["g"][r].float(), s["u"][r].float()
            dh, sg = dy @ s["wd"][e].float().T, torch.sigmoid(ge)
            dg[r], du[r] = dh * ue * sg * (1 + ge * (1 - sg)), dh * ge * sg
            dwd[e] = s["h"][r].float().T @ dy
    return {"g": g, "u": u, "h": h} if op == "up" else {"dx": dx, "dwg": dwg, "dwu": dwu} if op == "up_grad" else {"y": y} if op == "down" else {"dg": dg, "du": du, "dwd": dwd}


def _plain_gate_grad(s):
    c = s["case"]
    T, N, k = c["T"], c["N"], c["k"]
    prob, here = s["prob"], s["idx"] >= 0
    at = torch.clamp(s["idx"], min=0).long()
    dgate = torch.where(here, s["dgate"], 0.0)
    if c["renorm"]:
        p = torch.where(here, prob.gather(1, at), 0.0)
        total = p.sum(1, keepdim=True)
        total = torch.where(total > 0, total, 1.0)
        dgate = torch.where(here, (dgate - (dgate * p / total).sum(1, keepdim=True)) / total, 0.0)
    dprob = torch.zeros_like(prob).scatter_add_(1, at, dgate)
    load = torch.zeros(N, device=prob.device).scatter_add_(0, at.reshape(-1), here.reshape(-1).float()) / (T * k)
    loss = c["balance"] * N * (load * prob.mean(0)).sum()
    dprob = dprob + c["balance"] * N / T * load
    return {"dlogits": prob * (dprob - (dprob * prob).sum(1, keepdim=True)), "loss": loss.reshape(1)}


# ---------------------------------------------------------------- the definition, in 64 bits


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    T, N, k, rows = case["T"], case["N"], case["k"], case["T"] * case["k"]
    f64 = dict(dtype=torch.float64, device="cuda")
    if op == "dispatch":  # expert by expert: its slots in order, as many as it may take
        idx = s["idx"].reshape(-1).cpu().numpy()
        mine = [np.nonzero(idx == e)[0][: case["capacity"] or None] for e in range(N)]
        slots = torch.from_numpy(np.concatenate(mine)).cuda()
        x_perm = torch.zeros(rows, case["d"], **f64)
        x_perm[: slots.numel()] = s["x"].double()[slots // k]
        return {"x_perm": x_perm, "offsets": None, "perm": None, "inv": None}
    if op == "gate_grad":
        # per token: J^T dgate with J the Jacobian of the softmax, diag(p) - p p^T
        p = s["prob"].double()
        chosen = torch.zeros(T, N + 1, **f64)
        slot = torch.where(s["idx"] < 0, N, s["idx"]).long()
        taken = chosen.clone().scatter_(1, slot, 1.0)[:, :N]
        v = chosen.scatter_add_(1, slot, s["dgate"].double())[:, :N] * taken
        if case["renorm"]:
            total = (p * taken).sum(1, keepdim=True).clamp_min(1e-300)
            v = (v / total - taken * (v * p).sum(1, keepdim=True) / total**2)
        load = taken.sum(0) / (T * k)
        v = v + case["balance"] * N / T * load
        return {"dlogits": p * v - p * torch.einsum("te,te->t", p, v)[:, None], "loss": (case["balance"] * N / T * torch.einsum("te,e->", p, load)).reshape(1)}
    perm = s["perm"].long()
    live = perm >= 0
    slot = perm[live]
    token = slot // k
    if op in ("dispatch_grad", "combine"):
        out = s["add"].double()
        r = s["dx_perm" if op == "dispatch_grad" else "y"][live].double()
        if op == "combine":
            r *= s["gate"].reshape(-1)[slot].double()[:, None]
        out.index_add_(0, token, r)
        return {"dx" if op == "dispatch_grad" else "out": out}
    if op == "combine_grad":
        dy, dgate = torch.zeros(rows, case["d"], **f64), torch.zeros(rows, **f64)
        dout = s["dout"].double()[token]
        dgate[slot] = torch.einsum("rd,rd->r", dout, s["y"][live].double())
        dy[live] = dout * s["gate"].reshape(-1)[slot].double()[:, None]
        return {"dy": dy, "dgate": dgate.reshape(T, k)}
    n = {"up": ("g", "u", "h"), "up_grad": ("dx", "dwg", "dwu"), "down": ("y",), "down_grad": ("dg", "du", "dwd")}[op]
    like = {"dx": "dx_perm"}
    got = {x: torch.zeros(s[like.get(x, x)].shape, **f64) for x in n}
    expert = torch.repeat_interleave(torch.arange(N, device="cuda"), s["offsets"][1:].long() - s["offsets"][:-1].long())
    for e in torch.unique(expert).tolist():
        at = torch.nonzero(expert == e)[:, 0]
        if op == "up":
            x = s["x_perm"][at].double()
            a, b = torch.einsum("rd,id->ri", x, s["wg"][e].double()), torch.einsum("rd,id->ri", x, s["wu"][e].double())
            got["g"][at], got["u"][at], got["h"][at] = a, b, a / (1 + torch.exp(-a)) * b
        elif op == "up_grad":
            x, a, b = s["x_perm"][at].double(), s["dg"][at].double(), s["du"][at].double()
            got["dx"][at] = torch.einsum("ri,id->rd", a, s["wg"][e].double()) + torch.einsum("ri,id->rd", b, s["wu"][e].double())
            got["dwg"][e], got["dwu"][e] = torch.einsum("ri,rd->id", a, x), torch.einsum("ri,rd->id", b, x)
        elif op == "down":
            got["y"][at] = torch.einsum("ri,id->rd", s["h"][at].double(), s["wd"][e].double())
        else:
            dy, a, b = s["dy"][at].double(), s["g"][at].double(), s["u"][at].double()
            dh, sig = torch.einsum("rd,id->ri", dy, s["wd"][e].double()), 1 / (1 + torch.exp(-a))
            got["dg"][at], got["du"][at] = dh * b * (sig + a * sig * (1 - sig)), dh * a * sig
            got["dwd"][e] = torch.einsum("ri,rd->id", s["h"][at].double(), dy)
    return got


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    T, d, N, k, I, op = (case[x] for x in ("T", "d", "N", "k", "I", "op"))
    size = 2 if case["type"] == "bf16" else 4
    slots = T * k * (1 - case["drop"])
    ints = 4 * (2 * T * k + N + 1)
    if op == "dispatch":
        return {"bytes": size * d * (T + T * k) + ints + 4 * T * k, "flops": 0}
    if op in ("dispatch_grad", "combine"):
        return {"bytes": size * d * (2 * T + slots) + 8 * T * k, "flops": 2 * slots * d}
    if op == "combine_grad":
        return {"bytes": size * d * (T + slots + T * k) + 12 * T * k, "flops": 3 * slots * d}
    if op == "gate_grad":
        return {"bytes": 8 * T * N + 8 * T * k, "flops": 4 * T * N}
    # experts that get a row, of T tokens that each take k of N alike; a skewed load leaves some of them out
    hit = N * (1 - (1 - k / N) ** T) if k < N else N
    if case["zipf"]:
        hit = min(hit, max(1.0, 0.75 * N))
    w = size * hit * I * d
    rows = slots * size
    if op == "up":
        return {"bytes": 2 * w + rows * d + 3 * rows * I, "flops": 4 * slots * I * d}
    if op == "up_grad":
        return {"bytes": 2 * w + 2 * size * N * I * d + 2 * rows * d + 2 * rows * I, "flops": 8 * slots * I * d}
    if op == "down":
        return {"bytes": w + rows * d + rows * I, "flops": 2 * slots * I * d}
    return {"bytes": w + size * N * I * d + rows * d + 5 * rows * I, "flops": 4 * slots * I * d}
