"""Cases that time the operators around an MoE block: tokens sorted by expert
(dispatch) and back (combine), their gradients, the norms before and after a
block with its gate and residual scale, their gradients, and the router's
gradient.

``run`` computes the plain form (elementary torch operations in 32 bits,
rounded once at the end) or, with ``own`` set, makes the library's calls.
``exact`` gives the same outputs from the definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}

# Scratch memory that a program keeps for the calls that need some.
SCRATCH_BYTES = 128 << 20


def listed():
    return [
        # one decoded token goes to its 8 of 256 experts
        dict(name="dispatch_1", op="dispatch", T=1, H=6144, E=256, K=8, held=256, rows="bf16", x="bf16"),
        # a prompt of 2048 tokens, hot and cold experts
        dict(name="dispatch_2048", op="dispatch", T=2048, H=6144, E=256, K=8, held=256, rows="bf16", x="bf16"),
        # gradient of the dispatch on one of two expert-parallel ranks, ragged width
        dict(name="dispatch_grad_1000", op="dispatch_grad", T=1000, H=1030, E=64, K=6, held=32, rows="f32", x="f32"),
        # a decode batch of 64 on the fp32 residual stream, shared experts' output as the base
        dict(name="combine_64", op="combine", T=64, H=6144, E=256, K=8, held=256, rows="f32", x="f32", base=True),
        # the largest: a long prompt's expert rows back into its tokens
        dict(name="combine_8192", op="combine", T=8192, H=6144, E=256, K=8, held=256, rows="bf16", x="bf16",
             base=False),
        # training step: gradients of the experts' rows and of the routing weights
        dict(name="combine_grad_2048", op="combine_grad", T=2048, H=6144, E=256, K=8, held=256, rows="bf16",
             x="bf16"),
        # one decoded token between two blocks
        dict(name="norm_1", op="norm", T=1, H=6144, x="f32", y="f32", n="f32", post=True, gate=True, token=False),
        # a prompt between two blocks
        dict(name="norm_2048", op="norm", T=2048, H=6144, x="bf16", y="bf16", n="bf16", post=True, gate=True,
             token=False),
        # training step between two blocks: all gradients
        dict(name="norm_grad_2048", op="norm_grad", T=2048, H=6144, x="bf16", y="bf16", n="bf16", post=True,
             gate=True, token=False),
        # odd width, few rows, a gate for each token, fp32 residual stream
        dict(name="norm_grad_333", op="norm_grad", T=333, H=1537, x="f32", y="bf16", n="bf16", post=True, gate=False,
             token=True),
        # router gradient of a small layer
        dict(name="route_grad_64", op="route_grad", T=64, H=512, E=16, K=2, x="f32"),
        # router gradient of the full-size layer
        dict(name="route_grad_2048", op="route_grad", T=2048, H=6144, E=256, K=8, x="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["dispatch", "dispatch_grad", "combine", "combine_grad", "norm", "norm_grad", "route_grad"])
    types = ["f32", "bf16"]
    if op in ("norm", "norm_grad"):
        T = _log_int(rng, 1, 8192)
        H = _log_int(rng, 64, 8192)
        if rng.random() < 0.6:
            H = max(64, H // 64 * 64)
        post = rng.random() < 0.7
        T = min(T, (1 << (25 if op == "norm" else 24)) // H)
        x = rng.choice(types)
        # the norm of a bf16 residual stream is not wider than the stream
        return dict(op=op, T=T, H=H, x=x, y=rng.choice(types), n="bf16" if x == "bf16" else rng.choice(types),
                    post=post, gate=rng.random() < 0.5, token=rng.random() < 0.3)
    E = _log_int(rng, 4, 512)
    K = rng.randint(1, min(8, E))
    T = _log_int(rng, 1, 8192 if op != "route_grad" else 4096)
    H = _log_int(rng, 128, 6144)
    if op == "route_grad":
        return dict(op=op, T=T, H=max(128, H // 128 * 128), E=E, K=K, x=rng.choice(types))
    if rng.random() < 0.6:
        H = max(128, H // 128 * 128)
    held = E if rng.random() < 0.7 else max(1, E // 2)
    x = rng.choice(types)
    c = dict(op=op, T=T, H=H, E=E, K=K, held=held, rows="bf16" if x == "bf16" else rng.choice(types), x=x)
    if op == "combine":
        c["base"] = rng.random() < 0.5
    most = 8192 * 8 * 6144 * (1 if op == "combine_grad" else 2)  # bytes of rows: the largest listed case's
    c["T"] = max(1, min(T, most // (K * H * SIZE[c["rows"]])))
    return c


# ----------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda").mul_(scale).to(dtype)


def _routing(g, T, E, K, held):
    """Top-K of scores with Zipf-like popularity; experts that another rank holds are empty slots (-1)."""
    popularity = -1.1 * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    popularity = popularity[torch.randperm(E, generator=g, device="cuda")]
    noise = -torch.log(-torch.log(torch.rand((T, E), generator=g, device="cuda").clamp_(1e-7, 1 - 1e-7)))
    top, ids = torch.topk(noise + popularity, K, dim=1)
    weights = torch.softmax(top, dim=1)
    ids = torch.where(ids < held, ids, torch.full_like(ids, -1))
    return ids.to(torch.int32).contiguous(), weights.contiguous()


def _plan(ids, E):
    """Counts, offsets, position of each slot, slot of each position (the sort is stable)."""
    flat = ids.reshape(-1).long()
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    srt, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(srt, torch.arange(E + 1, device=ids.device))
    pos = torch.empty_like(order)
    pos[order] = torch.arange(n, device=ids.device)
    pos = torch.where(key < E, pos, torch.full_like(pos, -1))
    slot = torch.where(srt < E, order, torch.full_like(order, -1))
    i32 = torch.int32
    return (offsets[1:] - offsets[:-1]).to(i32), offsets.to(i32), pos.to(i32).reshape(ids.shape), slot.to(i32)


def prepare(case, seed):
    c = dict(case)
    g = _generator(seed)
    T, H = c["T"], c["H"]
    s = dict(c=c, scratch=torch.empty(SCRATCH_BYTES, dtype=torch.uint8, device="cuda"))
    f32 = dict(dtype=torch.float32, device="cuda")
    if c["op"] in ("norm", "norm_grad"):
        xt, yt, nt = DT[c["x"]], DT[c["y"]], DT[c["n"]]
        s.update(x=_normal(g, (T, H), xt, 3.0), y=_normal(g, (T, H), yt, 0.5),
                 pre_gain=1 + _normal(g, (H,), torch.float32, 0.2),
                 post_gain=1 + _normal(g, (H,), torch.float32, 0.2) if c["post"] else None,
                 gate=_normal(g, (H,), torch.float32, 0.5) if c["gate"] else None,
                 token_gate=torch.rand((T,), generator=g, device="cuda") if c["token"] else None,
                 x_scale=0.75, y_scale=1.25, eps=1e-6)
        if c["op"] == "norm":
            s.update(x_out=torch.empty((T, H), dtype=xt, device="cuda"),
                     norm=torch.empty((T, H), dtype=nt, device="cuda"))
        else:
            s.update(dx_out=_normal(g, (T, H), xt), dn=_normal(g, (T, H), nt),
                     dx=torch.empty((T, H), dtype=xt, device="cuda"), dy=torch.empty((T, H), dtype=yt, device="cuda"),
                     dpre=torch.empty((H,), **f32), dpost=torch.empty((H,), **f32) if c["post"] else None,
                     dgate=torch.empty((H,), **f32) if c["gate"] else None,
                     dtoken=torch.empty((T,), **f32) if c["token"] else None)
        return s
    E, K = c["E"], c["K"]
    s["ids"], s["w"] = _routing(g, T, E, K, c.get("held", E))
    s["counts"], s["offsets"], s["pos"], s["slot"] = _plan(s["ids"], E)
    xt = DT[c["x"]]
    if c["op"] == "route_grad":
        s.update(x=_normal(g, (T, H), xt), wr=_normal(g, (E, H), torch.float32, H ** -0.5),
                 dw=_normal(g, (T, K), torch.float32), dlogits=torch.empty((T, K), **f32),
                 dx=torch.empty((T, H), dtype=xt, device="cuda"), dwr=torch.empty((E, H), **f32),
                 dbias=torch.empty((E,), **f32))
        return s
    rt = DT[c["rows"]]
    if c["op"] == "dispatch":
        i32 = dict(dtype=torch.int32, device="cuda")
        s.update(x=_normal(g, (T, H), xt), rows=torch.zeros((T * K, H), dtype=rt, device="cuda"),
                 counts=torch.empty((E,), **i32), offsets=torch.empty((E + 1,), **i32),
                 pos=torch.empty((T, K), **i32), slot=torch.empty((T * K,), **i32))
    elif c["op"] == "dispatch_grad":
        s.update(rows=_normal(g, (T * K, H), rt), dx=torch.empty((T, H), dtype=xt, device="cuda"))
    elif c["op"] == "combine":
        s.update(rows=_normal(g, (T * K, H), rt), y=torch.empty((T, H), dtype=xt, device="cuda"),
                 base=_normal(g, (T, H), xt) if c["base"] else None)
    else:
        s.update(rows=_normal(g, (T * K, H), rt), dy=_normal(g, (T, H), xt),
                 drows=torch.zeros((T * K, H), dtype=rt, device="cuda"), dw=torch.empty((T, K), **f32))
    return s


# ----------------------------------------------------------- the plain form

def _gathered(rows, pos):
    """The rows of every slot in 32 bits [T][K][H]; empty slots are zero."""
    r = rows[pos.clamp(min=0).long()].float()
    return torch.where((pos >= 0).unsqueeze(-1), r, torch.zeros((), device=r.device))


def _placed(values, pos, like):
    """Rows at their positions; the others stay zero."""
    out = torch.zeros((like.shape[0] + 1, like.shape[1]), dtype=like.dtype, device=like.device)
    at = torch.where(pos >= 0, pos, torch.full_like(pos, like.shape[0])).reshape(-1).long()
    out[at] = values.reshape(-1, like.shape[1]).to(like.dtype)
    return out[:-1]


def _plain(s):
    c = s["c"]
    op = c["op"]
    if op == "dispatch":
        counts, offsets, pos, slot = _plan(s["ids"], c["E"])
        x = s["x"].float().unsqueeze(1).expand(-1, c["K"], -1)
        rows = torch.zeros((c["T"] * c["K"] + 1, c["H"]), dtype=s["rows"].dtype, device="cuda")
        at = torch.where(pos >= 0, pos, torch.full_like(pos, c["T"] * c["K"])).long()
        rows[at] = x.to(rows.dtype)
        return dict(counts=counts, offsets=offsets, pos=pos, slot=slot, rows=rows[:-1])
    if op == "dispatch_grad":
        return dict(dx=_gathered(s["rows"], s["pos"]).sum(1).to(s["dx"].dtype))
    if op == "combine":
        y = (_gathered(s["rows"], s["pos"]) * s["w"].unsqueeze(-1)).sum(1)
        if s["base"] is not None:
            y = y + s["base"].float()
        return dict(y=y.to(s["y"].dtype))
    if op == "combine_grad":
        dy = s["dy"].float().unsqueeze(1)
        dw = (_gathered(s["rows"], s["pos"]) * dy).sum(-1)
        return dict(drows=_placed(s["w"].unsqueeze(-1) * dy, s["pos"], s["drows"]), dw=dw)
    if op == "route_grad":
        ids = s["ids"].long()
        dl = s["w"] * (s["dw"] - (s["w"] * s["dw"]).sum(1, keepdim=True))
        dense = torch.zeros((c["T"], c["E"]), device="cuda").scatter_add_(1, ids, dl)
        x = s["x"].float()
        return dict(dlogits=dl, dx=(dense @ s["wr"]).to(s["x"].dtype), dwr=dense.t() @ x, dbias=dense.sum(0))
    # norms around a block
    y = s["y"].float()
    z, yh, rho = y, None, None
    if c["post"]:
        rho = torch.rsqrt(y.square().mean(1, keepdim=True) + s["eps"])
        yh = y * rho
        z = yh * s["post_gain"]
    gate = torch.full((), s["y_scale"], device="cuda")
    if s["gate"] is not None:
        gate = gate * s["gate"]
    if s["token_gate"] is not None:
        gate = gate * s["token_gate"].unsqueeze(1)
    if op == "norm":
        x_out = (s["x_scale"] * s["x"].float() + gate * z).to(s["x"].dtype)
        h = x_out.float()
        n = h * torch.rsqrt(h.square().mean(1, keepdim=True) + s["eps"]) * s["pre_gain"]
        return dict(x_out=x_out, n=n.to(s["norm"].dtype))
    h, dn = s["x"].float(), s["dn"].float()
    r = torch.rsqrt(h.square().mean(1, keepdim=True) + s["eps"])
    hh = h * r
    dnq = dn * s["pre_gain"]
    ds = s["dx_out"].float() + r * (dnq - hh * (hh * dnq).mean(1, keepdim=True))
    out = dict(dx=(s["x_scale"] * ds).to(s["x"].dtype), dpre=(hh * dn).sum(0))
    dz = gate * ds
    zds = s["y_scale"] * z * ds
    if s["gate"] is not None:
        out["dgate"] = (zds * s["token_gate"].unsqueeze(1) if s["token_gate"] is not None else zds).sum(0)
    if s["token_gate"] is not None:
        out["dtoken"] = (zds * s["gate"] if s["gate"] is not None else zds).sum(1)
    dy = dz
    if c["post"]:
        out["dpost"] = (yh * dz).sum(0)
        dzp = dz * s["post_gain"]
        dy = rho * (dzp - yh * (yh * dzp).mean(1, keepdim=True))
    out["dy"] = dy.to(s["y"].dtype)
    return out


# ------------------------------------------------------- the library's calls

def _own(s):
    import int4_expert_ffn_router_b200 as coli
    c = s["c"]
    op = c["op"]
    if op == "dispatch":
        coli.dispatch(s["ids"], s["x"], c["E"], s["counts"], s["offsets"], s["pos"], s["slot"], s["rows"],
                      s["scratch"])
        return dict(counts=s["counts"], offsets=s["offsets"], pos=s["pos"], slot=s["slot"], rows=s["rows"])
    if op == "dispatch_grad":
        coli.dispatch_backward(s["pos"], s["rows"], s["dx"])
        return dict(dx=s["dx"])
    if op == "combine":
        coli.combine(s["pos"], s["w"], s["rows"], s["y"], s["base"])
        return dict(y=s["y"])
    if op == "combine_grad":
        coli.combine_backward(s["pos"], s["w"], s["dy"], s["rows"], s["drows"], s["dw"])
        return dict(drows=s["drows"], dw=s["dw"])
    if op == "route_grad":
        coli.route_backward(s["wr"], s["x"], s["ids"], s["w"], s["dw"], s["offsets"], s["slot"], s["dlogits"],
                            s["dx"], s["dwr"], s["dbias"], s["scratch"])
        return dict(dlogits=s["dlogits"], dx=s["dx"], dwr=s["dwr"], dbias=s["dbias"])
    if "prev" not in s:  # the two blocks' parameters: a program makes them once, with its weights
        s["prev"] = coli.Block(post_norm=c["post"], post_gain=s["post_gain"], gate=s["gate"], x_scale=s["x_scale"],
                               y_scale=s["y_scale"], eps=s["eps"])
        s["next"] = coli.Block(pre_gain=s["pre_gain"], eps=s["eps"])
    if op == "norm":
        coli.block_norm(s["prev"], s["next"], s["x"], s["y"], s["x_out"], s["norm"], s["token_gate"])
        return dict(x_out=s["x_out"], n=s["norm"])
    coli.block_norm_backward(s["prev"], s["next"], s["x"], s["y"], s["dx_out"], s["dn"], s["dx"], s["dy"],
                             dpre_gain=s["dpre"], dpost_gain=s["dpost"], dgate=s["dgate"], token_gate=s["token_gate"],
                             dtoken_gate=s["dtoken"], work=s["scratch"])
    out = dict(dx=s["dx"], dy=s["dy"], dpre=s["dpre"])
    for name, key in (("dpost", "post"), ("dgate", "gate"), ("dtoken", "token")):
        if c[key]:
            out[name] = s[name]
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ the work

def work(case):
    c = case
    T, H = c["T"], c["H"]
    if c["op"] in ("norm", "norm_grad"):
        bx, by, bn = SIZE[c["x"]], SIZE[c["y"]], SIZE[c["n"]]
        gains = 4 * H * (1 + c["post"] + c["gate"]) + 4 * T * c["token"]
        if c["op"] == "norm":
            return dict(bytes=T * H * (2 * bx + by + bn) + gains, flops=T * H * 9)
        return dict(bytes=T * H * (3 * bx + 2 * by + bn) + 2 * gains, flops=T * H * 30)
    E, K = c["E"], c["K"]
    if c["op"] == "route_grad":
        return dict(bytes=2 * T * H * SIZE[c["x"]] + 8 * E * H + 4 * E + 20 * T * K, flops=4 * T * K * H)
    slots = T * K * c["held"] / E  # about the share of slots that this rank's experts take
    rows, x = slots * H * SIZE[c["rows"]], T * H * SIZE[c["x"]]
    if c["op"] == "dispatch":
        return dict(bytes=rows + x + 12 * T * K + 8 * E, flops=0)
    if c["op"] == "dispatch_grad":
        return dict(bytes=rows + x + 4 * T * K, flops=slots * H)
    if c["op"] == "combine":
        return dict(bytes=rows + x * (2 if c["base"] else 1) + 8 * T * K, flops=2 * slots * H)
    return dict(bytes=2 * rows + x + 12 * T * K, flops=3 * slots * H)


# ------------------------------------------------------- in 64 bits, by itself

def _exact_plan(ids, E):
    T, K = ids.shape
    flat = ids.reshape(-1).cpu().tolist()
    by_expert = [[] for _ in range(E)]
    for i, e in enumerate(flat):
        if 0 <= e < E:
            by_expert[e].append(i)
    counts = [len(b) for b in by_expert]
    slot = [i for b in by_expert for i in b]
    pos = [-1] * len(flat)
    for q, i in enumerate(slot):
        pos[i] = q
    offsets = [0]
    for n in counts:
        offsets.append(offsets[-1] + n)
    slot += [-1] * (len(flat) - len(slot))
    t = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    return t(counts), t(offsets), t(pos).reshape(T, K), t(slot)


def _held(pos, k):
    """Tokens whose slot k is not empty, and its positions."""
    tok = torch.nonzero(pos[:, k] >= 0).reshape(-1)
    return tok, pos[tok, k].long()


def exact(case, seed):
    s = prepare(case, seed)
    c, d = s["c"], torch.float64
    op, T, H = c["op"], c["T"], c["H"]
    zeros = lambda *shape: torch.zeros(shape, dtype=d, device="cuda")  # noqa: E731
    if op == "dispatch":
        counts, offsets, pos, slot = _exact_plan(s["ids"], c["E"])
        rows = zeros(T * c["K"], H)
        for k in range(c["K"]):
            tok, at = _held(pos, k)
            rows[at] = s["x"][tok].to(d)
        return dict(counts=counts, offsets=offsets, pos=pos, slot=slot, rows=rows)
    if op in ("dispatch_grad", "combine"):
        out = s["base"].to(d) if op == "combine" and c["base"] else zeros(T, H)
        for k in range(c["K"]):
            tok, at = _held(s["pos"], k)
            r = s["rows"][at].to(d)
            out[tok] += r if op == "dispatch_grad" else r * s["w"][tok, k].to(d).unsqueeze(1)
        return dict(dx=out) if op == "dispatch_grad" else dict(y=out)
    if op == "combine_grad":
        drows, dw = zeros(T * c["K"], H), zeros(T, c["K"])
        for k in range(c["K"]):
            tok, at = _held(s["pos"], k)
            dy = s["dy"][tok].to(d)
            drows[at] = dy * s["w"][tok, k].to(d).unsqueeze(1)
            dw[tok, k] = torch.linalg.vecdot(dy, s["rows"][at].to(d))
        return dict(drows=drows, dw=dw)
    if op == "route_grad":
        w, dw, x, wr, ids = s["w"].to(d), s["dw"].to(d), s["x"].to(d), s["wr"].to(d), s["ids"].long()
        # the weights are a softmax over the K selected logits: its Jacobian is diag(w) - w w^T
        jac = torch.diag_embed(w) - w.unsqueeze(2) * w.unsqueeze(1)
        dl = torch.einsum("tjk,tj->tk", jac, dw)
        dx, dwr, dbias = zeros(T, H), zeros(c["E"], H), zeros(c["E"])
        for k in range(c["K"]):
            dx += dl[:, k:k + 1] * wr[ids[:, k]]
            dbias.index_add_(0, ids[:, k], dl[:, k])
        sel = zeros(c["E"], T)
        for k in range(c["K"]):
            sel[ids[:, k], torch.arange(T, device="cuda")] += dl[:, k]
        torch.matmul(sel, x, out=dwr)
        return dict(dlogits=dl, dx=dx, dwr=dwr, dbias=dbias)
    x, y = s["x"].to(d), s["y"].to(d)
    one = torch.ones((), dtype=d, device="cuda")
    p = s["post_gain"].to(d) if c["post"] else one
    q = s["pre_gain"].to(d)
    g = s["gate"].to(d) if c["gate"] else one
    u = s["token_gate"].to(d).reshape(T, 1) if c["token"] else one
    a, b, eps = s["x_scale"], s["y_scale"], s["eps"]
    rho = 1 / torch.sqrt((y * y).sum(1, keepdim=True) / H + eps) if c["post"] else one
    if op == "norm":
        x_out = (a * x + b * u * g * p * y * rho).to(s["x"].dtype).to(d)
        n = x_out * q / torch.sqrt((x_out * x_out).sum(1, keepdim=True) / H + eps)
        return dict(x_out=a * x + b * u * g * p * y * rho, n=n)
    # gradients of L = <dx_out, s> + <dn, norm(s)>, with s = a x + b u g p (y rho)
    ss = (x * x).sum(1, keepdim=True) / H + eps
    dn, dxo = s["dn"].to(d), s["dx_out"].to(d)
    ds = dxo + q * dn / ss.sqrt() - x * (x * q * dn).sum(1, keepdim=True) / (H * ss * ss.sqrt())
    out = dict(dx=a * ds, dpre=(x * dn / ss.sqrt()).sum(0))
    v = b * u * g * p * ds  # gradient on y rho
    dy = v
    if c["post"]:
        dy = v * rho - y * rho ** 3 * (y * v).sum(1, keepdim=True) / H
        out["dpost"] = (b * u * g * ds * y * rho).sum(0)
    out["dy"] = dy
    if c["gate"]:
        out["dgate"] = (b * u * p * y * rho * ds).sum(0)
    if c["token"]:
        out["dtoken"] = (b * g * p * y * rho * ds).sum(1)
    return out
