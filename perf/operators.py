"""Timed cases of the operators around the experts' products of an MoE layer.

    rows        tokens sorted by expert (moe_dispatch) and back with the router's weights (moe_combine)
    rows_bwd    their gradient (moe_combine_backward, moe_dispatch_backward)
    router_bwd  the gradient of the top-k router's weights (moe_route_topk_backward)
    pre         the norm before a block with its gradient (moe_norm_pre, moe_norm_pre_backward)
    post        the norm after a block with its gate, the scaled residual and the next block's norm
                (moe_norm_post)
    post_bwd    the gradient of post (moe_norm_post_backward)
    fused       moe_combine and moe_norm_post in one launch (moe_combine_norm_post)

`own` false: elementary torch operations in 32 bits. `own` true: the package's kernels.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-5
ALPHA = 0.75


# --------------------------------------------------------------------------------------- cases

def _case(name, op, **kw):
    c = {"name": name, "op": op, "T": 1, "H": 2048, "dtype": "bf16", "pad": 0}
    if op in ("rows", "rows_bwd", "router_bwd", "fused"):
        c.update({"E": 64, "k": 8, "zipf": True, "drop": 0.0, "ydtype": "bf16"})
    if op in ("post", "post_bwd", "fused"):
        c.update({"norm_y": True, "gate": "none", "next": True})
    c.update(kw)
    return c


def listed():
    return [
        # one decoded token of the 64-expert top-8 layer: latency of the two calls
        _case("rows_decode_t1", "rows", T=1),
        # the 2048-token prefill of the same layer under skewed routing
        _case("rows_prefill_t2048", "rows", T=2048),
        # a long prompt through the wide layer (8 experts, top-2), the experts' rows kept in fp32
        _case("rows_large_t8192", "rows", T=8192, H=4096, E=8, k=2, zipf=False, ydtype="f32"),
        # a training step of the prefill-sized layer
        _case("rows_bwd_t2048", "rows_bwd", T=2048),
        # fp32 training on an odd width with a fifth of the choices dropped (expert capacity)
        _case("rows_bwd_odd_drop", "rows_bwd", T=183, H=1031, E=7, k=3, zipf=False, drop=0.2,
              dtype="f32", ydtype="f32", pad=3),
        # the router's gradient for one small micro-batch
        _case("router_bwd_t64", "router_bwd", T=64, dtype="f32"),
        # the router's gradient for a large batch over many experts
        _case("router_bwd_t16384", "router_bwd", T=16384, E=256, dtype="bf16"),
        # residual and norms between two blocks for one decoded token
        _case("post_decode_t1", "post", T=1),
        # the same for a prefill, with a per-channel gate on the block's output
        _case("post_prefill_t2048", "post", T=2048, gate="channel"),
        # sixteen decoded tokens: the experts' fp32 rows combined, normed and added in one call
        _case("fused_decode_t16", "fused", T=16, ydtype="f32"),
        # the gradient of post for a training batch of the wide model, gated per element
        _case("post_bwd_t8192", "post_bwd", T=8192, H=4096, gate="full"),
        # the first block's norm and its gradient: fp16, ragged batch, rows inside a wider buffer
        _case("pre_t511_f16", "pre", T=511, H=4096, dtype="f16", pad=64),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rows", "rows_bwd", "router_bwd", "pre", "post", "post_bwd", "fused"])
    H = rng.choice([rng.randrange(64, 1024), 128 * rng.randrange(1, 33), 8 * rng.randrange(16, 512)])
    T = _spread(rng, 1, 8192)
    kw = {"H": H, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]), "pad": rng.choice([0, 0, 8, 1])}
    wide = 2 if kw["dtype"] == "f32" else 1
    T = max(1, T // wide)
    if op in ("rows", "rows_bwd", "router_bwd", "fused"):
        E = _spread(rng, 2, 256)
        k = rng.randrange(1, min(E, 12) + 1)
        if op != "router_bwd":
            T = max(1, min(T, 11264 // wide // k))
        kw.update(E=E, k=k, zipf=rng.random() < 0.5, drop=rng.choice([0.0, 0.0, 0.1, 0.5]))
        kw["ydtype"] = rng.choice([kw["dtype"], "f32"])
        if op == "router_bwd":
            kw.update(drop=0.0)
    if op in ("post", "post_bwd", "fused"):
        kw.update(norm_y=rng.random() < 0.75, gate=rng.choice(["none", "channel", "token", "full"]),
                  next=rng.random() < 0.75)
    c = _case("", op, T=T, **kw)
    del c["name"]
    return c


# -------------------------------------------------------------------------------------- inputs

def _routing(c, g, dev):
    T, E, k = c["T"], c["E"], c["k"]
    z = torch.rand((T, E), generator=g, device=dev, dtype=torch.float64).clamp_(1e-12, 1 - 1e-12)
    z = -torch.log(-torch.log(z))
    if c["zipf"]:     # expert popularity of rank r goes with r**-1.1, ranks shuffled over the experts
        rank = torch.rand(E, generator=g, device=dev).argsort().double() + 1
        z = z - 1.1 * rank.log()
    z = z.to(torch.bfloat16).double() - torch.arange(E, device=dev) * 1e-9    # ties to the lower id
    v, i = z.topk(k, dim=1)
    idx = i.to(torch.int32)
    wts = torch.softmax(v, dim=1).float()
    if c["drop"]:
        idx[torch.rand((T, k), generator=g, device=dev) < c["drop"]] = -1
    return idx, wts


def prepare(case, seed):
    c = case
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    T, H, dt = c["T"], c["H"], DT[c["dtype"]]

    def rows(n, scale=1.0, dtype=dt, mean=0.0):
        """n rows of H values inside rows of H + pad."""
        b = torch.randn((n, H + c["pad"]), generator=g, device=dev)
        return (b * scale + mean).to(dtype)[:, :H]

    def room(n, dtype=dt):
        return torch.zeros((n, H + c["pad"]), dtype=dtype, device=dev)[:, :H]

    s = {"case": c}
    op = c["op"]
    if op in ("rows", "rows_bwd", "router_bwd", "fused"):
        s["idx"], s["wts"] = _routing(c, g, dev)
        T, k, E, P = c["T"], c["k"], c["E"], c["T"] * c["k"]
        ydt = DT[c["ydtype"]]
    if op == "rows":
        s["x"] = rows(T)
        s["yp"] = rows(P, 0.05, ydt)
        s["counts"] = torch.zeros(E, dtype=torch.int32, device=dev)
        s["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device=dev)
        s["perm"] = torch.full((P,), -1, dtype=torch.int32, device=dev)
        s["inv"] = torch.full((T, k), -1, dtype=torch.int32, device=dev)
        s["xp"] = room(P)
        s["out"] = room(T)
    elif op in ("rows_bwd", "fused"):
        # what the forward pass left: each pair's place in expert order, -1 where it was dropped
        e = torch.where(s["idx"] < 0, E, s["idx"].long()).reshape(-1)
        place = torch.empty(P, dtype=torch.int64, device=dev)
        place[e.argsort(stable=True)] = torch.arange(P, device=dev)
        s["inv"] = torch.where(e < E, place, -1).to(torch.int32).view(T, k)
        s["yp"] = rows(P, 0.05, ydt)
        if op == "rows_bwd":
            s["dout"] = rows(T, 0.02)
            s["dxp"] = rows(P, 0.02)
            s["dx"] = room(T)
            s["dyp"] = room(P, ydt)
            s["dwts"] = torch.zeros((T, k), device=dev)
    elif op == "router_bwd":
        s["dwts"] = torch.randn((T, k), generator=g, device=dev) * 0.02
        s["dlogits"] = torch.zeros((T, E), dtype=dt, device=dev)
    elif op == "pre":
        s["h"], s["w"] = rows(T), rows(1, 0.1, mean=1.0)[0]
        s["dx"], s["dres"] = rows(T, 0.02), rows(T, 0.02)
        s["x"], s["dh"], s["dw"] = room(T), room(T), torch.zeros(H, device=dev)
    if op in ("post", "post_bwd", "fused"):
        s["h"] = rows(T)
        if op != "fused":
            s["y"] = rows(T, 0.05)
        s["w"] = rows(1, 0.1, mean=1.0)[0] if c["norm_y"] else None
        s["w_next"] = rows(1, 0.1, mean=1.0)[0] if c["next"] else None
        s["gate"] = {"none": lambda: None, "channel": lambda: rows(1, 0.2, mean=0.5)[0],
                     "token": lambda: torch.rand(T, generator=g, device=dev),
                     "full": lambda: rows(T, 0.2, mean=0.5)}[c["gate"]]()
        if op != "post_bwd":
            s["h_out"] = room(T)
            s["x_next"] = room(T) if c["next"] else None
            s["y_out"] = room(T) if op == "fused" else None
        else:
            s["h_out"] = s["h"]       # the residual stream that the forward pass left
            s["dh_out"] = rows(T, 0.02)
            s["dx_next"] = rows(T, 0.02) if c["next"] else None
            s["dh"], s["dy"] = room(T), room(T)
            s["dw"] = torch.zeros(H, device=dev) if c["norm_y"] else None
            s["dw_next"] = torch.zeros(H, device=dev) if c["next"] else None
            s["dgate"] = {"none": lambda: None, "channel": lambda: torch.zeros(H, device=dev),
                          "token": lambda: torch.zeros(T, device=dev), "full": lambda: room(T)}[c["gate"]]()
    return s


# ----------------------------------------------------------------------------------- one pass

def run(s):
    if own:
        return _kernels(s)
    return _PLAIN[s["case"]["op"]](s)


def _kernels(s):
    import quantized_mixture_experts_grouped_b200 as q
    c = s["case"]
    op = c["op"]
    if op == "rows":
        q.moe_dispatch(s["x"], s["idx"], c["E"], s["counts"], s["offsets"], s["perm"], s["inv"], s["xp"])
        q.moe_combine(s["yp"], s["inv"], s["wts"], s["out"])
        return {n: s[n] for n in ("counts", "offsets", "perm", "inv", "xp", "out")}
    if op == "rows_bwd":
        q.moe_combine_backward(s["dout"], s["yp"], s["inv"], s["wts"], s["dyp"], s["dwts"])
        q.moe_dispatch_backward(s["dxp"], s["inv"], s["dx"])
        return {n: s[n] for n in ("dyp", "dwts", "dx")}
    if op == "router_bwd":
        q.moe_route_topk_backward(s["idx"], s["wts"], s["dwts"], s["dlogits"])
        return {"dlogits": s["dlogits"]}
    if op == "post":
        q.moe_norm_post(s["y"], s["h"], s["h_out"], EPS, alpha=ALPHA, norm_y=c["norm_y"], w=s["w"], gate=s["gate"],
                        w_next=s["w_next"], x_next=s["x_next"])
        return {"h_out": s["h_out"], "x_next": s["x_next"]}
    if op == "fused":
        q.moe_combine_norm_post(s["yp"], s["inv"], s["wts"], s["h"], s["h_out"], EPS, alpha=ALPHA,
                                norm_y=c["norm_y"], w=s["w"], gate=s["gate"], w_next=s["w_next"],
                                x_next=s["x_next"], y_out=s["y_out"])
        return {"h_out": s["h_out"], "x_next": s["x_next"], "y_out": s["y_out"]}
    if "ws" not in s:     # scratch for the weights' gradients, kept by the program
        s["ws"] = torch.empty(q.moe_norm_workspace_bytes(c["T"], c["H"]), dtype=torch.uint8, device="cuda")
    if op == "pre":
        q.moe_norm_pre(s["h"], s["w"], EPS, s["x"])
        q.moe_norm_pre_backward(s["dx"], s["h"], s["w"], EPS, s["dh"], dres=s["dres"], dw=s["dw"], ws=s["ws"])
        return {n: s[n] for n in ("x", "dh", "dw")}
    q.moe_norm_post_backward(s["dh_out"], s["y"], s["dh"], s["dy"], EPS, alpha=ALPHA, norm_y=c["norm_y"], w=s["w"],
                             dw=s["dw"], gate=s["gate"], dgate=s["dgate"], h_out=s["h_out"] if c["next"] else None,
                             w_next=s["w_next"], dx_next=s["dx_next"], dw_next=s["dw_next"], ws=s["ws"])
    return {n: s[n] for n in ("dh", "dy", "dw", "dgate", "dw_next")}


def _back(yp, inv, wts, T, k, H):
    """sum over j of wts[t][j] * yp[inv[t][j]] in 32 bits; dropped choices add nothing."""
    rows = yp.float()[inv.clamp(min=0).long().view(-1)].view(T, k, H)
    rows = torch.where((inv >= 0)[:, :, None], rows, 0.0)
    return (rows * wts[:, :, None]).sum(1) if wts is not None else rows.sum(1)


def _plain_rows(s):
    c = s["case"]
    T, k, E, H = c["T"], c["k"], c["E"], c["H"]
    P, dev = T * k, s["x"].device
    e = s["idx"].reshape(-1).long()
    ok = (e >= 0) & (e < E)
    upto = (e == torch.arange(E, device=dev)[:, None]).cumsum(1, dtype=torch.int32)
    counts = upto[:, -1]
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=dev)
    offsets[1:] = counts.cumsum(0, dtype=torch.int32)
    ec = e.clamp(0, E - 1)
    pos = offsets[ec] + upto.gather(0, ec[None, :])[0] - 1
    inv = torch.where(ok, pos, -1).to(torch.int32)
    to = torch.where(ok, pos, P).long()          # dropped pairs go to a spare row
    perm = torch.full((P + 1,), -1, dtype=torch.int32, device=dev)
    perm[to] = torch.where(ok, torch.arange(P, device=dev), -1).to(torch.int32)
    xp = torch.zeros((P + 1, H), dtype=s["x"].dtype, device=dev)
    xp[to] = s["x"].repeat_interleave(k, 0)
    out = _back(s["yp"], inv.view(T, k), s["wts"], T, k, H)
    return {"counts": counts, "offsets": offsets, "perm": perm[:P], "inv": inv.view(T, k), "xp": xp[:P],
            "out": out.to(s["x"].dtype)}


def _plain_rows_bwd(s):
    c = s["case"]
    T, k, H = c["T"], c["k"], c["H"]
    P = T * k
    inv, ok = s["inv"], s["inv"] >= 0
    d = s["dout"].float()
    y = s["yp"].float()[inv.clamp(min=0).long().view(-1)].view(T, k, H)
    dw = torch.where(ok, (y * d[:, None, :]).sum(2), 0.0)
    dyp = torch.zeros((P + 1, H), device=d.device)
    dyp[torch.where(ok, inv, P).long().view(-1)] = (s["wts"][:, :, None] * d[:, None, :]).view(P, H)
    dx = _back(s["dxp"], inv, None, T, k, H)
    return {"dyp": dyp[:P].to(s["yp"].dtype), "dwts": dw, "dx": dx.to(s["dx"].dtype)}


def _plain_router_bwd(s):
    c = s["case"]
    w, d = s["wts"], s["dwts"]
    z = w * (d - (w * d).sum(1, keepdim=True))
    out = torch.zeros((c["T"], c["E"]), device=w.device)
    out.scatter_(1, s["idx"].long(), z)
    return {"dlogits": out.to(s["dlogits"].dtype)}


def _rms(v):
    return torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)


def _rms_bwd(d, v, w):
    """Gradients of rms(v) * w towards v and w."""
    r = _rms(v)
    n = v * r
    dn = d if w is None else d * w.float()
    return r * (dn - n * (dn * n).mean(1, keepdim=True)), (d * n).sum(0)


def _plain_pre(s):
    h, d = s["h"].float(), s["dx"].float()
    dh, dw = _rms_bwd(d, h, s["w"])
    return {"x": (h * _rms(h) * s["w"].float()).to(s["x"].dtype),
            "dh": (dh + s["dres"].float()).to(s["dh"].dtype), "dw": dw}


def _gate(s):
    g = s["gate"]
    if g is None:
        return 1.0
    return g.float()[:, None] if s["case"]["gate"] == "token" else g.float()


def _after(s, y):
    c = s["case"]
    u = y * _rms(y) * s["w"].float() if c["norm_y"] else y
    h = ALPHA * s["h"].float() + _gate(s) * u
    x = (h * _rms(h) * s["w_next"].float()).to(s["h"].dtype) if c["next"] else None
    return {"h_out": h.to(s["h"].dtype), "x_next": x}


def _plain_post(s):
    return _after(s, s["y"].float())


def _plain_fused(s):
    c = s["case"]
    y = _back(s["yp"], s["inv"], s["wts"], c["T"], c["k"], c["H"])
    return {**_after(s, y), "y_out": y.to(s["h"].dtype)}


def _plain_post_bwd(s):
    c = s["case"]
    y, d = s["y"].float(), s["dh_out"].float()
    dw = dw_next = dgate = None
    if c["next"]:
        dn, dw_next = _rms_bwd(s["dx_next"].float(), s["h_out"].float(), s["w_next"])
        d = d + dn
    u = y * _rms(y) * s["w"].float() if c["norm_y"] else y
    du = _gate(s) * d
    if c["gate"] == "channel":
        dgate = (d * u).sum(0)
    elif c["gate"] == "token":
        dgate = (d * u).sum(1)
    elif c["gate"] == "full":
        dgate = (d * u).to(s["dh"].dtype)
    if c["norm_y"]:
        dy, dw = _rms_bwd(du, y, s["w"])
    else:
        dy = du
    return {"dh": (ALPHA * d).to(s["dh"].dtype), "dy": dy.to(s["dy"].dtype), "dw": dw, "dgate": dgate,
            "dw_next": dw_next}


_PLAIN = {"rows": _plain_rows, "rows_bwd": _plain_rows_bwd, "router_bwd": _plain_router_bwd, "pre": _plain_pre,
          "post": _plain_post, "post_bwd": _plain_post_bwd, "fused": _plain_fused}


# ------------------------------------------------------------------------------- least of work

def work(case):
    c = case
    op, T, H, z = c["op"], c["T"], c["H"], SIZE[c["dtype"]]
    row = T * H * z
    if op in ("rows", "rows_bwd", "router_bwd", "fused"):
        P, E, zy = T * c["k"], c["E"], SIZE[c["ydtype"]]
        live = int(P * (1 - c["drop"]))
        ids = 4 * P
    if op == "rows":      # idx, x -> rows, counts, offsets, perm, inv; rows, weights -> out
        return {"bytes": row + live * H * z + 3 * ids + 8 * E + live * H * zy + ids + row, "flops": 2 * live * H}
    if op == "rows_bwd":  # dout, y, weights -> dy, dweights; drows -> dx
        return {"bytes": row + 2 * live * H * zy + 3 * ids + live * H * z + row, "flops": 4 * live * H}
    if op == "router_bwd":
        return {"bytes": 3 * ids + T * E * z, "flops": 4 * P}
    if op == "pre":       # h -> x; dx, h, dres -> dh, dw (h is read again a pass later)
        return {"bytes": 6 * row + 2 * H * z + 4 * H, "flops": 14 * T * H}
    gate = {"none": 0, "channel": H * z, "token": 4 * T, "full": row}[c["gate"]]
    if op == "post":
        return {"bytes": 3 * row + gate + (row if c["next"] else 0) + 2 * H * z, "flops": 9 * T * H}
    if op == "fused":
        return {"bytes": live * H * zy + 2 * ids + 3 * row + gate + (row if c["next"] else 0) + 2 * H * z,
                "flops": (2 * c["k"] + 9) * T * H}
    return {"bytes": 4 * row + 2 * gate + (2 * row if c["next"] else 0) + 12 * H, "flops": 24 * T * H}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    c = case
    T, H = c["T"], c["H"]
    f = {n: v.double() for n, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    op = c["op"]

    def unit(v):          # v over its root mean square
        return v / torch.sqrt(v.pow(2).sum(1, keepdim=True) / H + EPS)

    def unit_grad(d, v):  # the same map's transposed Jacobian at v, applied to d
        m = v.pow(2).sum(1, keepdim=True) / H + EPS
        return d / m.sqrt() - v * ((d * v).sum(1, keepdim=True) / (H * m * m.sqrt()))

    def gate():
        if c["gate"] == "none":
            return torch.ones((), dtype=torch.float64, device=s["h"].device)
        return f["gate"].view(T, 1) if c["gate"] == "token" else f["gate"]

    def joined(rows, inv, weights):
        out = torch.zeros((T, H), dtype=torch.float64, device=rows.device)
        for j in range(c["k"]):
            t = torch.nonzero(inv[:, j] >= 0)[:, 0]
            v = rows.index_select(0, inv[t, j].long())
            out.index_add_(0, t, v if weights is None else v * weights[t, j, None])
        return out

    def after(y):
        u = unit(y) * f["w"] if c["norm_y"] else y
        h = torch.addcmul(ALPHA * f["h"], gate(), u)
        return {"h_out": h, "x_next": unit(h) * f["w_next"] if c["next"] else None}

    if op == "rows":
        E, P = c["E"], T * c["k"]
        pairs = s["idx"].reshape(-1).tolist()
        lists = [[] for _ in range(E)]
        for p, e in enumerate(pairs):
            if e >= 0:
                lists[e].append(p)
        perm = [p for ps in lists for p in ps]
        inv = [-1] * P
        for n, p in enumerate(perm):
            inv[p] = n
        counts = [len(ps) for ps in lists]
        offsets = [0]
        for n in counts:
            offsets.append(offsets[-1] + n)
        dev = s["x"].device
        ints = {"counts": counts, "offsets": offsets, "perm": perm + [-1] * (P - len(perm)), "inv": inv}
        ints = {n: torch.tensor(v, dtype=torch.int32, device=dev) for n, v in ints.items()}
        ints["inv"] = ints["inv"].view(T, c["k"])
        xp = torch.zeros((P, H), dtype=torch.float64, device=dev)
        xp[:len(perm)] = f["x"][torch.tensor(perm, dtype=torch.int64, device=dev) // c["k"]]
        return {**ints, "xp": xp, "out": joined(f["yp"], ints["inv"], f["wts"])}
    if op == "rows_bwd":
        dyp = torch.zeros_like(f["yp"])
        dwts = torch.zeros_like(f["wts"])
        for j in range(c["k"]):
            t = torch.nonzero(s["inv"][:, j] >= 0)[:, 0]
            r = s["inv"][t, j].long()
            dyp[r] = f["dout"][t] * f["wts"][t, j, None]
            dwts[t, j] = torch.linalg.vecdot(f["dout"][t], f["yp"][r])
        return {"dyp": dyp, "dwts": dwts, "dx": joined(f["dxp"], s["inv"], None)}
    if op == "router_bwd":
        out = torch.zeros((T, c["E"]), dtype=torch.float64, device=s["wts"].device)
        mean = torch.linalg.vecdot(f["wts"], f["dwts"])
        for j in range(c["k"]):
            out[torch.arange(T, device=out.device), s["idx"][:, j].long()] += f["wts"][:, j] * (f["dwts"][:, j] - mean)
        return {"dlogits": out}
    if op == "pre":
        return {"x": unit(f["h"]) * f["w"], "dh": unit_grad(f["dx"] * f["w"], f["h"]) + f["dres"],
                "dw": torch.einsum("th,th->h", f["dx"], unit(f["h"]))}
    if op == "post":
        return after(f["y"])
    if op == "fused":
        y = joined(f["yp"], s["inv"], f["wts"])
        return {**after(y), "y_out": y}
    d = f["dh_out"]
    out = {"dh": None, "dy": None, "dw": None, "dgate": None, "dw_next": None}
    if c["next"]:
        d = d + unit_grad(f["dx_next"] * f["w_next"], f["h_out"])
        out["dw_next"] = torch.einsum("th,th->h", f["dx_next"], unit(f["h_out"]))
    out["dh"] = ALPHA * d
    u = unit(f["y"]) * f["w"] if c["norm_y"] else f["y"]
    if c["gate"] != "none":
        out["dgate"] = {"channel": lambda: torch.einsum("th,th->h", d, u), "full": lambda: d * u,
                        "token": lambda: torch.linalg.vecdot(d, u)}[c["gate"]]()
    du = d * gate()
    out["dy"] = unit_grad(du * f["w"], f["y"]) if c["norm_y"] else du
    if c["norm_y"]:
        out["dw"] = torch.einsum("th,th->h", du, unit(f["y"]))
    return out
