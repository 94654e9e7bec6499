"""What is measured of the block operators: routing with scores and groups, the
norms around a block, the gradient of the combine, and the linear layer with its
epilogue, each forward and backward where it has both.

A case names one call of one operator. ``run`` makes it in elementary torch
operations (``own`` false) or through the package (``own`` true), on the same
inputs and into the same kind of outputs.
"""
import math

import torch

own = False

HID = 4096          # hidden size of the repository's bf16 layers
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ----------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------
def _route(name, back, T, E, K, score, groups, kept, top, renorm, bias, masked=0):
    return {"name": name, "op": "route", "back": back, "T": T, "E": E, "K": K, "score": score,
            "groups": groups, "kept": kept, "top": top, "renorm": renorm, "bias": bias,
            "masked": masked, "scale": 2.5 if renorm else 1.0}


def _norm(name, back, T, H, dtype, block, post, gate, pre, alpha=1.0):
    return {"name": name, "op": "norm", "back": back, "T": T, "H": H, "dtype": dtype,
            "block": block, "post": post, "gate": gate, "pre": pre, "alpha": alpha}


def _combine(name, T, K, H, E, dtype):
    return {"name": name, "op": "combine", "back": True, "T": T, "K": K, "H": H, "E": E,
            "dtype": dtype}


def _linear(name, back, T, n_in, n_out, dtype, act, bias, residual):
    return {"name": name, "op": "linear", "back": back, "T": T, "in": n_in, "out": n_out,
            "dtype": dtype, "act": act, "bias": bias, "residual": residual}


def listed():
    return [
        # one token of a 256-expert layer: the latency of a decode step's routing
        _route("route_one_token", False, 1, 256, 8, "sigmoid", 8, 4, 2, True, True),
        # a prefill batch of the same layer
        _route("route_prefill", False, 16384, 256, 8, "sigmoid", 8, 4, 2, True, True),
        # training: softmax scores without renormalisation reach every logit of the row
        _route("route_softmax_back", True, 16383, 128, 8, "softmax", 1, 1, 1, False, True),
        # one token between two blocks: post-norm, residual and the next block's pre-norm
        _norm("norm_one_token", False, 1, HID, "bf16", True, True, "none", True),
        # the same over a prefill batch
        _norm("norm_prefill", False, 16384, HID, "bf16", True, True, "channel", True, 0.5),
        # its training backward: every gradient, the weights' and the gate's summed over tokens
        _norm("norm_train_back", True, 16384, HID, "bf16", True, True, "channel", True, 0.5),
        # an fp32 layer, an odd batch and width, a gate of its own for every element
        _norm("norm_odd_f32_back", True, 777, 1004, "f32", True, True, "full", True, 0.7),
        # training of the fine-grained layer: 8 copies of every token
        _combine("combine_back", 4096, 8, HID, 128, "bf16"),
        # a small fp32 layer with two copies, an odd batch
        _combine("combine_odd_f32_back", 129, 2, 256, 16, "f32"),
        # one token through a square projection with its bias, activation and residual
        _linear("linear_one_token", False, 1, HID, HID, "bf16", "gelu", True, True),
        # a prefill batch through the wide layer of a dense feed-forward
        _linear("linear_prefill", False, 4096, HID, 14336, "bf16", "gelu", True, False),
        # training: input, weight and bias gradients of that layer
        _linear("linear_train_back", True, 4096, HID, 14336, "bf16", "gelu", True, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "norm", "combine", "linear", "route", "norm", "linear"])
    back = rng.random() < 0.5
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8, 16])
        E = groups * rng.randint(4, max(4, min(512 // groups, 256)))
        E = min(E, 512 // groups * groups)
        kept = rng.randint(1, groups)
        most = kept * (E // groups)
        K = rng.randint(1, min(16, most))
        T = max(1, min(_log(rng, 1, 16384), 16384 * 256 // E))
        score = rng.choice(["softmax", "sigmoid"])
        masked = rng.randint(1, E // 2) if rng.random() < 0.25 else 0
        return _route("", back, T, E, K, score, groups, kept, rng.choice([1, 2]),
                      rng.random() < 0.5, rng.random() < 0.7, masked)
    if op == "norm":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        H = 8 * _log(rng, 16, 1024)
        T = _log(rng, 1, 16384 * HID // H if dtype == "bf16" else 8192 * HID // H)
        T = max(1, min(T, 16384))
        block = rng.random() < 0.8
        gate = rng.choice(["none", "channel", "token", "full"]) if block else "none"
        return _norm("", back, T, H, dtype, block, block and rng.random() < 0.7, gate,
                     (not block) or rng.random() < 0.7, rng.choice([1.0, 0.5, 0.22]))
    if op == "combine":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        H = 128 * _log(rng, 1, 64)
        K = rng.randint(1, 16)
        T = max(1, _log(rng, 1, max(1, 4096 * 8 * HID // (H * K))))
        T = min(T, 16384)
        return _combine("", T, K, H, rng.randint(K, 256), dtype)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    cap = HID * 14336 if dtype == "bf16" else 1 << 20
    n_in = 8 * _log(rng, 16, 1792 if dtype == "bf16" else 256)
    n_out = 8 * _log(rng, 16, max(17, min(1792, cap // n_in // 8)))
    T = _log(rng, 1, 4096 if dtype == "bf16" else 512)
    act = rng.choice(["none", "gelu", "silu"])
    return _linear("", back, T, n_in, n_out, dtype, act, rng.random() < 0.7, rng.random() < 0.5)


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------
def _normal(g, shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(int(seed))
    st = {"case": dict(case)}
    T = case["T"]
    if case["op"] == "route":
        E, K = case["E"], case["K"]
        # gate logits of a normalised input, experts unevenly popular
        skew = -math.log(10.0) / 3 * torch.log10(torch.arange(1, E + 1, device="cuda").float())
        logits = _normal(g, (T, E)) + skew[torch.randperm(E, generator=g, device="cuda")]
        if case["masked"]:   # experts taken out of service
            off = torch.randperm(E, generator=g, device="cuda")[:case["masked"]]
            logits[:, off] = -math.inf
        st["logits"] = logits
        st["bias"] = ((torch.rand(E, generator=g, device="cuda") - 0.5) * 0.2
                      * (1.0 if case["score"] == "sigmoid" else 0.05)) if case["bias"] else None
        if case["back"]:
            st["idx"], _ = _plain_route(case, logits, st["bias"])
            st["d_w"] = _normal(g, (T, K))
            st["d_logits"] = torch.empty((T, E), device="cuda")
        else:
            st["idx"] = torch.empty((T, K), dtype=torch.int32, device="cuda")
            st["w"] = torch.empty((T, K), device="cuda")
        return st
    dt = DTYPES[case["dtype"]]
    if case["op"] == "norm":
        H = case["H"]
        st["h"] = _normal(g, (T, H), 2.0, dt)      # residual stream (backward: as left by the forward)
        st["y"] = _normal(g, (T, H), 0.5, dt) if case["block"] else None
        st["w_post"] = (1 + _normal(g, (H,), 0.1)).to(dt) if case["post"] else None
        shape = {"none": None, "channel": (H,), "token": (T,), "full": (T, H)}[case["gate"]]
        st["gate"] = None if shape is None else _normal(g, shape, 0.5, dt)
        st["w_pre"] = (1 + _normal(g, (H,), 0.1)).to(dt) if case["pre"] else None
        if case["back"]:
            st["d_h_out"] = _normal(g, (T, H), 1.0, dt)
            st["d_x"] = _normal(g, (T, H), 1.0, dt) if case["pre"] else None
            st["d_h"] = torch.empty((T, H), dtype=dt, device="cuda")
            st["d_y"] = torch.empty((T, H), dtype=dt, device="cuda") if case["block"] else None
            f32 = {"device": "cuda", "dtype": torch.float32}
            st["d_w_post"] = torch.empty(H, **f32) if case["post"] else None
            st["d_w_pre"] = torch.empty(H, **f32) if case["pre"] else None
            st["d_gate"] = (None if shape is None else torch.empty(shape, dtype=dt, device="cuda")
                            if case["gate"] == "full" else torch.empty(shape, **f32))
        else:
            st["h_out"] = torch.empty((T, H), dtype=dt, device="cuda") if case["block"] else None
            st["x"] = torch.empty((T, H), dtype=dt, device="cuda") if case["pre"] else None
        return st
    if case["op"] == "combine":
        K, H, E = case["K"], case["H"], case["E"]
        # the dispatch's order: copies sorted by expert, ascending token inside an expert
        idx = torch.rand((T, E), generator=g, device="cuda").topk(K, dim=1).indices.reshape(-1)
        perm = torch.sort(idx, stable=True).indices
        inv = torch.empty_like(perm)
        inv[perm] = torch.arange(T * K, device="cuda")
        st["inv"] = inv.to(torch.int32)
        st["w"] = torch.softmax(_normal(g, (T, K)), dim=1)
        st["y_rows"] = _normal(g, (T * K, H))
        st["d_out"] = _normal(g, (T, H), 1.0, dt)
        st["d_rows"] = torch.empty((T * K, H), dtype=dt, device="cuda")
        st["d_w"] = torch.empty((T, K), device="cuda")
        return st
    n_in, n_out = case["in"], case["out"]
    st["x"] = _normal(g, (T, n_in), 1.0, dt)
    st["w"] = _normal(g, (n_out, n_in), n_in ** -0.5, dt)
    if case["back"]:
        st["d_out"] = _normal(g, (T, n_out), 1.0, dt)
        st["pre"] = _normal(g, (T, n_out), 1.0, dt) if case["act"] != "none" else None
        st["d_x"] = torch.empty((T, n_in), dtype=dt, device="cuda")
        st["d_weight"] = torch.empty((n_out, n_in), dtype=dt, device="cuda")
        st["d_bias"] = torch.empty(n_out, device="cuda") if case["bias"] else None
    else:
        st["bias"] = _normal(g, (n_out,), 0.5, dt) if case["bias"] else None
        st["residual"] = _normal(g, (T, n_out), 1.0, dt) if case["residual"] else None
        st["out"] = torch.empty((T, n_out), dtype=dt, device="cuda")
    return st


# ----------------------------------------------------------------------------
# Plain forms
# ----------------------------------------------------------------------------
def _plain_route(c, logits, bias):
    # which experts are chosen is decided on 64-bit values: scores of different
    # experts come closer to one another than 32 bits tell apart
    l = logits.double()
    if c["score"] == "sigmoid":
        s = 1 / (1 + torch.exp(-l))
    else:
        z = torch.exp(l - l.max(dim=1, keepdim=True).values)
        s = z / z.sum(dim=1, keepdim=True)
    choice = s if bias is None else s + bias.double()
    choice = torch.where(l == -math.inf, -math.inf, choice)
    T, E = l.shape
    by_group = choice.view(T, c["groups"], E // c["groups"])
    value = by_group.sort(dim=2, descending=True).values[:, :, :c["top"]].sum(dim=2)
    best = value.sort(dim=1, descending=True, stable=True).indices[:, :c["kept"]]
    kept = torch.zeros_like(value).scatter_(1, best, 1.0).repeat_interleave(E // c["groups"], dim=1)
    order = choice.sort(dim=1, descending=True, stable=True).indices
    first = kept.gather(1, order).sort(dim=1, descending=True, stable=True).indices
    idx = order.gather(1, first)[:, :c["K"]]
    w = s.gather(1, idx)
    if c["renorm"]:
        total = w.sum(dim=1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return idx.to(torch.int32), (w * c["scale"]).float()


def _plain_route_back(c, logits, idx, d_w):
    l = logits.float()
    if c["score"] == "sigmoid":
        s = 1 / (1 + torch.exp(-l))
    else:
        z = torch.exp(l - l.max(dim=1, keepdim=True).values)
        s = z / z.sum(dim=1, keepdim=True)
    at = idx.long()
    chosen = s.gather(1, at)
    d = d_w * c["scale"]
    if c["renorm"]:
        total = chosen.sum(dim=1, keepdim=True)
        share = torch.where(total > 0, chosen / total, 0.0)
        d = torch.where(total > 0, (d - (d * share).sum(dim=1, keepdim=True)) / total, 0.0)
    ds = torch.zeros_like(s).scatter_add_(1, at, d)
    if c["score"] == "sigmoid":
        return ds * s * (1 / (1 + torch.exp(l)))
    return s * (ds - (ds * s).sum(dim=1, keepdim=True))


def _rstd(v):
    return torch.rsqrt((v * v).mean(dim=1, keepdim=True) + EPS)


def _wide_gate(c, gate):
    if gate is None:
        return 1.0
    return gate.float()[:, None] if c["gate"] == "token" else gate.float()


def _plain_norm(c, st):
    h = st["h"].float()
    dt = st["h"].dtype
    outs = []
    if c["block"]:
        u = st["y"].float()
        if c["post"]:
            u = u * _rstd(u) * st["w_post"].float()
        h = h + c["alpha"] * (_wide_gate(c, st["gate"]) * u)
        outs.append(h.to(dt))
    if c["pre"]:
        outs.append((h * _rstd(h) * st["w_pre"].float()).to(dt))
    return outs


def _plain_norm_back(c, st):
    dt = st["h"].dtype
    g = st["d_h_out"].float()
    out = {}
    if c["pre"]:
        h, d = st["h"].float(), st["d_x"].float()
        r = _rstd(h)
        n = h * r
        out["d_w_pre"] = (d * n).sum(dim=0)
        d = d * st["w_pre"].float()
        g = g + r * (d - n * (d * n).mean(dim=1, keepdim=True))
    out["d_h"] = g.to(dt)
    if c["block"]:
        y = st["y"].float()
        gate = _wide_gate(c, st["gate"])
        n = y
        if c["post"]:
            r = _rstd(y)
            n = y * r
        u = n * st["w_post"].float() if c["post"] else n
        d = g * c["alpha"]
        if c["gate"] == "channel":
            out["d_gate"] = (d * u).sum(dim=0)
        elif c["gate"] == "token":
            out["d_gate"] = (d * u).sum(dim=1)
        elif c["gate"] == "full":
            out["d_gate"] = (d * u).to(dt)
        d = d * gate
        if c["post"]:
            out["d_w_post"] = (d * n).sum(dim=0)
            d = d * st["w_post"].float()
            d = r * (d - n * (d * n).mean(dim=1, keepdim=True))
        out["d_y"] = d.to(dt)
    return out


def _plain_combine_back(c, st):
    T, K, H = c["T"], c["K"], c["H"]
    d = st["d_out"].float()
    inv = st["inv"].long()
    d_w = (st["y_rows"][inv].view(T, K, H) * d[:, None, :]).sum(dim=2)
    rows = (st["w"][:, :, None] * d[:, None, :]).reshape(T * K, H).to(st["d_out"].dtype)
    d_rows = torch.empty_like(rows)
    d_rows[inv] = rows
    return {"d_rows": d_rows, "d_w": d_w}


def _act(c, z):
    if c["act"] == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if c["act"] == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _plain_linear(c, st):
    z = st["x"].float() @ st["w"].float().t()
    if c["bias"]:
        z = z + st["bias"].float()
    z = _act(c, z)
    if c["residual"]:
        z = z + st["residual"].float()
    return z.to(st["x"].dtype)


def _plain_linear_back(c, st):
    d = st["d_out"].float()
    if c["act"] != "none":
        z = st["pre"].float()
        if c["act"] == "gelu":
            d = d * (0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
                     + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi)))
        else:
            s = 1 / (1 + torch.exp(-z))
            d = d * s * (1 + z * (1 - s))
    out = {"d_x": (d @ st["w"].float()).to(st["x"].dtype),
           "d_weight": (d.t() @ st["x"].float()).to(st["x"].dtype)}
    if c["bias"]:
        out["d_bias"] = d.sum(dim=0)
    return out


# ----------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------
def _plan(M, c):
    """The descriptor and workspace that a user's program keeps for a shape."""
    if c["op"] == "route":
        return M.make_route(c["T"], c["E"], c["K"], score=c["score"], groups=c["groups"],
                            topk_groups=c["kept"], group_top=c["top"], renorm=c["renorm"],
                            scale=c["scale"]), None
    code = M.dtype_code(DTYPES[c["dtype"]])
    if c["op"] == "norm":
        d = M.make_norm(c["T"], c["H"], code, gate=c["gate"], alpha=c["alpha"], eps=EPS)
        return d, M.alloc_workspace(d) if c["back"] else None
    if c["op"] == "combine":
        return M.make_desc(c["T"], c["H"], c["E"], c["K"], 128, 0, code), None
    d = M.make_linear(c["T"], c["in"], c["out"], code, act=c["act"])
    return d, M.alloc_workspace(d)


def _own(st):
    import fine_grained_moe_router_b200 as M
    c = st["case"]
    if "plan" not in st:
        st["plan"] = _plan(M, c)
    d, ws = st["plan"]
    if c["op"] == "route":
        if c["back"]:
            M.moe_route_backward(d, st["logits"], st["idx"], st["d_w"], st["d_logits"])
            return st["d_logits"]
        M.moe_route(d, st["logits"], st["bias"], st["idx"], st["w"])
        return st["idx"], st["w"]
    if c["op"] == "norm":
        if c["back"]:
            M.moe_block_norm_backward(d, st["d_h_out"], st["d_x"], st["h"], st["y"], st["w_post"],
                                      st["gate"], st["w_pre"], st["d_h"], st["d_y"],
                                      st["d_w_post"], st["d_gate"], st["d_w_pre"], ws)
            names = ("d_w_pre", "d_h", "d_gate", "d_w_post", "d_y")
            return {k: st[k] for k in names if st[k] is not None}
        M.moe_block_norm(d, st["h"], st["y"], st["w_post"], st["gate"], st["w_pre"], st["h_out"],
                         st["x"])
        return [st[k] for k in ("h_out", "x") if st[k] is not None]
    if c["op"] == "combine":
        M.moe_combine_backward(d, st["d_out"], st["y_rows"], st["w"], st["inv"], st["d_rows"],
                               st["d_w"])
        return {"d_rows": st["d_rows"], "d_w": st["d_w"]}
    if c["back"]:
        M.moe_linear_backward(d, st["d_out"], st["x"], st["w"], st["pre"], st["d_x"],
                              st["d_weight"], st["d_bias"], ws)
        return {k: st[k] for k in ("d_x", "d_weight", "d_bias") if st[k] is not None}
    M.moe_linear(d, st["x"], st["w"], st["bias"], st["residual"], None, st["out"], ws)
    return st["out"]


def run(state):
    if own:
        return _own(state)
    c = state["case"]
    if c["op"] == "route":
        if c["back"]:
            return _plain_route_back(c, state["logits"], state["idx"], state["d_w"])
        return _plain_route(c, state["logits"], state["bias"])
    if c["op"] == "norm":
        return _plain_norm_back(c, state) if c["back"] else _plain_norm(c, state)
    if c["op"] == "combine":
        return _plain_combine_back(c, state)
    return _plain_linear_back(c, state) if c["back"] else _plain_linear(c, state)


# ----------------------------------------------------------------------------
# What a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    T = case["T"]
    if case["op"] == "route":
        E, K = case["E"], case["K"]
        if not case["back"]:
            return {"bytes": 4 * (T * E + (E if case["bias"] else 0) + 2 * T * K),
                    "flops": T * E * 4 + T * K * 4}
        # only softmax scores without renormalisation depend on the whole row
        read = E if case["score"] == "softmax" and not case["renorm"] else K
        return {"bytes": 4 * (T * read + 2 * T * K + T * E), "flops": T * (4 * read + 6 * K)}
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        H = case["H"]
        rows = T * H
        gate = {"none": 0, "channel": H, "token": T, "full": rows}[case["gate"]]
        weights = H * (case["post"] + case["pre"])
        if not case["back"]:
            moved = rows * (1 + 2 * case["block"] + case["pre"])
            return {"bytes": size * (moved + gate + weights),
                    "flops": rows * (4 * case["post"] + 3 * case["block"] + 4 * case["pre"])}
        # d_h_out and d_h; d_x and h; y and d_y
        moved = rows * (2 + 2 * case["pre"] + 2 * case["block"])
        grads = 4 * weights + (size if case["gate"] == "full" else 4) * gate
        return {"bytes": size * (moved + gate + weights) + grads,
                "flops": rows * (10 * case["post"] + 4 * case["block"] + 10 * case["pre"])}
    if case["op"] == "combine":
        K, H = case["K"], case["H"]
        return {"bytes": T * K * H * (4 + size) + T * H * size + 12 * T * K,
                "flops": 3 * T * K * H}
    n_in, n_out = case["in"], case["out"]
    if not case["back"]:
        return {"bytes": size * (T * n_in + n_in * n_out + T * n_out * (1 + case["residual"])
                                 + (n_out if case["bias"] else 0)),
                "flops": 2 * T * n_in * n_out}
    return {"bytes": size * (2 * T * n_in + 2 * n_in * n_out
                             + T * n_out * (1 + (case["act"] != "none")))
            + (4 * n_out if case["bias"] else 0),
            "flops": 4 * T * n_in * n_out}


# ----------------------------------------------------------------------------
# The definitions in 64 bits. Selections are repeated maxima; gradients come
# from differentiating the forward definition.
# ----------------------------------------------------------------------------
def _first_max(v):
    m = v.amax(dim=1, keepdim=True)
    at = torch.arange(v.shape[1], device=v.device).expand_as(v)
    return torch.where(v == m, at, v.shape[1]).amin(dim=1)


def _scores64(c, l):
    return torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, dim=1)


def _weights64(c, l, idx):
    w = _scores64(c, l).gather(1, idx)
    if c["renorm"]:
        total = w.sum(dim=1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    return w * c["scale"]


def _exact_route(c, st):
    l = st["logits"].double()
    T, E = l.shape
    if c["back"]:
        l.requires_grad_(True)
        w = _weights64(c, l, st["idx"].long())
        (w * st["d_w"].double()).sum().backward()
        return l.grad
    choice = _scores64(c, l) + (0 if st["bias"] is None else st["bias"].double())
    choice = choice.masked_fill(l == -math.inf, -math.inf)
    size = E // c["groups"]
    values = []
    for g in range(c["groups"]):
        values.append(choice[:, g * size:(g + 1) * size].topk(c["top"], dim=1).values.sum(dim=1))
    values = torch.stack(values, dim=1)
    rows = torch.arange(T, device=l.device)
    # below every choice: what is used up (-3e300), above it what is masked (-2e300)
    out = torch.ones((T, c["groups"]), dtype=torch.bool, device=l.device)
    for _ in range(c["kept"]):
        taken = ~out
        v = torch.where(taken, -math.inf, values)
        at = _first_max(torch.where(taken, -3e300, v.clamp_min(-2e300)))
        out[rows, at] = False
    left = torch.where(out.repeat_interleave(size, dim=1), -3e300, choice.clamp_min(-2e300))
    idx = []
    for _ in range(c["K"]):
        at = _first_max(left)
        left[rows, at] = -3e300
        idx.append(at)
    idx = torch.stack(idx, dim=1)
    return idx.to(torch.int32), _weights64(c, l, idx)


def _rms64(v, w):
    return v / torch.sqrt((v ** 2).mean(dim=-1, keepdim=True) + EPS) * w


def _exact_norm(c, st):
    t = {k: st[k].double() for k in ("h", "y", "w_post", "gate", "w_pre")
         if st.get(k) is not None}
    if c["back"]:
        for v in t.values():
            v.requires_grad_(True)

    def step():
        u = _rms64(t["y"], t["w_post"]) if c["post"] else t["y"]
        if c["gate"] != "none":
            u = u * (t["gate"].unsqueeze(1) if c["gate"] == "token" else t["gate"])
        return u * c["alpha"]

    if not c["back"]:
        h = t["h"] + step() if c["block"] else t["h"]
        return ([h] if c["block"] else []) + ([_rms64(h, t["w_pre"])] if c["pre"] else [])
    # the gradient at the given sum h: into it from both of its uses, then on into the block
    g = st["d_h_out"].double()
    out = {}
    if c["pre"]:
        into, out["d_w_pre"] = torch.autograd.grad(_rms64(t["h"], t["w_pre"]),
                                                   [t["h"], t["w_pre"]], st["d_x"].double())
        g = g + into
    out["d_h"] = g
    if c["block"]:
        names = ["y"] + (["w_post"] if c["post"] else []) + (["gate"] if c["gate"] != "none" else [])
        got = dict(zip(names, torch.autograd.grad(step(), [t[k] for k in names], g)))
        out["d_y"] = got["y"]
        if c["post"]:
            out["d_w_post"] = got["w_post"]
        if c["gate"] != "none":
            out["d_gate"] = got["gate"]
    return {k: out[k] for k in ("d_w_pre", "d_h", "d_gate", "d_w_post", "d_y") if k in out}


def _exact_combine(c, st):
    rows = st["y_rows"].double().requires_grad_(True)
    w = st["w"].double().requires_grad_(True)
    picked = rows.index_select(0, st["inv"].long()).view(c["T"], c["K"], c["H"])
    total = torch.einsum("tk,tkh->th", w, picked)
    d_rows, d_w = torch.autograd.grad(total, [rows, w], st["d_out"].double())
    return {"d_rows": d_rows, "d_w": d_w}


def _exact_linear(c, st):
    f = {"none": lambda z: z, "silu": lambda z: z * torch.sigmoid(z),
         "gelu": lambda z: z * torch.special.ndtr(z)}[c["act"]]
    x, w = st["x"].double(), st["w"].double()
    if not c["back"]:
        z = torch.einsum("ti,oi->to", x, w)
        if c["bias"]:
            z = z + st["bias"].double()
        z = f(z)
        return z + st["residual"].double() if c["residual"] else z
    d = st["d_out"].double()
    if c["act"] != "none":
        z = st["pre"].double().requires_grad_(True)
        d, = torch.autograd.grad(f(z), [z], d)
    out = {"d_x": torch.einsum("to,oi->ti", d, w), "d_weight": torch.einsum("to,ti->oi", d, x)}
    if c["bias"]:
        out["d_bias"] = d.sum(dim=0)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return {"route": _exact_route, "norm": _exact_norm, "combine": _exact_combine,
            "linear": _exact_linear}[case["op"]](case, st)
