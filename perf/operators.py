"""The operators around the indexer loss, as cases that can be run in their plain form (elementary torch operations
in 32 bits) or through the framework: the projections that make q_idx, k_idx and w out of hidden states, the rotary
positions on them, and the AdamW step on the projections' weights.

`own` chooses between the two.  A case is a dict of plain values; `prepare` makes its inputs from a seed, `run` is
one pass, `work` what a pass cannot do without, `exact` the result by the definition in 64 bits.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
BLOCK = 256          # elements that share one scale of an 8-bit state
E4M3_MAX, E4M3_TINY = 448.0, 2.0 ** -9


# ------------------------------------------------------------------------------------------------ the cases

def _linear(name, direction, rows, k, n, dtype="bf16", out="", act="none", bias=True, residual=False, alpha=1.0):
    return {"name": name, "op": "linear", "direction": direction, "rows": rows, "in": k, "out": n, "dtype": dtype,
            "out_dtype": out or dtype, "act": act, "bias": bias, "residual": residual, "alpha": alpha}


def _rope(name, rows, heads, dim, rot, offset=0, axes=1, dtype="bf16", interleaved=False, inverse=False, far=1 << 17):
    return {"name": name, "op": "rope", "rows": rows, "heads": heads, "dim": dim, "rot": rot, "offset": offset,
            "axes": axes, "dtype": dtype, "interleaved": interleaved, "inverse": inverse, "far": far}


def _adamw(name, tensors, most, param="bf16", grad="bf16", state="e4m3", master=False, layers=0):
    return {"name": name, "op": "adamw", "tensors": tensors, "most": most, "param": param, "grad": grad,
            "state": state, "master": master, "layers": layers}


def listed():
    return [
        # one new token through the indexer's query projection (64 heads of 128): a pass over the weight
        _linear("linear one token", "fwd", 1, 2048, 8192),
        # a serving batch of an odd size through the same projection
        _linear("linear batch of 37", "fwd", 37, 2048, 8192, act="none", bias=False),
        # the query projection of a whole 64k context, the largest product
        _linear("linear 64k rows", "fwd", 65536, 2048, 8192, act="none"),
        # a gated-off branch with everything in the epilogue: bias, activation, residual
        _linear("linear gelu residual", "fwd", 8192, 4096, 2048, act="gelu_tanh", residual=True),
        # training: gradients through an activation, two sequences of 4096
        _linear("linear backward silu", "bwd", 8192, 2048, 8192, act="silu"),
        # the head weights w: 64 outputs in fp32, scaled, and their gradient
        _linear("linear head weights bwd", "bwd", 16384, 2048, 64, out="f32", bias=False, alpha=0.125),
        # sizes that no tile and no 16-byte row fits, gradients in fp32
        _linear("linear odd f32 backward", "bwd", 1013, 1023, 777, dtype="f32", act="relu"),
        # indexer queries, 64 heads of 128 of which 64 values rotate, time/height/width positions
        _rope("rope indexer queries", 16384, 64, 128, 64, axes=3),
        # the main heads' rotated tail, backward (the inverse rotation), adjacent pairs
        _rope("rope main heads bwd", 8192, 64, 192, 64, offset=128, interleaved=True, inverse=True),
        # decode: one new token for each of 5 sequences, far positions
        _rope("rope decode", 5, 64, 128, 128, axes=1, far=1 << 24),
        # the projections of 24 layers, 8-bit states, fp32 master weights
        _adamw("adamw 24 layers 8-bit", 72, 8192 * 2048, master=True, layers=24),
        # many small tensors of odd sizes, fp32 throughout
        _adamw("adamw small f32", 96, 70001, param="f32", grad="f32", state="f32"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "rope", "adamw"])
    if op == "linear":
        while True:
            c = _linear("", rng.choice(["fwd", "bwd"]), _log(rng, 1, 65536), _log(rng, 16, 8192), _log(rng, 16, 8192),
                        dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]), act=rng.choice(["none", "relu", "silu", "gelu_tanh"]),
                        bias=rng.random() < 0.7, residual=rng.random() < 0.4, alpha=rng.choice([1.0, 0.25]))
            if rng.random() < 0.6:      # sizes of real layers are mostly multiples of 8
                c["in"], c["out"] = 8 * max(2, c["in"] // 8), 8 * max(2, c["out"] // 8)
            c["residual"] = c["residual"] and c["direction"] == "fwd"
            if c["dtype"] == "bf16" and rng.random() < 0.3:
                c["out_dtype"] = "f32"
            if work(c)["flops"] <= (2e11 if c["dtype"] == "f32" else 2e12):
                break
    elif op == "rope":
        while True:
            dim = rng.choice([64, 72, 128, 192, 512, 8 * rng.randint(4, 64)])
            rot = min(dim, rng.choice([64, 128, dim, 2 * rng.randint(4, 64)]))
            c = _rope("", _log(rng, 1, 65536), rng.choice([1, 4, 64, 128, rng.randint(1, 128)]), dim, rot,
                      offset=rng.choice([0, dim - rot]), axes=rng.randint(1, 4), dtype=rng.choice(["bf16", "f32"]),
                      interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5, far=_log(rng, 64, 1 << 30))
            if work(c)["bytes"] <= 1.2e9:
                break
    else:
        c = _adamw("", _log(rng, 1, 150), _log(rng, 1, 1 << 22), param=rng.choice(["bf16", "f32"]),
                   grad=rng.choice(["bf16", "f32"]), state=rng.choice(["e4m3", "f32"]), master=False)
        c["master"] = c["param"] == "bf16" and rng.random() < 0.5
    del c["name"]
    return c


def _sizes(case):
    """Element counts of an AdamW case's tensors: the projections of `layers` layers, or sizes spread over the
    logarithm from 1 to `most`."""
    if case["layers"]:
        return [case["most"], case["most"] // 64, case["most"] // 128] * case["layers"]
    n, most = case["tensors"], case["most"]
    return [max(1, int(most ** ((i + 1) / n))) for i in range(n)]


def _sections(case):
    """How many of the frequency pairs each axis takes."""
    pairs, axes = case["rot"] // 2, case["axes"]
    s = [pairs // axes] * axes
    s[0] += pairs - sum(s)
    return s


# ------------------------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    s = {"case": case}
    if case["op"] == "linear":
        m, k, n, t, to = case["rows"], case["in"], case["out"], DT[case["dtype"]], DT[case["out_dtype"]]
        s["x"] = normal(m, k, dtype=t)
        s["weight"] = normal(n, k, scale=k ** -0.5, dtype=t)
        s["bias"] = normal(n, scale=0.1) if case["bias"] else None
        if case["direction"] == "fwd":
            s["residual"] = normal(m, n, dtype=to) if case["residual"] else None
        else:
            s["dy"] = normal(m, n, scale=0.01, dtype=to)
            s["preact"] = normal(m, n, dtype=t) if case["act"] != "none" else None
    elif case["op"] == "rope":
        s["x"] = normal(case["rows"], case["heads"], case["dim"], dtype=DT[case["dtype"]])
        s["positions"] = torch.randint(0, case["far"], (case["axes"], case["rows"]), generator=g, device="cuda",
                                       dtype=torch.int32)
        pairs = case["rot"] // 2
        s["inv_freq"] = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64, device="cuda") / pairs)
        s["sections"] = _sections(case)
    else:
        sizes = _sizes(case)
        at = [0]
        for n in sizes:  # each tensor starts on a scale block of the buffers
            at.append(at[-1] + (n + BLOCK - 1) // BLOCK * BLOCK)
        total = at[-1]
        master = normal(total, scale=0.02)
        param = master.to(DT[case["param"]])
        flat = {"param": param, "grad": normal(total, scale=1e-3, dtype=DT[case["grad"]])}
        if case["master"]:
            flat["master"] = master
        m = normal(total, scale=3e-4)
        r = normal(total, scale=3e-4).abs_().add_(8e-4)
        if case["state"] == "f32":
            flat["m"], flat["v"] = m, r * r
        else:
            for key, scale, x in (("m", "m_scale", m), ("v", "v_scale", r)):
                b = x.view(-1, BLOCK)
                top = b.abs().amax(1) / E4M3_MAX
                flat[scale] = top
                flat[key] = (b / top[:, None]).to(torch.float8_e4m3fn).view(-1)
        s["flat"] = flat
        s["tensors"] = [{key: (buf[a // BLOCK:(a + n + BLOCK - 1) // BLOCK] if key.endswith("scale") else buf[a:a + n])
                         for key, buf in flat.items()} for a, n in zip(at, sizes)]
        s["hyper"] = {"lr": 1e-4, "beta1": 0.9, "beta2": 0.99, "eps": 1e-8, "weight_decay": 0.1, "step": 100}
        s["grad_scale"] = torch.full((), 0.75, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"linear": _linear_own, "rope": _rope_own, "adamw": _adamw_own}[op](state)
    return {"linear": _linear_plain, "rope": _rope_plain, "adamw": _adamw_plain}[op](state)


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    c = 2 * math.sqrt(2 / math.pi)
    s = 1 / (1 + torch.exp(-c * (z + 0.044715 * z * z * z)))
    return s + z * s * (1 - s) * c * (1 + 3 * 0.044715 * z * z)


def _linear_form(s, f):
    """The product and its gradients, computed in the type `f`."""
    c, x, w = s["case"], s["x"].to(f), s["weight"].to(f)
    if c["direction"] == "fwd":
        z = c["alpha"] * (x @ w.t())
        if s["bias"] is not None:
            z = z + s["bias"].to(f)
        y = _act(z, c["act"])
        return {"y": y + s["residual"].to(f) if s["residual"] is not None else y}
    dz = s["dy"].to(f)
    if c["act"] != "none":
        dz = dz * _act_grad(s["preact"].to(f), c["act"])
    return {"dx": c["alpha"] * (dz @ w), "dw": c["alpha"] * (dz.t() @ x), "db": dz.sum(0) if c["bias"] else None}


def _linear_plain(s):
    c, r = s["case"], _linear_form(s, torch.float32)
    if c["direction"] == "fwd":
        return {"y": r["y"].to(DT[c["out_dtype"]])}
    return {"dx": r["dx"].to(DT[c["dtype"]]), "dw": r["dw"].to(DT[c["dtype"]]), "db": r["db"]}


def _linear_own(s):
    from sparse_attention_indexer_tcgen05_gb300 import binding as B
    c = s["case"]
    p = s.get("plan")
    if p is None:  # what a program makes once for a layer
        p = s["plan"] = B.LinearParams(rows=c["rows"], in_features=c["in"], out_features=c["out"], dtype=c["dtype"],
                                       out_dtype=c["out_dtype"], activation=c["act"], alpha=c["alpha"])
        need = p.fwd_workspace_bytes if c["direction"] == "fwd" else p.bwd_workspace_bytes
        s["workspace"] = torch.empty(max(1, need), dtype=torch.uint8, device="cuda")
    if c["direction"] == "fwd":
        return {"y": B.csa_linear_fwd(p, s["x"], s["weight"], bias=s["bias"], residual=s["residual"], workspace=s["workspace"])}
    dx, dw, db = B.csa_linear_bwd(p, s["dy"], s["x"], s["weight"], preact=s["preact"], need_db=c["bias"],
                                  workspace=s["workspace"])
    return {"dx": dx, "dw": dw, "db": db}


def _rope_form(s, f):
    c, x = s["case"], s["x"]
    lo, half = c["offset"], c["rot"] // 2
    axis = torch.cat([torch.full((n,), i, device="cuda", dtype=torch.int64) for i, n in enumerate(s["sections"])])
    angle = s["positions"].t().double()[:, axis] * s["inv_freq"]          # [rows, pairs], far positions need 64 bits
    cos, sin = torch.cos(angle).to(f)[:, None], torch.sin(angle).to(f)[:, None]
    if c["inverse"]:
        sin = -sin
    out = x.to(f, copy=True)
    part = out[..., lo:lo + c["rot"]]
    a, b = (part[..., 0::2], part[..., 1::2]) if c["interleaved"] else (part[..., :half], part[..., half:])
    u, v = a * cos - b * sin, a * sin + b * cos
    a.copy_(u)
    b.copy_(v)
    return out


def _rope_plain(s):
    return {"out": _rope_form(s, torch.float32).to(s["x"].dtype)}


def _rope_own(s):
    from sparse_attention_indexer_tcgen05_gb300 import binding as B
    c = s["case"]
    p = s.get("plan")
    if p is None:
        p = s["plan"] = B.RopeParams(rows=c["rows"], heads=c["heads"], head_dim=c["dim"], dtype=c["dtype"],
                                     rot_dim=c["rot"], rot_offset=c["offset"], sections=s["sections"],
                                     interleaved=c["interleaved"], inverse=c["inverse"])
    return {"out": B.csa_rope(p, s["x"], s["positions"], s["inv_freq"])}


def _codes(x, scale):
    """8-bit codes of one tensor's values and its scales, which it writes."""
    n = x.numel()
    b = torch.nn.functional.pad(x, (0, -n % BLOCK)).view(-1, BLOCK)
    top = b.abs().amax(1) / E4M3_MAX
    scale.copy_(top)
    return (b / torch.where(top > 0, top, torch.ones_like(top))[:, None]).view(-1)[:n]


def _values(codes, scale, f):
    return codes.to(f) * scale.to(f).repeat_interleave(BLOCK)[:codes.numel()]


def _adamw_tensor(t, h, gscale, f):
    """The step of one tensor in the type `f`, in place."""
    eight = "m_scale" in t
    p = (t["master"] if "master" in t else t["param"]).to(f)
    g = t["grad"].to(f) * gscale.to(f)
    if eight:
        m, r = _values(t["m"], t["m_scale"], f), _values(t["v"], t["v_scale"], f)
        v = r * r
    else:
        m, v = t["m"].to(f), t["v"].to(f)
    m = h["beta1"] * m + (1 - h["beta1"]) * g
    v = h["beta2"] * v + (1 - h["beta2"]) * g * g
    r = torch.sqrt(v)
    bc1, bc2 = 1 - h["beta1"] ** h["step"], 1 - h["beta2"] ** h["step"]
    p = p - h["lr"] * h["weight_decay"] * p - h["lr"] * (m / bc1) / (r / math.sqrt(bc2) + h["eps"])
    t["param"].copy_(p)
    if "master" in t:
        t["master"].copy_(p)
    if eight:
        t["m"].copy_(_codes(m, t["m_scale"]))
        c = _codes(r, t["v_scale"])
        t["v"].copy_(torch.where(r > 0, torch.clamp_min(c, E4M3_TINY), c))
    else:
        t["m"].copy_(m)
        t["v"].copy_(v)


def _adamw_plain(s):
    [_adamw_tensor(t, s["hyper"], s["grad_scale"], torch.float32) for t in s["tensors"]]
    return {k: v for k, v in s["flat"].items() if k != "grad"}


def _adamw_own(s):
    from sparse_attention_indexer_tcgen05_gb300 import binding as B
    table = s.get("plan")
    if table is None:  # the optimizer's list of tensors, made once
        table = s["plan"] = B.AdamWTensors(**{k: [t[k] for t in s["tensors"]] for k in s["tensors"][0]})
    h = s["hyper"]
    B.csa_adamw(table, step=h["step"], lr=h["lr"], beta1=h["beta1"], beta2=h["beta2"], eps=h["eps"],
                weight_decay=h["weight_decay"], grad_scale=s["grad_scale"])
    return {k: v for k, v in s["flat"].items() if k != "grad"}


# ------------------------------------------------------------------------------------------------ what a pass needs

def work(case):
    if case["op"] == "linear":
        m, k, n, e, eo = case["rows"], case["in"], case["out"], SIZE[case["dtype"]], SIZE[case["out_dtype"]]
        if case["direction"] == "fwd":
            return {"bytes": e * (m * k + n * k) + eo * m * n * (2 if case["residual"] else 1) + 4 * n * case["bias"],
                    "flops": 2.0 * m * n * k}
        return {"bytes": 2 * e * (m * k + n * k) + eo * m * n + (e * m * n if case["act"] != "none" else 0) + 4 * n * case["bias"],
                "flops": 4.0 * m * n * k}
    if case["op"] == "rope":
        n = case["rows"] * case["heads"]
        return {"bytes": 2 * SIZE[case["dtype"]] * n * case["dim"] + 4 * case["axes"] * case["rows"] + 4 * case["rot"],
                "flops": 3.0 * n * case["rot"]}
    total = sum(_sizes(case))
    p, g = SIZE[case["param"]], SIZE[case["grad"]]
    moved = (p + 8 if case["master"] else 2 * p) + g
    moved += 16 if case["state"] == "f32" else 4 + 16 / BLOCK
    return {"bytes": moved * total, "flops": 15.0 * total}


# ------------------------------------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        return _linear_exact(case, s)
    if case["op"] == "rope":
        return _rope_exact(case, s)
    return _adamw_exact(s)


def _linear_exact(c, s):
    x, w = s["x"].double(), s["weight"].double()
    k0, k1 = math.sqrt(2 / math.pi), 0.044715
    if c["direction"] == "fwd":
        z = torch.einsum("mk,nk->mn", x, w).mul_(c["alpha"])
        if s["bias"] is not None:
            z += s["bias"].double()
        if c["act"] == "relu":
            z = z.clamp(min=0)
        elif c["act"] == "silu":
            z = z * torch.sigmoid(z)
        elif c["act"] == "gelu_tanh":
            z = 0.5 * z * (1 + torch.tanh(k0 * (z + k1 * z ** 3)))
        return {"y": z if s["residual"] is None else z + s["residual"].double()}
    d = s["dy"].double()
    if c["act"] != "none":
        z = s["preact"].double()
        if c["act"] == "relu":
            d = d * (z > 0)
        elif c["act"] == "silu":
            q = torch.sigmoid(z)
            d = d * (q + z * q * (1 - q))
        else:
            t = torch.tanh(k0 * (z + k1 * z ** 3))
            d = d * (0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k0 * (1 + 3 * k1 * z * z))
    return {"dx": torch.einsum("mn,nk->mk", d, w) * c["alpha"], "dw": torch.einsum("mn,mk->nk", d, x) * c["alpha"],
            "db": d.sum(0) if c["bias"] else None}


def _rope_exact(c, s):
    x = s["x"].double()
    out = x.clone()
    sign, half, lo, pair = (-1.0 if c["inverse"] else 1.0), c["rot"] // 2, c["offset"], 0
    for axis, n in enumerate(s["sections"]):
        for i in range(pair, pair + n):
            turn = sign * s["positions"][axis].double() * s["inv_freq"][i]
            e = torch.polar(torch.ones_like(turn), turn)[:, None]
            ia, ib = (lo + 2 * i, lo + 2 * i + 1) if c["interleaved"] else (lo + i, lo + half + i)
            z = torch.complex(x[:, :, ia], x[:, :, ib]) * e
            out[:, :, ia], out[:, :, ib] = z.real, z.imag
        pair += n
    return {"out": out}


def _adamw_exact(s):
    h, q = s["hyper"], float(s["grad_scale"])
    out = {k: v.double() for k, v in s["flat"].items() if k != "grad"}
    for t in s["tensors"]:
        n, eight = t["param"].numel(), "m_scale" in t
        at = t["param"].storage_offset()
        g = t["grad"].double() * q
        w = (t["master"] if "master" in t else t["param"]).double()
        m, r = t["m"].double(), t["v"].double()
        if eight:
            blocks = torch.arange(n, device="cuda") // BLOCK
            m, r = m * t["m_scale"].double()[blocks], r * t["v_scale"].double()[blocks]
        else:
            r = r.sqrt()
        m = m * h["beta1"] + g * (1 - h["beta1"])
        r = torch.sqrt(r * r * h["beta2"] + g * g * (1 - h["beta2"]))
        step = m / (1 - h["beta1"] ** h["step"]) / (r / (1 - h["beta2"] ** h["step"]) ** 0.5 + h["eps"])
        w = w * (1 - h["lr"] * h["weight_decay"]) - h["lr"] * step
        out["param"][at:at + n] = w
        if "master" in t:
            out["master"][at:at + n] = w
        if not eight:
            out["m"][at:at + n], out["v"][at:at + n] = m, r * r
            continue
        b0, nb = at // BLOCK, t["m_scale"].numel()
        for key, y in (("m", m), ("v", r)):
            top = torch.zeros(nb, dtype=torch.float64, device="cuda").scatter_reduce_(0, blocks, y.abs(), "amax") / E4M3_MAX
            out[key + "_scale"][b0:b0 + nb] = top
            code = (y / top[blocks]).nan_to_num(0.0).to(torch.float8_e4m3fn).double()
            out[key][at:at + n] = torch.where(y > 0, code.clamp(min=E4M3_TINY), code) if key == "v" else code
    return out
