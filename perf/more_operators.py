"""The operators at the ends of a training step, as cases that can be run in their plain form (elementary torch operations
in 32 bits) or through the framework: the layer norm of the indexer's keys and of hidden states, and the losses of the
vocabulary's logits, softmax cross entropy with labels and distillation from a teacher's top logits, from hidden states
and the vocabulary's weight, with their gradients.

`own` chooses between the two.  A case is a dict of plain values; `prepare` makes its inputs from a seed, `run` is
one pass, `work` what a pass cannot do without, `exact` the result by the definition in 64 bits.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------------------------------------ the cases

def _norm(name, direction, rows, cols, dtype="bf16", param="f32", stats=True):
    return {"name": name, "op": "norm", "direction": direction, "rows": rows, "cols": cols, "dtype": dtype, "param": param,
            "stats": stats, "eps": 1e-6}


def _vocab(name, direction, rows, features, vocab, dtype="bf16", labels=True, slots=0, lse=False, alpha=1.0):
    return {"name": name, "op": "vocab", "direction": direction, "rows": rows, "features": features, "vocab": vocab,
            "dtype": dtype, "labels": labels, "slots": slots, "lse": lse, "alpha": alpha}


def listed():
    return [
        # one new token's hidden state before the vocabulary's weight: latency, no statistics kept
        _norm("norm one token", "fwd", 1, 4096, stats=False),
        # the indexer's keys of a 64k context at ratio 4: 128 values each, statistics kept for training
        _norm("norm indexer keys", "fwd", 16384, 128),
        # hidden states of a 64k context, backward with both parameters' gradients
        _norm("norm backward 64k rows", "bwd", 65536, 4096),
        # the indexer's keys backward: short rows, the gradients of 128 parameters from 16384 rows
        _norm("norm indexer keys bwd", "bwd", 16384, 128),
        # odd rows that no vector fits, in fp32
        _norm("norm odd f32 backward", "bwd", 5003, 1537, dtype="f32"),
        # the loss of one token: a pass over the vocabulary's weight
        _vocab("labels one token", "fwd", 1, 2048, 32000),
        # evaluation: the loss of 2048 tokens, no gradient
        _vocab("labels evaluation", "fwd", 2048, 4096, 131072),
        # training: loss and gradients of two sequences of 4096 tokens, a fifth of them without a label
        _vocab("labels training", "bwd", 8192, 2048, 131072),
        # an odd vocabulary and odd rows in fp32
        _vocab("labels odd f32", "bwd", 517, 768, 50257, dtype="f32"),
        # how far a sparse model is from the dense one, 32 candidates a token
        _vocab("distill evaluation", "fwd", 1000, 2048, 65536, labels=False, slots=32, lse=True),
        # distilling the dense model into the sparse one: 64 candidates a token and their share of the teacher's sum
        _vocab("distill training", "bwd", 4096, 4096, 131072, labels=False, slots=64, lse=True),
        # both losses at temperature 2 over an odd vocabulary
        _vocab("labels and distill", "bwd", 3001, 1024, 50257, slots=100, alpha=0.5),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


MOST_FLOPS = {"bf16": 1.3e13, "f32": 6e11}


def draw(rng):
    if rng.random() < 0.4:
        while True:
            c = _norm("", rng.choice(["fwd", "bwd"]), _log(rng, 1, 131072), _log(rng, 1, 16384),
                      dtype=rng.choice(["bf16", "bf16", "f32"]), param=rng.choice(["bf16", "f32"]))
            if rng.random() < 0.6:      # sizes of real layers are mostly multiples of 8
                c["cols"] = 8 * max(1, c["cols"] // 8)
            c["stats"] = c["direction"] == "bwd" or rng.random() < 0.5
            if work(c)["bytes"] <= 1.6e9:
                break
    else:
        while True:
            c = _vocab("", rng.choice(["fwd", "bwd"]), _log(rng, 1, 16384), _log(rng, 32, 8192), _log(rng, 256, 262144),
                       dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]), labels=rng.random() < 0.6,
                       alpha=rng.choice([1.0, 1.0, 0.5]))
            if rng.random() < 0.8:
                c["features"] = 8 * max(4, c["features"] // 8)
            if rng.random() < 0.5:
                c["vocab"] = 64 * (c["vocab"] // 64)
            if not c["labels"] or rng.random() < 0.3:
                c["slots"] = min(c["vocab"], _log(rng, 1, 256))
                c["lse"] = rng.random() < 0.5
            if c["rows"] * c["vocab"] <= 1 << 30 and work(c)["flops"] <= MOST_FLOPS[c["dtype"]]:
                break
    del c["name"]
    return c


# ------------------------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s, m, t = {"case": case}, case["rows"], DT[case["dtype"]]
    if case["op"] == "norm":
        n, tp = case["cols"], DT[case["param"]]
        x = normal(m, n, scale=1.5) + 0.3
        x[:, n // 3] *= 20.0                      # hidden states have a few large features
        s["x"] = x.to(t)
        s["weight"] = (1 + normal(n, scale=0.1)).to(tp)
        s["bias"] = normal(n, scale=0.1, dtype=tp)
        if case["direction"] == "bwd":
            s["dy"] = normal(m, n, scale=0.01, dtype=t)
            x = s["x"].float()
            mean = x.mean(1)                      # what the forward pass kept
            rstd = 1 / torch.sqrt(((x - mean[:, None]) ** 2).mean(1) + case["eps"])
            s["stats"] = torch.stack([mean, rstd])
        return s
    k, v, slots = case["features"], case["vocab"], case["slots"]
    s["weight"] = normal(v, k, scale=2 * k ** -0.5, dtype=t)
    token = torch.randint(0, v, (m,), generator=g, device="cuda")
    # the tokens are likely ones: a trained model's logits
    s["x"] = (normal(m, k) + 2.0 * s["weight"][token].float()).to(t)
    if case["labels"]:                            # prompts carry no label
        s["labels"] = torch.where((uniform(m) < 0.2) & (m > 1), torch.full_like(token, -100), token)
    if slots:
        # distinct candidates, the likeliest first; as many of them as the teacher's nucleus holds, -1 behind them
        width = v // slots
        ids = torch.arange(slots, device="cuda") * width + torch.randint(0, width, (m, slots), generator=g, device="cuda")
        ids = torch.gather(ids, 1, torch.argsort(uniform(m, slots), dim=1))
        logits = torch.sort(normal(m, slots, scale=3.0), dim=1, descending=True).values
        held = torch.floor(1 + uniform(m, 1) * slots)
        held = torch.where((uniform(m, 1) < 0.05) & (m > 1), torch.zeros_like(held), held)   # padding rows
        s["ids"] = torch.where(torch.arange(slots, device="cuda") < held, ids, torch.full_like(ids, -1))
        s["logits"] = logits
        if case["lse"]:                           # the candidates hold 80 to 100 % of the teacher's sum
            s["lse"] = torch.logsumexp(logits, 1) - torch.log(0.8 + 0.2 * uniform(m))
    return s


# ------------------------------------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _norm_own, "vocab": _vocab_own}[op](state)
    return {"norm": _norm_plain, "vocab": _vocab_plain}[op](state)


def _norm_plain(s):
    c, x, w = s["case"], s["x"].float(), s["weight"].float()
    if c["direction"] == "fwd":
        mean = x.mean(1, keepdim=True)
        d = x - mean
        rstd = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + c["eps"])
        y = (d * rstd * w + s["bias"].float()).to(s["x"].dtype)
        return {"y": y, "mean": mean[:, 0], "rstd": rstd[:, 0]} if c["stats"] else {"y": y}
    dy, mean, rstd = s["dy"].float(), s["stats"][0][:, None], s["stats"][1][:, None]
    xhat = (x - mean) * rstd
    a = dy * w
    dx = rstd * (a - a.mean(1, keepdim=True) - xhat * (a * xhat).mean(1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xhat).sum(0).to(DT[c["param"]]),
            "dbias": dy.sum(0).to(DT[c["param"]])}


def _norm_own(s):
    from sparse_attention_indexer_tcgen05_gb300 import binding as B
    c = s["case"]
    p = s.get("plan")
    if p is None:  # what a program makes once for a layer
        p = s["plan"] = B.LayerNormParams(rows=c["rows"], cols=c["cols"], dtype=c["dtype"], param_dtype=c["param"], eps=c["eps"])
        s["workspace"] = torch.empty(max(1, p.bwd_workspace_bytes), dtype=torch.uint8, device="cuda")
    if c["direction"] == "fwd":
        if not c["stats"]:
            return {"y": B.csa_layernorm_fwd(p, s["x"], s["weight"], s["bias"])}
        stats = torch.empty(2, c["rows"], dtype=torch.float32, device="cuda")
        y = B.csa_layernorm_fwd(p, s["x"], s["weight"], s["bias"], stats=stats)
        return {"y": y, "mean": stats[0], "rstd": stats[1]}
    dx, dw, db = B.csa_layernorm_bwd(p, s["dy"], s["x"], s["weight"], s["stats"], workspace=s["workspace"])
    return {"dx": dx, "dweight": dw, "dbias": db}


def _vocab_plain(s):
    c = s["case"]
    x, w, m = s["x"].float(), s["weight"].float(), c["rows"]
    z = c["alpha"] * (x @ w.t())
    top = z.amax(1, keepdim=True)
    lse = (top + torch.log(torch.exp(z - top).sum(1, keepdim=True)))[:, 0]
    loss, row_label, row_teacher = 0.0, torch.zeros_like(lse), torch.zeros_like(lse)
    scale = torch.zeros_like(lse)                 # dz = scale softmax(z) - targets
    if c["labels"]:
        held = s["labels"] >= 0
        label = torch.where(held, s["labels"], torch.zeros_like(s["labels"]))[:, None]
        row_label = torch.where(held, lse - z.gather(1, label)[:, 0], torch.zeros_like(lse))
        count = held.sum().clamp(min=1).float()
        loss = loss + row_label.sum() / count
        on_label = held.float() / count
        scale = scale + on_label
    if c["slots"]:
        held = s["ids"] >= 0
        ids = torch.where(held, s["ids"], torch.zeros_like(s["ids"]))
        logits = torch.where(held, s["logits"], torch.full_like(s["logits"], -1e30))
        if c["lse"]:
            t = torch.exp(logits - s["lse"][:, None])
        else:
            t = torch.exp(logits - logits.amax(1, keepdim=True)) * held
            t = t / t.sum(1, keepdim=True).clamp(min=1e-30)
        log_t = torch.log(torch.where(t > 0, t, torch.ones_like(t)))
        row_teacher = (t * (log_t - z.gather(1, ids) + lse[:, None])).sum(1)
        count = held.any(1).sum().clamp(min=1).float()
        loss = loss + row_teacher.sum() / count
        t = t / count
        scale = scale + t.sum(1)
    if c["direction"] == "fwd":
        return {"loss": loss, "row_label": row_label, "row_teacher": row_teacher}
    dz = torch.exp(z - lse[:, None]) * scale[:, None]
    if c["labels"]:
        dz.scatter_add_(1, label, -on_label[:, None])
    if c["slots"]:
        dz.scatter_add_(1, ids, -t)
    dt = s["x"].dtype
    return {"loss": loss, "dx": (c["alpha"] * (dz @ w)).to(dt), "dw": (c["alpha"] * (dz.t() @ x)).to(dt)}


def _vocab_own(s):
    from sparse_attention_indexer_tcgen05_gb300 import binding as B
    c = s["case"]
    p = s.get("plan")
    if p is None:
        p = s["plan"] = B.VocabLossParams(rows=c["rows"], features=c["features"], vocab=c["vocab"], dtype=c["dtype"],
                                          slots=c["slots"], alpha=c["alpha"], labels_64=True, ids_64=True)
        need = p.fwd_workspace_bytes if c["direction"] == "fwd" else p.bwd_workspace_bytes
        s["workspace"] = torch.empty(max(1, need), dtype=torch.uint8, device="cuda")
    targets = dict(labels=s.get("labels"), teacher_ids=s.get("ids"), teacher_logits=s.get("logits"), teacher_lse=s.get("lse"))
    if c["direction"] == "fwd":
        rows = torch.empty(2, c["rows"], dtype=torch.float32, device="cuda")
        loss = B.csa_vocab_loss_fwd(p, s["x"], s["weight"], **targets, row_loss=rows, workspace=s["workspace"])
        return {"loss": loss, "row_label": rows[0], "row_teacher": rows[1]}
    loss, dx, dw = B.csa_vocab_loss_bwd(p, s["x"], s["weight"], **targets, workspace=s["workspace"])
    return {"loss": loss, "dx": dx, "dw": dw}


# ------------------------------------------------------------------------------------------------ what a pass needs

def work(case):
    m, e = case["rows"], SIZE[case["dtype"]]
    if case["op"] == "norm":
        n = case["cols"]
        passes, params = (2, 2) if case["direction"] == "fwd" else (3, 3)
        return {"bytes": passes * e * m * n + params * SIZE[case["param"]] * n + (8 * m if case["stats"] else 0),
                "flops": (8.0 if case["direction"] == "fwd" else 14.0) * m * n}
    k, v = case["features"], case["vocab"]
    targets = m * (8 * case["labels"] + 12 * case["slots"] + 4 * case["lse"])
    passes = 1 if case["direction"] == "fwd" else 2
    return {"bytes": passes * e * k * (m + v) + targets + (8 * m if passes == 1 else 0), "flops": (2.0 if passes == 1 else 6.0) * m * k * v}


# ------------------------------------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    if case["op"] == "vocab" and work(case)["flops"] > 1.5e13:
        return None
    s = prepare(case, seed)
    return _norm_exact(case, s) if case["op"] == "norm" else _vocab_exact(case, s)


def _norm_exact(c, s):
    n = c["cols"]
    if c["direction"] == "fwd":
        y, means, rstds = [], [], []
        for x in s["x"].split(8192):
            x = x.double()
            var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
            rstd = (var + c["eps"]) ** -0.5
            y.append((x - mean) * rstd * s["weight"].double() + s["bias"].double())
            means.append(mean[:, 0])
            rstds.append(rstd[:, 0])
        out = {"y": torch.cat(y)}
        return {**out, "mean": torch.cat(means), "rstd": torch.cat(rstds)} if c["stats"] else out
    dx, dw, db = [], 0.0, 0.0
    for x, dy, st in zip(s["x"].split(8192), s["dy"].split(8192), s["stats"].t().split(8192)):
        st = st.double()
        h = (x.double() - st[:, :1]) * st[:, 1:]
        d = dy.double()
        a = d * s["weight"].double()
        b = a.sum(1, keepdim=True) + h * torch.einsum("mn,mn->m", a, h)[:, None]
        dx.append(st[:, 1:] * (a - b / n))
        dw = dw + torch.einsum("mn,mn->n", d, h)
        db = db + d.sum(0)
    return {"dx": torch.cat(dx), "dweight": dw, "dbias": db}


def _vocab_exact(c, s):
    m, w = c["rows"], s["weight"].double()
    zero = torch.zeros(m, dtype=torch.float64, device="cuda")
    labelled = (s["labels"] >= 0).double() if c["labels"] else zero
    per_label = labelled / max(1.0, float(labelled.sum()))
    if c["slots"]:
        held = s["ids"] >= 0
        t = s["logits"].double().masked_fill(~held, -math.inf)
        taught = held.any(1)
        norm = s["lse"].double() if c["lse"] else torch.logsumexp(t, 1)
        t = torch.where(held, torch.exp(t - norm[:, None]), torch.zeros_like(t))
        per_row = 1.0 / max(1, int(taught.sum()))
    rows_label, rows_teacher, dx, dw = zero.clone(), zero.clone(), [], 0.0
    step = max(1, (1 << 27) // c["vocab"])
    for r in range(0, m, step):
        part = slice(r, min(m, r + step))
        x = s["x"][part].double()
        logp = torch.log_softmax(c["alpha"] * torch.einsum("mk,vk->mv", x, w), 1)
        here = torch.arange(x.shape[0], device="cuda")
        weight, aims = zero[part].clone(), []
        if c["labels"]:
            label = s["labels"][part].clamp(min=0)
            rows_label[part] = -logp[here, label] * labelled[part]
            weight += per_label[part]
            aims.append((label[:, None], per_label[part][:, None]))
        if c["slots"]:
            ids, tt = s["ids"][part].clamp(min=0), t[part]
            rows_teacher[part] = (torch.xlogy(tt, tt) - tt * logp[here[:, None], ids]).sum(1)
            weight += tt.sum(1) * per_row
            aims.append((ids, tt * per_row))
        if c["direction"] == "bwd":
            d = logp.exp_().mul_(weight[:, None])
            for ids, a in aims:
                d.index_put_((here[:, None].expand_as(ids), ids), -a, accumulate=True)
            dx.append(c["alpha"] * torch.einsum("mv,vk->mk", d, w))
            dw = dw + c["alpha"] * torch.einsum("mv,mk->vk", d, x)
    loss = rows_label.sum() / max(1.0, float(labelled.sum())) + (rows_teacher.sum() * per_row if c["slots"] else 0.0)
    if c["direction"] == "fwd":
        return {"loss": loss, "row_label": rows_label, "row_teacher": rows_teacher}
    return {"loss": loss, "dx": torch.cat(dx), "dw": dw}
