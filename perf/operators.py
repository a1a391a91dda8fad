"""The cases on which the operators of an MoE block's training and serving
step are measured: products grouped by expert in 16 bits with their
gradients, the norms before and after the block with its gate and residual
scale, and the global gradient norm with clipping.

listed() and draw() give cases, prepare() makes their inputs on the GPU,
run() makes one pass and work() says what the pass cannot do without. With
`own` false run() computes the operators in elementary torch operations in
32 bits; with `own` true it calls the framework.
"""
import math
import random

import torch

own = False

TYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32}
EPS = 1e-6
CLIP_EPS = 1e-6


# ------------------------------------------------------------------- cases
def listed():
    def grouped(name, way, groups, rows, n, k, dtype="bfloat16", skew=0.0, align=1):
        return {"name": name, "op": "grouped", "way": way, "groups": groups, "rows": rows, "n": n,
                "k": k, "dtype": dtype, "skew": skew, "align": align}

    def norm(name, way, rows, h, dtype="bfloat16", res="bfloat16", z=True, post=True, pre=True,
             gate="none", scale=False, wide=False):
        return {"name": name, "op": "norm", "way": way, "rows": rows, "h": h, "dtype": dtype,
                "res": res, "z": z, "post": post, "pre": pre, "gate": gate, "scale": scale,
                "wide": wide}

    def clip(name, tensors, elements, dtype, max_norm, inplace):
        return {"name": name, "op": "clip", "tensors": tensors, "elements": elements,
                "dtype": dtype, "max_norm": max_norm, "inplace": inplace}

    return [
        # one token decoded: its eight experts' up/gate rows out of a shard of 64
        grouped("grouped one token", "forward", 64, 8, 4096, 7168),
        # a decode batch of 128 tokens: the down projections of the same shard
        grouped("grouped decode batch", "forward", 64, 1024, 7168, 2048),
        # a prompt of 4096 tokens through a shard of 32 experts, up/gate, ragged
        grouped("grouped prompt", "forward", 32, 32768, 4096, 7168, skew=0.3),
        # the input gradient of the up/gate projection at half that batch, in
        # fp16, with groups on 128-row boundaries as the permutation lays them
        grouped("grouped input gradient", "input_grad", 32, 16384, 7168, 4096, "float16", 0.3, 128),
        # the weight gradient of the down projection of the same step
        grouped("grouped weight gradient", "weight_grad", 32, 16384, 7168, 2048, skew=0.3),
        # the last norm, gate and residual of a decoded token, with the next norm
        norm("norm one token", "forward", 1, 7168, gate="row"),
        # a prompt of 4096 tokens, residual and next norm in one pass
        norm("norm prompt", "forward", 4096, 7168, scale=True),
        # training, the backward of the same with an fp32 residual stream
        norm("norm backward", "backward", 16384, 7168, res="float32", gate="row", scale=True,
             wide=True),
        # an odd width, as after pruning channels
        norm("norm backward odd", "backward", 777, 1409, "float16", "float16", gate="full"),
        # gradients of a tiny layer, where the launches count
        clip("clip tiny", 6, 1 << 20, "float32", 1.0, False),
        # a shard's expert gradients in fp32, clipped out of place
        clip("clip experts", 8, 700_000_000, "float32", 1.0, False),
        # many tensors of both types in flat buffers, below the limit: in place
        clip("clip many", 512, 150_000_000, "mixed", 1e9, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["grouped", "grouped", "norm", "clip"])
    if op == "grouped":
        way = rng.choice(["forward", "input_grad", "weight_grad"])
        while True:
            groups, rows = _log(rng, 1, 160), _log(rng, 1, 32768)
            n, k = 8 * _log(rng, 8, 896), 8 * _log(rng, 8, 896)
            skew = rng.choice([0.0, 0.3, 0.8])
            if groups * n * k <= 64 * 4096 * 7168 / 2 and _cap_guess(groups, rows, skew) * n * k <= 32768 * 4096 * 7168:
                break
        return {"op": "grouped", "way": way, "groups": groups, "rows": rows, "n": n, "k": k,
                "dtype": rng.choice(["bfloat16", "bfloat16", "float16"]), "skew": skew,
                "align": rng.choice([1, 1, 128])}
    if op == "norm":
        h = _log(rng, 64, 8192)
        h = h if rng.random() < 0.25 else 8 * max(8, h // 8)
        dtype = rng.choice(["bfloat16", "float16", "float32"])
        res = rng.choice([dtype, "float32"])
        z = rng.random() < 0.8
        return {"op": "norm", "way": rng.choice(["forward", "backward"]), "rows": _log(rng, 1, 16384),
                "h": h, "dtype": dtype, "res": res, "z": z, "post": z and rng.random() < 0.7,
                "pre": not z or rng.random() < 0.7,
                "gate": rng.choice(["none", "row", "full"]) if z else "none",
                "scale": z and rng.random() < 0.5, "wide": rng.random() < 0.5}
    tensors = _log(rng, 1, 512)
    return {"op": "clip", "tensors": tensors, "elements": max(tensors, _log(rng, 1000, 500_000_000)),
            "dtype": rng.choice(["float32", "bfloat16", "float16", "mixed"]),
            "max_norm": rng.choice([0.1, 1.0, 1e9]), "inplace": False}


def _shares(groups, skew):
    w = [(g + 1.0) ** -skew for g in range(groups)]
    return [x / sum(w) for x in w]


def _cap_guess(groups, rows, skew):
    """Rows of all groups when each is as long as the longest one."""
    return groups * rows * _shares(groups, skew)[0]


def work(case):
    if case["op"] == "grouped":
        g, r, n, k = case["groups"], case["rows"], case["n"], case["k"]
        if case["way"] == "weight_grad":
            moved = r * (n + k) * 2 + g * n * k * 4
        else:
            busy = sum(1.0 - (1.0 - p) ** r for p in _shares(g, case["skew"]))
            moved = r * (n + k) * 2 + busy * n * k * 2
        return {"bytes": moved, "flops": 2.0 * r * n * k}
    if case["op"] == "norm":
        t, h = case["rows"], case["h"]
        act, res = TYPES[case["dtype"]].itemsize, TYPES[case["res"]].itemsize
        per = 0
        if case["way"] == "forward":
            per += res + (act + res if case["z"] else 0) + (act if case["pre"] else 0)
            per += act if case["gate"] == "full" else 0
        else:
            per += res + (res if case["pre"] else 0) + (res + act if case["pre"] else 0)
            per += 2 * act if case["z"] else 0
            per += 2 * act if case["gate"] == "full" else 0
        return {"bytes": per * t * h, "flops": 0}
    size = {"float32": 4, "mixed": 3}.get(case["dtype"], 2)
    return {"bytes": size * case["elements"] * (1 if case["inplace"] else 2), "flops": 0}


# ------------------------------------------------------------------ inputs
def _normal(gen, shape, dtype, std=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"grouped": _prepare_grouped, "norm": _prepare_norm, "clip": _prepare_clip}[case["op"]](
        case, seed, gen)


def _prepare_grouped(case, seed, gen):
    groups, n, k = case["groups"], case["n"], case["k"]
    dtype = TYPES[case["dtype"]]
    # tokens choose their experts at random; which experts are popular too
    cpu = torch.Generator().manual_seed(seed)
    shares = torch.tensor(_shares(groups, case["skew"]))[torch.randperm(groups, generator=cpu)]
    chosen = torch.multinomial(shares, case["rows"], replacement=True, generator=cpu)
    rows = torch.bincount(chosen, minlength=groups)
    step = (rows + case["align"] - 1) // case["align"] * case["align"]
    start = torch.cumsum(step, 0) - step
    total = int(step.sum())
    state = {"case": case, "cap": int(rows.max()),
             "group_rows": rows.to(torch.int32).cuda(), "group_start": start.to(torch.int32).cuda()}
    if case["way"] == "weight_grad":
        state["dy"] = _normal(gen, (total, n), dtype, 0.5)
        state["x"] = _normal(gen, (total, k), dtype)
        state["out"] = torch.zeros((groups, n, k), dtype=torch.float32, device="cuda")
    else:
        shape = (groups, n, k) if case["way"] == "forward" else (groups, k, n)
        state["a"] = _normal(gen, (total, k), dtype)
        state["w"] = _normal(gen, shape, dtype, k ** -0.5)
        state["out"] = torch.zeros((total, n), dtype=dtype, device="cuda")
    return state


def _prepare_norm(case, seed, gen):
    t, h = case["rows"], case["h"]
    act, res = TYPES[case["dtype"]], TYPES[case["res"]]
    wtype = torch.float32 if case["wide"] else act
    state = {"case": case}
    # the residual stream grows with depth, and a few channels are large
    x = _normal(gen, (t, h), torch.float32, 3.0)
    x[:, :: 97] *= 8.0
    state["x"] = x.to(res)
    del x

    def vector(at):
        return (at + 0.2 * torch.randn(h, generator=gen, device="cuda")).to(wtype)

    state["pre_weight"] = vector(1.0) if case["pre"] else None
    state["post_weight"] = vector(0.6) if case["post"] else None
    state["scale"] = vector(0.3) if case["scale"] else None
    state["z"] = _normal(gen, (t, h), act, 1.5) if case["z"] else None
    state["gate"] = None
    if case["gate"] == "row":
        state["gate"] = torch.sigmoid(_normal(gen, (t,), torch.float32))
    elif case["gate"] == "full":
        state["gate"] = torch.sigmoid(_normal(gen, (t, h), torch.float32)).to(act)
    state["alpha"] = 0.7
    new = lambda like: None if like is None else torch.zeros_like(like)  # noqa: E731
    if case["way"] == "forward":
        state["r"] = new(state["x"]) if case["z"] else None
        state["u"] = torch.zeros((t, h), dtype=act, device="cuda") if case["pre"] else None
        return state
    state["dr"] = _normal(gen, (t, h), res, 0.01)
    state["du"] = _normal(gen, (t, h), act, 0.02) if case["pre"] else None
    state["dx"] = new(state["x"]) if case["pre"] else None
    state["dz"] = new(state["z"])
    state["dgate"] = new(state["gate"])
    state.update({"d" + name: None if state[name] is None else torch.zeros(h, device="cuda")
                  for name in ("pre_weight", "post_weight", "scale")})
    # the column sums' scratch: partial sums of two vectors for up to 1024 parts
    state["ws"] = torch.empty(2 * 1024 * h * 4 + 1024, dtype=torch.uint8, device="cuda")
    return state


def _sizes(case):
    """The tensors' sizes: spread over orders of magnitude, odd ones among them."""
    rng = random.Random(case["tensors"] * 1000003 + case["elements"])
    w = [math.exp(rng.uniform(0, 6)) for _ in range(case["tensors"])]
    left = case["elements"] - case["tensors"]
    sizes = [1 + int(left * x / sum(w)) for x in w]
    sizes[0] += case["elements"] - sum(sizes)
    return sizes


def _prepare_clip(case, seed, gen):
    sizes = _sizes(case)
    kinds = ["float32", "bfloat16"] if case["dtype"] == "mixed" else [case["dtype"]]
    state = {"case": case}
    mine = {kind: sizes[i::len(kinds)] for i, kind in enumerate(kinds) if sizes[i::len(kinds)]}
    flat = {kind: _normal(gen, (sum(m),), TYPES[kind], 1e-2) for kind, m in mine.items()}
    out = flat if case["inplace"] else {kind: torch.zeros_like(f) for kind, f in flat.items()}
    state["flat"], state["flat_out"] = flat, out
    state["grads"] = [g for kind, m in mine.items() for g in flat[kind].split(m)]
    state["out"] = [o for kind, m in mine.items() for o in out[kind].split(m)]
    state["norm"] = torch.zeros(1, device="cuda")
    # what a program keeps between steps: one partial sum of squares per block
    state["partials"] = torch.zeros(1024, dtype=torch.float64, device="cuda")
    state["list"] = None
    return state


# ------------------------------------------------------------------ a pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"grouped": _own_grouped, "norm": _own_norm, "clip": _own_clip}[op](state)
    return {"grouped": _plain_grouped, "norm": _plain_norm, "clip": _plain_clip}[op](state)


def _own_grouped(s):
    from mixture_experts_layer_40_b200 import capi
    if s["case"]["way"] == "weight_grad":
        capi.moe_grouped_wgrad(s["dy"], s["x"], s["group_rows"], s["group_start"], s["out"])
    else:
        capi.moe_grouped_matmul(s["a"], s["w"], s["group_rows"], s["group_start"], s["out"],
                                trans_b=s["case"]["way"] == "forward")
    return s["out"]


def _own_norm(s):
    from mixture_experts_layer_40_b200 import capi
    if s["case"]["way"] == "forward":
        capi.moe_block_norm(s["x"], EPS, pre_weight=s["pre_weight"], u=s["u"], z=s["z"],
                            post_weight=s["post_weight"], gate=s["gate"], scale=s["scale"],
                            alpha=s["alpha"], r=s["r"])
        return {"r": s["r"], "u": s["u"]}
    capi.moe_block_norm_backward(
        s["x"], EPS, s["ws"], dr=s["dr"], du=s["du"], pre_weight=s["pre_weight"], z=s["z"],
        post_weight=s["post_weight"], gate=s["gate"], scale=s["scale"], alpha=s["alpha"],
        dx=s["dx"], dz=s["dz"], dgate=s["dgate"], dscale=s["dscale"], dpost=s["dpost_weight"],
        dpre=s["dpre_weight"])
    return {"dx": s["dx"], "dz": s["dz"], "dgate": s["dgate"], "dscale": s["dscale"],
            "dpost": s["dpost_weight"], "dpre": s["dpre_weight"]}


def _own_clip(s):
    from mixture_experts_layer_40_b200 import capi
    if s["list"] is None:  # the table of the program's own gradient buffers
        s["list"] = capi.make_grad_list(s["grads"], None if s["case"]["inplace"] else s["out"])
    capi.moe_grad_sumsq(s["list"], s["partials"])
    capi.moe_grad_clip(s["list"], s["partials"], s["case"]["max_norm"], s["norm"])
    return {"norm": s["norm"], "grads": s["flat_out"]}


def _padded(state, m):
    """[groups, cap, width]: each group's rows of m in 32 bits, zeros behind."""
    at = torch.arange(state["cap"], device=m.device)
    live = at < state["group_rows"][:, None]
    index = torch.where(live, state["group_start"][:, None] + at, 0)
    return torch.where(live[..., None], m[index].float(), 0.0), torch.where(live, index, m.shape[0])


def _plain_grouped(s):
    if s["case"]["way"] == "weight_grad":
        return torch.bmm(_padded(s, s["dy"])[0].transpose(1, 2), _padded(s, s["x"])[0])
    a, index = _padded(s, s["a"])
    w = s["w"].float()
    prod = torch.bmm(a, w.transpose(1, 2) if s["case"]["way"] == "forward" else w)
    total, n = s["out"].shape
    out = torch.zeros((total + 1, n), dtype=s["out"].dtype, device=a.device)
    out[index.flatten()] = prod.flatten(0, 1).to(out.dtype)
    return out[:total]


def _unit(v):
    return v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)


def _times(a, b):
    return a if b is None else a * b


def _plain_norm(s):
    case, f = s["case"], lambda v: None if v is None else v.float()
    x, z, pre, post, scale, gate = (f(s[k]) for k in
                                    ("x", "z", "pre_weight", "post_weight", "scale", "gate"))
    gate = gate[:, None] if case["gate"] == "row" else gate
    if case["way"] == "forward":
        r = x
        if z is not None:
            r = x + s["alpha"] * _times(_times(_unit(z) * post if case["post"] else z, scale), gate)
        return {"r": r.to(s["x"].dtype) if case["z"] else None,
                "u": (_unit(r) * pre).to(s["u"].dtype) if case["pre"] else None}
    out = dict.fromkeys(("dx", "dz", "dgate", "dscale", "dpost", "dpre"))
    e = f(s["dr"])
    if case["pre"]:
        du, h, scale_r = f(s["du"]), _unit(x), torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
        dh = du * pre
        e = e + scale_r * (dh - h * (dh * h).mean(1, keepdim=True))
        out["dx"], out["dpre"] = e.to(s["x"].dtype), (du * h).sum(0)
    if case["z"]:
        y = _unit(z) if case["post"] else z
        q = _times(_times(s["alpha"] * e, scale), gate)
        out["dz"] = q
        if case["post"]:
            scale_z, dy = torch.rsqrt((z * z).mean(1, keepdim=True) + EPS), q * post
            out["dz"] = scale_z * (dy - y * (dy * y).mean(1, keepdim=True))
            out["dpost"] = (q * y).sum(0)
        out["dz"] = out["dz"].to(s["z"].dtype)
        branch = _times(y, post)
        if case["scale"]:
            out["dscale"] = (_times(s["alpha"] * e, gate) * branch).sum(0)
        if case["gate"] != "none":
            dgate = s["alpha"] * e * _times(branch, scale)
            dgate = dgate.sum(1) if case["gate"] == "row" else dgate
            out["dgate"] = dgate.to(s["gate"].dtype)
    return out


def _plain_clip(s):
    total = torch.stack([(g.float() ** 2).sum() for g in s["grads"]]).sum()
    norm = total.sqrt()
    c = (s["case"]["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0)
    [o.copy_(g.float() * c) for o, g in zip(s["out"], s["grads"])]
    return {"norm": norm[None], "grads": s["flat_out"]}


# ------------------------------------------------------- the values in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(case, s)
    if case["op"] == "clip":
        total = sum(v.double().pow(2).sum().item() for v in s["flat"].values())
        factor = min(1.0, case["max_norm"] / (math.sqrt(total) + CLIP_EPS))
        return {"norm": torch.tensor([math.sqrt(total)], dtype=torch.float64, device="cuda"),
                "grads": {k: v.double() * factor for k, v in s["flat"].items()}}
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    spans = zip(s["group_start"].tolist(), s["group_rows"].tolist())
    for g, (at, count) in enumerate(spans):
        part = slice(at, at + count)
        if case["way"] == "weight_grad":
            out[g] = s["dy"][part].double().T @ s["x"][part].double()
        elif count:
            w = s["w"][g].double()
            out[part] = s["a"][part].double() @ (w.T if case["way"] == "forward" else w)
    return out


def _exact_norm(case, s):
    """By the definition, and its gradients by the chain rule on whole rows."""
    d = {k: (v.double() if isinstance(v, torch.Tensor) else v) for k, v in s.items() if k != "ws"}
    one = torch.ones((), dtype=torch.float64, device="cuda")
    gate = one if d["gate"] is None else d["gate"][:, None] if case["gate"] == "row" else d["gate"]
    scale = one if d["scale"] is None else d["scale"]
    post = one if d["post_weight"] is None else d["post_weight"]
    length = lambda v: torch.sqrt(v.square().mean(dim=1, keepdim=True) + EPS)  # noqa: E731
    if case["way"] == "forward":
        r = d["x"]
        if case["z"]:
            branch = d["z"] / length(d["z"]) if case["post"] else d["z"]
            r = r + d["alpha"] * gate * scale * post * branch
        return {"r": r if case["z"] else None,
                "u": r / length(r) * d["pre_weight"] if case["pre"] else None}

    def through(v, up):
        """The gradient of v / length(v) against `up`."""
        n = length(v)
        return up / n - v * (up * v).mean(dim=1, keepdim=True) / n ** 3

    out = dict.fromkeys(("dx", "dz", "dgate", "dscale", "dpost", "dpre"))
    e = d["dr"]
    if case["pre"]:
        e = e + through(d["x"], d["du"] * d["pre_weight"])
        out["dx"] = e
        out["dpre"] = (d["du"] * d["x"] / length(d["x"])).sum(dim=0)
    if case["z"]:
        branch = d["z"] / length(d["z"]) if case["post"] else d["z"]
        up = d["alpha"] * gate * scale * post * e
        out["dz"] = through(d["z"], up) if case["post"] else up
        plain = d["alpha"] * e * branch
        if case["post"]:
            out["dpost"] = (plain * gate * scale).sum(dim=0)
        if case["scale"]:
            out["dscale"] = (plain * gate * post).sum(dim=0)
        if case["gate"] == "row":
            out["dgate"] = (plain * scale * post).sum(dim=1)
        elif case["gate"] == "full":
            out["dgate"] = plain * scale * post
    return out
