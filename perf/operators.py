"""What the layer's operators beside the recurrence cost, and what they answer: the gated norm behind the mixer and the
residual norm before the next block (forward and backward), the drafted token tree over the state cache, the ragged
recurrence over cache slots, and the cache's own copies.

`run` computes a case either in its plain form (elementary torch operations in 32 bits, 64 for the sums of log decays) or,
where `own` is true, through the framework's entry points.  `exact` gives the same answers in 64 bits, by another route:
token by token and node by node from the recurrence itself.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of 256 sequences: the mixer's output through its gated norm (16 heads of 128)
        {"name": "gated norm, decode", "op": "gated_norm", "rows": 256 * 16, "d": 128, "dtype": "bf16", "act": "silu",
         "train": False},
        # a training step's norm and its gradients over the prefill workload B8 H16 T4096
        {"name": "gated norm, training", "op": "gated_norm", "rows": 8 * 4096 * 16, "d": 128, "dtype": "bf16",
         "act": "silu", "train": True},
        # one decode step of 256 sequences: residual sum and norm at the model's width (16 heads x 128)
        {"name": "residual norm, decode", "op": "add_norm", "rows": 256, "width": 2048, "dtype": "bf16", "scaled": True,
         "train": False},
        # a training step's residual norm and its gradients, B8 T4096
        {"name": "residual norm, training", "op": "add_norm", "rows": 8 * 4096, "width": 2048, "dtype": "bf16",
         "scaled": True, "train": True},
        # one user: a draft of eight nodes
        {"name": "tree, one user", "op": "tree", "batch": 1, "heads": 16, "d_k": 128, "d_v": 128, "dtype": "bf16",
         "nodes": 8, "ragged": False, "back": 4, "slots": 8},
        # a small batch with trees of uneven size
        {"name": "tree, batch", "op": "tree", "batch": 32, "heads": 16, "d_k": 128, "d_v": 128, "dtype": "bf16",
         "nodes": 32, "ragged": True, "back": 8, "slots": 48},
        # a full batch with full trees
        {"name": "tree, full", "op": "tree", "batch": 128, "heads": 16, "d_k": 128, "d_v": 128, "dtype": "bf16",
         "nodes": 64, "ragged": False, "back": 12, "slots": 160},
        # one token for each of 256 sequences, the old states kept until the tokens are accepted
        {"name": "recurrent, decode", "op": "recurrent", "batch": 256, "heads": 16, "d_k": 128, "d_v": 128,
         "dtype": "bf16", "tokens": 1, "ragged": False, "gather": False, "slots": 512},
        # the accepted paths of 64 drafts, gathered out of the drafted tokens
        {"name": "recurrent, accepted", "op": "recurrent", "batch": 64, "heads": 16, "d_k": 128, "d_v": 128,
         "dtype": "bf16", "tokens": 9, "ragged": True, "gather": True, "slots": 160},
        # uneven prompt tails in fp32, heads of 64 (the fp32 parity workload's)
        {"name": "recurrent, fp32 runs", "op": "recurrent", "batch": 8, "heads": 16, "d_k": 64, "d_v": 64,
         "dtype": "f32", "tokens": 201, "ragged": True, "gather": False, "slots": 24},
        # three continuations of one sequence
        {"name": "copy, fork", "op": "copy", "pairs": 3, "heads": 16, "d_k": 128, "d_v": 128, "slots": 16, "forks": 3,
         "freed": 0},
        # a batch after a round: sequences moved together, others forked, the ended ones cleared
        {"name": "copy, compaction", "op": "copy", "pairs": 192, "heads": 16, "d_k": 128, "d_v": 128, "slots": 448,
         "forks": 2, "freed": 24},
    ]


def _log(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(["gated_norm", "add_norm", "tree", "recurrent", "copy"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "gated_norm":
        return {"op": op, "rows": _log(rng, 1, 260000), "d": rng.choice([64, 128]), "dtype": dtype,
                "act": rng.choice(["silu", "sigmoid"]), "train": rng.random() < 0.6}
    if op == "add_norm":
        width = 8 * _log(rng, 8, 1024)
        return {"op": op, "rows": _log(rng, 1, max(1, (1 << 25) // width)), "width": width, "dtype": dtype,
                "scaled": rng.random() < 0.7, "train": rng.random() < 0.6}
    d_k, d_v = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (128, 64)])
    heads = rng.choice([1, 2, 3, 4, 5, 8, 16])
    if op == "copy":
        pairs = _log(rng, 1, 300)
        return {"op": op, "pairs": pairs, "heads": heads, "d_k": d_k, "d_v": d_v, "slots": 2 * pairs + rng.randint(2, 40),
                "forks": rng.randint(1, 4), "freed": rng.randint(0, pairs // 4)}
    batch = _log(rng, 1, 96)
    if op == "tree":
        return {"op": op, "batch": batch, "heads": heads, "d_k": d_k, "d_v": d_v, "dtype": dtype,
                "nodes": _log(rng, 1, 64), "ragged": rng.random() < 0.7, "back": rng.randint(1, 16),
                "slots": batch + rng.randint(0, 16)}
    tokens = _log(rng, 1, max(1, 600 // batch))
    return {"op": op, "batch": batch, "heads": heads, "d_k": d_k, "d_v": d_v, "dtype": dtype, "tokens": tokens,
            "ragged": rng.random() < 0.7, "gather": rng.random() < 0.4, "slots": 2 * batch + rng.randint(0, 16)}


# ---------------------------------------------------------------- inputs

def _rand(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _tokens(gen, n, heads, d_k, d_v, dtype):
    """n tokens of the mixer: q and k of unit length, decay exp(-softplus(N(1, 1))), sigmoid gates."""
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    alpha = torch.exp(-torch.nn.functional.softplus(_rand(gen, n, heads, d_k) + 1.0))
    return {"q": unit(_rand(gen, n, heads, d_k)).to(dtype), "k": unit(_rand(gen, n, heads, d_k)).to(dtype),
            "v": _rand(gen, n, heads, d_v).to(dtype), "alpha": alpha,
            "b": torch.sigmoid(_rand(gen, n, heads, d_k)).to(dtype),
            "w": torch.sigmoid(_rand(gen, n, heads, d_v)).to(dtype)}


def _lengths(rng, batch, most, ragged):
    if not ragged:
        return [most] * batch
    got = [rng.integers(1, most + 1) for _ in range(batch)]
    got[int(rng.integers(batch))] = most
    return [int(n) for n in got]


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _sizes(case):
    """Lengths of a case's sequences: they are part of the case, not of the seed."""
    rng = np.random.default_rng([case["batch"], case.get("nodes", case.get("tokens"))])
    return _lengths(rng, case["batch"], case.get("nodes", case.get("tokens")), case["ragged"])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    op, s = case["op"], {"case": case}
    if own:
        import gated_delta_rule_96_b200 as g
        g.load_library()
    if op == "gated_norm":
        t, shape = TYPES[case["dtype"]], (case["rows"], case["d"])
        s |= {"o": (0.3 * _rand(gen, *shape)).to(t), "gate": _rand(gen, *shape).to(t),
              "weight": 1.0 + 0.1 * _rand(gen, case["d"]), "dy": _rand(gen, *shape).to(t)}
        if own and case["train"]:
            s["workspace"] = g.new_workspace(g.gdn2_gated_norm_bwd_workspace_bytes(case["rows"], case["d"]))
        return s
    if op == "add_norm":
        t, shape = TYPES[case["dtype"]], (case["rows"], case["width"])
        s |= {"x": _rand(gen, *shape).to(t), "residual": (2.0 * _rand(gen, *shape)).to(t),
              "scale": 0.5 + 0.1 * _rand(gen, case["width"]) if case["scaled"] else None,
              "weight": 1.0 + 0.1 * _rand(gen, case["width"])}
        if case["train"]:   # the backward of another layer's call, with the sum that its forward stored
            s |= {"h": (2.0 * _rand(gen, *shape)).to(t), "dy": _rand(gen, *shape).to(t),
                  "dh": _rand(gen, *shape).to(t)}
            if own:
                s["workspace"] = g.new_workspace(g.gdn2_add_norm_bwd_workspace_bytes(case["rows"], case["width"]))
        return s
    heads, d_k, d_v, slots = case["heads"], case["d_k"], case["d_v"], case["slots"]
    s["pool"] = 0.1 * _rand(gen, slots, heads, d_k, d_v)
    if own:
        s["workspace"] = g.new_workspace(0)
    if op == "copy":
        # distinct destinations, none of them a source; one source serves `forks` pairs; -1 clears its slot
        order = rng.permutation(slots)
        dst, rest = order[: case["pairs"]], order[case["pairs"]:]
        src = rest[(np.arange(case["pairs"]) // case["forks"]) % len(rest)]
        src[rng.permutation(case["pairs"])[: case["freed"]]] = -1
        return s | {"src": _ints(src.tolist()), "dst": _ints(dst.tolist())}
    lens = _sizes(case)
    cu, total = np.concatenate([[0], np.cumsum(lens)]).tolist(), int(sum(lens))
    s["cu"] = _ints(cu)
    order = rng.permutation(slots).tolist()
    if op == "tree":
        parents = []
        for n in lens:   # node 0 is the last token; the others hang on one of the `back` nodes before them
            parents += [-1] + [int(rng.integers(max(0, i - case["back"]), i)) for i in range(1, n)]
        s |= _tokens(gen, total, heads, d_k, d_v, TYPES[case["dtype"]])
        return s | {"slots": _ints(order[: case["batch"]]), "parents": _ints(parents), "most": max(lens)}
    rows, index = total, None
    if case["gather"]:   # every third drafted token was accepted
        rows = 3 * total
        index = _ints(np.sort(rng.permutation(rows)[:total]).tolist())
    s |= _tokens(gen, rows, heads, d_k, d_v, TYPES[case["dtype"]])
    return s | {"slots_in": _ints(order[: case["batch"]]), "slots_out": _ints(order[case["batch"]: 2 * case["batch"]]),
                "index": index, "most": max(lens)}


# ---------------------------------------------------------------- the passes

def run(s):
    return (_own if own else _plain)(s)


def _own(s):
    import gated_delta_rule_96_b200 as g
    case, op = s["case"], s["case"]["op"]
    if op == "gated_norm":
        y = g.gated_norm_fwd(s["o"], s["gate"], s["weight"], act=case["act"], eps=EPS)
        if not case["train"]:
            return y
        return (y, *g.gated_norm_bwd(s["o"], s["gate"], s["weight"], s["dy"], act=case["act"], eps=EPS,
                                     workspace=s["workspace"]))
    if op == "add_norm":
        out = g.add_norm_fwd(s["x"], s["residual"], s["scale"], s["weight"], eps=EPS)
        if case["train"]:
            out += g.add_norm_bwd(s["h"], s["x"], s["scale"], s["weight"], s["dy"], s["dh"], eps=EPS,
                                  workspace=s["workspace"])
        return out
    if op == "copy":
        g.gdn2_state_copy(s["pool"], s["pool"], s["dst"], s["src"], workspace=s["workspace"])
        return s["pool"]
    tokens = [s[name] for name in ("q", "k", "v", "alpha", "b", "w")]
    if op == "tree":
        return g.tree_fwd(*tokens, s["pool"], s["slots"], s["cu"], s["parents"], s["most"], workspace=s["workspace"])
    o = g.recurrent_fwd(*tokens, s["pool"], s["slots_in"], s["slots_out"], s["cu"], index=s["index"],
                        workspace=s["workspace"])
    return o, s["pool"]


def _plain(s):
    op = s["case"]["op"]
    if op == "gated_norm":
        return _plain_gated_norm(s)
    if op == "add_norm":
        return _plain_add_norm(s)
    if op == "copy":
        src, dst = s["src"].long(), s["dst"].long()
        moved = s["pool"][src.clamp(min=0)] * (src >= 0).float().view(-1, 1, 1, 1)
        s["pool"][dst] = moved
        return s["pool"]
    return _plain_chunk(s)


def _plain_gated_norm(s):
    case, o, gate, w = s["case"], s["o"].float(), s["gate"].float(), s["weight"]
    sig = torch.sigmoid(gate)
    act = gate * sig if case["act"] == "silu" else sig
    r = torch.rsqrt(o.square().mean(-1, keepdim=True) + EPS)
    xn = o * r
    y = (xn * w * act).to(s["o"].dtype)
    if not case["train"]:
        return y
    dy = s["dy"].float()
    slope = sig * (1 + gate * (1 - sig)) if case["act"] == "silu" else sig * (1 - sig)
    dgate = dy * xn * w * slope
    dn = dy * act
    dx = dn * w
    do = r * (dx - xn * (dx * xn).mean(-1, keepdim=True))
    return y, do.to(y.dtype), dgate.to(y.dtype), (dn * xn).sum(0)


def _plain_add_norm(s):
    case, t = s["case"], s["x"].dtype
    scale = 1.0 if s["scale"] is None else s["scale"]
    h = s["residual"].float() + scale * s["x"].float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["weight"]
    out = (y.to(t), h.to(t))
    if not case["train"]:
        return out
    h, dy = s["h"].float(), s["dy"].float()
    r = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    xn, dx = h * r, dy * s["weight"]
    dres = s["dh"].float() + r * (dx - xn * (dx * xn).mean(-1, keepdim=True))
    dscale = None if s["scale"] is None else (dres * s["x"].float()).sum(0)
    return out + (dres.to(t), (scale * dres).to(t), dscale, (dy * xn).sum(0))


def _plain_chunk(s):
    """Tree and runs alike, in the chunk form: with G the product of the decays from the state to a node,
    (I + A) D = u - (e G) S,  A[n, i] = sum_c e_n G_n / G_i k_i over the ancestors i of n,  o = (q G) S + P D."""
    case, tree = s["case"], s["case"]["op"] == "tree"
    n, batch, heads = s["most"], case["batch"], case["heads"]
    cu, at = s["cu"].long(), torch.arange(n, device="cuda")
    lens = cu[1:] - cu[:-1]
    real = at[None, :] < lens[:, None]                                     # [batch, n]
    row = torch.where(real, cu[:-1, None] + at, 0)
    token = row if tree or s["index"] is None else s["index"].long()[row]
    pad = lambda x, fill=0.0: torch.where(real[..., None, None], x[token].float(), fill).transpose(1, 2)  # noqa: E731
    q, k, v, b, w = (pad(s[name]) for name in ("q", "k", "v", "b", "w"))     # [batch, heads, n, d]
    loga = pad(s["alpha"], 1.0).double().log()
    e, u = b * k, w * v
    if tree:
        up = torch.where(real, s["parents"].long()[row], -1)
        path = torch.eye(n, device="cuda") + (up[:, :, None] == at).float()  # self and parent, then all ancestors
        for _ in range(max(1, (n - 1).bit_length())):
            path = (path @ path).clamp(max=1.0)
        S = s["pool"][s["slots"].long()]
    else:
        path = torch.ones(n, n, device="cuda").tril().expand(batch, n, n)
        S = s["pool"][s["slots_in"].long()]
    path = path[:, None]
    g = path.double() @ loga
    apart = torch.where(path[..., None] > 0, g[:, :, :, None] - g[:, :, None], -math.inf)
    fall = torch.exp(apart.float()) * k[:, :, None]                         # [batch, heads, n, n, d_k]
    A = (fall * e[:, :, :, None]).sum(-1) * (1 - torch.eye(n, device="cuda"))
    P = (fall * q[:, :, :, None]).sum(-1)
    G = torch.exp(g).float()
    inverse, power = torch.eye(n, device="cuda") - A, A @ A
    for _ in range((n - 1).bit_length()):                                   # (I - A)(I + A^2)(I + A^4) ...
        inverse, power = inverse + inverse @ power, power @ power
    D = inverse @ (u - (e * G) @ S)
    o = ((q * G) @ S + P @ D).transpose(1, 2)[real].to(s["q"].dtype)
    if tree:
        return o
    last = (lens - 1).view(batch, 1, 1, 1).expand(batch, heads, 1, case["d_k"])
    keys = fall[torch.arange(batch, device="cuda"), :, lens - 1]             # decayed to the last token
    s["pool"][s["slots_out"].long()] = G.gather(2, last).transpose(2, 3) * S + keys.transpose(2, 3) @ D
    return o, s["pool"]


# ---------------------------------------------------------------- sizes of the work

def work(case):
    op = case["op"]
    if op in ("gated_norm", "add_norm"):
        size = 2 if case["dtype"] == "bf16" else 4
        n = case["rows"] * case.get("d", case.get("width"))
        if op == "gated_norm":
            # o, gate -> y; then o, gate, dy -> do, dgate
            return {"bytes": n * size * (3 + (5 if case["train"] else 0)), "flops": n * (12 + (30 if case["train"] else 0))}
        # x, residual -> h, y; then h, x, dy, dh -> dresidual, dx
        grads = (6 if case["scaled"] else 5) if case["train"] else 0
        return {"bytes": n * size * (4 + grads), "flops": n * (6 + 3 * grads)}
    state = 4 * case["heads"] * case["d_k"] * case["d_v"]
    if op == "copy":
        kept = case["pairs"] - case["freed"]
        return {"bytes": state * (case["pairs"] + -(-kept // case["forks"])), "flops": 0}
    size = 2 if case["dtype"] == "bf16" else 4
    lens, d_k, d_v = _sizes(case), case["d_k"], case["d_v"]
    token = case["heads"] * (size * (3 * d_k + 3 * d_v) + 4 * d_k)           # q k b, v w o, alpha
    states = 1 if op == "tree" else 2
    # a node: two products with the state (tree), with the state's update besides (run)
    flops = sum(lens) * case["heads"] * d_k * d_v * (4 if op == "tree" else 8)
    return {"bytes": states * state * case["batch"] + token * sum(lens), "flops": flops}


# ---------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    op = case["op"]
    if op == "gated_norm":
        o, gate = (s[name].double().requires_grad_() for name in ("o", "gate"))
        weight = s["weight"].double().requires_grad_()
        norm = o / torch.sqrt((o * o).sum(-1, keepdim=True) / case["d"] + EPS)
        y = norm * weight / (1 + torch.exp(-gate)) * (gate if case["act"] == "silu" else 1)
        if not case["train"]:
            return y.detach()
        return (y.detach(), *torch.autograd.grad(y, (o, gate, weight), s["dy"].double()))
    if op == "add_norm":
        def forward(x, residual, scale):
            h = residual + x * scale
            return h, h / torch.sqrt((h * h).sum(-1, keepdim=True) / case["width"] + EPS) * s["weight"].double()
        scale = torch.ones(case["width"], device="cuda").double() if s["scale"] is None else s["scale"].double()
        h, y = forward(s["x"].double(), s["residual"].double(), scale)
        if not case["train"]:
            return y, h
        # the gradients at the stored sum: scale as it is, the sum's other part whatever makes it that
        x, scale, weight = s["x"].double(), scale.requires_grad_(), s["weight"].double().requires_grad_()
        h2 = s["h"].double().requires_grad_()
        y2 = h2 / torch.sqrt((h2 * h2).sum(-1, keepdim=True) / case["width"] + EPS) * weight
        dres, dweight = torch.autograd.grad(y2, (h2, weight), s["dy"].double())
        dres = dres + s["dh"].double()
        dscale = None if s["scale"] is None else torch.einsum("rc,rc->c", dres, x)
        return y, h, dres, dres * scale.detach(), dscale, dweight
    pool = s["pool"].double()
    if op == "copy":
        old, src, dst = pool.clone(), s["src"].tolist(), s["dst"].tolist()
        for i, j in zip(src, dst):
            pool[j] = old[i] if i >= 0 else 0.0
        return pool
    q, k, v, alpha, b, w = (s[name].double() for name in ("q", "k", "v", "alpha", "b", "w"))
    cu = s["cu"].tolist()
    o = torch.zeros(cu[-1], case["heads"], case["d_v"], dtype=torch.float64, device="cuda")

    def step(S, t):
        S = alpha[t][..., None] * S
        read = (S * (b[t] * k[t])[..., None]).sum(-2)
        S = S + k[t][..., None] * (w[t] * v[t] - read)[..., None, :]
        return S, (S * q[t][..., None]).sum(-2)

    if op == "tree":
        parents, slots, levels = s["parents"].tolist(), s["slots"].tolist(), {}
        for i, first in enumerate(cu[:-1]):
            depth = []
            for n in range(cu[i + 1] - first):
                p = parents[first + n]
                depth.append(0 if p < 0 else depth[p] + 1)
                levels.setdefault(depth[n], []).append((first + n, first + p if p >= 0 else -1, slots[i]))
        before, place = None, {}
        for d in sorted(levels):   # the states of one level of every tree at a time
            nodes = levels[d]
            t = torch.tensor([n for n, _, _ in nodes], device="cuda")
            S = pool[[slot for _, _, slot in nodes]] if d == 0 else before[[place[p] for _, p, _ in nodes]]
            before, o[t] = step(S, t)
            place = {n: j for j, (n, _, _) in enumerate(nodes)}
        return o
    lens = [hi - lo for lo, hi in zip(cu, cu[1:])]
    S, index = pool[s["slots_in"].long()], None if s["index"] is None else s["index"].long()
    for t in range(max(lens)):
        live = [i for i, n in enumerate(lens) if n > t]
        at = torch.tensor([cu[i] + t for i in live], device="cuda")
        S[live], o[at] = step(S[live], at if index is None else index[at])
    pool[s["slots_out"].long()] = S
    return o, pool
