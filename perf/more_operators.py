"""Cases of the residual stream's norm and of the loss over the vocabulary, for timing and comparison.

Operators: the sum of the residual stream and a block's output with the norm before the next block, and the norm, gate
and scale after this one (``norm``), its backward pass (``norm_grad``), the softmax cross entropy over a vocabulary with
the z-loss from the hidden states and the output embedding (``loss``), and its gradients (``loss_grad``).  ``own``
chooses between the framework's calls and the plain form of the same formulas in elementary torch operations.

Formulas, for rows x (residual stream), u (block), y, z of D elements, with r(v) = 1 / sqrt(mean(v^2) + eps):
    p = u r(u) block_gain, or u without the norm after the block;  t = gate p (or p)
    y = x_scale x + block_scale t, rounded to the tensors' type;   z = y r(y) gain
backward for upstream dy (of y) and dz (of z), with r = r(y), n = y r:
    dn = dz gain;  dY = dy + (dn - n mean(dn n)) r;  dgain = sum over rows of dz n
    dx = x_scale dY;  dt = block_scale dY;  dgate = dt p (summed over rows where the gate is one for all of them)
    dp = dt gate;  du = dp, or the same gradient of the norm of u;  dblock_gain = sum over rows of dp u r(u)
loss, for hidden states x (N, D), output embedding w (V, D) and labels:
    l = x w^T;  lse = log sum exp l;  loss = lse - l[label] + z_weight lse^2, or 0 where the label is ignored
    dl = dloss (softmax(l) (1 + 2 z_weight lse) - onehot(label)), or 0;  dx = dl w;  dw = dl^T x
"""
import math

import torch

own = False

DEVICE = "cuda"
EPS = 1e-6
IGNORED = -100
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # One step of generation: a single token's residual row of the pages' model, latency counts.
        {"name": "norm one token bf16", "op": "norm", "batch": 1, "seq": 1, "dim": 2048, "gain": True,
         "block_norm": False, "gate": "none", "x_scale": 1.0, "block_scale": 1.0, "type": "bf16", "layout": "plain"},
        # Between two blocks of the pages' model, on its microbatch of 4 windows of 4096 tokens.
        {"name": "norm microbatch bf16", "op": "norm", "batch": 4, "seq": 4096, "dim": 2048, "gain": True,
         "block_norm": False, "gate": "none", "x_scale": 1.0, "block_scale": 1.0, "type": "bf16", "layout": "plain"},
        # Norms on both sides of the block, a gate for each channel and a scaled residual, in FP32, odd sizes, the
        # residual and the block's output side by side in wider rows.
        {"name": "norm both gated ragged f32", "op": "norm", "batch": 3, "seq": 1037, "dim": 1001, "gain": True,
         "block_norm": True, "gate": "channel", "x_scale": 0.9, "block_scale": 0.5, "type": "f32",
         "layout": "packed"},
        # The backward pass between two blocks, on the microbatch.
        {"name": "norm grad microbatch bf16", "op": "norm_grad", "batch": 4, "seq": 4096, "dim": 2048, "gain": True,
         "block_norm": False, "gate": "none", "x_scale": 1.0, "block_scale": 1.0, "type": "bf16", "layout": "plain"},
        # The FP32 replay of a step with both norms and a learned gate for each channel.
        {"name": "norm grad both gated f32", "op": "norm_grad", "batch": 4, "seq": 2048, "dim": 2048, "gain": True,
         "block_norm": True, "gate": "channel", "x_scale": 1.0, "block_scale": 0.7, "type": "f32",
         "layout": "plain"},
        # A short batch of odd sizes, a gate for each element (another projection's output), tokens before the batch.
        {"name": "norm grad gated ragged bf16", "op": "norm_grad", "batch": 5, "seq": 333, "dim": 1111, "gain": True,
         "block_norm": True, "gate": "element", "x_scale": 1.0, "block_scale": 1.0, "type": "bf16",
         "layout": "seq_first"},
        # A single token scored against the whole vocabulary of the pages' model.
        {"name": "loss one token bf16", "op": "loss", "tokens": 1, "dim": 2048, "vocab": 128256, "ignored": 0.0,
         "z_weight": 0.0, "weighted": False, "type": "bf16", "padded": False},
        # The microbatch of the pages' model with its z-loss.
        {"name": "loss microbatch bf16", "op": "loss", "tokens": 16384, "dim": 2048, "vocab": 128256, "ignored": 0.0,
         "z_weight": 1e-4, "weighted": False, "type": "bf16", "padded": False},
        # Odd sizes in FP32, padded tokens whose labels are ignored, rows wider than the width.
        {"name": "loss ragged f32", "op": "loss", "tokens": 517, "dim": 1001, "vocab": 32003, "ignored": 0.2,
         "z_weight": 1e-4, "weighted": False, "type": "f32", "padded": True},
        # The gradients of the microbatch: the largest.
        {"name": "loss grad microbatch bf16", "op": "loss_grad", "tokens": 16384, "dim": 2048, "vocab": 128256,
         "ignored": 0.0, "z_weight": 1e-4, "weighted": False, "type": "bf16", "padded": False},
        # Half a window in the FP32 replay of a step, every token with a weight of its own.
        {"name": "loss grad f32", "op": "loss_grad", "tokens": 2048, "dim": 2048, "vocab": 128256, "ignored": 0.1,
         "z_weight": 0.0, "weighted": True, "type": "f32", "padded": False},
        # A short batch of odd sizes with padding over a smaller vocabulary.
        {"name": "loss grad ragged bf16", "op": "loss_grad", "tokens": 333, "dim": 1111, "vocab": 49999,
         "ignored": 0.2, "z_weight": 1e-4, "weighted": True, "type": "bf16", "padded": True},
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "norm_grad", "loss", "loss_grad", "loss_grad"])
    kind = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("loss"):
        dim = rng.choice([64 * _spread(rng, 4, 64), _spread(rng, 100, 4096)])
        vocab = rng.choice([128256, _spread(rng, 500, 200000)])
        # FP32 costs six times the products of BF16: an eighth of the tokens.
        most = 16384 * 2048 * 128256 // (dim * vocab * (8 if kind == "f32" else 1))
        return {"op": op, "tokens": _spread(rng, 1, min(16384, max(1, most))), "dim": dim, "vocab": vocab,
                "ignored": rng.choice([0.0, 0.0, 0.1, 0.5]), "z_weight": rng.choice([0.0, 1e-4, 1e-3]),
                "weighted": rng.random() < 0.5, "type": kind, "padded": rng.random() < 0.3}
    dim = rng.choice([64 * _spread(rng, 2, 128), _spread(rng, 50, 8192)])
    tokens = _spread(rng, 1, min(65536, 16384 * 2048 // (dim * (2 if kind == "f32" else 1))))
    batch = min(tokens, _spread(rng, 1, 64))
    block_norm = rng.random() < 0.5
    return {"op": op, "batch": batch, "seq": tokens // batch, "dim": dim, "gain": rng.random() < 0.7,
            "block_norm": block_norm, "gate": rng.choice(["none", "channel", "element"]),
            "x_scale": rng.choice([1.0, 1.0, 0.9]), "block_scale": rng.choice([1.0, 1.0, 0.5]), "type": kind,
            "layout": rng.choice(["plain", "packed", "seq_first"])}


def _rows(case, count):
    """`count` empty tensors (batch, seq, dim) in the case's layout of memory."""
    b, s, d, t = case["batch"], case["seq"], case["dim"], TYPES[case["type"]]
    if case["layout"] == "packed":
        return list(torch.empty(b, s, count * d, dtype=t, device=DEVICE).split(d, dim=-1))
    if case["layout"] == "seq_first":
        return [torch.empty(s, b, d, dtype=t, device=DEVICE).transpose(0, 1) for _ in range(count)]
    return [torch.empty(b, s, d, dtype=t, device=DEVICE) for _ in range(count)]


def _prepare_norm(case, gen):
    def normal(t, std, mean=0.0):
        return t.copy_(torch.randn(t.shape, generator=gen, device=DEVICE) * std + mean)

    def channel(std, mean, kind=TYPES[case["type"]]):
        return normal(torch.empty(case["dim"], dtype=kind, device=DEVICE), std, mean)

    state = {"case": case, "gain": channel(0.1, 1.0) if case["gain"] else None,
             "block_gain": channel(0.1, 1.0) if case["gain"] and case["block_norm"] else None, "gate": None}
    x, u = _rows(case, 2)
    state["x"], state["block"] = normal(x, 2.0), normal(u, 0.6)
    if case["gate"] == "channel":
        state["gate"] = channel(0.2, 0.5)
    elif case["gate"] == "element":
        state["gate"] = normal(_rows(case, 1)[0], 0.3, 0.5)
    if case["op"] == "norm_grad":
        # What the forward pass leaves behind: the sum, here of values like its own.
        state["y"] = state.pop("x")
        dy, dz = _rows(case, 2)
        state["dy"], state["dz"] = normal(dy, 1e-3), normal(dz, 1e-3)
    state["out"] = _rows(case, 2)  # where a program keeps the results
    return state


def _prepare_loss(case, gen):
    n, d, v, t = case["tokens"], case["dim"], case["vocab"], TYPES[case["type"]]
    wide = d + (13 if case["padded"] else 0)  # rows that are a part of wider ones
    w = (torch.randn(v, wide, generator=gen, device=DEVICE) * (0.9 / math.sqrt(d))).to(t)[:, :d]
    labels = torch.randint(v, (n,), generator=gen, device=DEVICE)
    # Hidden states that lean towards their labels, from not at all to certainty.
    lean = torch.rand(n, 1, generator=gen, device=DEVICE) * 16
    x = torch.empty(n, wide, dtype=t, device=DEVICE)[:, :d]
    x.copy_(torch.randn(n, d, generator=gen, device=DEVICE) + lean * w[labels].float())
    labels[torch.rand(n, generator=gen, device=DEVICE) < case["ignored"]] = IGNORED
    state = {"case": case, "x": x, "weight": w, "labels": labels}
    if case["op"] == "loss_grad":
        # The mean over the tokens that count, or weights of their own; the forward pass has left its statistics.
        counted = (labels != IGNORED).sum().clamp(min=1)
        state["dloss"] = torch.rand(n, generator=gen, device=DEVICE) / counted if case["weighted"] else 1.0 / counted
        state["lse"] = torch.empty(n, device=DEVICE)
        for first in range(0, n, 2048):  # prepared in 64 bits, so that both sides start from the same statistics
            part = slice(first, first + 2048)
            logits = x[part].double() @ w.double().T
            state["lse"][part] = logits.logsumexp(-1)
    return state


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    return _prepare_loss(case, gen) if case["op"].startswith("loss") else _prepare_norm(case, gen)


def _root(v):
    return torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)


def _after(state):
    """The block's output after its norm, and the norm's parts, in 32 bits."""
    u = state["block"].float()
    if not state["case"]["block_norm"]:
        return u, None, None
    root = _root(u)
    n = u * root
    return (n if state["block_gain"] is None else n * state["block_gain"].float()), n, root


def _plain_norm(state):
    case = state["case"]
    t = _after(state)[0]
    if state["gate"] is not None:
        t = t * state["gate"].float()
    kind = state["x"].dtype
    y = (state["x"].float() * case["x_scale"] + t * case["block_scale"]).to(kind)
    z = y.float() * _root(y.float())
    if state["gain"] is not None:
        z = z * state["gain"].float()
    return {"y": y, "z": z.to(kind)}


def _norm_back(n, root, dz, gain):
    """Gradients of n * gain at the normed input and at the gain."""
    dn = dz if gain is None else dz * gain.float()
    dgain = None if gain is None else (dz * n).sum((0, 1))
    return (dn - n * (dn * n).mean(-1, keepdim=True)) * root, dgain


def _plain_norm_grad(state):
    case, kind, outs = state["case"], state["y"].dtype, {}
    y = state["y"].float()
    root = _root(y)
    through, outs["dgain"] = _norm_back(y * root, root, state["dz"].float(), state["gain"])
    total = state["dy"].float() + through
    outs["dx"] = (total * case["x_scale"]).to(kind)
    p, n, root = _after(state)
    dt = total * case["block_scale"]
    dp = dt if state["gate"] is None else dt * state["gate"].float()
    if case["gate"] == "channel":
        outs["dgate"] = (dt * p).sum((0, 1))
    elif case["gate"] == "element":
        outs["dgate"] = (dt * p).to(kind)
    if case["block_norm"]:
        dp, outs["dblock_gain"] = _norm_back(n, root, dp, state["block_gain"])
    outs["dblock"] = dp.to(kind)
    return {name: t for name, t in outs.items() if t is not None}


def _plain_loss(state):
    case, labels = state["case"], state["labels"]
    logits = state["x"].float() @ state["weight"].float().T
    most = logits.amax(-1)
    counted = labels != IGNORED
    picked = logits.gather(1, labels.clamp(min=0)[:, None])[:, 0]
    lse = most + (logits - most[:, None]).exp_().sum(-1).log()
    loss = lse - picked + case["z_weight"] * lse.square()
    return {"loss": torch.where(counted, loss, 0.0), "lse": lse}


def _plain_loss_grad(state):
    case, labels, lse = state["case"], state["labels"], state["lse"]
    x, w = state["x"].float(), state["weight"].float()
    dlogits = (x @ w.T).sub_(lse[:, None]).exp_().mul_((1 + 2 * case["z_weight"] * lse)[:, None])
    dlogits[torch.arange(len(labels), device=DEVICE), labels.clamp(min=0)] -= 1.0
    dlogits *= torch.where(labels != IGNORED, state["dloss"], 0.0)[:, None]
    return {"dx": (dlogits @ w).to(state["x"].dtype), "dweight": (dlogits.T @ x).to(state["weight"].dtype)}


def _plain(state):
    return {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "loss": _plain_loss,
            "loss_grad": _plain_loss_grad}[state["case"]["op"]](state)


def _own(state):
    import bitwise_reproducible_amd as br
    case = state["case"]
    if case["op"] == "loss":
        loss, lse = br.repro_vocab_loss(state["x"], state["weight"], state["labels"], z_weight=case["z_weight"],
                                        ignore_index=IGNORED)
        return {"loss": loss, "lse": lse}
    if case["op"] == "loss_grad":
        dx, dweight = br.repro_vocab_loss_backward(state["x"], state["weight"], state["labels"], state["lse"],
                                                   state["dloss"], z_weight=case["z_weight"], ignore_index=IGNORED)
        return {"dx": dx, "dweight": dweight}
    form = {"gain": state["gain"], "block_gain": state["block_gain"], "gate": state["gate"],
            "block_norm": case["block_norm"], "x_scale": case["x_scale"], "block_scale": case["block_scale"],
            "eps": EPS}
    if case["op"] == "norm":
        y, z = br.repro_residual_norm(state["x"], state["block"], y=state["out"][0], out=state["out"][1], **form)
        return {"y": y, "z": z}
    plain_sum = not case["block_norm"] and case["gate"] == "none" and case["x_scale"] == case["block_scale"]
    dx, dblock, dgain, dblock_gain, dgate = br.repro_residual_norm_backward(
        state["y"], state["block"], state["dy"], state["dz"], dx=state["out"][0],
        dblock=None if plain_sum else state["out"][1], **form)
    outs = {"dgain": dgain, "dx": dx, "dgate": dgate, "dblock_gain": dblock_gain, "dblock": dblock}
    return {name: t for name, t in outs.items() if t is not None}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    """Every input read once and every output written once; operations as the formulas have them."""
    size = 2 if case["type"] == "bf16" else 4
    if case["op"].startswith("loss"):
        n, d, v = case["tokens"], case["dim"], case["vocab"]
        if case["op"] == "loss":
            return {"bytes": (n + v) * d * size + 16 * n, "flops": 2 * n * d * v + 3 * n * v}
        return {"bytes": 2 * (n + v) * d * size + 16 * n, "flops": 6 * n * d * v + 5 * n * v}
    elements = case["batch"] * case["seq"] * case["dim"]
    full = case["gate"] == "element"
    if case["op"] == "norm":
        return {"bytes": (4 + full) * elements * size, "flops": (8 + 4 * case["block_norm"]) * elements}
    # The block's output is read, and a gradient of its own written, only where they differ from the stream's.
    apart = case["block_norm"] or case["gate"] != "none"
    scaled = apart or case["x_scale"] != case["block_scale"]
    return {"bytes": (4 + apart + scaled + 2 * full) * elements * size, "flops": (12 + 12 * apart) * elements}


def _exact_norm(state):
    case = state["case"]
    wide = {name: state[name].double() for name in ("x", "y", "block", "gain", "block_gain", "gate", "dy", "dz")
            if state.get(name) is not None}

    def scale_of(v):
        return 1.0 / (torch.linalg.vector_norm(v, dim=-1, keepdim=True).pow(2) / case["dim"] + EPS).sqrt()

    u, gate = wide["block"], wide.get("gate", 1.0)
    gain, block_gain = wide.get("gain", 1.0), wide.get("block_gain", 1.0)
    at = scale_of(u) if case["block_norm"] else 1.0
    after = u * at * (block_gain if case["block_norm"] else 1.0)
    if case["op"] == "norm":
        y = case["x_scale"] * wide["x"] + case["block_scale"] * gate * after
        # The norm is that of the sum as it is stored; where the sum sits on the border of two stored values, that of
        # either is.
        stored = y.to(state["x"].dtype).double()
        return {"y": y, "z": stored * scale_of(stored) * gain}
    y, dz = wide["y"], wide["dz"]
    r = scale_of(y)
    dn = dz * gain
    total = wide["dy"] + dn * r - y * r.pow(3) * (dn * y).sum(-1, keepdim=True) / case["dim"]
    outs = {"dgain": (dz * y * r).flatten(0, 1).sum(0) if case["gain"] else None, "dx": case["x_scale"] * total}
    dt = case["block_scale"] * total
    if case["gate"] != "none":
        outs["dgate"] = (dt * after).flatten(0, 1).sum(0) if case["gate"] == "channel" else dt * after
    dp = dt * gate
    if case["block_norm"]:
        if "block_gain" in wide:
            outs["dblock_gain"] = (dp * u * at).flatten(0, 1).sum(0)
        dn = dp * block_gain
        dp = dn * at - u * at.pow(3) * (dn * u).sum(-1, keepdim=True) / case["dim"]
    outs["dblock"] = dp
    return {name: t for name, t in outs.items() if t is not None}


def _exact_loss(state):
    """In blocks of tokens, from torch's own softmax in 64 bits."""
    case, labels = state["case"], state["labels"]
    w = state["weight"].double()
    outs = {name: [] for name in (("loss", "lse") if case["op"] == "loss" else ("dx",))}
    dweight = torch.zeros_like(w)
    for first in range(0, case["tokens"], 1024):
        part = slice(first, first + 1024)
        x, label = state["x"][part].double(), labels[part]
        counted = label != IGNORED
        logits = x @ w.T
        if case["op"] == "loss":
            lse = torch.logsumexp(logits, -1)
            nll = torch.nn.functional.cross_entropy(logits, label, ignore_index=IGNORED, reduction="none")
            outs["loss"].append(nll + counted * case["z_weight"] * lse * lse)
            outs["lse"].append(lse)
            continue
        lse = state["lse"][part].double()
        factor = state["dloss"].double().expand(case["tokens"])[part] * counted
        prob = torch.exp(logits - lse[:, None]) * (1 + 2 * case["z_weight"] * lse)[:, None]
        prob.scatter_add_(1, label.clamp(min=0)[:, None], -torch.ones_like(prob[:, :1]))
        prob *= factor[:, None]
        outs["dx"].append(prob @ w)
        dweight += prob.T @ x
    outs = {name: torch.cat(parts) for name, parts in outs.items()}
    return outs if case["op"] == "loss" else {**outs, "dweight": dweight}


def exact(case, seed):
    """run()'s outputs from the definitions in 64 bits."""
    state = prepare(case, seed)
    return _exact_loss(state) if case["op"].startswith("loss") else _exact_norm(state)
