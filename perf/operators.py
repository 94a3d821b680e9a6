"""Cases of the operators around one attention layer and one optimizer step, for timing and comparison.

Operators: the rotation table of the positions (``table``), the norm of every query and key head with the
position rotation (``heads``), its backward pass (``heads_grad``), and the global l2 norm of a model's gradient
tensors with clipping (``clip``).  ``own`` chooses between the framework's calls and the plain form of the same
formulas in elementary torch operations.

Formulas, for one head x of D elements (rotary dimension R <= D, both even, h = R/2):
    r = 1 / sqrt(mean(x^2) + eps)     n = x r     z = n * gain (or n)
    pair (a, b) = (z[i], z[i + h]), or (z[2i], z[2i + 1]) when interleaved, for i < h:
    y_a = a cos - b sin               y_b = b cos + a sin           z[R..D) passes unchanged
backward of it for an upstream gradient dy:
    dz = the rotation by the negative angle of dy
    dgain = sum over batch, tokens and heads of dz * n
    dn = dz * gain (or dz)            dx = (dn - n mean(dn * n)) r
table:  angle = position * inv_freq[i];  cos(angle), sin(angle)
clip:   norm = sqrt(sum over all tensors of g^2);  c = min(1, max_norm / (norm + 1e-6));  out = c g
"""
import math

import torch

own = False

DEVICE = "cuda"
EPS = 1e-6
THETA = 5e5  # the rotation base of the pages' model
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # One step of generation: a single token at a far position, the pages' 16 query and 4 key heads of 128.
        {"name": "heads one token bf16", "op": "heads", "batch": 1, "seq": 1, "q_heads": 16, "k_heads": 4, "dim": 128,
         "rotary": 128, "interleaved": False, "gain": False, "type": "bf16", "layout": "packed", "given": True,
         "far": 4095},
        # The pages' microbatch, 4 windows of 4096 tokens, queries and keys side by side in one projection's output.
        {"name": "heads microbatch bf16", "op": "heads", "batch": 4, "seq": 4096, "q_heads": 16, "k_heads": 4,
         "dim": 128, "rotary": 128, "interleaved": False, "gain": False, "type": "bf16", "layout": "packed",
         "given": False, "far": 0},
        # Odd sizes in FP32: learned gains, a part of each head rotated in interleaved pairs, heads before tokens.
        {"name": "heads ragged f32", "op": "heads", "batch": 3, "seq": 1037, "q_heads": 12, "k_heads": 4, "dim": 80,
         "rotary": 64, "interleaved": True, "gain": True, "type": "f32", "layout": "heads_first", "given": True,
         "far": 700},
        # The backward pass of the microbatch, into one packed gradient that the weight gradient's product reads.
        {"name": "heads grad microbatch bf16", "op": "heads_grad", "batch": 4, "seq": 4096, "q_heads": 16,
         "k_heads": 4, "dim": 128, "rotary": 128, "interleaved": False, "gain": False, "type": "bf16",
         "layout": "packed", "given": False, "far": 0},
        # FP32 replay of a step (batch 4 x 2048 tokens) with learned gains and their gradients.
        {"name": "heads grad gains f32", "op": "heads_grad", "batch": 4, "seq": 2048, "q_heads": 16, "k_heads": 4,
         "dim": 128, "rotary": 128, "interleaved": False, "gain": True, "type": "f32", "layout": "plain",
         "given": False, "far": 0},
        # Odd sizes: one key head shared by seven query heads, half of each head rotated, gains, a short batch.
        {"name": "heads grad ragged bf16", "op": "heads_grad", "batch": 5, "seq": 333, "q_heads": 7, "k_heads": 1,
         "dim": 96, "rotary": 48, "interleaved": False, "gain": True, "type": "bf16", "layout": "heads_first",
         "given": True, "far": 100},
        # The norm gains of the pages' model alone (two per layer and the last): latency counts.
        {"name": "clip gains f32", "op": "clip", "tensors": "gains", "layers": 24, "width": 2048, "ffn": 5632,
         "vocab": 0, "shard": 1, "type": "f32", "tight": False, "max_norm": 1.0},
        # One rank's FP32 shard of the pages' model, an eighth of every tensor.
        {"name": "clip shard f32", "op": "clip", "tensors": "model", "layers": 24, "width": 2048, "ffn": 5632,
         "vocab": 128256, "shard": 8, "type": "f32", "tight": False, "max_norm": 1.0},
        # All of the pages' model (1.61e9 parameters) in BF16: the largest.
        {"name": "clip model bf16", "op": "clip", "tensors": "model", "layers": 24, "width": 2048, "ffn": 5632,
         "vocab": 128256, "shard": 1, "type": "bf16", "tight": False, "max_norm": 1.0},
        # Odd sizes of both types, laid out without padding, so that most tensors start off any vector's border.
        {"name": "clip ragged mixed", "op": "clip", "tensors": "ragged", "layers": 113, "width": 999, "ffn": 700001,
         "vocab": 0, "shard": 1, "type": "mixed", "tight": True, "max_norm": 0.5},
        # The table of one 4096-token window, and that of a long context read from far positions on.
        {"name": "table 4096", "op": "table", "length": 4096, "start": 0, "rotary": 128, "theta": THETA},
        {"name": "table 131072 far", "op": "table", "length": 131072, "start": 1 << 20, "rotary": 128,
         "theta": THETA},
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["heads", "heads", "heads_grad", "heads_grad", "clip", "clip", "table"])
    if op == "table":
        return {"op": op, "length": _spread(rng, 1, 131072), "start": rng.choice([0, _spread(rng, 1, 1 << 20)]),
                "rotary": 2 * _spread(rng, 1, 64), "theta": rng.choice([1e4, THETA])}
    if op == "clip":
        if rng.random() < 0.5:
            return {"op": op, "tensors": "ragged", "layers": _spread(rng, 1, 600), "width": _spread(rng, 1, 2500),
                    "ffn": _spread(rng, 2500, 1000000), "vocab": 0, "shard": 1,
                    "type": rng.choice(["f32", "bf16", "mixed"]), "tight": rng.random() < 0.5,
                    "max_norm": rng.choice([0.1, 0.5, 1.0, 1e4])}
        width = 64 * _spread(rng, 1, 32)
        return {"op": op, "tensors": "model", "layers": _spread(rng, 1, 24), "width": width,
                "ffn": width * rng.randint(5, 11) // 4, "vocab": _spread(rng, 256, 128256),
                "shard": rng.choice([1, 2, 8]), "type": rng.choice(["f32", "bf16"]) if width <= 1024 else "bf16",
                "tight": False, "max_norm": rng.choice([0.1, 1.0, 1.0, 1e4])}
    dim = rng.choice([64, 80, 96, 128, 128, 256, 2 * _spread(rng, 8, 128)])
    rotary = dim if rng.random() < 0.7 else 2 * rng.randint(1, dim // 2)
    k_heads = rng.choice([1, 2, 4, 5, 8])
    q_heads = k_heads * rng.choice([1, 2, 3, 4, 7, 8])
    most = 16384 * 20 * 128 // ((q_heads + k_heads) * dim)
    tokens = _spread(rng, 1, min(most, 65536))
    batch = min(tokens, _spread(rng, 1, 64))
    return {"op": op, "batch": batch, "seq": tokens // batch, "q_heads": q_heads, "k_heads": k_heads, "dim": dim,
            "rotary": rotary, "interleaved": rng.random() < 0.3, "gain": rng.random() < 0.5,
            "type": rng.choice(["bf16", "bf16", "f32"]), "layout": rng.choice(["packed", "plain", "heads_first"]),
            "given": rng.random() < 0.5, "far": _spread(rng, 1, 4096)}


def _sizes(case):
    """Elements and type of every gradient tensor of a clip case."""
    if case["tensors"] == "ragged":
        # A fixed walk over odd sizes between 1 and ffn; every third tensor is large, the others small.
        sizes, x = [], case["width"] * 2 + 1
        for i in range(case["layers"]):
            x = (x * 48271 + 11) % 2147483647
            sizes.append(1 + x % (case["ffn"] if i % 3 == 0 else case["width"]))
    else:
        w, f = case["width"], case["ffn"]
        layer = [w, w] if case["tensors"] == "gains" else [w, w, w * w, w * w // 4, w * w // 4, w * w, w * f, w * f, f * w]
        sizes = layer * case["layers"] + [w] + [w * case["vocab"]] * (2 if case["vocab"] else 0)
        sizes = [-(-s // case["shard"]) for s in sizes]
    kinds = [case["type"] if case["type"] != "mixed" else ("bf16", "f32")[i % 2] for i in range(len(sizes))]
    return list(zip(sizes, kinds))


def _views(sizes, tight):
    """One flat buffer for each type and every tensor's view of it, padded to 16 bytes unless tight."""
    starts, total = [], {"f32": 0, "bf16": 0}
    for n, kind in sizes:
        starts.append(total[kind])
        total[kind] += n if tight else -(-n // 8) * 8
    flat = {kind: torch.zeros(n, dtype=TYPES[kind], device=DEVICE) for kind, n in total.items() if n}
    return flat, [flat[kind][s:s + n] for (n, kind), s in zip(sizes, starts)]


def _head_views(case, kind):
    """Empty q and k (batch, seq, heads, dim) in the case's layout of memory."""
    b, s, hq, hk, d = case["batch"], case["seq"], case["q_heads"], case["k_heads"], case["dim"]
    if case["layout"] == "packed":
        both = torch.empty(b, s, hq + hk, d, dtype=TYPES[kind], device=DEVICE)
        return both[:, :, :hq], both[:, :, hq:]
    if case["layout"] == "heads_first":
        return tuple(torch.empty(b, h, s, d, dtype=TYPES[kind], device=DEVICE).transpose(1, 2) for h in (hq, hk))
    return tuple(torch.empty(b, s, h, d, dtype=TYPES[kind], device=DEVICE) for h in (hq, hk))


def _normal(t, gen, std):
    """Fills t with normal values (in place, from the generator alone)."""
    return t.copy_(torch.randn(t.shape, generator=gen, device=DEVICE) * std)


def _inv_freq(rotary, theta):
    return theta ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device=DEVICE) / rotary)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    state = {"case": case}
    if case["op"] == "table":
        # A user's frequencies: the usual powers, scaled a little as long-context recipes do.
        scale = 1 + 0.01 * torch.rand(case["rotary"] // 2, generator=gen, device=DEVICE, dtype=torch.float64)
        state["inv_freq"] = _inv_freq(case["rotary"], case["theta"]) * scale
        return state
    if case["op"] == "clip":
        sizes = _sizes(case)
        flat, state["grads"] = _views(sizes, case["tight"])
        for t in flat.values():
            # Gradients of the usual size with a few far larger ones; zero padding would be part of no tensor.
            for part in t.split(1 << 28):
                _normal(part, gen, 1e-3)
            t[torch.randint(t.numel(), (1 + t.numel() // 1000,), generator=gen, device=DEVICE)] *= 300.0
        state["flat"], state["outs"] = _views(sizes, case["tight"])
        if own:
            # The list's handle, which a training program makes once for its buffers.
            import bitwise_reproducible_amd as br
            state["list"] = br.GradList(state["grads"], outs=state["outs"])
        return state
    q, k = _head_views(case, case["type"])
    state["q"], state["k"] = _normal(q, gen, 1.5), _normal(k, gen, 0.7)
    length = case["far"] + case["seq"] + 1
    angle = torch.arange(length, dtype=torch.float64, device=DEVICE)[:, None] * _inv_freq(case["rotary"], THETA)
    state["cos"], state["sin"] = angle.cos().float(), angle.sin().float()
    state["positions"] = None
    if case["given"]:
        first = torch.randint(0, case["far"] + 1, (case["batch"], 1), generator=gen, device=DEVICE)
        state["positions"] = (first + torch.arange(case["seq"], device=DEVICE)).to(torch.int32)
    state["q_gain"] = state["k_gain"] = None
    if case["gain"]:
        for name in ("q_gain", "k_gain"):
            state[name] = (1 + 0.1 * torch.randn(case["dim"], generator=gen, device=DEVICE)).to(TYPES[case["type"]])
    state["q_out"], state["k_out"] = _head_views(case, case["type"])
    if case["op"] == "heads_grad":
        dq, dk = _head_views(dict(case, layout="heads_first"), case["type"])
        state["dq_out"], state["dk_out"] = _normal(dq, gen, 1e-2), _normal(dk, gen, 1e-2)
    return state


def _turn(x, cos, sin, interleaved):
    """The rotation of the first 2 * cos.shape[-1] elements of every head; the others pass."""
    h = cos.shape[-1]
    if interleaved:
        a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = x[..., :h], x[..., h:2 * h]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((turned, x[..., 2 * h:]), dim=-1) if 2 * h < x.shape[-1] else turned


def _angles(state):
    where = state["positions"]
    if where is None:
        where = torch.arange(state["case"]["seq"], device=DEVICE)[None]
    where = where.long()
    return state["cos"][where][:, :, None], state["sin"][where][:, :, None]


def _heads(x, gain, cos, sin, interleaved):
    x32 = x.float()
    n = x32 * torch.rsqrt(x32.square().mean(-1, keepdim=True) + EPS)
    z = n if gain is None else n * gain.float()
    return _turn(z, cos, sin, interleaved).to(x.dtype)


def _heads_grad(x, dy, gain, cos, sin, interleaved):
    x32 = x.float()
    r = torch.rsqrt(x32.square().mean(-1, keepdim=True) + EPS)
    n = x32 * r
    dz = _turn(dy.float(), cos, -sin, interleaved)
    dgain = None if gain is None else (dz * n).sum((0, 1, 2))
    dn = dz if gain is None else dz * gain.float()
    return ((dn - n * (dn * n).mean(-1, keepdim=True)) * r).to(x.dtype), dgain


def _plain(state):
    case = state["case"]
    if case["op"] == "table":
        at = torch.arange(case["start"], case["start"] + case["length"], dtype=torch.float64, device=DEVICE)
        angle = at[:, None] * state["inv_freq"]
        return {"cos": angle.cos().float(), "sin": angle.sin().float()}
    if case["op"] == "clip":
        squares = torch.stack([g.float().square().sum(dtype=torch.float64) for g in state["grads"]])
        norm = squares.sum().sqrt()
        coef = (case["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
        [o.copy_(g.float() * coef) for g, o in zip(state["grads"], state["outs"])]
        return {"norm": norm.float(), "coef": coef, "flat": state["flat"]}
    cos, sin = _angles(state)
    if case["op"] == "heads":
        return {x: _heads(state[x], state[x + "_gain"], cos, sin, case["interleaved"]) for x in ("q", "k")}
    dq, dq_gain = _heads_grad(state["q"], state["dq_out"], state["q_gain"], cos, sin, case["interleaved"])
    dk, dk_gain = _heads_grad(state["k"], state["dk_out"], state["k_gain"], cos, sin, case["interleaved"])
    return {"dq": dq, "dk": dk} | ({"dq_gain": dq_gain, "dk_gain": dk_gain} if case["gain"] else {})


def _own(state):
    import bitwise_reproducible_amd as br
    case = state["case"]
    if case["op"] == "table":
        cos, sin = br.repro_rope_table(state["inv_freq"], case["length"], start=case["start"])
        return {"cos": cos, "sin": sin}
    if case["op"] == "clip":
        norm = br.repro_clip_grad_list(state["list"], case["max_norm"])
        return {"norm": norm[0], "coef": norm[2], "flat": state["flat"]}
    if case["op"] == "heads":
        q, k = br.repro_qk_norm_rope(state["q"], state["k"], state["cos"], state["sin"], positions=state["positions"],
                                     q_gain=state["q_gain"], k_gain=state["k_gain"], eps=EPS,
                                     interleaved=case["interleaved"], q_out=state["q_out"], k_out=state["k_out"])
        return {"q": q, "k": k}
    dq, dk, dq_gain, dk_gain = br.repro_qk_norm_rope_backward(
        state["q"], state["k"], state["dq_out"], state["dk_out"], state["cos"], state["sin"],
        positions=state["positions"], q_gain=state["q_gain"], k_gain=state["k_gain"], eps=EPS,
        interleaved=case["interleaved"], dq=state["q_out"], dk=state["k_out"])
    return {"dq": dq, "dk": dk} | ({"dq_gain": dq_gain, "dk_gain": dk_gain} if case["gain"] else {})


def run(state):
    return _own(state) if own else _plain(state)


def _sizeof(kind):
    return 2 if kind == "bf16" else 4


def work(case):
    """Every input read once and every output written once; operations as the formulas have them."""
    if case["op"] == "table":
        half = case["rotary"] // 2
        return {"bytes": 8 * half * case["length"] + 8 * half, "flops": 60 * half * case["length"]}
    if case["op"] == "clip":
        sizes = _sizes(case)
        return {"bytes": sum(2 * n * _sizeof(kind) for n, kind in sizes), "flops": 3 * sum(n for n, _ in sizes)}
    tokens = case["batch"] * case["seq"]
    elements = tokens * (case["q_heads"] + case["k_heads"]) * case["dim"]
    positions = tokens if case["given"] else case["seq"]  # rows of the table: at most one for each position
    table = 8 * (case["rotary"] // 2) * min(positions, case["far"] + case["seq"] + 1)
    moved, each = (2, 8) if case["op"] == "heads" else (3, 16)
    return {"bytes": moved * elements * _sizeof(case["type"]) + table, "flops": each * elements}


def exact(case, seed):
    """run()'s outputs from the definitions in 64 bits, element by element over pairs instead of halves."""
    state = prepare(case, seed)
    if case["op"] == "table":
        import numpy as np
        # 80-bit products and functions: the angle of a far position keeps 64 bits' accuracy after its reduction.
        f = state["inv_freq"].cpu().numpy().astype(np.longdouble)
        at = np.arange(case["start"], case["start"] + case["length"]).astype(np.longdouble)
        cos, sin = (np.empty((len(at), len(f))) for _ in range(2))
        for first in range(0, len(at), 8192):
            angle = at[first:first + 8192, None] * f
            cos[first:first + 8192], sin[first:first + 8192] = np.cos(angle), np.sin(angle)
        return {"cos": cos, "sin": sin}
    if case["op"] == "clip":
        total = 0.0
        for g in state["grads"]:
            for part in g.split(1 << 27):
                d = part.double()
                total += float(torch.dot(d, d))
        norm = math.sqrt(total)
        coef = min(1.0, case["max_norm"] / (norm + 1e-6))
        flat = {}
        for kind, f in state["flat"].items():
            flat[kind] = torch.zeros(f.numel(), dtype=torch.float64, device=DEVICE)
        seen = {kind: f.data_ptr() for kind, f in state["flat"].items()}
        for g, o in zip(state["grads"], state["outs"]):
            kind = "bf16" if g.dtype == torch.bfloat16 else "f32"
            at = (o.data_ptr() - seen[kind]) // o.element_size()
            flat[kind][at:at + o.numel()].copy_(g).mul_(coef)
        return {"norm": torch.tensor(norm, dtype=torch.float64), "coef": torch.tensor(coef, dtype=torch.float64),
                "flat": flat}
    rotary, dim = case["rotary"], case["dim"]
    half = rotary // 2
    i = torch.arange(half, device=DEVICE)
    first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
    outs = {}
    for x in ("q", "k"):
        v = state[x].double()
        where = state["positions"]
        if where is None:
            where = torch.arange(case["seq"], device=DEVICE).expand(case["batch"], -1)
        turn = torch.complex(state["cos"].double(), state["sin"].double())[where.long()].unsqueeze(2)
        gain = torch.ones(dim, dtype=torch.float64, device=DEVICE)
        if case["gain"]:
            gain = state[x + "_gain"].double()
        scale = 1.0 / (torch.linalg.vector_norm(v, dim=-1, keepdim=True).pow(2) / dim + EPS).sqrt()
        if case["op"] == "heads":
            out = v * scale * gain
            pair = torch.complex(out[..., first], out[..., second]) * turn
            out[..., first], out[..., second] = pair.real, pair.imag
            outs[x] = out
            continue
        dz = state["d%s_out" % x].double().clone(memory_format=torch.contiguous_format)
        pair = torch.complex(dz[..., first], dz[..., second]) * turn.conj()
        dz[..., first], dz[..., second] = pair.real, pair.imag
        if case["gain"]:
            outs["d%s_gain" % x] = (dz * v * scale).flatten(0, 2).sum(0)
        dn = dz * gain
        along = (dn * v).sum(-1, keepdim=True)
        outs["d" + x] = dn * scale - v * scale.pow(3) * along / dim
    return outs
