"""The layers around the products and the step's clipping, as measured cases.

What makes the gradients that are no linear layer's (an embedding's table, the
gains and gates of a block's norms), added into the fp32 accumulators of the
deferred reduction, and what happens to the reduced gradients before the
owner's update (their global norm, and clipping by it).

`own` False computes the plain form in elementary torch operations in 32
bits; True makes the framework's calls.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
MAX_NORM, CLIP_EPS = 1.0, 1e-6
NORM_EPS = 1e-6


def clip(name, shapes, dtype="f32"):
    """shapes: count*numel or count*rows x cols, joined by +."""
    return {"name": name, "op": "clip", "shapes": shapes, "dtype": dtype}


def lookup(name, T, V, D, dtype="bf16", pad=0.0, wide=True):
    """T tokens of a table [V, D]; `pad` of them outside it; ids in 64 bits if wide, else 32."""
    return {"name": name, "op": "embedding", "T": T, "V": V, "D": D, "dtype": dtype, "pad": pad, "wide": wide}


def lookup_backward(name, T, V, D, dtype="bf16", grad="f32", accumulate=True, pad=0.0, wide=True):
    return {"name": name, "op": "embedding_backward", "T": T, "V": V, "D": D, "dtype": dtype, "grad": grad,
            "accumulate": accumulate, "pad": pad, "wide": wide}


def norms(name, T, D, dtype="bf16", block=True, gates=0, scale=1.0, offset=0.0):
    """The norm after a block (with its gate rows, 0: none) and the norm before the next; without `block` the
    latter alone."""
    return {"name": name, "op": "norm", "T": T, "D": D, "dtype": dtype, "block": block, "gates": gates,
            "scale": scale, "offset": offset}


def norms_backward(name, T, D, dtype="bf16", block=True, gates=0, scale=1.0, offset=0.0, grad="f32",
                   accumulate=True):
    return {"name": name, "op": "norm_backward", "T": T, "D": D, "dtype": dtype, "block": block, "gates": gates,
            "scale": scale, "offset": offset, "grad": grad, "accumulate": accumulate}


def listed():
    return [
        # the reduced gains of a hidden-1024 model's norms alone: many small vectors, latency
        clip("clip_gains", "57*1024+56*128"),
        # an owner's share of that model, reduced in bf16
        clip("clip_owner", "16*1024+32*1024x1024+8*4096x1024+8*1024x4096", "bf16"),
        # the whole model with its 151936 x 1024 embedding, reduced in fp32
        clip("clip_model", "1*151936x1024+39*1024+76*1024x1024+19*1024x4096+19*4096x1024"),
        # the next token of one sequence
        lookup("embedding_token", 1, 151936, 1024),
        # a training micro-batch of eight sequences, scaled by the square root of the width
        lookup("embedding_batch", 8 * 4096, 151936, 1024),
        # that micro-batch's gradient, added to a replica's accumulators
        lookup_backward("embedding_backward_batch", 8 * 4096, 151936, 1024),
        # a shorter batch of a 7B-class model, its table's gradient written anew
        lookup_backward("embedding_backward_7b", 8192, 32000, 4096, accumulate=False),
        # odd sizes in fp32, sequences padded to one length
        lookup_backward("embedding_backward_odd_f32", 1511, 5003, 515, "f32", pad=0.2, wide=False),
        # one token between two blocks of the 7B-class model
        norms("norm_token", 1, 4096),
        # a training batch there, the block's output scaled for its depth
        norms("norm_batch_7b", 8192, 4096, scale=0.25),
        # the gradient of that batch, with a gate for every channel, added to the accumulators
        norms_backward("norm_backward_7b", 8192, 4096, gates=1, scale=0.25),
        # odd sizes in fp32, a gate row for each of seven sequences, gains about one
        norms_backward("norm_backward_odd_f32", 777, 1003, "f32", gates=7, offset=1.0, accumulate=False),
    ]


def _size(rng, lo, hi):
    """Spread over the logarithm; every other one odd-sized."""
    v = int(round(lo * (hi / lo) ** rng.random()))
    if rng.random() < 0.5:
        v = v // 64 * 64 if v >= 128 else v
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["clip", "embedding", "embedding_backward", "norm", "norm_backward"])
    dtype = "f32" if rng.random() < 0.4 else "bf16"
    grad = "bf16" if dtype == "bf16" and rng.random() < 0.3 else "f32"
    if op == "clip":
        groups, left = [], 200_000_000
        for _ in range(rng.randint(1, 5)):
            n = min(_size(rng, 1, 20_000_000), max(1, left))
            count = rng.randint(1, max(1, min(60, left // n)))
            left -= n * count
            groups.append("%d*%d" % (count, n))
        c = clip("", "+".join(groups), dtype)
    elif op in ("embedding", "embedding_backward"):
        T, V, D = _size(rng, 1, 32768), _size(rng, 64, 151936), _size(rng, 16, 4096)
        while T * D > 32768 * 1024:
            T //= 2
        while V * D > 151936 * 1024:
            V //= 2
        pad, wide = rng.choice([0.0, 0.0, 0.1, 0.5]), rng.random() < 0.7
        if op == "embedding":
            c = lookup("", T, V, D, dtype, pad, wide)
        else:
            c = lookup_backward("", T, V, D, dtype, grad, rng.random() < 0.6, pad, wide)
    else:
        T, D = _size(rng, 1, 16384), _size(rng, 16, 8192)
        while T * D > 8192 * 4096:
            T //= 2
        gates = rng.choice([0, 1, 1, rng.randint(1, 12), T])
        T = max(1, T // gates) * gates if gates else T
        block, scale, offset = rng.random() < 0.8, rng.choice([1.0, 0.25, 0.5 ** 0.5]), rng.choice([0.0, 1.0])
        if op == "norm":
            c = norms("", T, D, dtype, block, gates if block else 0, scale, offset)
        else:
            c = norms_backward("", T, D, dtype, block, gates if block else 0, scale, offset, grad,
                               rng.random() < 0.6)
    del c["name"]
    return c


def _shapes(case):
    out = []
    for g in case["shapes"].split("+"):
        count, size = g.split("*")
        out += [tuple(int(v) for v in size.split("x"))] * int(count)
    return out


def _ids(gen, case):
    """Tokens by a natural text's frequencies (the k-th most frequent one's falls as 1 / k), anywhere in the
    table; padding at the end of the batch is -1."""
    T, V = case["T"], case["V"]
    u = torch.rand(T, device="cuda", generator=gen, dtype=torch.float64)
    rank = (torch.exp(u * math.log(V + 1)).long() - 1).clamp_(0, V - 1)
    step = next(p for p in (611953, 15485863, 32452843) if math.gcd(p, V) == 1)
    ids = rank * step % V
    if case["pad"]:
        ids[T - int(T * case["pad"]):] = -1
    return ids if case["wide"] else ids.int()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 17)
    dt = DTYPES[case["dtype"]]

    def randn(*shape, scale=1.0, dtype=dt, mean=0.0):
        return (torch.randn(*shape, device="cuda", generator=gen) * scale + mean).to(dtype)

    s = {"case": dict(case)}
    if case["op"] == "clip":
        # each tensor of its own size, as layers at different depths have
        s["grads"] = [randn(*shape, scale=1e-2 * 2.0 ** (k % 5 - 2)) for k, shape in enumerate(_shapes(case))]
        # the owner's flat partition, which the clipped gradients go to: every pass then clips the same ones
        s["flat"] = torch.zeros(sum(g.numel() for g in s["grads"]), dtype=dt, device="cuda")
        s["out"], at = [], 0
        for g in s["grads"]:
            s["out"].append(s["flat"][at:at + g.numel()].view(g.shape))
            at += g.numel()
        return s
    if case["op"] in ("embedding", "embedding_backward"):
        T, V, D = case["T"], case["V"], case["D"]
        s["ids"], s["scale"] = _ids(gen, case), D ** 0.5
        if case["op"] == "embedding":
            s["table"] = randn(V, D, scale=0.02)
        else:
            s["dy"] = randn(T, D, scale=1e-2)
            s["dtable"] = randn(V, D, scale=1e-2, dtype=DTYPES[case["grad"]])
        return s
    T, D = case["T"], case["D"]
    mean = 1.0 - case["offset"]
    s["gain"] = randn(D, scale=0.1, mean=mean)
    s["post_gain"], s["gate"], s["h"] = None, None, None
    if case["block"]:
        s["post_gain"], s["h"] = randn(D, scale=0.1, mean=mean), randn(T, D, scale=0.5)
        if case["gates"]:
            s["gate"] = randn(*((D,) if case["gates"] == 1 else (case["gates"], D)), scale=0.3, mean=0.5)
    if case["op"] == "norm":
        s["x"] = randn(T, D, scale=2.0)
        return s
    gt = DTYPES[case["grad"]]
    s["s"], s["dy"], s["ds"] = randn(T, D, scale=2.0), randn(T, D, scale=1e-2), randn(T, D, scale=1e-2)
    s["dgain"] = randn(D, scale=1e-2, dtype=gt)
    s["dpost_gain"] = randn(D, scale=1e-2, dtype=gt) if case["block"] else None
    s["dgate"] = randn(*s["gate"].shape, scale=1e-2, dtype=gt) if s["gate"] is not None else None
    return s


def _rms(v):
    return v / (v.square().mean(dim=-1, keepdim=True) + NORM_EPS).sqrt()


def _gate_rows(gate, T):
    """A row of the gate for every token."""
    if gate is None:
        return 1.0
    rows = gate.float().view(-1, gate.shape[-1])
    return rows.repeat_interleave(T // rows.shape[0], dim=0) if rows.shape[0] > 1 else rows


def _store(to, value, accumulate):
    to.copy_(to.float() + value.view(to.shape) if accumulate else value.view(to.shape))


def run(s):
    c = s["case"]
    if own:
        from gradient_reduction_amd import clip as clipping
        from gradient_reduction_amd import embedding, norm
        if c["op"] == "clip":
            return clipping.clip_grad_norm(s["grads"], MAX_NORM, eps=CLIP_EPS, out=s["out"]), s["flat"]
        if c["op"] == "embedding":
            return embedding.forward(s["ids"], s["table"], scale=s["scale"])
        if c["op"] == "embedding_backward":
            return embedding.backward(s["dy"], s["ids"], scale=s["scale"], dtable=s["dtable"],
                                      accumulate=c["accumulate"])
        if c["op"] == "norm":
            return norm.forward(s["x"], s["gain"], h=s["h"], post_gain=s["post_gain"], gate=s["gate"],
                                scale=c["scale"], offset=c["offset"], eps=NORM_EPS)
        return norm.backward(s["dy"], s["s"], s["gain"], ds=s["ds"], h=s["h"], post_gain=s["post_gain"],
                             gate=s["gate"], scale=c["scale"], offset=c["offset"], eps=NORM_EPS,
                             dgain=s["dgain"], dpost_gain=s["dpost_gain"], dgate=s["dgate"],
                             accumulate=c["accumulate"])

    dt = DTYPES[c["dtype"]]
    if c["op"] == "clip":
        squares = sum(g.float().square().sum(dtype=torch.float64) for g in s["grads"])
        norm_ = squares.sqrt()
        coef = (MAX_NORM / (norm_ + CLIP_EPS)).clamp(max=1.0).float()
        for g, o in zip(s["grads"], s["out"]):
            o.copy_(g.float() * coef)
        return norm_.float(), s["flat"]
    if c["op"] == "embedding":
        ids, inside = s["ids"].long(), (s["ids"] >= 0) & (s["ids"] < c["V"])
        rows = s["table"][ids.clamp(0, c["V"] - 1)].float() * s["scale"]
        return torch.where(inside[:, None], rows, torch.zeros_like(rows)).to(dt)
    if c["op"] == "embedding_backward":
        inside = (s["ids"] >= 0) & (s["ids"] < c["V"])
        total = s["dtable"].float() if c["accumulate"] else torch.zeros_like(s["dtable"], dtype=torch.float32)
        rows = s["dy"].float() * s["scale"] * inside[:, None]
        total.index_add_(0, s["ids"].long().clamp(0, c["V"] - 1), rows)
        if total is not s["dtable"]:
            s["dtable"].copy_(total)
        return s["dtable"]
    gain = s["gain"].float() + c["offset"]
    post = s["post_gain"].float() + c["offset"] if c["block"] else None
    gate = _gate_rows(s["gate"], c["T"])
    if c["op"] == "norm":
        if not c["block"]:
            return s["x"], (_rms(s["x"].float()) * gain).to(dt)
        total = s["x"].float() + c["scale"] * gate * (_rms(s["h"].float()) * post)
        return total.to(dt), (_rms(total) * gain).to(dt)

    def through(v, g):
        """A norm's gradient from g = that of its result, gain taken in."""
        r = 1 / (v.square().mean(dim=-1, keepdim=True) + NORM_EPS).sqrt()
        n = v * r
        return r * (g - n * (g * n).mean(dim=-1, keepdim=True)), n

    dy = s["dy"].float()
    d, n = through(s["s"].float(), dy * gain)
    d = d + s["ds"].float()
    _store(s["dgain"], (dy * n).sum(dim=0), c["accumulate"])
    if not c["block"]:
        return d.to(dt), None, s["dgain"], None, None
    du = c["scale"] * gate * d
    dh, n = through(s["h"].float(), du * post)
    _store(s["dpost_gain"], (du * n).sum(dim=0), c["accumulate"])
    if s["gate"] is not None:
        each = c["scale"] * d * (n * post)
        _store(s["dgate"], each.view(c["gates"], -1, c["D"]).sum(dim=1), c["accumulate"])
    return d.to(dt), dh.to(dt), s["dgain"], s["dpost_gain"], s["dgate"]


def _distinct(case):
    """Rows of the table that the tokens are expected to name."""
    T, V = case["T"] - int(case["T"] * case["pad"]), case["V"]
    k = torch.arange(1, V + 1, dtype=torch.float64)
    p = torch.log1p(1 / k) / math.log(V + 1)
    return float((1 - torch.exp(T * torch.log1p(-p))).sum())


def work(case):
    """Each input read once, each output written once (a table's rows that a token names, unless the whole table is
    written)."""
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "clip":
        n = sum(math.prod(shape) for shape in _shapes(case))
        return {"bytes": 2 * e * n, "flops": 3.0 * n}
    if case["op"] in ("embedding", "embedding_backward"):
        T, V, D = case["T"], case["V"], case["D"]
        real, rows = T - int(T * case["pad"]), _distinct(case)
        ids = T * (8 if case["wide"] else 4)
        if case["op"] == "embedding":
            return {"bytes": ids + e * D * (rows + T), "flops": 1.0 * T * D}
        ge = 2 if case["grad"] == "bf16" else 4
        table = 2 * rows if case["accumulate"] else V
        return {"bytes": ids + e * real * D + ge * D * table, "flops": 2.0 * real * D}
    T, D = case["T"], case["D"]
    vectors = 1 + (1 + case["gates"] if case["block"] else 0)
    if case["op"] == "norm":
        return {"bytes": e * (T * D * (4 if case["block"] else 2) + vectors * D),
                "flops": T * D * (10.0 if case["block"] else 4.0)}
    ge = 2 if case["grad"] == "bf16" else 4
    return {"bytes": e * (T * D * (6 if case["block"] else 4) + vectors * D) +
            ge * vectors * D * (1 + case["accumulate"]),
            "flops": T * D * (28.0 if case["block"] else 12.0)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        total = torch.zeros((), dtype=torch.float64, device="cuda")
        for g in s["grads"]:
            total += torch.linalg.vector_norm(g.double()).square()
        length = torch.sqrt(total)
        factor = torch.where(length + CLIP_EPS > MAX_NORM, MAX_NORM / (length + CLIP_EPS), torch.ones_like(length))
        return length, torch.cat([torch.mul(g.double(), factor).reshape(-1) for g in s["grads"]])
    if case["op"] == "embedding":
        # a row of zeros stands behind the table for whatever lies outside
        table = torch.cat([s["table"].double(), torch.zeros(1, case["D"], dtype=torch.float64, device="cuda")])
        ids = s["ids"].long()
        ids = torch.where((ids < 0) | (ids >= case["V"]), torch.full_like(ids, case["V"]), ids)
        return torch.index_select(table, 0, ids) * s["scale"]
    if case["op"] == "embedding_backward":
        keep = (s["ids"] >= 0).nonzero()[:, 0]
        ids, rows = s["ids"].long()[keep], s["dy"].double()[keep]
        out = torch.zeros(case["V"], case["D"], dtype=torch.float64, device="cuda")
        out.scatter_add_(0, ids[:, None].expand_as(rows), rows)
        out *= s["scale"]
        return out + s["dtable"].double() if case["accumulate"] else out

    def leaf(name):
        return None if s[name] is None else s[name].double().requires_grad_()

    def normed(v, w):
        return (case["offset"] + w) * v * torch.rsqrt(torch.mean(v * v, -1, keepdim=True) + NORM_EPS)

    def branch(h, w, g):
        out = case["scale"] * normed(h, w)
        if g is None:
            return out
        T, D = out.shape
        return (out.view(case["gates"], T // case["gates"], D) * g.view(case["gates"], 1, D)).view(T, D)

    h, post, gain, gate = leaf("h"), leaf("post_gain"), leaf("gain"), leaf("gate")
    if case["op"] == "norm":
        x = s["x"].double()
        with torch.no_grad():
            total = x + branch(h, post, gate) if case["block"] else x
            return total, normed(total, gain)
    keep = 1.0 if case["accumulate"] else 0.0
    v = leaf("s")
    dv, dgain = torch.autograd.grad(normed(v, gain), (v, gain), s["dy"].double())
    d = dv + s["ds"].double()
    dgain = dgain + keep * s["dgain"].double()
    if not case["block"]:
        return d, None, dgain, None, None
    wanted = (h, post) if gate is None else (h, post, gate)
    dh, dpost, *rest = torch.autograd.grad(branch(h, post, gate), wanted, d)
    dpost = dpost + keep * s["dpost_gain"].double()
    return d, dh, dgain, dpost, rest[0] + keep * s["dgate"].double() if rest else None
