"""The products and updates around the gradient reduction, as measured cases.

What makes a gradient (a linear layer's product with its epilogue, and its
backward, whose weight gradient goes into the fp32 accumulators of the
deferred reduction) and what uses it on the owner after the reduction
(orthogonalising by Newton-Schulz products, and the whole momentum update).

`own` False computes the plain form in elementary torch operations in 32
bits; True makes the framework's calls.
"""
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ("none", "relu", "gelu", "silu")
COEFFS = (3.4445, -4.7750, 2.0315)   # quintic step that lifts small singular values fast
STEPS, EPS = 5, 1e-7
MU, LR, DECAY = 0.95, 3e-4, 0.1


def linear(name, T, N, K, dtype="bf16", act="none", bias=True, residual=False, pre=False):
    return {"name": name, "op": "linear", "T": T, "N": N, "K": K, "dtype": dtype, "act": act, "bias": bias,
            "residual": residual, "pre": pre}


def bias_act(name, T, N, dtype="bf16", act="gelu"):
    return {"name": name, "op": "bias_act_backward", "T": T, "N": N, "dtype": dtype, "act": act}


def backward(name, T, N, K, dtype="bf16", grad="f32", accumulate=True, bias=True):
    return {"name": name, "op": "linear_backward", "T": T, "N": N, "K": K, "dtype": dtype, "grad": grad,
            "accumulate": accumulate, "bias": bias}


def orth(name, shapes, dtype="bf16"):
    return {"name": name, "op": "orthogonalize", "shapes": shapes, "dtype": dtype}


def update(name, shapes, dtype="bf16", weight="f32", nesterov=True):
    return {"name": name, "op": "muon_update", "shapes": shapes, "dtype": dtype, "weight": weight,
            "nesterov": nesterov}


def listed():
    return [
        # one token through an up projection of the hidden-1024 model: latency, the weight read once
        linear("linear_token", 1, 4096, 1024, act="gelu"),
        # sixteen sequences' next tokens through the 7B-class layer's down projection, residual added
        linear("linear_decode16", 16, 4096, 11008, bias=False, residual=True),
        # a training batch through the 7B-class layer's gate projection, the backward's input kept
        linear("linear_batch_7b", 8192, 11008, 4096, act="silu", bias=False, pre=True),
        # fp32 with odd sizes on every side
        linear("linear_odd_f32", 777, 1003, 515, dtype="f32", act="gelu", residual=True, pre=True),
        # activation and bias gradients of that layer's batch; and a short odd one
        bias_act("bias_act_batch_7b", 8192, 11008, act="silu"),
        bias_act("bias_act_odd", 333, 1003, act="gelu"),
        # a micro-batch of the 7B-class layer's gate projection, added into the fp32 accumulators
        backward("backward_batch_7b", 8192, 11008, 4096, bias=False),
        # odd sizes in fp32, gradients written anew
        backward("backward_odd_f32", 777, 1003, 515, dtype="f32", accumulate=False),
        # one square matrix of the hidden-1024 model
        orth("orth_1024", "1*1024x1024"),
        # every matrix of one 7B-class layer
        orth("orth_layer_7b", "4*4096x4096+2*11008x4096+1*4096x11008"),
        # an owner's share of the hidden-1024 model: eight layers' matrices, one update
        update("update_owner", "32*1024x1024+8*4096x1024+8*1024x4096"),
        # small and odd matrices of an fp32 gradient
        update("update_odd_f32", "2*128x128+3*768x130+2*257x1025+1*5x1+1*1x333", dtype="f32"),
    ]


def _size(rng, lo, hi):
    """Spread over the logarithm; every other one odd-sized."""
    v = int(round(lo * (hi / lo) ** rng.random()))
    if rng.random() < 0.5:
        v = v // 64 * 64 if v >= 128 else v
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["linear", "bias_act_backward", "linear_backward", "orthogonalize", "muon_update"])
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    if op in ("linear", "linear_backward"):
        T, N, K = _size(rng, 1, 8192), _size(rng, 16, 11008), _size(rng, 16, 11008)
        while 2 * T * N * K > (7e11 if dtype == "bf16" else 5e10):
            T = max(1, T // 2)
        if op == "linear":
            c = linear("", T, N, K, dtype, rng.choice(ACTS), rng.random() < 0.5, rng.random() < 0.5,
                       rng.random() < 0.5)
        else:
            c = backward("", T, N, K, dtype, "bf16" if dtype == "bf16" and rng.random() < 0.3 else "f32",
                         rng.random() < 0.7, rng.random() < 0.5)
    elif op == "bias_act_backward":
        c = bias_act("", _size(rng, 1, 8192), _size(rng, 16, 11008), dtype, rng.choice(ACTS[1:]))
    else:
        groups = []
        for _ in range(rng.randint(1, 3)):
            r, k = _size(rng, 1, 4096), _size(rng, 1, 4096)
            most = max(1, int(3e10 / (min(r, k) ** 2 * max(r, k))))
            groups.append("%d*%dx%d" % (rng.randint(1, min(12, most)), r, k))
        shapes = "+".join(groups)
        if op == "orthogonalize":
            c = orth("", shapes, dtype)
        else:
            c = update("", shapes, dtype, "bf16" if dtype == "bf16" and rng.random() < 0.3 else "f32",
                       rng.random() < 0.5)
    del c["name"]
    return c


def _groups(shapes):
    out = []
    for g in shapes.split("+"):
        count, size = g.split("*")
        r, k = size.split("x")
        out.append((int(count), int(r), int(k)))
    return out


def _gradients(gen, count, r, k, dt):
    """Noise and a few strong directions, as a batch's weight gradient has."""
    rank = min(4, r, k)
    g = torch.randn(count, r, k, device="cuda", generator=gen)
    u = torch.randn(count, r, rank, device="cuda", generator=gen)
    v = torch.randn(count, rank, k, device="cuda", generator=gen)
    return ((g + 2.0 / rank ** 0.5 * torch.bmm(u, v) * (r + k) ** 0.5 / (r * k) ** 0.5) * 1e-3).to(dt)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 17)
    dt = DTYPES[case["dtype"]]

    def randn(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, device="cuda", generator=gen) * scale).to(dtype)

    s = {"case": dict(case)}
    if case["op"] == "linear":
        T, N, K = case["T"], case["N"], case["K"]
        s["x"], s["w"] = randn(T, K), randn(N, K, scale=K ** -0.5)
        s["bias"] = randn(N, scale=0.1) if case["bias"] else None
        s["residual"] = randn(T, N) if case["residual"] else None
    elif case["op"] == "bias_act_backward":
        T, N = case["T"], case["N"]
        s["dy"], s["pre"] = randn(T, N, scale=1e-2), randn(T, N)
        s["db"] = randn(N, scale=1e-2, dtype=torch.float32)
    elif case["op"] == "linear_backward":
        T, N, K = case["T"], case["N"], case["K"]
        gt = DTYPES[case["grad"]]
        s["x"], s["w"], s["dy"] = randn(T, K), randn(N, K, scale=K ** -0.5), randn(T, N, scale=1e-2)
        s["dw"] = randn(N, K, scale=1e-2, dtype=gt)
        s["db"] = randn(N, scale=1e-2, dtype=gt) if case["bias"] else None
    else:
        gs = _groups(case["shapes"])
        s["grads"] = [_gradients(gen, c, r, k, dt) for c, r, k in gs]
        if case["op"] == "muon_update":
            wt = DTYPES[case["weight"]]
            s["momentum"] = [randn(c, r, k, scale=1e-3, dtype=torch.float32) for c, r, k in gs]
            s["weights"] = [randn(c, r, k, scale=0.02, dtype=wt) for c, r, k in gs]
    return s


def _act(v, act):
    if act == "relu":
        return v * (v > 0)
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * 0.5 ** 0.5))
    if act == "silu":
        return v / (1 + torch.exp(-v))
    return v


def _act_slope(v, act):
    if act == "relu":
        return (v > 0).to(v.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(v * 0.5 ** 0.5)) + v * torch.exp(-0.5 * v * v) * (0.5 / torch.pi) ** 0.5
    if act == "silu":
        p = 1 / (1 + torch.exp(-v))
        return p * (1 + v * (1 - p))
    return torch.ones_like(v)


def _newton_schulz(g):
    """[count, r, k] in 32 bits."""
    a, b, c = COEFFS
    wide = g.shape[1] <= g.shape[2]
    x = g if wide else g.transpose(1, 2).contiguous()
    x = x / (x.square().sum(dim=(1, 2), keepdim=True).sqrt() + EPS)
    for _ in range(STEPS):
        gram = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.bmm(b * gram + c * torch.bmm(gram, gram), x)
    return x if wide else x.transpose(1, 2)


def run(s):
    c = s["case"]
    if own:
        from gradient_reduction_amd import linear as lin
        from gradient_reduction_amd import muon
        if c["op"] == "linear":
            return lin.forward(s["x"], s["w"], s["bias"], s["residual"], act=c["act"], save_pre=c["pre"])
        if c["op"] == "bias_act_backward":
            return lin.bias_act_backward(s["dy"], s["pre"], act=c["act"], db=s["db"], accumulate=True)
        if c["op"] == "linear_backward":
            return lin.backward(s["dy"], s["x"], s["w"], dw=s["dw"], db=s["db"], accumulate=c["accumulate"])
        if c["op"] == "orthogonalize":
            return muon.orthogonalize(s["grads"], steps=STEPS, coeffs=COEFFS, eps=EPS)
        muon.update(s["weights"], s["grads"], s["momentum"], lr=LR, mu=MU, nesterov=c["nesterov"],
                    weight_decay=DECAY, scale="rms", steps=STEPS, coeffs=COEFFS, eps=EPS)
        return s["weights"], s["momentum"]

    dt = DTYPES[c["dtype"]]
    if c["op"] == "linear":
        pre = s["x"].float() @ s["w"].float().t()
        if c["bias"]:
            pre = pre + s["bias"].float()
        y = _act(pre, c["act"])
        if c["residual"]:
            y = y + s["residual"].float()
        return (y.to(dt), pre.to(dt)) if c["pre"] else y.to(dt)
    if c["op"] == "bias_act_backward":
        dz = s["dy"].float() * _act_slope(s["pre"].float(), c["act"])
        s["db"] += dz.sum(dim=0)
        return dz.to(dt), s["db"]
    if c["op"] == "linear_backward":
        dy, x = s["dy"].float(), s["x"].float()
        dx = (dy @ s["w"].float()).to(dt)
        dw = dy.t() @ x
        s["dw"].copy_(s["dw"].float() + dw if c["accumulate"] else dw)
        if not c["bias"]:
            return dx, s["dw"], None
        db = dy.sum(dim=0)
        s["db"].copy_(s["db"].float() + db if c["accumulate"] else db)
        return dx, s["dw"], s["db"]
    if c["op"] == "orthogonalize":
        return [_newton_schulz(g.float()).to(dt).contiguous() for g in s["grads"]]
    for w, g, m in zip(s["weights"], s["grads"], s["momentum"]):
        m.mul_(MU).add_(g.float())
        o = _newton_schulz(g.float() + MU * m if c["nesterov"] else m)
        w.copy_(w.float() * (1 - LR * DECAY) - LR * 0.2 * max(w.shape[1:]) ** 0.5 * o)
    return s["weights"], s["momentum"]


def work(case):
    """Each input read once, each output written once; the products' operations, a symmetric product's
    half counted."""
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "linear":
        T, N, K = case["T"], case["N"], case["K"]
        n = T * K + N * K + T * N * (1 + case["residual"] + case["pre"]) + N * case["bias"]
        return {"bytes": e * n, "flops": 2.0 * T * N * K}
    if case["op"] == "bias_act_backward":
        T, N = case["T"], case["N"]
        return {"bytes": 3 * e * T * N + 8 * N, "flops": 10.0 * T * N}
    if case["op"] == "linear_backward":
        T, N, K = case["T"], case["N"], case["K"]
        ge = 2 if case["grad"] == "bf16" else 4
        grads = (N * K + N * case["bias"]) * ge * (1 + case["accumulate"])
        return {"bytes": e * (T * N + 2 * T * K + N * K) + grads, "flops": 4.0 * T * N * K}
    n = sum(c * r * k for c, r, k in _groups(case["shapes"]))
    flops = 0.0
    for c, r, k in _groups(case["shapes"]):
        m, l = min(r, k), max(r, k)
        flops += c * STEPS * (3.0 * m * m * l + 1.0 * m * m * m)
    if case["op"] == "orthogonalize":
        return {"bytes": 2 * e * n, "flops": flops}
    return {"bytes": n * (e + 8 + 2 * (2 if case["weight"] == "bf16" else 4)), "flops": flops}


def _exact_orthogonal(u):
    """R X0 with R the polynomial of H = X0 X0T that the steps compose to: R <- R (a + b P + c P P),
    P = H R R."""
    a, b, c = COEFFS
    flip = u.shape[0] > u.shape[1]
    x = (u.t() if flip else u).contiguous()
    x = x / (torch.linalg.vector_norm(x) + EPS)
    h = x @ x.t()
    eye = torch.eye(h.shape[0], dtype=h.dtype, device=h.device)
    p, r = h, eye
    for k in range(STEPS):
        if k:
            p = h @ (r @ r)
        r = r @ (a * eye + b * p + c * (p @ p))
    o = r @ x
    return o.t() if flip else o


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() if torch.is_tensor(v) else [x.double() for x in v] if isinstance(v, list) else v
         for k, v in s.items()}
    if case["op"] == "linear":
        pre = torch.matmul(d["x"], d["w"].t())
        if d["bias"] is not None:
            pre += d["bias"]
        if case["act"] == "relu":
            y = torch.maximum(pre, torch.zeros_like(pre))
        elif case["act"] == "gelu":
            y = pre * torch.special.ndtr(pre)
        elif case["act"] == "silu":
            y = pre * torch.special.expit(pre)
        else:
            y = pre.clone()
        if d["residual"] is not None:
            y += d["residual"]
        return (y, pre) if case["pre"] else y
    if case["op"] == "bias_act_backward":
        z = d["pre"]
        if case["act"] == "relu":
            slope = torch.heaviside(z, torch.zeros_like(z))
        elif case["act"] == "gelu":
            slope = torch.special.ndtr(z) + z * torch.exp(-z.square() / 2) / (2 * torch.pi) ** 0.5
        else:
            p = torch.special.expit(z)
            slope = p + z * p * torch.special.expit(-z)
        dz = d["dy"] * slope
        return dz, d["db"] + torch.sum(dz, 0)
    if case["op"] == "linear_backward":
        keep = 1.0 if case["accumulate"] else 0.0
        dx = torch.matmul(d["dy"], d["w"])
        dw = keep * d["dw"] + torch.matmul(d["x"].t(), d["dy"]).t()
        db = keep * d["db"] + torch.sum(d["dy"], 0) if case["bias"] else None
        return dx, dw, db
    if case["op"] == "orthogonalize":
        return [torch.stack([_exact_orthogonal(m) for m in g]) for g in d["grads"]]
    ws, ms = [], []
    for w, g, m in zip(d["weights"], d["grads"], d["momentum"]):
        new = MU * m + g
        u = MU * new + g if case["nesterov"] else new
        o = torch.stack([_exact_orthogonal(x) for x in u])
        ws.append(w - LR * (DECAY * w + 0.2 * max(w.shape[1:]) ** 0.5 * o))
        ms.append(new)
    return ws, ms
