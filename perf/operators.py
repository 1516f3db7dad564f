"""Operator cases: linear layers with a fused epilogue, and orthogonalised (Muon) updates.

What a data-parallel training step needs on either side of the gradient
all-reduce: the layer products that make the gradients (forward with bias,
activation and residual; backward straight into gradient buffers), and the
update that uses them (Newton-Schulz orthogonalisation, alone and inside the
Muon step on every rank's parameters).

``run`` computes a case in plain torch operations in 32 bits where ``own`` is
false, and through the library's entry points where it is true; ``exact`` is
the same in 64 bits from the definitions.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
COEFFS = (3.4445, -4.7750, 2.0315)  # the quintic of the Muon update
STEPS = 5
EPS = 1e-7
LR, MOMENTUM, DECAY = 0.02, 0.95, 0.1


# -- the cases ---------------------------------------------------------------

def _forward(name, tokens, n_in, n_out, dtype, act, bias=True, residual=False, save_z=False):
    return {"name": name, "op": "forward", "tokens": tokens, "in": n_in, "out": n_out, "dtype": dtype, "act": act,
            "bias": bias, "residual": residual, "save_z": save_z}


def _backward(name, tokens, n_in, n_out, dtype, act, grad="f32", accumulate=True):
    return {"name": name, "op": "backward", "tokens": tokens, "in": n_in, "out": n_out, "dtype": dtype, "act": act,
            "grad": grad, "accumulate": accumulate}


def _ortho(name, shapes, dtype):
    return {"name": name, "op": "ortho", "shapes": shapes, "dtype": dtype}


def _muon(name, shapes, dtype, copies):
    return {"name": name, "op": "muon", "shapes": shapes, "dtype": dtype, "copies": copies}


def listed():
    return [
        # a classifier head (ResNet-50's fc, 2048 -> 1000) answering for one example: latency
        _forward("forward fc, 1 token", 1, 2048, 1000, "f16", "none"),
        # a few tokens through a wide layer: the weights are the traffic
        _forward("forward 16 tokens", 16, 4096, 8192, "bf16", "silu", bias=False),
        # a ragged batch through odd sizes, everything the epilogue has, ready for the backward pass
        _forward("forward ragged", 333, 1001, 777, "f16", "gelu", residual=True, save_z=True),
        # a training batch through a square layer of a language model
        _forward("forward training batch", 8192, 4096, 4096, "bf16", "gelu", residual=True, save_z=True),
        # the same head's backward pass on a worker's batch, adding to its binary32 gradient
        _backward("backward fc", 256, 2048, 1000, "f16", "none"),
        # ragged backward, gradients in the 16 bits that travel in half-precision communication
        _backward("backward ragged", 517, 771, 1029, "f16", "relu", grad="f16", accumulate=False),
        # a training batch backward through an expanding layer, binary32 gradients
        _backward("backward training batch", 8192, 2048, 8192, "bf16", "gelu"),
        # one small matrix (ResNet-50's stem, 64 x 147): latency
        _ortho("orthogonalise stem", "64x147", "f32"),
        # a stack of wide layers whose update is kept in 16 bits
        _ortho("orthogonalise wide x4", "4*1024x4096", "bf16"),
        # a tall odd matrix in binary16
        _ortho("orthogonalise tall odd", "2049x1023", "f16"),
        # the whole of ResNet-50's gradient, 16 workers' parameters
        _muon("muon resnet50, 16 workers", "resnet50", "f32", 16),
        # four blocks of a language model, binary16 gradients, two workers
        _muon("muon blocks", "4*2048x2048,2*8192x2048,2*2048x8192", "f16", 2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.4 else max(lo, n // 64 * 64) if n >= 64 else n


def draw(rng):
    op = rng.choice(["forward", "forward", "backward", "backward", "ortho", "muon"])
    if op in ("forward", "backward"):
        tokens, n_in, n_out = _size(rng, 1, 8192), _size(rng, 64, 4096), _size(rng, 64, 8192)
        act = rng.choice(["none", "relu", "gelu", "silu"])
        dtype = rng.choice(["f16", "bf16"])
        if op == "forward":
            c = _forward("", tokens, n_in, n_out, dtype, act, rng.random() < 0.7, rng.random() < 0.5, rng.random() < 0.5)
        else:
            c = _backward("", tokens, n_in, n_out, dtype, act, rng.choice(["f32", "f32", "f16"]), rng.random() < 0.5)
    else:
        shapes = ",".join("%d*%dx%d" % (rng.randint(1, 2), _size(rng, 16, 2048), _size(rng, 16, 4096))
                          for _ in range(rng.randint(1, 3)))
        if op == "ortho":
            c = _ortho("", shapes, rng.choice(["f32", "f16", "bf16"]))
        else:
            c = _muon("", shapes, rng.choice(["f32", "f16"]), _log(rng, 1, 6))
    del c["name"]
    return c


def _tensors(shapes):
    """(offset, rows, cols) of every matrix of a flat gradient buffer, and the buffer's elements."""
    mats, at = [], 0
    if shapes == "resnet50":
        # stem, bottleneck stages and fc in forward order; each convolution is followed by
        # its batch norm's two vectors, the fc by its bias, which the update leaves alone
        convs, cin = [(64, 147)], 64
        for stage, blocks in enumerate((3, 4, 6, 3)):
            width = 64 << stage
            for b in range(blocks):
                convs += [(width, cin), (width, 9 * width), (4 * width, width)]
                convs += [(4 * width, cin)] if b == 0 else []
                cin = 4 * width
        for rows, cols in convs:
            mats.append((at, rows, cols))
            at += rows * cols + 2 * rows
        mats.append((at, 1000, cin))
        return mats, at + 1000 * cin + 1000
    for part in shapes.split(","):
        count, shape = part.split("*") if "*" in part else ("1", part)
        rows, cols = (int(v) for v in shape.split("x"))
        for _ in range(int(count)):
            mats.append((at, rows, cols))
            at += rows * cols
    return mats, at


# -- inputs ------------------------------------------------------------------

def _gradient(mats, n, dtype, gen):
    """Gradients as a layer's matrix has them: a few strong directions over noise, at a small scale."""
    flat = torch.randn(n, generator=gen, device="cuda") * 1e-3
    for off, rows, cols in mats:
        r = min(16, rows, cols)
        left = torch.randn(rows, r, generator=gen, device="cuda")
        right = torch.randn(r, cols, generator=gen, device="cuda")
        flat[off:off + rows * cols].view(rows, cols).add_(left @ right, alpha=1e-3)
    return flat.to(DTYPES[dtype])


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, sigma=1.0, dtype=None):
        return (torch.randn(*shape, generator=gen, device="cuda") * sigma).to(DTYPES[dtype or case["dtype"]])

    s = {}
    if case["op"] in ("forward", "backward"):
        t, i, o = case["tokens"], case["in"], case["out"]
        s["x"] = normal(t, i)
        s["w"] = normal(o, i, sigma=i ** -0.5)
        if case["op"] == "forward":
            s["bias"] = normal(o, sigma=0.1) if case["bias"] else None
            s["residual"] = normal(t, o) if case["residual"] else None
            s["y"] = s["x"].new_empty(t, o)
            s["z"] = s["y"].new_empty(t, o) if case["save_z"] else None
        else:
            s["dy"] = normal(t, o)
            s["z"] = normal(t, o) if case["act"] != "none" else None
            s["dx"] = s["x"].new_empty(t, i)
            # the sums of a worker's earlier micro-batches, or space for the gradient
            s["dw"] = normal(o, i, sigma=t ** 0.5, dtype=case["grad"])
            s["db"] = normal(o, sigma=t ** 0.5, dtype=case["grad"])
    else:
        mats, n = _tensors(case["shapes"])
        s["mats"] = mats
        s["grad"] = _gradient(mats, n, case["dtype"], gen)
        if case["op"] == "ortho":
            s["out"] = torch.zeros_like(s["grad"])
        else:
            param = normal(n, sigma=0.02, dtype="f32")
            s["params"] = [param.clone() for _ in range(case["copies"])]
            s["mom"] = _gradient(mats, n, "f32", gen) * 10
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        from gradient_all_reduce_ddl_gb300 import ddl
        if case["op"] in ("forward", "backward"):
            s["layer"] = ddl.Linear(case["in"], case["out"], case["tokens"], case["dtype"], case["act"])
        else:
            s["ortho"] = ddl.Ortho(s["mats"], case["dtype"], steps=STEPS, coefficients=COEFFS, eps=EPS)
    return s


# -- the operators in plain torch --------------------------------------------

def _act(z, kind):
    if kind == "relu":
        return torch.clamp(z, min=0)
    if kind == "gelu":
        return z * (0.5 * (1 + torch.erf(z * math.sqrt(0.5))))
    if kind == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, kind):
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    sig = 1 / (1 + torch.exp(-z))
    return sig * (1 + z * (1 - sig))


def _forward_plain(s, c):
    z = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(z, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    s["y"].copy_(y)
    if s["z"] is not None:
        s["z"].copy_(z)
    return {"y": s["y"], "z": s["z"]}


def _backward_plain(s, c):
    dz = s["dy"].float()
    if s["z"] is not None:
        dz = dz * _act_grad(s["z"].float(), c["act"])
    s["dx"].copy_(dz @ s["w"].float())
    dw = dz.t() @ s["x"].float()
    db = dz.sum(0)
    if c["accumulate"]:
        dw, db = dw + s["dw"].float(), db + s["db"].float()
    s["dw"].copy_(dw)
    s["db"].copy_(db)
    return {"dx": s["dx"], "dw": s["dw"], "db": s["db"]}


def _newton_schulz(g):
    """g (binary32) with its singular values driven towards one."""
    a, b, c = COEFFS
    x = g if g.shape[0] <= g.shape[1] else g.t()
    x = x / (x.square().sum().sqrt() + EPS)
    for _ in range(STEPS):
        gram = x @ x.t()
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x if g.shape[0] <= g.shape[1] else x.t()


def _ortho_plain(s):
    for off, rows, cols in s["mats"]:
        g = s["grad"][off:off + rows * cols].view(rows, cols)
        s["out"][off:off + rows * cols].view(rows, cols).copy_(_newton_schulz(g.float()))
    return {"out": s["out"]}


def _muon_plain(s):
    for off, rows, cols in s["mats"]:
        at = slice(off, off + rows * cols)
        g = s["grad"][at].float()
        v = s["mom"][at]
        v.mul_(MOMENTUM).add_(g)
        step = _newton_schulz((g + MOMENTUM * v).view(rows, cols)).reshape(-1) * math.sqrt(max(1.0, rows / cols))
        for p in s["params"]:
            p[at] = p[at] * (1 - LR * DECAY) - LR * step
    return {"params": s["params"], "mom": s["mom"]}


def run(state):
    c = state["case"]
    if not own:
        if c["op"] == "forward":
            return _forward_plain(state, c)
        if c["op"] == "backward":
            return _backward_plain(state, c)
        return _ortho_plain(state) if c["op"] == "ortho" else _muon_plain(state)
    if c["op"] == "forward":
        state["layer"].forward(state["x"], state["w"], state["y"], bias=state["bias"], residual=state["residual"],
                               z=state["z"])
        return {"y": state["y"], "z": state["z"]}
    if c["op"] == "backward":
        state["layer"].backward(state["dy"], state["x"], state["w"], z=state["z"], dx=state["dx"], dw=state["dw"],
                                db=state["db"], accumulate=c["accumulate"])
        return {"dx": state["dx"], "dw": state["dw"], "db": state["db"]}
    if c["op"] == "ortho":
        state["ortho"].run(state["grad"], state["out"])
        return {"out": state["out"]}
    state["ortho"].muon(state["grad"], state["params"], state["mom"], LR, momentum=MOMENTUM, weight_decay=DECAY,
                        nesterov=True)
    return {"params": state["params"], "mom": state["mom"]}


# -- what a pass has to do, and its result in 64 bits --------------------------

def work(case):
    size = {"f32": 4, "f16": 2, "bf16": 2}
    e = size[case["dtype"]]
    if case["op"] == "forward":
        t, i, o = case["tokens"], case["in"], case["out"]
        moved = t * i + o * i + o * case["bias"] + t * o * (1 + case["residual"] + case["save_z"])
        return {"bytes": e * moved, "flops": 2 * t * i * o}
    if case["op"] == "backward":
        t, i, o = case["tokens"], case["in"], case["out"]
        moved = e * (2 * t * i + o * i + t * o * (1 + (case["act"] != "none")))
        return {"bytes": moved + size[case["grad"]] * (o * i + o) * (1 + case["accumulate"]), "flops": 4 * t * i * o}
    mats, _ = _tensors(case["shapes"])
    # the Gram matrix and its square are symmetric: half of each is enough
    flops = sum(STEPS * (min(r, c) * (min(r, c) + 1) * (max(r, c) + min(r, c)) + 2 * min(r, c) ** 2 * max(r, c))
                for _, r, c in mats)
    elems = sum(r * c for _, r, c in mats)
    moved = elems * 2 * e if case["op"] == "ortho" else elems * (e + 8 + 8 * case["copies"])
    return {"bytes": moved, "flops": flops}


def _exact_ortho(g):
    """Horner's form of the quintic in X, with the Gram matrix on the columns' side where that is shorter."""
    a, b, c = COEFFS
    x = g / (torch.linalg.vector_norm(g) + EPS)
    for _ in range(STEPS):
        if x.shape[0] <= x.shape[1]:
            m = torch.matmul(x, x.mT)
            x = torch.addmm(x, torch.addmm(m, m, m, beta=b, alpha=c), x, beta=a)
        else:
            m = torch.matmul(x.mT, x)
            x = torch.addmm(x, x, torch.addmm(m, m, m, beta=b, alpha=c), beta=a)
    return x


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] in ("forward", "backward"):
        x, w = s["x"].double(), s["w"].double()
        if case["op"] == "forward":
            z = torch.matmul(x, w.mT)
            z += s["bias"].double() if case["bias"] else 0
            y = {"none": lambda v: v.clone(), "relu": torch.relu, "gelu": torch.nn.functional.gelu,
                 "silu": torch.nn.functional.silu}[case["act"]](z)
            y += s["residual"].double() if case["residual"] else 0
            return {"y": y, "z": z if case["save_z"] else None}
        dz = s["dy"].double()
        if case["act"] != "none":
            z = s["z"].double()
            if case["act"] == "relu":
                dz = torch.where(z > 0, dz, torch.zeros_like(dz))
            elif case["act"] == "gelu":
                dz = dz * (torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
            else:
                dz = dz * (torch.sigmoid(z) + torch.sigmoid(z) * torch.sigmoid(-z) * z)
        keep = 1.0 if case["accumulate"] else 0.0
        return {"dx": torch.matmul(dz, w), "dw": torch.matmul(dz.mT, x) + keep * s["dw"].double(),
                "db": torch.sum(dz, 0) + keep * s["db"].double()}
    if case["op"] == "ortho":
        out = torch.zeros_like(s["grad"], dtype=torch.float64)
        for off, rows, cols in s["mats"]:
            out[off:off + rows * cols] = _exact_ortho(s["grad"][off:off + rows * cols].double().view(rows, cols)).reshape(-1)
        return {"out": out}
    mom = s["mom"].double()
    new = s["params"][0].double()
    for off, rows, cols in s["mats"]:
        at = slice(off, off + rows * cols)
        g = s["grad"][at].double()
        mom[at] = MOMENTUM * mom[at] + g
        o = _exact_ortho((g + MOMENTUM * mom[at]).view(rows, cols)).reshape(-1)
        new[at] -= LR * (DECAY * new[at] + math.sqrt(max(1.0, rows / cols)) * o)
    return {"params": [new] * case["copies"], "mom": mom}
