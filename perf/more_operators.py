"""Operator cases: softmax cross entropy of a linear head over a large vocabulary, and AdamW steps over many tensors.

The two ends of a data-parallel training step that the layers, the all-reduce and
the Muon update leave open: the loss, from which the gradients start (its logits
are too large to keep), and the update of the tensors that Muon leaves alone
(embeddings, heads, norms, biases), for every worker's copy of the parameters.

``run`` computes a case in plain torch operations in 32 bits where ``own`` is
false, and through the library's entry points where it is true; ``exact`` is
the same in 64 bits from the definitions.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BETA1, BETA2, EPS = 0.9, 0.999, 1e-8
LR, DECAY = 1e-4, 0.1
BLOCK = 128       # elements of an 8-bit state that share a scale
TOP = 448.0       # e4m3's largest number
STEPS_DONE = 1000


# -- the cases ---------------------------------------------------------------

def _loss(name, op, tokens, n_in, vocab, dtype, bias=False, smoothing=0.0, ignored=0.0, grad="f32", accumulate=False,
          weighted=False):
    return {"name": name, "op": op, "tokens": tokens, "in": n_in, "vocab": vocab, "dtype": dtype, "bias": bias,
            "smoothing": smoothing, "ignored": ignored, "grad": grad, "accumulate": accumulate, "weighted": weighted}


def _adam(name, tensors, state, grad="f32", copies=1, operands="", clip=0.0, scale=1.0):
    return {"name": name, "op": "adam", "tensors": tensors, "state": state, "grad": grad, "copies": copies,
            "operands": operands, "clip": clip, "scale": scale}


def listed():
    return [
        # scoring one example with a classifier's head (ResNet-50's fc, 2048 -> 1000): latency
        _loss("loss fc 1 token", "loss", 1, 2048, 1000, "f16", bias=True),
        # log probabilities of a few tokens over a large vocabulary: the weights are the traffic
        _loss("loss 16 tokens", "loss", 16, 4096, 65536, "bf16"),
        # a ragged validation batch with odd sizes, smoothed labels and padding
        _loss("loss ragged", "loss", 333, 1001, 20011, "f16", bias=True, smoothing=0.1, ignored=0.2),
        # a validation batch of a language model
        _loss("loss validation batch", "loss", 8192, 4096, 65536, "bf16", ignored=0.05),
        # the classifier's head in training, a worker's batch, added to its binary32 gradient
        _loss("train fc", "train", 256, 2048, 1000, "f16", bias=True, smoothing=0.1, accumulate=True),
        # ragged training batch, weighted tokens, gradients in the 16 bits that half-precision communication takes
        _loss("train ragged", "train", 517, 771, 5003, "f16", bias=True, ignored=0.3, grad="f16", weighted=True),
        # a language model's head in training
        _loss("train batch", "train", 8192, 2048, 65536, "bf16", ignored=0.05),
        # what Muon leaves of ResNet-50 (batch norms' vectors, the fc's bias), four workers: latency
        _adam("adamw vectors 4 workers", "resnet50 vectors", "f32", copies=4),
        # all of ResNet-50's tensors, 16 workers
        _adam("adamw resnet50 16 workers", "resnet50", "f32", copies=16),
        # a language model with 8-bit states, clipped, with the layers' bfloat16 weights
        _adam("adamw language model 8 bits", "lm", "8bit", operands="bf16", clip=1.0),
        # odd tensors packed one after the other, binary16 gradients with a loss scale, two workers, 8-bit states
        _adam("adamw ragged 8 bits", "4099,1001*777,31,777,1,5003*301,129", "8bit", grad="f16", copies=2, scale=1 / 1024),
        # four blocks of a language model, binary16 gradients with a loss scale, clipped, binary16 weights for the layers
        _adam("adamw blocks 2 workers", "2048*2048,2048*2048,8192*2048,2048*8192,2048", "f32", grad="f16", copies=2,
              operands="f16", clip=0.5, scale=1 / 1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.4 else max(lo, n // 64 * 64) if n >= 64 else n


def draw(rng):
    op = rng.choice(["loss", "loss", "train", "train", "adam", "adam"])
    if op != "adam":
        train = op == "train"
        c = _loss("", op, _size(rng, 1, 8192), _size(rng, 64, 2048 if train else 4096), _size(rng, 500, 65536),
                  rng.choice(["f16", "bf16"]), bias=rng.random() < 0.5, smoothing=rng.choice([0.0, 0.0, 0.1]),
                  ignored=rng.choice([0.0, 0.1, 0.5]))
        if train:
            c.update(grad=rng.choice(["f32", "f32", "f16"]), accumulate=rng.random() < 0.5, weighted=rng.random() < 0.5)
    else:
        parts = []
        for _ in range(rng.randint(1, 8)):
            n = _size(rng, 1, 4096)
            parts.append("%d*%d" % (n, _size(rng, 16, 4096)) if rng.random() < 0.5 else "%d" % n)
        c = _adam("", ",".join(parts), rng.choice(["f32", "8bit"]), rng.choice(["f32", "f16"]), _log(rng, 1, 8),
                  rng.choice(["", "f16", "bf16"]), rng.choice([0.0, 1.0]), rng.choice([1.0, 1 / 1024]))
    del c["name"]
    return c


def _resnet50():
    """Elements of ResNet-50's tensors in forward order: convolutions with their batch norms' two vectors, then the fc."""
    convs, cin = [64 * 147], 64
    widths = [64]
    for stage, blocks in enumerate((3, 4, 6, 3)):
        width = 64 << stage
        for b in range(blocks):
            convs += [width * cin, width * 9 * width, 4 * width * width] + ([4 * width * cin] if b == 0 else [])
            widths += [width, width, 4 * width] + ([4 * width] if b == 0 else [])
            cin = 4 * width
    sizes = [n for c, w in zip(convs, widths) for n in (c, w, w)]
    return sizes + [1000 * cin, 1000]


def _tensors(spec):
    """Elements of every tensor of the flat buffers, in order, and whether weight decay applies to it (matrices)."""
    if spec.startswith("resnet50"):
        sizes = _resnet50()
        decayed = [i % 3 == 0 for i in range(len(sizes))]
        decayed[-2:] = [True, False]
        if spec.endswith("vectors"):
            sizes, decayed = [n for n, d in zip(sizes, decayed) if not d], [False] * decayed.count(False)
        return sizes, decayed
    if spec == "lm":  # an embedding and 24 blocks of width 1024
        block = [1024, 1024 * 4096, 1024, 4 * 1024 * 1024, 4 * 1024 * 1024]
        sizes = [32768 * 1024] + block * 24 + [1024]
        return sizes, [n > 1024 for n in sizes]
    dims = [[int(v) for v in part.split("*")] for part in spec.split(",")]
    return [math.prod(d) for d in dims], [len(d) > 1 for d in dims]


# -- inputs ------------------------------------------------------------------

def _loss_inputs(case, gen):
    t, i, v = case["tokens"], case["in"], case["vocab"]

    def normal(*shape, sigma=1.0, dtype=case["dtype"]):
        return (torch.randn(*shape, generator=gen, device="cuda") * sigma).to(DTYPES[dtype])

    s = {"w": normal(v, i, sigma=i ** -0.5), "bias": normal(v, sigma=0.5) if case["bias"] else None}
    s["labels"] = torch.randint(0, v, (t,), generator=gen, device="cuda")
    # a model that knows something: from none of the label's logit standing out to about 0.9 of the probability on it
    sure = torch.rand(t, 1, generator=gen, device="cuda") * (math.log(v) + 2)
    s["x"] = (torch.randn(t, i, generator=gen, device="cuda") + sure * s["w"][s["labels"]].float()).to(DTYPES[case["dtype"]])
    s["labels"][torch.rand(t, generator=gen, device="cuda") < case["ignored"]] = -100
    s["loss"], s["lse"] = s["x"].new_empty(t, dtype=torch.float32), s["x"].new_empty(t, dtype=torch.float32)
    if case["op"] == "train":
        # the mean over the tokens that count, or their weights; in half precision with the loss scale that it needs
        count = (s["labels"] >= 0).sum().clamp(min=1)
        weight = torch.rand(t, generator=gen, device="cuda") + 0.5 if case["weighted"] else torch.ones(t, device="cuda")
        s["dloss"] = weight * (1024.0 if case["grad"] == "f16" else 1.0) / count
        s["dx"] = torch.empty_like(s["x"])
        # the sums of a worker's earlier micro-batches, or space for the gradient
        s["dw"] = normal(v, i, sigma=float(s["dloss"][0]), dtype=case["grad"])
        s["db"] = normal(v, sigma=float(s["dloss"][0]), dtype=case["grad"]) if case["bias"] else None
    return s


def _blocks(x, s):
    """A flat buffer as rows of BLOCK elements that share a scale; each tensor begins a row, its last one is filled with zeros."""
    if s["pad"] is None:
        return x.view(-1, BLOCK)
    return torch.cat([x, x.new_zeros(1)])[s["pad"]]


def _flat(rows, s):
    return rows.reshape(-1) if s["unpad"] is None else rows.reshape(-1)[s["unpad"]]


def _encode(rows):
    """Rows of BLOCK values as e4m3 codes and a scale each."""
    top = rows.abs().amax(1, keepdim=True)
    held = top >= 2.0 ** -100
    codes = torch.where(held, rows * (TOP / torch.where(held, top, torch.ones_like(top))), torch.zeros_like(rows))
    return codes.clamp(-TOP, TOP).to(torch.float8_e4m3fn), torch.where(held, top / TOP, torch.zeros_like(top))


def _encode_root(rows):
    """The same of square roots, of which none but zero becomes zero."""
    codes, scale = _encode(rows)
    return torch.where((rows > 0) & (scale > 0), codes.float().clamp(min=2.0 ** -9), codes.float()).to(torch.float8_e4m3fn), scale


def _places(sizes):
    """Where the rows' elements lie in the flat buffer (its length: nowhere), and where the buffer's elements lie in the rows."""
    n = sum(sizes)
    if all(k % BLOCK == 0 for k in sizes):
        return None, None
    counts = torch.tensor(sizes, device="cuda")
    rows = (counts + BLOCK - 1) // BLOCK
    begin = torch.cumsum(counts, 0) - counts
    first = torch.cumsum(rows, 0) - rows
    tensor = torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), counts)
    unpad = torch.arange(n, device="cuda") - begin[tensor] + first[tensor] * BLOCK
    pad = torch.full((int(rows.sum()) * BLOCK,), n, device="cuda")
    pad[unpad] = torch.arange(n, device="cuda")
    return pad.view(-1, BLOCK), unpad


def _adam_inputs(case, gen):
    sizes, decayed = _tensors(case["tensors"])
    n, counts = sum(sizes), torch.tensor(sizes, device="cuda")

    def per_tensor(values):
        return torch.repeat_interleave(values, counts)

    def normal():
        return torch.randn(n, generator=gen, device="cuda")

    s = {"sizes": sizes, "decayed": decayed}
    # gradients of 1e-5 to 1e-2 by tensor; of an embedding's first half most rows were not met
    sigma = per_tensor(10 ** (torch.rand(len(sizes), generator=gen, device="cuda") * 3 - 5))
    grad = normal().mul_(sigma)
    m = normal().mul_(sigma).mul_(0.3)
    root = torch.rand(n, generator=gen, device="cuda").add_(0.5).mul_(sigma)
    if case["tensors"] == "lm":
        met = torch.rand(16384, generator=gen, device="cuda") < 0.2
        for x in (grad, m, root):
            x[:16384 * 1024].view(16384, 1024).mul_(met.unsqueeze(1))
    del sigma
    s["grad"] = grad.div_(case["scale"]).to(DTYPES[case["grad"]])
    param = normal().mul_(0.02)
    s["params"] = [param] + [param.clone() for _ in range(case["copies"] - 1)]
    s["operands"] = [torch.zeros(n, dtype=DTYPES[case["operands"]], device="cuda") for _ in s["params"]] if case["operands"] else None
    s["step"] = torch.tensor([STEPS_DONE], device="cuda")
    s["norm"] = torch.zeros(1, device="cuda") if case["clip"] else None
    if case["state"] == "f32":
        s["m"], s["v"], s["scales"] = m, root.square_(), None
    else:
        s["pad"], s["unpad"] = _places(sizes)
        (cm, sm), (cr, sr) = _encode(_blocks(m, s)), _encode_root(_blocks(root, s))
        s["m"], s["v"] = _flat(cm.view(torch.uint8), s).view(torch.float8_e4m3fn), _flat(cr.view(torch.uint8), s).view(torch.float8_e4m3fn)
        s["scales"] = torch.cat([sm, sr], 1).t().contiguous()
    return s


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return _adam_inputs(case, gen) if case["op"] == "adam" else _loss_inputs(case, gen)


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        from gradient_all_reduce_ddl_gb300 import ddl
        if case["op"] == "adam":
            begin = [sum(s["sizes"][:k]) for k in range(len(s["sizes"]))]
            s["adam"] = ddl.Adam([(at, n, 1.0, float(d)) for at, n, d in zip(begin, s["sizes"], s["decayed"])],
                                 dtype=case["grad"], state=case["state"], betas=(BETA1, BETA2), eps=EPS)
        else:
            s["head"] = ddl.CrossEntropy(case["in"], case["vocab"], case["tokens"], case["dtype"], smoothing=case["smoothing"])
    elif case["op"] == "adam":
        s["decay"] = torch.repeat_interleave(torch.tensor(s["decayed"], device="cuda").float(), torch.tensor(s["sizes"], device="cuda"))
    return s


# -- the operators in plain torch --------------------------------------------

def _logits_plain(s, c):
    """The logits, and what the loss needs of them."""
    z = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        z += s["bias"].float()
    top = z.amax(1, keepdim=True)
    # the difference of two near numbers where the label is likely: in 64 bits
    lse = (top.double() + torch.log(torch.exp(z - top).sum(1, keepdim=True, dtype=torch.float64))).squeeze(1)
    s["lse"].copy_(lse)
    valid, eps = s["labels"] >= 0, c["smoothing"]
    picked = z.gather(1, s["labels"].clamp(min=0).unsqueeze(1)).squeeze(1)
    loss = lse - (1 - eps) * picked.double()
    if eps:
        loss = loss - eps * z.mean(1, dtype=torch.float64)
    s["loss"].copy_(torch.where(valid, loss, torch.zeros_like(loss)))
    return z, valid


def _train_plain(s, c):
    z, valid = _logits_plain(s, c)
    p = z.sub_(s["lse"].unsqueeze(1)).exp_()
    rows = torch.arange(len(valid), device=p.device)
    p[rows, s["labels"].clamp(min=0)] -= 1 - c["smoothing"]
    if c["smoothing"]:
        p -= c["smoothing"] / c["vocab"]
    p *= torch.where(valid, s["dloss"], torch.zeros_like(s["dloss"])).unsqueeze(1)
    s["dx"].copy_(p @ s["w"].float())
    dw = p.t() @ s["x"].float()
    s["dw"].copy_(dw + s["dw"].float() if c["accumulate"] else dw)
    if s["db"] is not None:
        db = p.sum(0)
        s["db"].copy_(db + s["db"].float() if c["accumulate"] else db)
    return {"loss": s["loss"], "lse": s["lse"], "dx": s["dx"], "dw": s["dw"], "db": s["db"]}


def _adam_plain(s, c):
    scale = c["scale"]
    g = s["grad"].float()
    if c["clip"]:
        norm = torch.sqrt(g.double().square().sum()) * scale
        s["norm"].copy_(norm)
        scale = (scale * torch.clamp(c["clip"] / (norm + 1e-6), max=1.0)).float()
    g = g * scale
    s["step"] += 1
    t = s["step"].double()
    if c["state"] == "f32":
        m, v = s["m"], s["v"]
    else:
        m = _flat(_blocks(s["m"].float(), s) * s["scales"][0].unsqueeze(1), s)
        v = _flat(_blocks(s["v"].float(), s) * s["scales"][1].unsqueeze(1), s).square_()
    m.mul_(BETA1).add_(g * (1 - BETA1))
    v.mul_(BETA2).add_(g * (1 - BETA2) * g)
    size, root = (LR / (1 - BETA1 ** t)).float(), torch.sqrt(1 - BETA2 ** t).float()
    change = m / (torch.sqrt(v) / root + EPS) * size
    keep = 1 - LR * DECAY * s["decay"]
    for k, p in enumerate(s["params"]):
        p.mul_(keep).sub_(change)
        if s["operands"]:
            s["operands"][k].copy_(p)
    if c["state"] == "8bit":
        (cm, sm), (cr, sr) = _encode(_blocks(m, s)), _encode_root(_blocks(torch.sqrt(v), s))
        s["m"].view(torch.uint8).copy_(_flat(cm.view(torch.uint8), s))
        s["v"].view(torch.uint8).copy_(_flat(cr.view(torch.uint8), s))
        s["scales"].copy_(torch.cat([sm, sr], 1).t())
    return _adam_outputs(s)


def _adam_outputs(s):
    return {"params": s["params"], "operands": s["operands"], "m": s["m"], "v": s["v"], "scales": s["scales"], "step": s["step"],
            "norm": s["norm"]}


def run(state):
    c, s = state["case"], state
    if c["op"] == "adam":
        if not own:
            return _adam_plain(s, c)
        s["adam"].step(s["grad"], s["params"], s["m"], s["v"], s["step"], LR, weight_decay=DECAY, scales=s["scales"],
                       operands=s["operands"], grad_scale=c["scale"], max_norm=c["clip"], norm=s["norm"])
        return _adam_outputs(s)
    if not own:
        if c["op"] == "train":
            return _train_plain(s, c)
        _logits_plain(s, c)
        return {"loss": s["loss"], "lse": s["lse"]}
    s["head"].forward(s["x"], s["w"], s["labels"], s["loss"], s["lse"], bias=s["bias"])
    if c["op"] == "loss":
        return {"loss": s["loss"], "lse": s["lse"]}
    s["head"].backward(s["x"], s["w"], s["labels"], s["lse"], dloss=s["dloss"], bias=s["bias"], dx=s["dx"], dw=s["dw"],
                       db=s["db"], accumulate=c["accumulate"])
    return {"loss": s["loss"], "lse": s["lse"], "dx": s["dx"], "dw": s["dw"], "db": s["db"]}


# -- what a pass has to do, and its result in 64 bits --------------------------

def work(case):
    size = {"f32": 4, "f16": 2, "bf16": 2, "": 0}
    if case["op"] == "adam":
        n = sum(_tensors(case["tensors"])[0])
        state = 16 if case["state"] == "f32" else 4 + 16 / BLOCK
        return {"bytes": n * (size[case["grad"]] + state + case["copies"] * (8 + size[case["operands"]])), "flops": 0}
    t, i, v, e = case["tokens"], case["in"], case["vocab"], size[case["dtype"]]
    moved = e * (t * i + v * i + v * case["bias"]) + 16 * t
    if case["op"] == "loss":
        return {"bytes": moved, "flops": 2 * t * i * v}
    moved += e * t * i + 4 * t + size[case["grad"]] * (v * i + v * case["bias"]) * (1 + case["accumulate"])
    return {"bytes": moved, "flops": 6 * t * i * v}


def _exact_loss(case, s):
    x, w = s["x"].double(), s["w"].double()
    z = torch.matmul(x, w.mT)
    if case["bias"]:
        z += s["bias"].double()
    lse = torch.logsumexp(z, 1)
    eps, valid = case["smoothing"], s["labels"] >= 0
    target = torch.full_like(z, eps / case["vocab"])
    target[valid, s["labels"][valid]] += 1 - eps
    # sum of the targets' logits, entry by entry
    loss = torch.where(valid, lse - torch.einsum("tv,tv->t", target, z), 0.0)
    out = {"loss": loss, "lse": lse}
    if case["op"] == "loss":
        return out
    dz = torch.softmax(z, 1) - target
    del z, target
    dz = torch.where(valid.unsqueeze(1), dz * s["dloss"].double().unsqueeze(1), 0.0)
    keep = 1.0 if case["accumulate"] else 0.0
    out["dx"] = torch.matmul(dz, w)
    out["dw"] = torch.addmm(s["dw"].double(), dz.mT, x, beta=keep)
    out["db"] = torch.sum(dz, 0) + keep * s["db"].double() if case["bias"] else None
    return out


def _exact_codes(rows):
    """Values of e4m3 codes, scaled by the largest of each row: rounded to 3 bits behind the first, 2^-9 at the finest."""
    top = rows.abs().max(1, keepdim=True).values
    u = torch.where(top >= 2.0 ** -100, rows / top * TOP, torch.zeros_like(rows))
    grid = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(u / grid) * grid, torch.where(top >= 2.0 ** -100, top / TOP, torch.zeros_like(top))


def _exact_adam(case, s):
    g = s["grad"].double() * case["scale"]
    norm = torch.linalg.vector_norm(g)
    if case["clip"]:
        g = g * min(1.0, case["clip"] / (float(norm) + 1e-6))
    if case["state"] == "f32":
        m, v = s["m"].double(), s["v"].double()
    else:
        m = _flat(_blocks(s["m"].double(), s) * s["scales"][0].double().unsqueeze(1), s)
        v = _flat(_blocks(s["v"].double(), s) * s["scales"][1].double().unsqueeze(1), s) ** 2
    m = torch.lerp(g, m, BETA1)
    v = torch.lerp(g * g, v, BETA2)
    t = STEPS_DONE + 1
    change = LR * (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt() + EPS)
    decayed = torch.repeat_interleave(torch.tensor(s["decayed"], device="cuda").double(), torch.tensor(s["sizes"], device="cuda"))
    new = s["params"][0].double()
    new = new - LR * DECAY * decayed * new - change
    out = {"params": [new] * case["copies"], "operands": [new] * case["copies"] if case["operands"] else None, "m": m, "v": v,
           "scales": None, "step": None, "norm": norm.reshape(1) if case["clip"] else None}
    if case["state"] == "8bit":
        (cm, sm), (cr, sr) = _exact_codes(_blocks(m, s)), _exact_codes(_blocks(v.sqrt(), s))
        root = _flat(cr, s)
        floor = (v > 0) & (_flat((sr > 0).double().expand_as(cr), s) > 0)
        out.update(m=_flat(cm, s), v=torch.where(floor, root.clamp(min=2.0 ** -9), root), scales=torch.cat([sm, sr], 1).mT)
    return out


def exact(case, seed):
    s = _inputs(case, seed)
    return _exact_adam(case, s) if case["op"] == "adam" else _exact_loss(case, s)
