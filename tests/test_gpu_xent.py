"""Softmax cross entropy of a linear head on the GPU against the same formulas in 64 bits.

Element-wise bounds, from the arithmetic (U = the storage type's unit roundoff,
2^-11 binary16, 2^-8 bfloat16; u = 2^-24):
 - a logit: each of the K additions loses at most one unit in the last place (2^-23)
   of a partial sum that the sum of magnitudes bounds: e_z = (K + 16) 2^-23 sum |x||w|,
   and of the bias once more;
 - with e the largest e_z of the token: sums of exp(z - largest) are off by the
   factor 1 + e + 2^-16 (2^-20 each term, up to 256 additions in a row at 2^-24
   each, which leaves a factor of 3 for joining them), so lse by e + 2^-16 and its
   rounding, and the loss log(1 + r) by r / (1 + r) = 1 - p of twice that and its own
   rounding (4 u); smoothing adds its share of e + 2^-16 mean |z| + 8 u |z|;
 - exp(z - lse) by its own 2 e + 2^-16 + 2^-22 |z - lse| + u |lse|;
 - dz in planes: U of itself (one), 2^-16 (bfloat16, two) or 2^-22 (binary16, two) and,
   for binary16's subnormals at a scale where the largest coefficient is above 2^14,
   2^-39 of that;
 - dx and dw: the sums' own additions as for the logits, of V or T terms; storing
   rounds once: U |value|, or half of 2^-24 below binary16's normal range; accumulation
   adds 2^-23 of what was there.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = {"f16": 2.0 ** -24, "bf16": 2.0 ** -130, "f32": 2.0 ** -140}


@pytest.fixture(scope="module")
def ddl():
    assert torch.cuda.is_available(), "GPU test needs a CUDA device"
    import __graft_entry__
    __graft_entry__.build()
    from gradient_all_reduce_ddl_gb300 import ddl as mod
    return mod


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(seed, rows, cols, dtype, sigma=1.0, ld=None, offset=0):
    """rows x cols view with the given row stride, `offset` elements into its storage, NaN around it."""
    ld = ld or cols
    flat = torch.full((offset + rows * ld,), float("nan"), dtype=TYPES[dtype], device="cuda")
    view = flat[offset:].view(rows, ld)[:, :cols]
    view.copy_(torch.randn(rows, cols, generator=_gen(seed), device="cuda") * sigma)
    return view


def _blank(rows, cols, dtype, ld=None, offset=0):
    """A view into storage full of a marker, and a check that nothing outside the view changed."""
    ld = ld or cols
    flat = torch.full((offset + rows * ld + 64,), 7.0, dtype=TYPES[dtype], device="cuda")
    view = flat[offset:offset + rows * ld].view(rows, ld)[:, :cols]

    def untouched():
        keep = flat.clone()
        keep[offset:offset + rows * ld].view(rows, ld)[:, :cols] = 7.0
        return bool((keep == 7.0).all())
    return view, untouched


def _within(got, want, bound):
    assert bool(torch.isfinite(got.double()).all())
    err = (got.double() - want).abs()
    worst = float((err / bound).max()) if err.numel() else 0.0
    assert worst <= 1.0, f"error is {worst:.2f} times its bound"


class Head:
    """Inputs of one call, its results in 64 bits, and their bounds."""

    def __init__(self, t, k, v, dtype="bf16", bias=False, smoothing=0.0, ignored=0.2, seed=0, sure=None, ldx=None, ldw=None,
                 offset=0, dloss=None):
        self.t, self.k, self.v, self.dtype, self.smoothing = t, k, v, dtype, smoothing
        gen = _gen(seed)
        self.w = _normal(seed + 1, v, k, dtype, k ** -0.5, ldw, offset)
        self.bias = _normal(seed + 2, 1, v, dtype, 0.5)[0] if bias else None
        self.labels = torch.randint(0, v, (t,), generator=gen, device="cuda")
        self.x = _normal(seed + 3, t, k, dtype, 1.0, ldx, offset)
        sure = torch.rand(t, 1, generator=gen, device="cuda") * (math.log(v) + 3) if sure is None else sure
        self.x.copy_(self.x.float() + sure * self.w[self.labels].float())
        self.labels[torch.rand(t, generator=gen, device="cuda") < ignored] = -100
        self.dloss = (torch.rand(t, generator=gen, device="cuda") + 0.5) / t if dloss is None else dloss

    def solve(self):
        x, w = self.x.double(), self.w.double()
        self.z = x @ w.t()
        mag = x.abs() @ w.abs().t()
        if self.bias is not None:
            self.z += self.bias.double()
            mag += self.bias.double().abs()
        self.ez = (self.k + 16) * 2.0 ** -23 * mag
        self.e = self.ez.amax(1)
        self.lse = torch.logsumexp(self.z, 1)
        self.valid = self.labels >= 0
        y = self.labels.clamp(min=0)
        q = torch.full_like(self.z, self.smoothing / self.v)
        q[torch.arange(self.t, device="cuda"), y] += 1 - self.smoothing
        p = torch.exp(self.z - self.lse[:, None])
        # lse - z_y as log(1 + the others), which keeps small losses
        zy = self.z.gather(1, y[:, None])
        others = self.z.scatter(1, y[:, None], float("-inf")) - zy
        r = torch.logsumexp(others, 1)
        own = torch.nn.functional.softplus(r)
        loss = own + self.smoothing * (zy[:, 0] - self.z.mean(1))
        self.loss = torch.where(self.valid, loss, 0.0)
        miss = torch.sigmoid(r)  # 1 - p of the label
        self.loss_bound = (2 * self.e + 2.0 ** -16) * miss + 4 * U["f32"] * own + 1e-30
        if self.smoothing:
            self.loss_bound += self.smoothing * (2 * self.e + 2.0 ** -16 * self.z.abs().mean(1)) + 8 * U["f32"] * (
                zy[:, 0].abs() + self.z.abs().mean(1) + own)
        self.lse_bound = self.e + 2.0 ** -16 + 2 * U["f32"] * self.lse.abs()
        c = torch.where(self.valid, self.dloss.double(), 0.0)[:, None]
        self.dz = torch.where(self.valid[:, None], (p - q) * c, 0.0)
        rel = (2 * self.e + 2.0 ** -16 + 2 * U["f32"] * self.lse.abs())[:, None] + 2.0 ** -22 * (self.z - self.lse[:, None]).abs()
        self.dz_err = c.abs() * (p * rel + 4 * U["f32"] * (p + q))
        self.floor = 2.0 ** -39 * float(c.abs().max()) if self.dtype == "f16" else 0.0
        return self

    def plane_err(self, planes):
        u = U[self.dtype] if planes == 1 else 2.0 ** -16 if self.dtype == "bf16" else 2.0 ** -22
        return self.dz_err + u * self.dz.abs() + self.floor

    def forward(self, ddl, head, stream=None):
        loss, lse = (torch.full((self.t,), 7.0, device="cuda") for _ in range(2))
        head.forward(self.x, self.w, self.labels, loss, lse, bias=self.bias, stream=stream)
        return loss, lse

    def check_forward(self, loss, lse):
        _within(lse, self.lse, self.lse_bound)
        _within(loss, self.loss, self.loss_bound)
        assert bool((loss[~self.valid] == 0).all())

    def check_backward(self, dx=None, dw=None, db=None, old_w=0.0, old_b=0.0):
        mag = self.dz.abs()
        if dx is not None:
            want = self.dz @ self.w.double()
            bound = (self.plane_err(1) + (self.v + 16) * 2.0 ** -23 * mag) @ self.w.double().abs() + U[self.dtype] * want.abs()
            _within(dx, want, bound + TINY[self.dtype])
        name = {torch.float32: "f32", torch.float16: "f16"}
        if dw is not None:
            g = name[dw.dtype]
            want = self.dz.t() @ self.x.double() + old_w
            err = self.plane_err(1 if self.dtype == "f16" and g == "f16" else 2)
            bound = (err + (self.t + 16) * 2.0 ** -23 * mag).t() @ self.x.double().abs()
            _within(dw, want, bound + 2.0 ** -23 * (want.abs() + abs(old_w)) + U[g] * want.abs() + TINY[g])
        if db is not None:
            g = name[db.dtype]
            want = self.dz.sum(0) + old_b
            bound = (self.dz_err + (self.t + 16) * 2.0 ** -24 * mag).sum(0)
            _within(db, want, bound + 2.0 ** -23 * (want.abs() + abs(old_b)) + U[g] * want.abs() + TINY[g])


def _run(ddl, h, grad="f32", accumulate=False, ldg=None, goff=0, ldd=None):
    """Forward and backward of one call, everything asked for, and checked."""
    h.solve()
    with ddl.CrossEntropy(h.k, h.v, h.t, h.dtype, smoothing=h.smoothing) as head:
        loss, lse = h.forward(ddl, head)
        h.check_forward(loss, lse)
        dx, keep_x = _blank(h.t, h.k, h.dtype, ldd, goff)
        dw, keep_w = _blank(h.v, h.k, grad, ldg, goff)
        db, keep_b = _blank(1, h.v, grad, None, goff)
        head.backward(h.x, h.w, h.labels, lse, dloss=h.dloss, bias=h.bias, dx=dx, dw=dw, db=db[0], accumulate=accumulate)
        head.check()
        old = 7.0 if accumulate else 0.0
        h.check_backward(dx, dw, db[0], old, old)
        assert keep_x() and keep_w() and keep_b()


SIZES = [(1, 1, 1), (1, 64, 1000), (2, 8, 5), (16, 130, 300), (31, 64, 128), (32, 1024, 5000), (33, 72, 129), (64, 200, 777),
         (65, 64, 777), (127, 63, 255), (128, 64, 128), (129, 65, 513), (256, 2048, 1000), (300, 520, 2049), (1000, 96, 257),
         (1030, 256, 4100), (2500, 64, 3)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("t, k, v", SIZES)
def test_sizes(ddl, t, k, v, dtype):
    _run(ddl, Head(t, k, v, dtype, bias=(t + v) % 2 == 1, smoothing=0.1 if t % 3 == 0 else 0.0, seed=t + v))


@pytest.mark.parametrize("t, k, v", [(1, 64, 65536), (16, 320, 40000), (32, 72, 19457), (33, 130, 20011), (64, 1032, 70001)])
def test_few_tokens_large_vocabularies(ddl, t, k, v):
    """More tiles than SMs: several in a row, of 128 rows or fewer, the last ones cut."""
    h = Head(t, k, v, "bf16", bias=True, smoothing=0.1, seed=t + v).solve()
    with ddl.CrossEntropy(k, v, t, "bf16", smoothing=0.1) as head:
        h.check_forward(*h.forward(ddl, head))
        head.check()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("grad, accumulate", [("f16", False), ("f16", True), ("f32", True)])
@pytest.mark.parametrize("t, k, v", [(7, 40, 33), (200, 96, 515), (700, 1030, 1100)])
def test_gradient_types_and_accumulation(ddl, t, k, v, dtype, grad, accumulate):
    scale = 64.0 if grad == "f16" else 1.0
    h = Head(t, k, v, dtype, bias=True, smoothing=0.1, seed=5)
    h.dloss *= scale
    _run(ddl, h, grad, accumulate)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("ldx, ldw, offset, ldg, goff, ldd", [(101, 103, 1, 105, 3, 107), (104, 112, 8, 112, 4, 104), (100, 100, 2, 100, 1, 100),
                                                            (128, 128, 0, 100, 0, 101)])
def test_strides_and_alignments(ddl, dtype, ldx, ldw, offset, ldg, goff, ldd):
    for t in (20, 150):
        _run(ddl, Head(t, 100, 333, dtype, bias=True, seed=6, ldx=ldx, ldw=ldw, offset=offset), "f16", False, ldg, goff, ldd)
        _run(ddl, Head(t, 100, 333, dtype, bias=True, seed=6, ldx=ldx, ldw=ldw, offset=offset), "f32", True, ldg, goff, ldd)


def test_operands_in_one_buffer(ddl):
    """x and dx as column blocks of one buffer, the weights' and the bias's gradients at any element of a flat one."""
    h = Head(90, 72, 200, "f16", bias=True, seed=7).solve()
    wide = torch.full((90, 160), 7.0, dtype=torch.float16, device="cuda")
    wide[:, :72] = h.x
    flat = torch.zeros(200 * 72 + 200 + 9, device="cuda")
    h.x = wide[:, :72]
    with ddl.CrossEntropy(72, 200, 90, "f16") as head:
        loss, lse = h.forward(ddl, head)
        head.backward(h.x, h.w, h.labels, lse, dloss=h.dloss, bias=h.bias, dx=wide[:, 80:152], dw=flat[5:5 + 14400].view(200, 72),
                      db=flat[14405:14605])
    h.check_forward(loss, lse)
    h.check_backward(wide[:, 80:152], flat[5:14405].view(200, 72), flat[14405:14605])
    assert bool((wide[:, 72:80] == 7).all()) and bool((wide[:, 152:] == 7).all())
    assert not flat[:5].any() and not flat[14605:].any()


@pytest.mark.parametrize("wanted", ["dx", "dw", "db", "dx dw", "dw db", "dx db"])
def test_any_of_the_gradients(ddl, wanted):
    h = Head(140, 96, 300, "bf16", bias=True, seed=8).solve()
    out = {"dx": torch.empty_like(h.x), "dw": torch.empty(300, 96, device="cuda"), "db": torch.empty(300, device="cuda")}
    out = {n: x for n, x in out.items() if n in wanted.split()}
    with ddl.CrossEntropy(96, 300, 140, "bf16") as head:
        _, lse = h.forward(ddl, head)
        head.backward(h.x, h.w, h.labels, lse, dloss=h.dloss, bias=h.bias, **out)
        head.check()
    h.check_backward(**out)


def test_fewer_tokens_than_the_most(ddl):
    with ddl.CrossEntropy(80, 400, 600, "f16", smoothing=0.05) as head:
        for t in (600, 1, 77, 64, 599, 0, 3):
            h = Head(t, 80, 400, "f16", bias=True, smoothing=0.05, seed=t)
            loss, lse = h.forward(ddl, head)
            dx, dw, db = torch.empty_like(h.x), torch.full((400, 80), 7.0, device="cuda"), torch.full((400,), 7.0, device="cuda")
            head.backward(h.x, h.w, h.labels, lse, dloss=h.dloss, bias=h.bias, dx=dx, dw=dw, db=db)
            if t:
                h.solve()
                h.check_forward(loss, lse)
                h.check_backward(dx, dw, db)
            else:  # empty sums
                assert not dw.any() and not db.any()
                dw.fill_(7.0)
                head.backward(h.x, h.w, h.labels, lse, dw=dw, accumulate=True)
                assert bool((dw == 7).all())
        head.check()


def test_no_weights_of_the_tokens(ddl):
    """dloss left out is ones."""
    h = Head(100, 64, 90, "f16", seed=9, dloss=torch.ones(100, device="cuda")).solve()
    dx, dw = torch.empty_like(h.x), torch.empty(90, 64, device="cuda")
    with ddl.CrossEntropy(64, 90, 100, "f16") as head:
        _, lse = h.forward(ddl, head)
        head.backward(h.x, h.w, h.labels, lse, dx=dx, dw=dw)
    h.check_backward(dx, dw)


def test_either_result_of_the_forward_pass(ddl):
    h = Head(70, 64, 500, "bf16", seed=10).solve()
    with ddl.CrossEntropy(64, 500, 70, "bf16") as head:
        loss, lse = h.forward(ddl, head)
        one, other = torch.empty_like(loss), torch.empty_like(lse)
        head.forward(h.x, h.w, h.labels, one)
        head.forward(h.x, h.w, h.labels, None, other)
    assert torch.equal(loss, one) and torch.equal(lse, other)


@pytest.mark.parametrize("t", [5, 40, 300])
def test_small_losses_keep_their_precision(ddl, t):
    """Labels up to 40 above the rest: losses from 1 to 1e-14, each within the relative error of its bound."""
    h = Head(t, 256, 1500, "bf16", seed=11, ignored=0.0, sure=torch.linspace(0, 40, t, device="cuda")[:, None]).solve()
    with ddl.CrossEntropy(256, 1500, t, "bf16") as head:
        loss, lse = h.forward(ddl, head)
    h.check_forward(loss, lse)
    assert float(h.loss.min()) < 1e-9


@pytest.mark.parametrize("dtype, size", [("f16", 1e-12), ("f16", 1e-30), ("f16", 1e8), ("bf16", 1e-12), ("bf16", 1e20)])
def test_small_and_large_token_weights(ddl, dtype, size):
    h = Head(150, 64, 200, dtype, bias=True, seed=12, dloss=torch.rand(150, generator=_gen(1), device="cuda") * size).solve()
    dw, db = torch.empty(200, 64, device="cuda"), torch.empty(200, device="cuda")
    with ddl.CrossEntropy(64, 200, 150, dtype) as head:
        _, lse = h.forward(ddl, head)
        head.backward(h.x, h.w, h.labels, lse, dloss=h.dloss, bias=h.bias, dw=dw, db=db)
    h.check_backward(None, dw, db)


@pytest.mark.parametrize("t", [3, 50, 200])
def test_ignored_tokens_do_not_count(ddl, t):
    """Their weights may be anything; all of them ignored gives zeros."""
    h = Head(t, 64, 300, "f16", bias=True, seed=13, ignored=0.5).solve()
    with ddl.CrossEntropy(64, 300, t, "f16") as head:
        _, lse = h.forward(ddl, head)
        out = []
        for bad in (None, float("inf"), float("nan")):
            c = h.dloss.clone()
            if bad is not None:
                c[~h.valid] = bad
            dx, dw, db = torch.empty_like(h.x), torch.empty(300, 64, device="cuda"), torch.empty(300, device="cuda")
            head.backward(h.x, h.w, h.labels, lse, dloss=c, bias=h.bias, dx=dx, dw=dw, db=db)
            out.append((dx, dw, db))
        for got in out[1:]:
            assert all(torch.equal(a, b) for a, b in zip(got, out[0]))
        none = torch.full_like(h.labels, -1)
        loss = torch.empty(t, device="cuda")
        head.forward(h.x, h.w, none, loss, lse, bias=h.bias)
        _within(lse, h.lse, h.lse_bound)
        head.backward(h.x, h.w, none, lse, dloss=h.dloss, bias=h.bias, dx=dx, dw=dw, db=db)
        assert not loss.any() and not dx.any() and not dw.any() and not db.any()
        head.check()


@pytest.mark.parametrize("t", [4, 150])
def test_masked_entries(ddl, t):
    """A bias of -infinity takes entries out: the rest is as if they were not there."""
    h = Head(t, 64, 400, "bf16", bias=True, seed=14)
    out = torch.rand(400, generator=_gen(2), device="cuda") < 0.5
    out[h.labels.clamp(min=0)] = False
    small = Head(t, 64, 400, "bf16", bias=True, seed=14)
    small.w, small.bias, small.v = h.w[~out].contiguous(), h.bias[~out].contiguous(), int((~out).sum())
    place = torch.cumsum((~out).long(), 0) - 1
    small.labels = torch.where(h.labels >= 0, place[h.labels.clamp(min=0)], h.labels)
    small.solve()
    h.bias = torch.where(out, float("-inf"), h.bias.float()).bfloat16()
    with ddl.CrossEntropy(64, 400, t, "bf16") as head:
        loss, lse = h.forward(ddl, head)
        dx, dw, db = torch.empty_like(h.x), torch.empty(400, 64, device="cuda"), torch.empty(400, device="cuda")
        head.backward(h.x, h.w, h.labels, lse, dloss=h.dloss, bias=h.bias, dx=dx, dw=dw, db=db)
    small.check_forward(loss, lse)
    small.check_backward(dx, dw[~out], db[~out])
    assert not dw[out].any() and not db[out].any()


@pytest.mark.parametrize("t", [4, 150])
def test_nothing_left_and_infinities(ddl, t):
    """All entries masked: lse is -infinity, the loss NaN, as the formula has it.  +infinity: lse is +infinity.  A row with a
    NaN spoils its own results alone."""
    h = Head(t, 64, 400, "bf16", bias=True, seed=15, ignored=0.0).solve()
    with ddl.CrossEntropy(64, 400, t, "bf16") as head:
        loss, lse = torch.empty(t, device="cuda"), torch.empty(t, device="cuda")
        head.forward(h.x, h.w, h.labels, loss, lse, bias=torch.full_like(h.bias, float("-inf")))
        assert bool((lse == float("-inf")).all()) and bool(loss.isnan().all())
        top = h.bias.clone()
        free = [v for v in range(400) if not bool((h.labels == v).any())][0]
        top[free] = float("inf")
        head.forward(h.x, h.w, h.labels, loss, lse, bias=top)
        assert bool((lse == float("inf")).all()) and bool((loss == float("inf")).all())
        x = h.x.clone()
        x[1, 3] = float("nan")
        head.forward(x, h.w, h.labels, loss, lse, bias=h.bias)
        others = torch.arange(t, device="cuda") != 1
        assert bool(loss[1].isnan()) and bool(lse[1].isnan())
        _within(loss[others], h.loss[others], h.loss_bound[others])
        _within(lse[others], h.lse[others], h.lse_bound[others])


def test_one_entry(ddl):
    """A vocabulary of one: nothing to lose."""
    h = Head(40, 64, 1, "f16", seed=16, ignored=0.0).solve()
    dw, dx = torch.empty(1, 64, device="cuda"), torch.empty_like(h.x)
    with ddl.CrossEntropy(64, 1, 40, "f16") as head:
        loss, lse = h.forward(ddl, head)
        head.backward(h.x, h.w, h.labels, lse, dx=dx, dw=dw)
    assert not loss.any()
    assert torch.equal(lse.isfinite(), torch.ones_like(lse, dtype=torch.bool))


@pytest.mark.parametrize("t", [5, 150])
def test_labels_past_the_vocabulary_are_reported(ddl, t):
    h = Head(t, 64, 400, "f16", seed=17, ignored=0.0)
    good = h.labels.clone()
    h.solve()
    h.labels = good.clone()
    h.labels[2], h.labels[3] = 400, 1 << 40
    with ddl.CrossEntropy(64, 400, t, "f16") as head:
        loss, lse = h.forward(ddl, head)
        bad = torch.zeros(t, dtype=torch.bool, device="cuda")
        bad[2:4] = True
        assert bool(loss[bad].isnan().all())
        _within(loss[~bad], h.loss[~bad], h.loss_bound[~bad])
        with pytest.raises(ddl.DDLError) as e:
            head.check()
        assert e.value.status == ddl.DDL_ERR_DEVICE_CHECK
        head.check()  # reported once
        dx = torch.full_like(h.x, 7.0)
        head.backward(h.x, h.w, h.labels, lse, dx=dx)
        assert not dx[bad].any()


@pytest.mark.parametrize("t, k, v, dtype", [(16384, 64, 40001, "bf16"), (16384, 65, 20001, "f16")])
def test_pieces_of_the_vocabulary(ddl, t, k, v, dtype):
    """More logits than a piece holds: three or two pieces, the last one ragged; dx is added over them, in odd rows, too."""
    h = Head(t, k, v, dtype, bias=True, seed=18).solve()
    with ddl.CrossEntropy(k, v, t, dtype) as head:
        loss, lse = h.forward(ddl, head)
        dx, dw, db = torch.empty_like(h.x), torch.empty(v, k, device="cuda"), torch.empty(v, device="cuda")
        head.backward(h.x, h.w, h.labels, lse, dloss=h.dloss, bias=h.bias, dx=dx, dw=dw, db=db)
        head.check()
    h.check_forward(loss, lse)
    h.check_backward(dx, dw, db)


@pytest.mark.parametrize("t", [3, 64, 65, 500, 4096, 4097])
@pytest.mark.parametrize("k, v", [(96, 1500), (1030, 333)])
def test_binary32_dw_of_bfloat16_heads(ddl, t, k, v):
    """As exact as sums in binary32: the 2-norm of the error, with weights that differ, in two or three planes of dz.  Two keep
    dz to 2^-17 of itself, uniformly off (2^-17 / sqrt 3 of the norm); the logits are off by 16 roundings of 2^-24 of their
    size, up to 16, twice."""
    h = Head(t, k, v, "bf16", bias=True, seed=25).solve()
    dw = torch.empty(v, k, device="cuda")
    with ddl.CrossEntropy(k, v, t, "bf16") as head:
        _, lse = h.forward(ddl, head)
        head.backward(h.x, h.w, h.labels, lse, dloss=h.dloss, bias=h.bias, dw=dw)
    h.check_backward(None, dw)
    want = h.dz.t() @ h.x.double()
    off = float((dw.double() - want).norm() / want.norm())
    assert off <= 2.0 ** -17 / math.sqrt(3) * (t > 4096) + 2 * 16 * 16 * 2.0 ** -24


@pytest.mark.parametrize("t", [16384, 16385, 20000])
def test_many_tokens(ddl, t):
    """On either side of the number up to which the gradient launch makes dz's scale itself."""
    h = Head(t, 40, 50, "f16", bias=True, seed=24, dloss=torch.rand(t, generator=_gen(4), device="cuda") * 1e-9)
    h.dloss[-1] = 1e-3  # the largest is the last
    h.labels[-1] = 7
    _run(ddl, h)


def test_bands_of_tokens(ddl):
    """The largest vocabulary: two launches share out the tokens, the second has a few."""
    t, k, v = 1030, 16, 1 << 22
    h = Head(t, k, v, "f16", seed=19)
    with ddl.CrossEntropy(k, v, t, "f16") as head:
        loss, lse = h.forward(ddl, head)
        head.check()
    for at in (0, 500, 1020):
        part = Head(10, k, v, "f16", seed=19)
        part.x, part.w, part.labels, part.dloss = h.x[at:at + 10], h.w, h.labels[at:at + 10], h.dloss[at:at + 10]
        part.solve()
        part.check_forward(loss[at:at + 10], lse[at:at + 10])


def test_formula_is_torchs(ddl):
    """The 64-bit reference is torch's own cross entropy and its gradient."""
    h = Head(60, 32, 70, "f16", bias=True, smoothing=0.2, seed=20).solve()
    x, w, b = (a.double().clone().requires_grad_() for a in (h.x, h.w, h.bias))
    loss = torch.nn.functional.cross_entropy(x @ w.t() + b, h.labels, reduction="none", label_smoothing=0.2)
    assert torch.allclose(loss, h.loss, rtol=1e-12, atol=1e-12)
    (loss * h.dloss.double()).sum().backward()
    assert torch.allclose(x.grad, h.dz @ w.detach(), rtol=1e-10, atol=1e-14)
    assert torch.allclose(w.grad, h.dz.t() @ x.detach(), rtol=1e-10, atol=1e-14)
    assert torch.allclose(b.grad, h.dz.sum(0), rtol=1e-10, atol=1e-14)


def test_gradient_against_differences(ddl):
    """The weighted loss at x + d and x - d differs by twice dx . d, up to a third of the cube of the logits' spread along d."""
    h = Head(80, 64, 150, "f16", bias=True, smoothing=0.1, seed=21).solve()
    step = (torch.sign(h.dz @ h.w.double()) * 0.02).half()  # along the gradient, where the difference is large
    up = (h.x + step).half()
    down = (h.x - step).half()
    mid, d = (up.double() + down.double()) / 2, (up.double() - down.double()) / 2
    h.x = mid.half()
    exactly = bool((h.x.double() == mid).all())
    d = torch.where(h.x.double() == mid, d, 0.0)  # where the midpoint is a binary16 number, too
    up, down = (h.x.double() + d).half(), (h.x.double() - d).half()
    assert exactly or bool((d != 0).float().mean() > 0.3)
    h.solve()
    with ddl.CrossEntropy(64, 150, 80, "f16", smoothing=0.1) as head:
        _, lse = h.forward(ddl, head)
        dx = torch.empty_like(h.x)
        dl = h.dloss * 1024
        head.backward(h.x, h.w, h.labels, lse, dloss=dl, bias=h.bias, dx=dx)
        ends = []
        for x in (up, down):
            loss = torch.empty(80, device="cuda")
            head.forward(x, h.w, h.labels, loss, bias=h.bias)
            ends.append(loss.double())
    c = torch.where(h.valid, dl.double(), 0.0)
    got = (c * (ends[0] - ends[1])).sum()
    want = 2 * (dx.double() * d).sum()
    spread = (d @ h.w.double().t())
    spread = spread.amax(1) - spread.amin(1)
    bound = (c * spread ** 3).sum() / 3 + (c * 4 * h.loss_bound).sum() + 2 * (dx.double().abs() * d.abs()).sum() * 2.0 ** -9
    assert abs(float(got - want)) <= float(bound)
    assert abs(float(want)) > 3 * float(bound)


def _everything(ddl, head, h, stream=None):
    loss, lse = h.forward(ddl, head, stream)
    dx, dw, db = torch.empty_like(h.x), torch.zeros(h.v, h.k, device="cuda"), torch.zeros(h.v, device="cuda")
    head.backward(h.x, h.w, h.labels, lse, dloss=h.dloss, bias=h.bias, dx=dx, dw=dw, db=db, stream=stream)
    return loss, lse, dx, dw, db


@pytest.mark.parametrize("t, k, v", [(3, 100, 1000), (256, 1024, 1000), (1500, 128, 3000)])
def test_repeats_bit_for_bit(ddl, t, k, v):
    h = Head(t, k, v, "f16", bias=True, smoothing=0.1, seed=22)
    with ddl.CrossEntropy(k, v, t, "f16", smoothing=0.1) as head:
        first = _everything(ddl, head, h)
        for _ in range(5):
            assert all(torch.equal(a, b) for a, b in zip(first, _everything(ddl, head, h)))


def test_two_handles_on_two_streams(ddl):
    hs = [Head(700, 256, 2000, "bf16", bias=True, seed=23 + i) for i in range(2)]
    heads = [ddl.CrossEntropy(256, 2000, 700, "bf16") for _ in hs]
    alone = [_everything(ddl, a, h) for a, h in zip(heads, hs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in hs]
    together = [None, None]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                together[i] = _everything(ddl, heads[i], hs[i], s)
    torch.cuda.synchronize()
    for a, b in zip(alone, together):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    for head in heads:
        head.check()
        head.close()


def test_captured_calls_replay_on_new_inputs(ddl):
    a, b = (Head(200, 96, 1500, "f16", bias=True, seed=30 + i) for i in range(2))
    with ddl.CrossEntropy(96, 1500, 200, "f16") as head:
        want = _everything(ddl, head, b)
        _everything(ddl, head, a)
        x, w, labels, bias, dloss = a.x.clone(), a.w.clone(), a.labels.clone(), a.bias.clone(), a.dloss.clone()
        out = [torch.empty_like(t) for t in want]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            head.forward(x, w, labels, out[0], out[1], bias=bias)
            head.backward(x, w, labels, out[1], dloss=dloss, bias=bias, dx=out[2], dw=out[3], db=out[4])
        for to, new in zip((x, w, labels, bias, dloss), (b.x, b.w, b.labels, b.bias, b.dloss)):
            to.copy_(new)
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(out, want))
        head.check()


STOPS = [dict(products=0), dict(products=1), dict(loads_even=0), dict(loads_even=3), dict(loads_odd=0), dict(loads_odd=2)]


@pytest.mark.parametrize("stop", STOPS)
@pytest.mark.parametrize("t, k, v", [(16, 512, 2000), (100, 1024, 500), (2048, 512, 4096)])
def test_waits_that_run_out_are_reported(ddl, t, k, v, stop):
    """A role of the product kernel stops early, the others' waits run out: the call ends, the check reports it, and the
    next call gives the bits of one before."""
    h = Head(t, k, v, "bf16", bias=True, seed=40)
    with ddl.CrossEntropy(k, v, t, "bf16") as head:
        want = _everything(ddl, head, h)
        for which in (0, 1):
            ddl.ddl_xent_selftest_wait_timeout(head.handle, 300, **stop)
            if which == 0:
                h.forward(ddl, head)
            else:
                head.backward(h.x, h.w, h.labels, want[1], dx=torch.empty_like(h.x), dw=torch.empty(v, k, device="cuda"))
            torch.cuda.synchronize()
            try:
                head.check()
                reported = False
            except ddl.DDLError as e:
                assert e.status == ddl.DDL_ERR_DEVICE_CHECK
                reported = True
            # stops of odd CTAs' loads reach pairs only; a CTA of a split contraction may have no second chunk or fourth block
            assert reported or stop not in (dict(products=0), dict(loads_even=0))
            assert all(torch.equal(a, b) for a, b in zip(want, _everything(ddl, head, h)))
            head.check()


def test_memory_that_is_short(ddl, monkeypatch):
    """A failed allocation is reported and queues nothing; the next call makes up for it."""
    h = Head(100, 63, 90, "f16", bias=True, seed=51).solve()
    with ddl.CrossEntropy(63, 90, 100, "f16") as head:
        dx, dw = torch.empty_like(h.x), torch.full((90, 63), 7.0, device="cuda")
        monkeypatch.setenv("DDL_INJECT_ALLOC_FAILURE", "1")
        with pytest.raises(ddl.DDLError) as e:
            h.forward(ddl, head)
        assert e.value.status == ddl.DDL_ERR_OOM
        monkeypatch.delenv("DDL_INJECT_ALLOC_FAILURE")
        loss, lse = h.forward(ddl, head)
        h.check_forward(loss, lse)
        monkeypatch.setenv("DDL_INJECT_ALLOC_FAILURE", "1")
        with pytest.raises(ddl.DDLError) as e:
            head.backward(h.x, h.w, h.labels, lse, dloss=h.dloss, bias=h.bias, dx=dx, dw=dw)
        assert e.value.status == ddl.DDL_ERR_OOM
        torch.cuda.synchronize()
        assert bool((dw == 7).all())
        monkeypatch.delenv("DDL_INJECT_ALLOC_FAILURE")
        head.backward(h.x, h.w, h.labels, lse, dloss=h.dloss, bias=h.bias, dx=dx, dw=dw)
        h.check_backward(dx, dw)


def test_checks_of_the_object(ddl):
    h = Head(20, 64, 100, "f16", bias=True, seed=50)
    with ddl.CrossEntropy(64, 100, 20, "f16") as head:
        loss = torch.empty(20, device="cuda")
        ok = dict(x=h.x, w=h.w, labels=h.labels, loss=loss, bias=h.bias)
        head.forward(**ok)
        for change in (dict(x=h.x.bfloat16()), dict(w=h.w[:99]), dict(labels=h.labels.int()), dict(loss=loss.double()),
                       dict(loss=loss[:19]), dict(bias=h.bias.float()), dict(labels=h.labels.cpu()), dict(x=h.x.t().contiguous().t())):
            with pytest.raises(ValueError):
                head.forward(**{**ok, **change})
        with pytest.raises(ddl.DDLError) as e:
            head.forward(**{**ok, "loss": None})
        assert e.value.status == ddl.DDL_ERR_INVALID_ARG
        with pytest.raises(ddl.DDLError) as e:
            head.forward(torch.zeros(21, 64, dtype=torch.float16, device="cuda"), h.w, torch.zeros(21, dtype=torch.long, device="cuda"),
                         torch.empty(21, device="cuda"))
        assert e.value.status == ddl.DDL_ERR_INVALID_ARG
        with pytest.raises(ValueError):
            head.backward(h.x, h.w, h.labels, loss, dw=torch.empty(100, 64, device="cuda", dtype=torch.bfloat16))


def test_a_training_step_of_all_operators(ddl):
    """Two workers: a layer, the head's loss, both backward passes into flat gradients, the all-reduce, and AdamW with the
    16-bit weights of the next step; against the same in 64 bits with the bounds of its parts."""
    width, vocab, batch, workers, lr = 64, 300, 96, 2, 1e-2
    n1, n2 = width * width, vocab * width
    n = n1 + n2 + vocab
    start = torch.cat([torch.randn(n1 + n2, generator=_gen(60), device="cuda") * width ** -0.5, torch.zeros(vocab, device="cuda")])
    params = [start.clone() for _ in range(workers)]
    weights = [p.bfloat16() for p in params]
    grads = [torch.zeros(n, device="cuda") for _ in range(workers)]
    layer = ddl.Linear(width, width, batch, "bf16", "gelu")
    head = ddl.CrossEntropy(width, vocab, batch, "bf16")
    adam = ddl.Adam([(0, n1), (n1, n2), (n1 + n2, vocab, 1.0, 0.0)])
    state, plan = adam.new_state(), ddl.Plan(workers, n, "f32", "ring")
    xs = [torch.randn(batch, width, generator=_gen(61 + r), device="cuda").bfloat16() for r in range(workers)]
    ys = [torch.randint(0, vocab, (batch,), generator=_gen(71 + r), device="cuda") for r in range(workers)]
    loss, lse, dloss = torch.empty(batch, device="cuda"), torch.empty(batch, device="cuda"), torch.full((batch,), 1 / batch, device="cuda")
    ref = torch.zeros(n, dtype=torch.float64, device="cuda")
    losses = []
    for _ in range(2):
        ref.zero_()
        for x, y, g, o in zip(xs, ys, grads, weights):
            w1, w2, b2 = o[:n1].view(width, width), o[n1:n1 + n2].view(vocab, width), o[n1 + n2:]
            h, z, dh = (torch.empty(batch, width, dtype=torch.bfloat16, device="cuda") for _ in range(3))
            layer.forward(x, w1, h, z=z)
            losses.append(float(head.forward(h, w2, y, loss, lse, bias=b2).mean()))
            head.backward(h, w2, y, lse, dloss=dloss, bias=b2, dx=dh, dw=g[n1:n1 + n2].view(vocab, width), db=g[n1 + n2:])
            layer.backward(dh, x, z=z, dw=g[:n1].view(width, width))
            flat = o.double().requires_grad_()
            hid = torch.nn.functional.gelu(x.double() @ flat[:n1].view(width, width).t())
            out = hid @ flat[n1:n1 + n2].view(vocab, width).t() + flat[n1 + n2:]
            torch.nn.functional.cross_entropy(out, y).backward()
            ref += flat.grad / workers
        plan.allreduce(grads, 1 / workers)
        torch.cuda.synchronize()
        for part in (slice(0, n1), slice(n1, n1 + n2), slice(n1 + n2, n)):
            # h, dh and z, and dz within dh's product, are rounded to bfloat16 on the way: 2^-8 of their norms each
            assert float((grads[0][part].double() - ref[part]).norm() / ref[part].norm()) < 4 * 2.0 ** -8
        before = params[0].clone()
        adam.step(grads[0], params, lr=lr, operands=weights, **state)
        for p, o in zip(params, weights):
            assert torch.equal(p, params[0]) and torch.equal(o, p.bfloat16())
        assert float((params[0] - before).abs().max()) <= lr * 1.01 * (1 + 4)
    assert int(state["step"]) == 2 and all(math.isfinite(v) for v in losses)
    for handle in (layer, head, plan):
        handle.check()
    for handle in (layer, head, adam, plan):
        handle.close()


class LowHead(Head):
    """A head whose bias is far below zero on some entries.  Its sum with the products rounds to binary32 (and loses them where
    its half unit is above them, from 2^30 on): the reference's logits are rounded likewise, and off by the products' own error
    and, below that, one rounding more.  Gradients are those of the call's own lse."""

    def __init__(self, t, k, v, dtype, low, entries, masked=0, **more):
        super().__init__(t, k, v, dtype, bias=True, ignored=0.1, **more)
        self.bias[entries] = low
        self.bias[:masked] = float("-inf")
        if masked:
            self.labels = torch.where(self.labels >= 0, self.labels.clamp(min=masked), self.labels)

    def solve(self):
        x, w = self.x.double(), self.w.double()
        self.z = (x @ w.t() + self.bias.double()).float().double()
        size = torch.where(self.z.abs() < 2.0 ** 30, self.z.abs(), 0.0)
        self.ez = torch.where(self.z.isfinite(), (self.k + 16) * 2.0 ** -23 * (x.abs() @ w.abs().t()) + 2.0 ** -23 * size, 0.0)
        top = self.z.amax(1, keepdim=True)
        near = self.z > top - 40 - self.ez  # what is left of the others is less than 2^-24 of any sum
        self.e = torch.where(near, self.ez, 0.0).amax(1)
        self.lse = torch.logsumexp(self.z, 1)
        self.valid = self.labels >= 0
        y = torch.where(self.valid, self.labels, self.v - 1)  # (an entry that is never masked)
        zy = self.z.gather(1, y[:, None])
        r = torch.logsumexp(self.z.scatter(1, y[:, None], float("-inf")) - zy, 1)
        own = torch.nn.functional.softplus(r)
        self.loss = torch.where(self.valid, own, 0.0)
        e = torch.maximum(self.e, self.ez.gather(1, y[:, None])[:, 0])
        self.loss_bound = (2 * e + 2.0 ** -16) * torch.sigmoid(r) + 4 * U["f32"] * own + 1e-30
        self.lse_bound = self.e + 2.0 ** -16 + 2 * U["f32"] * self.lse.abs()
        return self

    def solve_backward(self, lse):
        """dz and its error, from the lse that the call is given."""
        d = self.z - lse.double()[:, None]
        q = torch.zeros_like(self.z)
        q[torch.arange(self.t, device="cuda"), self.labels.clamp(min=0)] = 1.0
        p = torch.exp(d)
        c = torch.where(self.valid, self.dloss.double(), 0.0)[:, None]
        self.dz = torch.where(self.valid[:, None], (p - q) * c, 0.0)
        rel = torch.where(p > 0, 2 * self.ez + 2.0 ** -22 * d.abs() + 2.0 ** -20, 0.0)
        self.dz_err = c.abs() * (p * torch.expm1(rel) + 4 * U["f32"] * (p + q))
        self.floor = 2.0 ** -39 * float(c.abs().max()) if self.dtype == "f16" else 0.0


def _check_low(ddl, t, k, v, dtype, low):
    """Low entries everywhere, neighbours from a tile's edge, on the last tile, and behind entries masked with -infinity."""
    with ddl.CrossEntropy(k, v, t, dtype) as head:
        for first, count, masked in ((0, v, 0), (0, 50, 0), (128, 128, 0), (256, 300, 0), (v // 256 * 256, 256, 0), (100, v, 100),
                                     (300, v, 300)):
            h = LowHead(t, k, v, dtype, low, slice(first, first + count), masked, seed=t + first).solve()
            loss, lse = h.forward(ddl, head)
            h.check_forward(loss, lse)
            h.solve_backward(lse)
            dx, dw, db = torch.empty_like(h.x), torch.empty(v, k, device="cuda"), torch.empty(v, device="cuda")
            head.backward(h.x, h.w, h.labels, lse, dloss=h.dloss, bias=h.bias, dx=dx, dw=dw, db=db)
            h.check_backward(dx, dw, db)
            head.check()


@pytest.mark.parametrize("dtype, low", [("bf16", -100.0), ("bf16", -1e4), ("f16", -300.0), ("f16", torch.finfo(torch.float16).min)])
@pytest.mark.parametrize("k, v", [(64, 700), (1024, 700), (64, 5003)])
@pytest.mark.parametrize("t", [4, 64, 65, 150, 333])
def test_finite_logits_far_below_zero(ddl, t, k, v, dtype, low):
    """A softmax does not change with a shift: entries that a large negative bias takes out leave finite losses and gradients."""
    _check_low(ddl, t, k, v, dtype, low)


@pytest.mark.parametrize("k, v", [(64, 700), (1024, 700), (64, 5003)])
@pytest.mark.parametrize("t", [4, 64, 65, 333])
@pytest.mark.parametrize("low", [-1e12, torch.finfo(torch.bfloat16).min])
def test_logits_as_low_as_numbers_go(ddl, t, k, v, low):
    """The same with a mask of the type's lowest number, whose product with log2 e is none."""
    _check_low(ddl, t, k, v, "bf16", low)


@pytest.mark.parametrize("t, k", [(4, 64), (64, 1024), (65, 64), (150, 1024), (333, 64)])
def test_mean_of_large_logits(ddl, t, k):
    """Smoothing takes the mean of the logits: it is a number where their sum is none.  Half of the entries at -2^127 make it
    -2^126 exactly, next to which the other logits are lost; 1 - smoothing is a power of two."""
    v = 512
    h = Head(t, k, v, "bf16", bias=True, seed=19, ignored=0.0)
    h.bias[::2] = -2.0 ** 127
    h.labels |= 1  # an entry that is left
    with ddl.CrossEntropy(k, v, t, "bf16", smoothing=0.5) as head:
        loss, lse = h.forward(ddl, head)
        head.check()
    assert bool(lse.isfinite().all())
    assert bool((loss == 2.0 ** 125).all())


@pytest.mark.parametrize("t, k, v", [(3, 64, 500), (200, 96, 1500), (700, 130, 2049)])
def test_calls_that_follow_each_other_at_once(ddl, t, k, v):
    """Launches begin while the one before them ends: a forward pass reads labels and a bias that were just written, a backward
    pass the lse of a forward pass, an optimizer's step the gradients, and the next forward pass the bias that it wrote.  The
    same bits as with a pause after each."""
    hs = [Head(t, k, v, "bf16", bias=True, smoothing=0.1, seed=31 + i) for i in range(3)]
    width = v + (v & 1)

    def chain(pause):
        x, w, labels, dloss = (a.clone() for a in (hs[0].x.contiguous(), hs[0].w.contiguous(), hs[0].labels, hs[0].dloss))
        bias32, bias16 = torch.zeros(width, device="cuda"), torch.zeros(width, dtype=torch.bfloat16, device="cuda")
        db, out = torch.zeros(width, device="cuda"), []
        with ddl.CrossEntropy(k, v, t, "bf16", smoothing=0.1) as head, ddl.Adam([(0, v)]) as adam:
            state = adam.new_state()
            for i in range(12):
                h = hs[i % 3]
                for to, new in ((x, h.x), (w, h.w), (dloss, h.dloss), (labels, h.labels)):
                    to.copy_(new)
                    pause()
                loss, lse = torch.empty(t, device="cuda"), torch.empty(t, device="cuda")
                dx, dw = torch.empty_like(x), torch.empty(v, k, device="cuda")
                pause()
                head.forward(x, w, labels, loss, lse, bias=bias16[:v])
                pause()
                head.backward(x, w, labels, lse, dloss=dloss, bias=bias16[:v], dx=dx, dw=dw, db=db[:v])
                pause()
                adam.step(db, [bias32], lr=0.1, operands=[bias16], **state)
                pause()
                out += [loss, lse, dx, dw, bias32.clone()]
                pause()
            torch.cuda.synchronize()
            head.check()
        return out
    want = chain(torch.cuda.synchronize)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(chain(lambda: None), want))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("t", [5, 150])
def test_an_infinite_weight_of_the_label(ddl, t, dtype):
    """A label whose logit is -infinity has dz = -dloss, a finite number (no rest where it is a power of two): dx is infinite where the
    label's weight is, as the products have it, and not NaN."""
    h = Head(t, 64, 300, dtype, seed=29, ignored=0.0, sure=0.0)
    h.labels[:] = 1 + h.labels % 299
    h.labels[1] = 0
    h.x[:, 7] = -h.x[:, 7].abs().clamp(min=0.5)
    h.w[0, 7] = float("inf")
    dloss = torch.full((t,), 0.5, device="cuda")
    dx = torch.empty_like(h.x)
    with ddl.CrossEntropy(64, 300, t, dtype) as head:
        loss, lse = h.forward(ddl, head)
        assert bool(lse.isfinite().all()) and float(loss[1]) == float("inf")
        head.backward(h.x, h.w, h.labels, lse, dloss=dloss, dx=dx)
    assert float(dx[1, 7]) == float("-inf")
    assert bool(dx[1, :7].isfinite().all()) and bool(dx[1, 8:].isfinite().all())


@pytest.mark.parametrize("k, v, c", [(512, 1000, 1), (2048, 1000, 1), (4096, 300, 1), (1024, 20011, 2), (4096, 20011, 2)])
@pytest.mark.parametrize("t", [1, 3, 8])
def test_losses_of_a_few_tokens(ddl, t, k, v, c):
    """They are not averaged: their logits leave the truncating accumulator after c blocks of 64.  With u = 2^-24 and n blocks, of
    a label's logit z that all blocks add to alike, each of the 4 c additions loses up to half a unit, a quarter on average, 0.36 u, of
    1/(4 c), 2/(4 c) ... of the c blocks' sum: 0.18 (4 c + 1) u z in all.  The n / c additions after that round 1, 2 ... of n / c parts
    of z by 0.42 u: root of 0.06 n / c, u z.  The root mean square over tokens is within 1.5 times both, times what a logit's error
    does to the loss."""
    square = count = 0
    n = -(-k // 64)
    with ddl.CrossEntropy(k, v, t, "bf16") as head:
        for seed in range(-(-96 // t)):
            h = Head(t, k, v, "bf16", seed=100 + 7 * seed, ignored=0.0, sure=torch.full((t, 1), 8.0, device="cuda")).solve()
            loss, _ = h.forward(ddl, head)
            zy = h.z.gather(1, h.labels[:, None])
            miss = torch.sigmoid(torch.logsumexp(h.z.scatter(1, h.labels[:, None], float("-inf")) - zy, 1))
            square += float((((loss.double() - h.loss) / (miss * zy[:, 0])) ** 2).sum())
            count += t
    off = math.sqrt(square / count)
    assert off <= 1.5 * math.sqrt((0.18 * (4 * c + 1)) ** 2 + 0.06 * n / c) * U["f32"], f"{off / U['f32']:.2f} u"


@pytest.mark.parametrize("t", [64, 500, 2000, 4096, 4097, 6145, 9000, 17000])
@pytest.mark.parametrize("k, v, ignored", [(96, 700, 0.0), (96, 700, 0.99), (1030, 333, 0.0), (1030, 333, 0.95)])
def test_binary32_dw_keeps_dz_by_the_tokens_that_count(ddl, t, k, v, ignored):
    """A bfloat16 head's, whatever tokens of the call are ignored or weigh nothing.  u = 2^-24; small logits, so that their own errors
    are far below it, and dz from the call's own lse.  dz takes 3 roundings; the tensor core truncates 4 sums of a block of 64
    tokens by half a unit at most, c blocks in a row (1, 2, 4 up to 640, 2048 and more tokens), and the rest are sums in binary32,
    whose roundings average out: (3 + 4 c + sqrt(t / 64 c)) u, 6e-7 to 1.6e-6 of the norm.  Where more than 4096 tokens count, dz
    has two planes: the second rounds what the first left to half a unit of it: 2^-16 of a power of two that is 0.72 of the number in
    both, evenly (1 / sqrt 3 each): 0.52 / 3 of 2^-16, 2.6e-6, which fails the first bound."""
    h = Head(t, k, v, "bf16", seed=26, ignored=ignored, sure=0.0)
    h.w.mul_(0.02)
    h.labels[0] = 5
    if ignored == 0.95:  # these weigh nothing instead
        h.dloss[h.labels < 0] = 0.0
        h.labels.clamp_(min=0)
    h.solve()
    dw = torch.empty(v, k, device="cuda")
    with ddl.CrossEntropy(k, v, t, "bf16") as head:
        _, lse = h.forward(ddl, head)
        head.backward(h.x, h.w, h.labels, lse, dloss=h.dloss, dw=dw)
        head.check()
    p = torch.exp(h.z - lse.double()[:, None])
    p[torch.arange(t, device="cuda"), h.labels.clamp(min=0)] -= 1.0
    dz = p * torch.where(h.valid, h.dloss.double(), 0.0)[:, None]
    want = dz.t() @ h.x.double()
    c = 1 if t <= 640 else 2 if t <= 2048 else 4
    off = float((dw.double() - want).norm() / want.norm())
    counted = int((h.valid & (h.dloss != 0)).sum())
    assert off <= (3 + 4 * c + math.sqrt(t / (64 * c))) * U["f32"] + (counted > 4096) * 0.52 / 3 * 2.0 ** -16


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("t, k, v", [(70, 256, 1500), (600, 1030, 2050)])
def test_dx_is_nearly_as_exact_as_its_rounding(ddl, t, k, v, dtype):
    """Of dx's plane of dz the label's value, which is most of dz here, is corrected: the rest, of norm 1 / sqrt(v) of it, adds
    less than a thousandth in quadrature to what storing dx rounds.  Without the correction the two are alike: 1.4."""
    h = Head(t, k, v, dtype, seed=27, ignored=0.0, sure=0.0)
    h.w.mul_(0.1)
    h.dloss *= 256.0
    h.solve()
    dx = torch.empty_like(h.x)
    with ddl.CrossEntropy(k, v, t, dtype) as head:
        _, lse = h.forward(ddl, head)
        head.backward(h.x, h.w, h.labels, lse, dloss=h.dloss, dx=dx)
    want = h.dz @ h.w.double()
    stored = want.to(dx.dtype).double()
    assert float((dx.double() - want).norm()) <= 1.05 * float((stored - want).norm())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_token_weights_of_many_sizes(ddl, dtype):
    """Weights from 2^-26 to 1 of the largest in one call: every token's dx is within the bound of its own dz and of 2^-39 of the
    largest weight (binary16)."""
    t = 300
    dloss = 2.0 ** (12 - 26 * torch.rand(t, generator=_gen(5), device="cuda"))
    h = Head(t, 96, 260, dtype, bias=True, smoothing=0.1, seed=28, ignored=0.1, dloss=dloss)
    _run(ddl, h)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("t", [11, 64, 200])
def test_gradients_of_tokens_that_are_nearly_sure(ddl, t, dtype):
    """x w^T with w the identity: exact logits, and dx is dz.  1 - p of the labels from 1e-3 to 1e-7, where what is left of dz is lse's and
    the exponential's rounding: 2^-23 |lse| + 2^-21 of the probability, 4 u of the difference, and the rounding of the plane (the
    label's dz excepted) and of dx."""
    v = 64
    x = torch.zeros(t, v, device="cuda")
    labels = torch.randint(0, v, (t,), generator=_gen(32), device="cuda")
    x[torch.arange(t), labels] = torch.linspace(11, 20, t, device="cuda")
    x, w = x.to(TYPES[dtype]), torch.eye(v, device="cuda").to(TYPES[dtype])
    loss, lse, dx = torch.empty(t, device="cuda"), torch.empty(t, device="cuda"), torch.empty_like(x)
    dloss = torch.full((t,), 1024.0, device="cuda")
    with ddl.CrossEntropy(v, v, t, dtype) as head:
        head.forward(x, w, labels, loss, lse)
        head.backward(x, w, labels, lse, dloss=dloss, dx=dx)
        head.check()
    z = x.double()
    p = torch.softmax(z, 1)
    q = torch.nn.functional.one_hot(labels, v).double()
    miss = (p * (1 - q)).sum(1, keepdim=True)
    want = torch.where(q > 0, -miss, p)
    bound = p * (2.0 ** -23 * (20 + math.log(v)) + 2.0 ** -21 + 2.0 ** -22 * (z - z.amax(1, keepdim=True)).abs()) + 4 * U["f32"] * q
    bound = 1024 * (bound + 2 * U[dtype] * want.abs()) + TINY[dtype] + 2.0 ** -29
    _within(dx, 1024 * want, bound)
    small = torch.nn.functional.softplus(torch.log(miss[:, 0]) - torch.log1p(-miss[:, 0]))
    _within(loss, small, small * 2.0 ** -15)


@pytest.mark.parametrize("t, k, v", [(8192, 64, 70001), (20000, 64, 30011)])
def test_few_tokens_that_count_over_pieces_of_the_vocabulary(ddl, t, k, v):
    """Every piece's products take the same number of planes, from a scale that the launch or a pass of its own made: the bound of
    three planes, (3 + 4 c + sqrt(t / 64 c)) u with c = 4, for each half of the vocabulary."""
    h = Head(t, k, v, "bf16", seed=33, ignored=0.98, sure=0.0)
    h.w.mul_(0.02)
    h.solve()
    dw, dx = torch.empty(v, k, device="cuda"), torch.empty_like(h.x)
    with ddl.CrossEntropy(k, v, t, "bf16") as head:
        _, lse = h.forward(ddl, head)
        head.backward(h.x, h.w, h.labels, lse, dloss=h.dloss, dx=dx, dw=dw)
        head.check()
    h.check_backward(dx)
    p = torch.exp(h.z - lse.double()[:, None])
    p[torch.arange(t, device="cuda"), h.labels.clamp(min=0)] -= 1.0
    want = (p * torch.where(h.valid, h.dloss.double(), 0.0)[:, None]).t() @ h.x.double()
    for part in (slice(0, v // 2), slice(v // 2, v)):
        assert float((dw[part].double() - want[part]).norm() / want[part].norm()) <= (3 + 16 + math.sqrt(t / 256)) * U["f32"]
