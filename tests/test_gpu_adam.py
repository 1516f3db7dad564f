"""The AdamW step on the GPU against the formulas in 64 bits.

Element-wise bounds, from the arithmetic (u = 2^-24, half a unit in the last place
of a binary32 number near one).  g' = c g: c takes up to 5 roundings (the norm, the
sum with 1e-6, the quotient, two products), g' one more.
 - m: 3 u of beta1 m (the constant, the product, the sum), 9 u of (1 - beta1) g';
 - v: 3 u of beta2 v, 16 u of (1 - beta2) g'^2;
 - p: 4 u of itself and, with U = lr / (1 - beta1^t) (beta1 |m| + (1 - beta1) |g'|) /
   (sqrt(v / (1 - beta2^t)) + eps), 34 u of U: 9 of m, 9 of sqrt(v), 4 of
   sqrt(1 - beta2^t), 2 of the quotient's denominator, 10 of the factors before it;
 - 16-bit copies round once more: u' of the value (2^-11, 2^-8), or half of the
   smallest subnormal;
 - 8-bit states: half a step of e4m3, 2^-4 of the value or 2^-10 of the scale; a
   root below that is at most 2^-9 of the scale off.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 128


@pytest.fixture(scope="module")
def ddl():
    assert torch.cuda.is_available(), "GPU test needs a CUDA device"
    import __graft_entry__
    __graft_entry__.build()
    from gradient_all_reduce_ddl_gb300 import ddl as mod
    return mod


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _shifted(t, shift):
    """A copy of t that begins `shift` elements into its storage."""
    flat = torch.empty(t.numel() + shift, dtype=t.dtype, device="cuda")
    flat[shift:].copy_(t)
    return flat[shift:]


class Problem:
    """Tensors in a flat buffer whose gaps hold NaN, states after some steps, and the step in 64 bits."""

    def __init__(self, ddl, tensors, state="f32", grad="f32", copies=1, operands=None, seed=0, sigma=1e-3, steps=7,
                 betas=(0.9, 0.999), eps=1e-8, shift=0):
        self.adam = ddl.Adam(tensors, dtype=grad, state=state, betas=betas, eps=eps)
        self.betas, self.eps, self.state = betas, eps, state
        n, gen = self.adam.extent + 5, _gen(seed)
        self.inside = torch.zeros(n, dtype=torch.bool, device="cuda")
        self.lr_scale, self.decay_scale = torch.zeros(n, device="cuda", dtype=torch.float64), torch.zeros(n, device="cuda", dtype=torch.float64)
        self.block = torch.zeros(n, dtype=torch.long, device="cuda")
        at = 0
        for t in tensors:
            sl = slice(t[0], t[0] + t[1])
            self.inside[sl] = True
            self.lr_scale[sl], self.decay_scale[sl] = t[2] if len(t) > 2 else 1.0, t[3] if len(t) > 3 else 1.0
            self.block[sl] = at + torch.arange(t[1], device="cuda") // BLOCK
            at += -(-t[1] // BLOCK)
        self.n_blocks = at
        assert at == self.adam.n_blocks

        def normal(s):
            x = torch.randn(n, generator=gen, device="cuda") * s
            return torch.where(self.inside, x, torch.full_like(x, float("nan")))
        self.grad = _shifted(normal(sigma).to(TYPES[grad]), shift)
        self.params = [_shifted(normal(0.02), shift) for _ in range(copies)]
        self.operands = None if operands is None else [_shifted(torch.full((n,), 7.0, dtype=TYPES[operands], device="cuda"), shift)
                                                       for _ in range(copies)]
        self.step_count = torch.tensor([steps], device="cuda")
        m, root = normal(0.3 * sigma), normal(sigma).abs()
        if state == "f32":
            self.m, self.v, self.scales = _shifted(m, shift), _shifted(root * root, shift), None
        else:
            self.scales = torch.rand(2, self.n_blocks, generator=gen, device="cuda") * sigma / 100
            codes = torch.randint(0, 256, (2, n), generator=gen, device="cuda").to(torch.uint8)
            codes[0][codes[0] % 128 == 127] = 1
            codes[1] %= 127
            codes[:, ~self.inside] = 0x55
            self.m, self.v = _shifted(codes[0], shift), _shifted(codes[1], shift)

    def states(self):
        """m and v in 64 bits."""
        if self.state == "f32":
            return self.m.double(), self.v.double()
        m = self.m.view(torch.float8_e4m3fn).float().double() * self.scales[0].double()[self.block]
        r = self.v.view(torch.float8_e4m3fn).float().double() * self.scales[1].double()[self.block]
        return m, r * r

    def run(self, lr=1e-2, wd=0.1, grad_scale=1.0, max_norm=0.0, want_norm=False, stream=None):
        """One step, checked."""
        m, v = self.states()
        p = [x.double() for x in self.params]
        g, t = self.grad.double(), int(self.step_count) + 1
        b1, b2 = self.betas
        norm_out = torch.zeros(1, device="cuda") if want_norm else None
        self.adam.step(self.grad, self.params, self.m, self.v, self.step_count, lr, weight_decay=wd, scales=self.scales,
                       operands=self.operands, grad_scale=grad_scale, max_norm=max_norm, norm=norm_out, stream=stream)
        torch.cuda.synchronize()
        assert int(self.step_count) == t
        ins = self.inside
        norm = float(torch.linalg.vector_norm(g[ins])) * abs(grad_scale)
        if want_norm:
            assert abs(float(norm_out) - norm) <= 4 * U * norm
        c = grad_scale * (min(1.0, max_norm / (norm + 1e-6)) if max_norm else 1.0)
        g = c * g
        m1, v1 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
        mag = b1 * m.abs() + (1 - b1) * g.abs()
        over = lr * self.lr_scale / (1 - b1 ** t) / ((v1 / (1 - b2 ** t)).sqrt() + self.eps)
        for x, old in zip(self.params, p):
            want = old * (1 - lr * self.lr_scale * wd * self.decay_scale) - over * m1
            self.within(x, want, 4 * U * old.abs() + 34 * U * over * mag + 1e-37)
        if self.operands:
            for o, x in zip(self.operands, self.params):
                assert torch.equal(o[ins], x.to(o.dtype)[ins])
                assert bool((o[~ins] == 7.0).all())
        if self.state == "f32":
            self.within(self.m, m1, 9 * U * mag + 2.0 ** -149)
            self.within(self.v, v1, 16 * U * v1 + 2.0 ** -148)
            assert bool(self.m[~ins].isnan().all()) and bool(self.v[~ins].isnan().all())
        else:
            self.codes_within(m1, v1, mag)
        for x in self.params:
            assert bool(x[~ins].isnan().all())

    def within(self, got, want, bound):
        err = (got.double() - want).abs()[self.inside]
        assert bool(torch.isfinite(got[self.inside]).all())
        worst = float((err / bound[self.inside]).max())
        assert worst <= 1.0, f"error is {worst:.2f} times its bound"

    def codes_within(self, m1, v1, mag):
        ins = self.inside
        assert bool((self.m[~ins] == 0x55).all()) and bool((self.v[~ins] == 0x55).all())
        m, r = (x.view(torch.float8_e4m3fn).float().double() for x in (self.m, self.v))
        top_m, top_r = (torch.zeros(self.n_blocks, device="cuda", dtype=torch.float64).scatter_reduce_(
            0, self.block[ins], x[ins], "amax") for x in (m1.abs(), v1.sqrt()))
        for k, top in enumerate((top_m, top_r)):
            s = self.scales[k].double()
            assert float(((s * 448 - top).abs() - 20 * U * top - 20 * U * float(mag[ins].max())).max()) <= 0
        sm, sr = self.scales[0].double()[self.block], self.scales[1].double()[self.block]
        half = torch.maximum(m1.abs() * 2.0 ** -4, sm * 2.0 ** -10)
        self.within(m * sm, m1, half * (1 + 1e-5) + 9 * U * mag + 1e-300)
        r1 = v1.sqrt()
        half = torch.where(r1 < sr * 2.0 ** -9, sr * 2.0 ** -9, torch.maximum(r1 * 2.0 ** -4, sr * 2.0 ** -10))
        self.within(r * sr, r1, half * (1 + 1e-5) + 1e-300)
        assert bool((r[ins] > 0)[(r1 > 0)[ins]].all())


ODD = [(3, 1), (4, 127), (131, 128), (260, 129), (400, 1000, 0.5, 0.0), (1401, 2), (1408, 3 * 128), (2001, 1025, 2.0, 1.0)]


@pytest.mark.parametrize("state", ["f32", "8bit"])
@pytest.mark.parametrize("grad", ["f32", "f16"])
@pytest.mark.parametrize("copies, operands", [(1, None), (2, "bf16"), (5, "f16")])
def test_odd_tensors(ddl, state, grad, copies, operands):
    Problem(ddl, ODD, state, grad, copies, operands, seed=1).run()


@pytest.mark.parametrize("state", ["f32", "8bit"])
@pytest.mark.parametrize("n", [1, 4, 31, 128, 129, 1023, 1024, 1025, 300_001, 6_000_000])
def test_lengths(ddl, state, n):
    Problem(ddl, [(0, n)], state, seed=n, operands="bf16").run(want_norm=True, max_norm=1e-3)


@pytest.mark.parametrize("state", ["f32", "8bit"])
@pytest.mark.parametrize("shift", [1, 2, 3])
def test_unaligned_buffers(ddl, state, shift):
    Problem(ddl, [(0, 640), (641, 300)], state, "f16", 2, "f16", seed=shift, shift=shift).run()


@pytest.mark.parametrize("copies", [16, 17, 256])
def test_many_copies(ddl, copies):
    Problem(ddl, [(0, 1000), (1001, 333)], "8bit", copies=copies, operands="bf16", seed=2).run()


def test_many_tensors(ddl):
    sizes, at, tensors = [1 + 37 * k % 300 for k in range(500)], 0, []
    for k, n in enumerate(sizes):
        tensors.append((at, n, 1.0, float(k % 2)))
        at += n + k % 3
    Problem(ddl, tensors[::-1], "8bit", seed=3).run(want_norm=True)
    Problem(ddl, tensors, "f32", seed=3).run(want_norm=True)


@pytest.mark.parametrize("state", ["f32", "8bit"])
@pytest.mark.parametrize("steps, betas, eps", [(0, (0.9, 0.999), 1e-8), (0, (0.0, 0.0), 1e-8), (100_000, (0.95, 0.98), 1e-3),
                                               (3, (0.9, 0.9999999), 1e-12)])
def test_constants_and_step_counts(ddl, state, steps, betas, eps):
    Problem(ddl, ODD, state, seed=4, steps=steps, betas=betas, eps=eps).run()


@pytest.mark.parametrize("grad_scale, max_norm", [(1 / 1024, 0.0), (1 / 1024, 1e-6), (1.0, 1e-3), (1.0, 1e3), (-2.0, 1e-3)])
def test_scaled_and_clipped(ddl, grad_scale, max_norm):
    for state in ("f32", "8bit"):
        Problem(ddl, ODD, state, seed=5).run(grad_scale=grad_scale, max_norm=max_norm, want_norm=True)


@pytest.mark.parametrize("size", [1e-30, 1e25])
def test_norm_outside_the_range_of_squares(ddl, size):
    with ddl.Adam([(0, 5000)]) as adam:
        g = torch.randn(5000, generator=_gen(6), device="cuda") * size
        p, s, norm = torch.zeros(5000, device="cuda"), adam.new_state(), torch.zeros(1, device="cuda")
        adam.step(g, [p], lr=0.0, norm=norm, max_norm=size, **s)
        want = float(torch.linalg.vector_norm(g.double()))
        assert abs(float(norm) - want) <= 4 * U * want


@pytest.mark.parametrize("state", ["f32", "8bit"])
def test_zero_gradients_of_new_states(ddl, state):
    with ddl.Adam([(0, 1000)], state=state) as adam:
        p = torch.randn(1000, generator=_gen(7), device="cuda")
        want, s = p.clone(), adam.new_state()
        g, norm = torch.zeros(1000, device="cuda"), torch.ones(1, device="cuda")
        adam.step(g, [p], lr=0.1, max_norm=1.0, norm=norm, **s)
        assert torch.equal(p, want) and float(norm) == 0 and int(s["step"]) == 1
        assert not s["m"].any() and not s["v"].any()


@pytest.mark.parametrize("state", ["f32", "8bit"])
def test_several_steps_follow_64_bits(ddl, state):
    """Chained steps, each checked from the states that the one before left."""
    pr = Problem(ddl, ODD, state, seed=8, operands="bf16")
    for k in range(5):
        pr.grad.copy_(torch.where(pr.inside, torch.randn(pr.grad.numel(), generator=_gen(80 + k), device="cuda") * 1e-3, pr.grad))
        pr.run(want_norm=True, max_norm=2e-2)


@pytest.mark.parametrize("state", ["f32", "8bit"])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_bad_gradient_spoils_its_own_element(ddl, state, bad):
    with ddl.Adam([(0, 512)], state=state) as adam:
        g = torch.randn(512, generator=_gen(10), device="cuda")
        results = []
        for value in (g[200].item(), bad):
            p, s = torch.zeros(512, device="cuda"), adam.new_state()
            h = g.clone()
            h[200] = value
            adam.step(h, [p], lr=0.1, **s)
            adam.step(g, [p], lr=0.1, **s)
            results.append(p)
        others = torch.arange(512, device="cuda") != 200
        if state == "f32":
            assert torch.equal(results[0][others], results[1][others])
        else:  # the block's scale may have been the element's own
            assert bool(torch.isfinite(results[1][others]).all())
            assert torch.equal(results[0][:128], results[1][:128]) and torch.equal(results[0][256:], results[1][256:])
        assert bool(results[1][200].isnan())


def test_captured_steps_count_on(ddl):
    pr = Problem(ddl, ODD, "8bit", seed=11, operands="f16")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        pr.run(want_norm=True, max_norm=1e-2, stream=s)  # tables are uploaded before the capture
    keep = [x.clone() for x in (pr.params[0], pr.m, pr.v, pr.scales, pr.step_count)]
    norm = torch.zeros(1, device="cuda")

    def call():
        pr.adam.step(pr.grad, pr.params, pr.m, pr.v, pr.step_count, 1e-2, weight_decay=0.1, scales=pr.scales,
                     operands=pr.operands, max_norm=1e-2, norm=norm)
    for _ in range(3):
        call()
    torch.cuda.synchronize()
    want = [x.clone() for x in (pr.params[0], pr.m, pr.v, pr.scales, pr.step_count)]
    for x, k in zip((pr.params[0], pr.m, pr.v, pr.scales, pr.step_count), keep):
        x.copy_(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for x, w in zip((pr.params[0], pr.m, pr.v, pr.scales, pr.step_count), want):
        ins = slice(None) if x.numel() != pr.inside.numel() else pr.inside
        assert torch.equal(x[ins], w[ins])


def test_repeats_bit_for_bit_and_on_two_streams(ddl):
    """Two handles step at once on two streams; each gives what it gives alone."""
    def make():
        return [Problem(ddl, [(0, 3_000_001)], "8bit", "f16", 2, seed=20 + k) for k in range(2)]
    alone, together = make(), make()
    for pr in alone:
        pr.run(max_norm=1e-2)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for pr, s in zip(together, streams):
        pr.adam.step(pr.grad, pr.params, pr.m, pr.v, pr.step_count, 1e-2, weight_decay=0.1, scales=pr.scales, max_norm=1e-2, stream=s)
    torch.cuda.synchronize()
    for a, b in zip(alone, together):
        for x, y in zip([a.m, a.v, a.scales, *a.params], [b.m, b.v, b.scales, *b.params]):
            assert torch.equal(x.nan_to_num(7.0) if x.is_floating_point() else x, y.nan_to_num(7.0) if y.is_floating_point() else y)


def test_against_torch_adamw(ddl):
    """Three steps of torch's own AdamW in 64 bits."""
    n, lr, wd = 1000, 1e-2, 0.1
    start = torch.randn(n, generator=_gen(12), device="cuda")
    ref = torch.nn.Parameter(start.double())
    opt = torch.optim.AdamW([ref], lr=lr, weight_decay=wd, betas=(0.9, 0.99), eps=1e-6)
    with ddl.Adam([(0, n)], betas=(0.9, 0.99), eps=1e-6) as adam:
        p, s = start.clone(), adam.new_state()
        for k in range(3):
            g = torch.randn(n, generator=_gen(13 + k), device="cuda")
            ref.grad = g.double()
            opt.step()
            adam.step(g, [p], lr=lr, weight_decay=wd, **s)
    # three steps of at most 4 u |p| + 34 u U each, |p| < 5 and U < 3.2 lr; m's and v's own errors are counted in U's
    assert float((p.double() - ref.detach()).abs().max()) <= 3 * (20 + 34 * 3.2 * lr + 50 * lr) * U
    assert math.isclose(float(s["step"]), 3)


def test_memory_that_is_short(ddl, monkeypatch):
    pr = Problem(ddl, ODD, "8bit", seed=14)
    before = [x.clone() for x in (pr.m, pr.v, pr.step_count)]
    monkeypatch.setenv("DDL_INJECT_ALLOC_FAILURE", "1")
    with pytest.raises(ddl.DDLError) as e:
        pr.adam.step(pr.grad, pr.params, pr.m, pr.v, pr.step_count, 1e-2, scales=pr.scales)
    assert e.value.status == ddl.DDL_ERR_OOM
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, (pr.m, pr.v, pr.step_count)))
    monkeypatch.delenv("DDL_INJECT_ALLOC_FAILURE")
    pr.run()


def test_checks_of_the_object(ddl):
    with ddl.Adam([(0, 64)], state="8bit") as adam:
        x, s = torch.zeros(64, device="cuda"), adam.new_state()
        adam.step(x, [x.clone()], lr=0.1, **s)
        for change in (dict(grad=x.half()), dict(params=[x.double()]), dict(m=x), dict(step=x), dict(scales=x), dict(grad=x[:63]),
                       dict(operands=[x]), dict(operands=[]), dict(norm=x.half()), dict(grad=torch.zeros(128, device="cuda")[::2])):
            a = dict(grad=x.clone(), params=[x.clone()], lr=0.1, **s)
            a.update(change)
            with pytest.raises(ValueError):
                adam.step(**a)
        pinned = torch.zeros(64).pin_memory()
        with pytest.raises(ddl.DDLError) as e:  # memory of another kind
            ddl.ddl_adam_step(adam.handle, pinned, [x.clone()], None, ddl.DDL_FP16, s["m"], s["v"], s["scales"], s["step"], 0.1)
        assert e.value.status == ddl.DDL_ERR_INVALID_ARG


@pytest.mark.parametrize("state", ["f32", "8bit"])
@pytest.mark.parametrize("eps", [2.0 ** -126, 1e-30, 1e-20])
@pytest.mark.parametrize("sigma", [1e-17, 1e-18, 1e-19])
def test_roots_of_tiny_second_moments(ddl, state, eps, sigma):
    """v of gradients that small is below binary32's normal range, where it has an absolute error of half of 2^-149; its root is an
    ordinary number, by which the step divides.  Of a new state (m = 0.1 g, v = 0.001 g^2 in binary32) the step is lr m / 0.1 /
    (sqrt(v / 0.001) + eps): 40 u of it, and what v's two roundings below the normal range, 2^-149 in all, are of its root."""
    n, lr = 1000, 1e-2
    g = torch.randn(n, generator=_gen(15), device="cuda") * sigma
    with ddl.Adam([(0, n)], state=state, eps=eps) as adam:
        p, s = torch.zeros(n, device="cuda"), adam.new_state()
        adam.step(g, [p], lr=lr, **s)
    g = g.double()
    v = 0.001 * g * g
    known = v > 2.0 ** -143
    assert bool(known.float().mean() > 0.5)
    want = -lr * g / ((v / 0.001).sqrt() + eps)
    bound = (40 * U + 2.0 ** -149 / v) * want.abs()
    assert float(((p.double() - want).abs() / bound)[known].max()) <= 1.0
    if state == "8bit":  # a root that is not zero is not kept as zero
        assert bool((s["v"][known] != 0).all())
    else:
        assert float(((s["v"].double() - v).abs() - 3 * U * v - 2.0 ** -149)[known].max()) <= 0
