"""The orthogonalised update on the GPU against its formulas in 64 bits.

Newton-Schulz multiplies early roundings by up to a^steps, by an amount that
depends on the matrix, so binary32 results are held to what a binary32
evaluation of the same formula loses on the same input: at most four times its
error in the Frobenius norm, plus 2^-19 (two roundings a step of 22-bit
operands, 2^-22 each, for five steps, rounded up).  16-bit results add their
storage rounding, 2^-11 or 2^-8 of each element.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ABC = (3.4445, -4.7750, 2.0315)
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module")
def ddl():
    assert torch.cuda.is_available(), "GPU test needs a CUDA device"
    import __graft_entry__
    __graft_entry__.build()
    from gradient_all_reduce_ddl_gb300 import ddl as mod
    return mod


def _newton_schulz(g, steps=5, abc=ABC, eps=1e-7):
    """In g's own precision."""
    a, b, c = abc
    tall = g.shape[0] > g.shape[1]
    x = g.t() if tall else g
    x = x / (x.square().sum().sqrt() + eps)
    for _ in range(steps):
        m = x @ x.t()
        x = a * x + (b * m + c * (m @ m)) @ x
    return x.t() if tall else x


def _gradient(rows, cols, seed=0, rank=16, noise=1.0, scale=1e-3):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = min(rank, rows, cols)
    g = torch.randn(rows, r, generator=gen, device="cuda") @ torch.randn(r, cols, generator=gen, device="cuda")
    return (g + noise * torch.randn(rows, cols, generator=gen, device="cuda")) * scale


def _view(flat, m):
    off, rows, cols = m[:3]
    ld = m[3] if len(m) > 3 else cols
    return torch.as_strided(flat, (rows, cols), (ld, 1), flat.storage_offset() + off)


def _allowed(g, want, **kw):
    """Frobenius error allowed to a binary32 result."""
    plain = _newton_schulz(g.float(), **kw).double()
    return 4 * (plain - want).norm() + 2.0 ** -19 * want.norm()


def _check(got, g, dtype, **kw):
    want = _newton_schulz(g.double(), **kw)
    got = got.double()
    assert torch.isfinite(got).all()
    tol = _allowed(g, want, **kw) + U[dtype] * want.norm()
    assert (got - want).norm() <= tol, f"off by {(got - want).norm() / want.norm():.2e}, allowed {tol / want.norm():.2e}"


SHAPES = [(1, 1), (1, 100), (100, 1), (2, 3), (16, 16), (64, 147), (147, 64), (127, 129), (129, 127), (128, 128),
          (128, 512), (33, 4608), (4608, 33), (257, 300), (300, 257), (512, 512), (640, 1000), (1000, 2048), (1025, 769),
          (2304, 2304), (1280, 5000), (3000, 1100)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows, cols", SHAPES)
def test_one_matrix(ddl, rows, cols, dtype):
    g = _gradient(rows, cols).to(TYPES[dtype])
    out = torch.empty_like(g)
    with ddl.Ortho([(0, rows, cols)], dtype) as o:
        o.run(g.view(-1), out.view(-1))
        o.check()
    _check(out, g, dtype)


@pytest.mark.parametrize("kind", ["noise only", "low rank", "large", "small", "one large element"])
def test_distributions(ddl, kind):
    g = {"noise only": lambda: torch.randn(200, 300, device="cuda", generator=torch.Generator("cuda").manual_seed(5)),
         "low rank": lambda: _gradient(200, 300, rank=3, noise=1e-3),
         "large": lambda: _gradient(200, 300, scale=1e30),      # squares overflow binary32
         "small": lambda: _gradient(200, 300, scale=1e-5),
         "one large element": lambda: _gradient(200, 300, noise=1e-2)}[kind]()
    if kind == "one large element":
        g[17, 33] = 50.0
    out = torch.empty_like(g)
    with ddl.Ortho([(0, 200, 300)]) as o:
        o.run(g.view(-1), out.view(-1))
        o.check()
    if kind == "large":  # the same direction at a scale that binary32 squares
        g = g * 2.0 ** -100
    _check(out, g, "f32")


MIXED = [(5, 64, 147), (9413, 100, 33, 40), (13500, 33, 100, 101), (17000, 1, 7), (17008, 256, 256), (82600, 300, 129)]
N_MIXED = 82600 + 300 * 129 + 11


def _mixed(dtype="f32", seed=3):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    flat = (torch.randn(N_MIXED, generator=gen, device="cuda") * 1e-3).to(TYPES[dtype])
    for k, m in enumerate(MIXED):
        _view(flat, m).copy_(_gradient(m[1], m[2], seed + k))
    return flat


def _inside():
    mask = torch.zeros(N_MIXED, dtype=torch.bool, device="cuda")
    for m in MIXED:
        _view(mask, m).fill_(True)
    return mask


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shift", [0, 1])
def test_many_matrices(ddl, dtype, shift):
    """Mixed shapes, strides and offsets in one handle; nothing outside the matrices is written."""
    flat = _mixed(dtype)
    out = torch.full((N_MIXED + shift,), 7.0, dtype=TYPES[dtype], device="cuda")[shift:]
    with ddl.Ortho(MIXED, dtype) as o:
        o.run(flat, out)
        o.check()
    for m in MIXED:
        _check(_view(out, m), _view(flat, m), dtype)
    assert bool((out[~_inside()] == 7.0).all())


def test_large_and_small_together(ddl):
    """Matrices that fill 256 x 256 tiles on CTA pairs beside ones that do not."""
    shapes = [(2048, 2048), (64, 147), (2048, 1024), (1000, 2048), (33, 20), (2048, 2050)]
    mats, at = [], 0
    for r, c in shapes:
        mats.append((at, r, c))
        at += r * c + 3
    flat = torch.zeros(at, device="cuda")
    for k, m in enumerate(mats):
        _view(flat, m).copy_(_gradient(m[1], m[2], k))
    out = torch.full_like(flat, 7.0)
    with ddl.Ortho(mats) as o:
        o.run(flat, out)
        again = o.run(flat, torch.full_like(flat, 7.0))
        o.check()
    assert torch.equal(out, again)
    for m in mats:
        _check(_view(out, m), _view(flat, m), "f32")


def test_in_place_and_repeats(ddl):
    flat = _mixed()
    a, b = flat.clone(), torch.zeros_like(flat)
    with ddl.Ortho(MIXED) as o:
        o.run(flat, b)
        o.run(a, a)
        o.check()
    inside = _inside()
    assert torch.equal(a[inside], b[inside]) and torch.equal(a[~inside], flat[~inside])


@pytest.mark.parametrize("steps, abc", [(1, ABC), (2, ABC), (10, (1.875, -1.25, 0.375)), (3, (1.5, -0.5, 0.0))])
def test_polynomials(ddl, steps, abc):
    g = _gradient(130, 200, rank=60)
    out = torch.empty_like(g)
    with ddl.Ortho([(0, 130, 200)], steps=steps, coefficients=abc, eps=1e-3) as o:
        o.run(g.view(-1), out.view(-1))
        o.check()
    _check(out, g, "f32", steps=steps, abc=abc, eps=1e-3)


def test_zero_nan_and_infinity_stay_in_their_matrix(ddl):
    mats = [(0, 40, 50), (2000, 40, 50), (4000, 40, 50), (6000, 40, 50)]
    flat = torch.cat([_gradient(40, 50, k).view(-1) for k in range(4)])
    alone = flat.clone()
    flat[:2000] = 0
    flat[2000 + 777] = float("nan")
    flat[4000 + 5] = float("inf")
    out = torch.empty_like(flat)
    with ddl.Ortho(mats) as o:
        o.run(flat, out)
        good = o.run(alone, torch.empty_like(alone))
        o.check()
    assert bool((out[:2000] == 0).all())
    assert bool(torch.isnan(out[2000:4000]).all()) and bool(torch.isnan(out[4000:6000]).all())
    assert torch.equal(out[6000:], good[6000:])


def _muon64(flat, params, mom, lr, mu, wd, nesterov):
    """The step in 64 bits: new momentum, new parameters, and what a parameter may be off by."""
    mom, params = mom.double(), [p.double() for p in params]
    slack = torch.zeros_like(mom)
    for m in MIXED:
        g, v = _view(flat, m).double(), _view(mom, m)
        v.copy_(mu * v + g)
        u = g + mu * v if nesterov else v.clone()
        o = _newton_schulz(u)
        s = max(1.0, m[1] / m[2]) ** 0.5
        # the binary32 step's error and the input's own rounding, through the same polynomial
        off = _allowed(u, o) + (_newton_schulz(u.float().double()) - o).norm()
        _view(slack, m).fill_(float(lr * s * off))
        for p in params:
            _view(p, m).mul_(1 - lr * wd).sub_(lr * s * o)
    return mom, params, slack


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("copies, nesterov, wd, shift", [(1, True, 0.0, 0), (3, False, 0.1, 0), (5, True, 0.1, 1), (17, True, 0.1, 0)])
def test_muon(ddl, dtype, copies, nesterov, wd, shift):
    lr, mu = 0.02, 0.95
    flat = _mixed(dtype)
    gen = torch.Generator(device="cuda").manual_seed(9)
    params = [torch.randn(N_MIXED + shift, generator=gen, device="cuda")[shift:] * 0.1 for _ in range(copies)]
    params = [torch.cat([torch.zeros(shift, device="cuda"), p])[shift:] for p in params]
    mom = _mixed("f32", 30) * 3
    m64, p64, slack = _muon64(flat, params, mom, lr, mu, wd, nesterov)
    before, mom_before, grad_before = [p.clone() for p in params], mom.clone(), flat.clone()
    with ddl.Ortho(MIXED, dtype) as o:
        o.muon(flat, params, mom, lr, momentum=mu, weight_decay=wd, nesterov=nesterov)
        o.check()
    inside = _inside()
    assert torch.equal(flat, grad_before)
    assert torch.equal(mom[~inside], mom_before[~inside])
    # one product and one sum, each rounded
    tol = 2.0 ** -23 * (mu * mom_before.double().abs() + flat.double().abs() + m64.abs())
    assert bool(((mom.double() - m64).abs() <= tol + 1e-30).all())
    for p, q, b in zip(params, p64, before):
        assert torch.equal(p[~inside], b[~inside])
        for m in MIXED:
            err = (_view(p, m).double() - _view(q, m)).norm()
            round_off = 2.0 ** -22 * (_view(q, m).norm() + _view(b, m).double().norm())
            assert err <= _view(slack, m).max() + round_off


def test_muon_on_a_stream_and_in_a_graph(ddl):
    flat, params, mom = _mixed(), [_mixed("f32", 40)], _mixed("f32", 30)
    want_p, want_m = params[0].clone(), mom.clone()
    got_p, got_m = params[0].clone(), mom.clone()
    with ddl.Ortho(MIXED) as o:
        for _ in range(3):
            o.muon(flat, [want_p], want_m, 0.02)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        o.muon(flat, [got_p], got_m, 0.02, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o.muon(flat, [got_p], got_m, 0.02)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        o.check()
    assert torch.equal(want_p, got_p) and torch.equal(want_m, got_m)


def test_refuses_host_memory_and_failed_allocation(ddl, monkeypatch):
    g = _gradient(32, 32)
    out = torch.empty_like(g)
    host = torch.zeros(32 * 32).pin_memory()
    with ddl.Ortho([(0, 32, 32)]) as o:
        monkeypatch.setenv("DDL_INJECT_ALLOC_FAILURE", "1")
        with pytest.raises(ddl.DDLError) as e:
            o.run(g.view(-1), out.view(-1))
        assert e.value.status == ddl.DDL_ERR_OOM
        monkeypatch.delenv("DDL_INJECT_ALLOC_FAILURE")
        with pytest.raises(ddl.DDLError) as e:
            ddl.ddl_ortho_run(o.handle, host.data_ptr(), out)
        assert e.value.status == ddl.DDL_ERR_INVALID_ARG
        o.run(g.view(-1), out.view(-1))
        o.check()
    _check(out, g, "f32")


@pytest.mark.parametrize("rows, cols", [(48, 507), (192, 3265), (256, 832), (1287, 384), (536, 1335), (768, 768), (1024, 3400)])
def test_no_less_exact_than_binary32(ddl, rows, cols):
    """22-bit operands and sums that are promoted in time: over several inputs no more than one and a half times a
    binary32 evaluation's error, and 2^-21 for the operands' and the result's own last bits."""
    own = plain = 0.0
    with ddl.Ortho([(0, rows, cols)]) as o:
        for seed in range(4):
            g = _gradient(rows, cols, seed)
            got = torch.empty_like(g)
            o.run(g.view(-1), got.view(-1))
            want = _newton_schulz(g.double())
            own += float((got.double() - want).norm() / want.norm())
            plain += float((_newton_schulz(g).double() - want).norm() / want.norm())
        o.check()
    assert own <= 1.5 * plain + 4 * 2.0 ** -21, (own / 4, plain / 4)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("power", [-117, -100, 100])
def test_without_eps_the_scale_does_not_matter(ddl, power, dtype):
    """eps = 0 is accepted: X = G / |G| then, however small or large G is (its elements stay normal numbers here)."""
    g = _gradient(64, 80).to(TYPES[dtype])
    scaled = (g.float() * 2.0 ** (power / 2) * 2.0 ** (power / 2)).to(TYPES[dtype])
    keep = scaled.float().abs() >= 2.0 ** -126
    g, scaled = torch.where(keep, g, 0), torch.where(keep, scaled, 0)
    out = torch.empty_like(scaled)
    with ddl.Ortho([(0, 64, 80)], dtype, eps=0.0) as o:
        o.run(scaled.view(-1), out.view(-1))
        o.check()
    _check(out, g, dtype, eps=0.0)


@pytest.mark.parametrize("stop", [dict(products=0), dict(products=2), dict(loads_even=0), dict(loads_even=6), dict(loads_odd=0),
                                  dict(loads_odd=6), dict(loads_even=3, loads_odd=8), dict(loads_even=8, loads_odd=3)], ids=str)
@pytest.mark.parametrize("shapes", [[(64, 147)], [(1024, 1024)], [(1024, 4096)] * 4, [(2049, 1023)], [(64, 64), (2048, 2050)]],
                         ids=str)
def test_waits_that_run_out_end_the_call(ddl, shapes, stop):
    """A role of the product kernels stops, what waits for it gives up: the call ends, the error word tells, and the calls
    after it are right.  (A stop beyond what a CTA has to do is none.)"""
    mats, at = [], 0
    for r, c in shapes:
        mats.append((at, r, c))
        at += r * c
    flat = torch.cat([_gradient(r, c, k).view(-1) for k, (r, c) in enumerate(shapes)])
    with ddl.Ortho(mats) as o:
        want = o.run(flat, torch.empty_like(flat))
        o.check()
        ddl.ddl_ortho_selftest_wait_timeout(o.handle, 300, **stop)
        o.run(flat, torch.empty_like(flat))
        if stop.get("products") == 0 or stop.get("loads_even") == 0:
            with pytest.raises(ddl.DDLError) as e:
                o.check()
            assert e.value.status == ddl.DDL_ERR_DEVICE_CHECK
        else:
            try:
                o.check()
            except ddl.DDLError as e:
                assert e.status == ddl.DDL_ERR_DEVICE_CHECK
        got = o.run(flat, torch.empty_like(flat))
        o.check()
    assert torch.equal(want, got)
