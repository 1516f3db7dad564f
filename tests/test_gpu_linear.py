"""Linear layers on the GPU against the same formulas in 64 bits.

Element-wise bounds, from the arithmetic (u = the storage type's unit roundoff,
2^-11 binary16, 2^-8 bfloat16):
 - a sum of K products of 16-bit numbers: each product is exact in binary32, and
   each of the K additions loses at most one unit in the last place (2^-23) of a
   partial sum that the sum of magnitudes bounds: (K + 16) 2^-23 sum |a||b|;
 - the activations are 1.13-Lipschitz and computed to 2^-20 of their value; a
   residual adds 2^-23 of itself;
 - storing rounds once: u |value|, or half of 2^-24 below binary16's normal range;
 - dz is computed to 2^-20 and kept to 2^-21 (two or three planes) or, for 16-bit
   results, to u of itself (exactly without activation and for ReLU).
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -23}
TINY = {"f16": 2.0 ** -24, "bf16": 2.0 ** -130, "f32": 2.0 ** -140}


@pytest.fixture(scope="module")
def ddl():
    assert torch.cuda.is_available(), "GPU test needs a CUDA device"
    import __graft_entry__
    __graft_entry__.build()
    from gradient_all_reduce_ddl_gb300 import ddl as mod
    return mod


def _act(z, kind):
    if kind == "relu":
        return torch.clamp(z, min=0)
    if kind == "gelu":
        return z * 0.5 * torch.special.erfc(-z * math.sqrt(0.5))
    if kind == "silu":
        return z * torch.sigmoid(z)
    return z


def _slope(z, kind):
    if kind == "relu":
        return (z > 0).double()
    if kind == "gelu":
        return 0.5 * torch.special.erfc(-z * math.sqrt(0.5)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if kind == "silu":
        return torch.sigmoid(z) * (1 + z * torch.sigmoid(-z))
    return torch.ones_like(z)


def _normal(seed, rows, cols, dtype, sigma=1.0, ld=None, offset=0):
    """rows x cols view with the given row stride, `offset` elements into its storage."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ld = ld or cols
    flat = torch.full((offset + rows * ld,), float("nan"), dtype=TYPES[dtype], device="cuda")
    view = flat[offset:].view(rows, ld)[:, :cols]
    view.copy_(torch.randn(rows, cols, generator=gen, device="cuda") * sigma)
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
    err = (got.double() - want).abs()
    assert torch.isfinite(got.double()).all()
    worst = (err / bound).max().item()
    assert worst <= 1.0, f"error is {worst:.2f} times its bound"


def _forward_bound(x, w, bias, z, r, y, dtype):
    mag = x.double().abs() @ w.double().abs().t() + (bias.double().abs() if bias is not None else 0)
    zerr = (x.shape[1] + 16) * 2.0 ** -23 * mag
    rmag = r.double().abs() if r is not None else 0
    return (zerr + U[dtype] * z.abs() + TINY[dtype],
            1.13 * zerr + 2.0 ** -20 * z.abs() + 2.0 ** -23 * rmag + U[dtype] * (y.abs() + 1.13 * zerr) + TINY[dtype])


SHAPES = [  # tokens, in, out: one token, each narrow tile, tile edges, odd sizes, split contractions
    (1, 1, 1), (1, 2048, 1000), (1, 77, 129), (2, 64, 128), (31, 512, 257), (32, 2048, 64), (33, 130, 128),
    (64, 4096, 300), (65, 63, 127), (128, 128, 128), (129, 4096, 130), (200, 65, 1), (333, 1001, 777), (1000, 264, 520),
    # 256 x 256 tiles, more than one a CTA pair; ragged edges of them; few of them with a long contraction
    (4101, 136, 3080), (2300, 512, 2304), (515, 8200, 520),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("tokens, n_in, n_out", SHAPES)
def test_forward(ddl, tokens, n_in, n_out, dtype):
    x, w = _normal(1, tokens, n_in, dtype), _normal(2, n_out, n_in, dtype, n_in ** -0.5)
    bias, r = _normal(3, 1, n_out, dtype)[0], _normal(4, tokens, n_out, dtype)
    z64 = x.double() @ w.double().t()
    for act in ("none", "relu", "gelu", "silu"):
        for b, res, save in ((None, None, False), (bias, r, True), (bias, None, True), (None, r, False)):
            y, clean = _blank(tokens, n_out, dtype)
            z, zclean = _blank(tokens, n_out, dtype) if save else (None, None)
            with ddl.Linear(n_in, n_out, tokens, dtype, act) as layer:
                layer.forward(x, w, y, bias=b, residual=res, z=z)
                layer.check()
            zz = z64 + (b.double() if b is not None else 0)
            yy = _act(zz, act) + (res.double() if res is not None else 0)
            zb, yb = _forward_bound(x, w, b, zz, res, yy, dtype)
            _within(y, yy, yb)
            assert clean()
            if save:
                _within(z, zz, zb)
                assert zclean()


@pytest.mark.parametrize("layout", [
    dict(x=(96, 0), w=(96, 0), y=(80, 0)),    # aligned rows, further apart than they are long
    dict(x=(91, 0), w=(96, 8), y=(77, 0)),    # x copied first
    dict(x=(96, 1), w=(93, 3), y=(80, 1)),    # both copied, y off any vector boundary
    dict(x=(90, 0), w=(90, 0), y=(73, 5)),
])
@pytest.mark.parametrize("tokens", [1, 40, 150])
def test_strides_and_alignment(ddl, tokens, layout):
    n_in, n_out, dtype = 90, 73, "f16"
    (lx, ox), (lw, ow), (ly, oy) = layout["x"], layout["w"], layout["y"]
    x, w = _normal(1, tokens, n_in, dtype, 1.0, lx, ox), _normal(2, n_out, n_in, dtype, 0.1, lw, ow)
    r = _normal(3, tokens, n_out, dtype, 1.0, ly, oy)
    bias = _normal(4, 1, n_out + 3, dtype)[0, 3:]
    z64 = x.double() @ w.double().t() + bias.double()
    y64 = _act(z64, "gelu") + r.double()
    zb, yb = _forward_bound(x, w, bias, z64, r, y64, dtype)
    y, clean = _blank(tokens, n_out, dtype, ly, oy)
    z, zclean = _blank(tokens, n_out, dtype, ly, oy)
    dy = _normal(5, tokens, n_out, dtype, 1.0, ly, oy)
    dw, wclean = _blank(n_out, n_in, "f32", lw, ow)
    db, bclean = _blank(1, n_out, "f32", None, 1)
    dx, xclean = _blank(tokens, n_in, dtype, lx, ox)
    with ddl.Linear(n_in, n_out, 200, dtype, "gelu") as layer:
        layer.forward(x, w, y, bias=bias, residual=r, z=z)
        layer.backward(dy, x, w, z=z, dx=dx, dw=dw, db=db[0])
        layer.check()
    _within(y, y64, yb)
    _within(z, z64, zb)
    _check_backward(dy, x, w, z, "gelu", dtype, "f32", dx, dw, db[0], None)
    assert clean() and zclean() and wclean() and bclean() and xclean()


def test_column_blocks_of_one_buffer(ddl):
    """x, residual, z and y side by side in one wider buffer, and dx beside them."""
    T, K, N = 140, 64, 40
    buf = torch.randn(T, 288, device="cuda").half()
    x, r, z, y, dx = buf[:, :64], buf[:, 64:104], buf[:, 104:144], buf[:, 144:184], buf[:, 184:248]
    w, dy = _normal(2, N, K, "f16", 0.1), _normal(3, T, N, "f16")
    before = buf.clone()
    dw, wclean = _blank(N, K, "f32")
    with ddl.Linear(K, N, T, "f16", "silu") as layer:
        layer.forward(x, w, y, residual=r, z=z)
        layer.backward(dy, x, w, z=z, dx=dx, dw=dw)
        layer.check()
    z64 = x.double() @ w.double().t()
    y64 = _act(z64, "silu") + r.double()
    zb, yb = _forward_bound(x, w, None, z64, r, y64, "f16")
    _within(z, z64, zb)
    _within(y, y64, yb)
    _check_backward(dy, x, w, z, "silu", "f16", "f32", dx, dw, None, None)
    assert torch.equal(buf[:, :104], before[:, :104]) and torch.equal(buf[:, 248:], before[:, 248:]) and wclean()


def test_residual_in_place(ddl):
    x, w, r = _normal(1, 150, 64, "bf16"), _normal(2, 96, 64, "bf16", 0.1), _normal(3, 150, 96, "bf16")
    with ddl.Linear(64, 96, 150, "bf16", "silu") as layer:
        apart, _ = _blank(150, 96, "bf16")
        layer.forward(x, w, apart, residual=r)
        layer.forward(x, w, r, residual=r)
        layer.check()
    assert torch.equal(apart, r)


def _check_backward(dy, x, w, z, act, dtype, grad, dx, dw, db, before):
    T, (N, K) = dy.shape[0], w.shape
    dz = dy.double() * (_slope(z.double(), act) if z is not None else 1)
    curved = act in ("gelu", "silu")
    keep16 = U[dtype] if curved else 0.0
    # GELU's and SiLU's slopes round to 2^-20 of terms up to 1.2, whatever they add up to
    slope_err = 2.0 ** -20 * 1.2 * dy.double().abs() if curved else torch.zeros_like(dz)
    half = TINY[dtype] * 2 if curved else 0.0
    if dx is not None:
        mag = dz.abs() @ w.double().abs()
        want = dz @ w.double()
        bound = ((N + 16) * 2.0 ** -23 + keep16) * mag + (slope_err + half) @ w.double().abs() + U[dtype] * want.abs()
        _within(dx, want, bound * 1.001 + TINY[dtype])
    if dw is not None:
        kept = (2.0 ** -21 if grad == "f32" else keep16) if curved else 0.0
        small = (2.0 ** -34 if dtype == "f16" and grad == "f32" else half) if curved else 0.0
        want = dz.t() @ x.double() + (before[0].double() if before else 0)
        mag = dz.abs().t() @ x.double().abs()
        bound = ((T + 16) * 2.0 ** -23 + kept) * mag + (slope_err + small).t() @ x.double().abs()
        bound = bound + U[grad] * (want.abs() + bound) + TINY[grad] + (2.0 ** -23 * before[0].double().abs() if before else 0)
        _within(dw, want, bound)
    if db is not None:
        want = dz.sum(0) + (before[1].double() if before else 0)
        bound = (T + 16) * 2.0 ** -23 * dz.abs().sum(0) + slope_err.sum(0) + U[grad] * want.abs() * 1.01 + TINY[grad]
        _within(db, want, bound + (2.0 ** -23 * before[1].double().abs() if before else 0))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("tokens, n_in, n_out", [
    (1, 1, 1), (1, 77, 33), (2, 128, 64), (63, 64, 128), (64, 200, 136), (129, 129, 129), (256, 2048, 1000),
    (517, 771, 1029), (1000, 64, 72), (3000, 136, 120),
    # 256 x 256 tiles on CTA pairs, whole and ragged; long sums of few tiles
    (2304, 1536, 2048), (2100, 1032, 2050), (9000, 264, 256),
])
def test_backward(ddl, tokens, n_in, n_out, dtype):
    dy, x = _normal(1, tokens, n_out, dtype), _normal(2, tokens, n_in, dtype)
    w, z = _normal(3, n_out, n_in, dtype, n_in ** -0.5), _normal(4, tokens, n_out, dtype)
    for act in ("none", "relu", "gelu", "silu"):
        zz = None if act == "none" else z
        with ddl.Linear(n_in, n_out, tokens, dtype, act) as layer:
            for grad in ("f32", "f16"):
                for accumulate in (False, True):
                    dx, xclean = _blank(tokens, n_in, dtype)
                    dw, wclean = _blank(n_out, n_in, grad)
                    db, bclean = _blank(1, n_out, grad)
                    before = None
                    if accumulate:
                        dw.copy_(torch.randn(n_out, n_in, device="cuda"))
                        db.copy_(torch.randn(1, n_out, device="cuda"))
                        before = (dw.clone(), db[0].clone())
                    layer.backward(dy, x, w, z=zz, dx=dx, dw=dw, db=db[0], accumulate=accumulate)
                    layer.check()
                    _check_backward(dy, x, w, zz, act, dtype, grad, dx, dw, db[0], before)
                    assert xclean() and wclean() and bclean()


@pytest.mark.parametrize("wanted", ["dx", "dw", "db", "dx dw", "dw db", "dx db"])
def test_backward_of_some(ddl, wanted):
    """Each result alone is the same result of a full call (layouts, hence the order of sums, may differ)."""
    T, K, N = 300, 200, 136
    dy, x, w, z = (_normal(1, T, N, "f16"), _normal(2, T, K, "f16"), _normal(3, N, K, "f16", 0.1), _normal(4, T, N, "f16"))

    def outs():  # every result on its own, against the same result of a full call
        return dict(dx=_blank(T, K, "f16")[0], dw=_blank(N, K, "f32")[0], db=_blank(1, N, "f32")[0][0])
    with ddl.Linear(K, N, T, "f16", "silu") as layer:
        full, part = outs(), outs()
        layer.backward(dy, x, w, z=z, **full)
        layer.backward(dy, x if "dw" in wanted else None, w if "dx" in wanted else None, z=z,
                       **{k: part[k] for k in wanted.split()})
        layer.check()
    for k, v in part.items():
        if k in wanted.split():
            bound = 1e-6 if k == "dw" else 2.0 ** -10
            assert (v.double() - full[k].double()).norm() <= bound * full[k].double().norm()
        else:
            assert bool((v == 7.0).all())


def test_gradient_against_differences(ddl):
    """dw, db and dx against central differences of the forward formula in 64 bits.  With step h
    the difference is off by h^2/6 times a third derivative (below 2 for GELU times |x|^3 |dy|)
    and by 2^-52 / h of the loss; h = 1e-4 keeps both under 1e-6 of the sums of magnitudes here."""
    T, K, N = 40, 24, 16
    x, w, dy = _normal(1, T, K, "bf16"), _normal(2, N, K, "bf16", 0.2), _normal(3, T, N, "bf16")
    bias = _normal(4, 1, N, "bf16")[0]
    z, y = _blank(T, N, "bf16")[0], _blank(T, N, "bf16")[0]
    dx, dw, db = _blank(T, K, "bf16")[0], _blank(N, K, "f32")[0], _blank(1, N, "f32")[0]
    with ddl.Linear(K, N, T, "bf16", "gelu") as layer:
        layer.forward(x, w, y, bias=bias, z=z)
        layer.backward(dy, x, w, z=z, dx=dx, dw=dw, db=db[0])
        layer.check()
    # the backward pass sees z rounded to bfloat16: the formula's z is moved there by a constant
    shift = z.double() - (x.double() @ w.double().t() + bias.double())

    def loss(xx, ww, bb):
        return (_act(xx @ ww.t() + bb + shift, "gelu") * dy.double()).sum()
    X, W, B, h = x.double(), w.double(), bias.double(), 1e-4
    scale = (dy.double().abs().t() @ x.double().abs()).max()
    for n, k in ((0, 0), (3, 7), (15, 23), (8, 11)):
        e = torch.zeros_like(W)
        e[n, k] = h
        diff = (loss(X, W + e, B) - loss(X, W - e, B)) / (2 * h)
        assert abs(diff - dw[n, k].double()) <= 1e-5 * scale
    for n in (0, 9, 15):
        e = torch.zeros_like(B)
        e[n] = h
        diff = (loss(X, W, B + e) - loss(X, W, B - e)) / (2 * h)
        assert abs(diff - db[0, n].double()) <= 1e-5 * dy.double().abs().sum(0).max()
    for t, k in ((0, 0), (17, 5), (39, 23)):
        e = torch.zeros_like(X)
        e[t, k] = h
        diff = (loss(X + e, W, B) - loss(X - e, W, B)) / (2 * h)
        mag = (dy[t].double().abs() * 1.13) @ W[:, k].abs()  # dz and dx are rounded to bfloat16 here
        assert abs(diff - dx[t, k].double()) <= 2.1 * 2.0 ** -8 * mag


def test_special_values(ddl):
    """Infinities and NaNs go where the formulas put them and nowhere else; huge slopes do not overflow."""
    T, K, N = 70, 64, 40
    x, w, dy, z = _normal(1, T, K, "f16"), _normal(2, N, K, "f16", 0.1), _normal(3, T, N, "f16"), _normal(4, T, N, "f16")
    x[3, 5], x[9, 0] = float("nan"), float("inf")
    y = _blank(T, N, "f16")[0]
    with ddl.Linear(K, N, T, "f16", "relu") as layer:
        layer.forward(x, w, y)
        layer.check()
    want = torch.clamp(x.double() @ w.double().t(), min=0)
    assert torch.equal(torch.isnan(y), torch.isnan(want)) and torch.equal(torch.isinf(y), torch.isinf(want))
    ok = torch.isfinite(want).all(1)
    assert int(ok.sum()) == T - 2 and bool(torch.isfinite(y[ok]).all())

    x = _normal(1, T, K, "f16")
    dy[4, 6], dy[5, 7] = 65504.0, float("inf")
    z[4, 6], z[5, 7] = 1.5, 1.0
    dw, db = _blank(N, K, "f32")[0], _blank(1, N, "f32")[0]
    with ddl.Linear(K, N, T, "f16", "gelu") as layer:
        layer.backward(dy, x, w, z=z, dw=dw, db=db[0])
        layer.check()
    dz = dy.double() * _slope(z.double(), "gelu")
    want = dz.t() @ x.double()
    rows = torch.arange(N, device="cuda") != 7
    assert bool(torch.isfinite(dw[rows]).all()) and not bool(torch.isfinite(dw[7]).any())
    assert (dw[rows].double() - want[rows]).norm() <= 1e-6 * want[rows].norm()
    assert torch.isinf(db[0, 7]) and bool(torch.isfinite(db[0, rows]).all())


def test_no_tokens(ddl):
    with ddl.Linear(16, 8, 4, "f16", "none") as layer:
        e = lambda n: torch.empty(0, n, dtype=torch.float16, device="cuda")  # noqa: E731
        layer.forward(e(16), _normal(1, 8, 16, "f16"), e(8))
        dw, clean = _blank(8, 16, "f32", 20, 3)
        db, bclean = _blank(1, 8, "f32")
        layer.backward(e(8), e(16), dw=dw, db=db[0], accumulate=True)
        assert bool((dw == 7.0).all()) and bool((db == 7.0).all())
        layer.backward(e(8), e(16), dw=dw, db=db[0])
        assert bool((dw == 0.0).all()) and bool((db == 0.0).all()) and clean() and bclean()


def test_repeats_and_streams(ddl):
    """The same call gives the same bits, also on a stream of its own behind an event, and replayed from a graph."""
    T, K, N = 900, 264, 520
    dy, x, w, z = _normal(1, T, N, "bf16"), _normal(2, T, K, "bf16"), _normal(3, N, K, "bf16", 0.1), _normal(4, T, N, "bf16")
    with ddl.Linear(K, N, T, "bf16", "gelu") as layer:
        def call(o, stream=None):
            layer.forward(x, w, o[0], z=o[1], stream=stream)
            layer.backward(dy, x, w, z=z, dx=o[2], dw=o[3], db=o[4][0], stream=stream)

        def outs():
            return [_blank(T, N, "bf16")[0], _blank(T, N, "bf16")[0], _blank(T, K, "bf16")[0], _blank(N, K, "f32")[0],
                    _blank(1, N, "f32")[0]]
        first, second, third = outs(), outs(), outs()
        call(first)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        call(second, side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(third)
        for _ in range(3):
            for o in third:
                o.fill_(0)
            graph.replay()
        torch.cuda.synchronize()
        layer.check()
    for a, b, c in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_more_than_2_31_elements(ddl):
    """Outputs past 2^31 elements: sampled rows against the formula."""
    T, K, N = 270_000, 64, 8192
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, K, generator=gen, device="cuda").half()
    w = _normal(2, N, K, "f16", 0.125)
    y = torch.empty(T, N, dtype=torch.float16, device="cuda")
    with ddl.Linear(K, N, T, "f16", "none") as layer:
        layer.forward(x, w, y)
        layer.check()
    at = torch.tensor([0, 1, 127, 128, 131_071, 262_143, 262_144, 262_145, T - 1], device="cuda")
    z = x[at].double() @ w.double().t()
    zb, yb = _forward_bound(x[at], w, None, z, None, z, "f16")
    _within(y[at], z, yb)


def test_refuses_host_memory_and_failed_allocation(ddl, monkeypatch):
    x, w = _normal(1, 8, 17, "f16"), _normal(2, 8, 17, "f16")
    y = _blank(8, 8, "f16")[0]
    host = torch.zeros(8, 17, dtype=torch.float16).pin_memory()
    with ddl.Linear(17, 8, 8, "f16") as layer:
        with pytest.raises(ddl.DDLError) as e:
            ddl.ddl_linear_forward(layer.handle, 8, host.data_ptr(), 17, w.data_ptr(), 17, None, None, 0, None, 0,
                                   y.data_ptr(), 8)
        assert e.value.status == ddl.DDL_ERR_INVALID_ARG
        monkeypatch.setenv("DDL_INJECT_ALLOC_FAILURE", "1")  # the rows are unaligned: workspace is needed
        with pytest.raises(ddl.DDLError) as e:
            layer.forward(x, w, y)
        assert e.value.status == ddl.DDL_ERR_OOM
        monkeypatch.delenv("DDL_INJECT_ALLOC_FAILURE")
        layer.forward(x, w, y)
        layer.check()
    z = x.double() @ w.double().t()
    _within(y, z, _forward_bound(x, w, None, z, None, z, "f16")[1])


@pytest.mark.parametrize("n_out", [8, 1])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_activations_of_every_number(ddl, dtype, n_out):
    """Every 16-bit number as a pre-activation: 2^-20 of its size for the activation, and the result's rounding."""
    x = torch.arange(1 << 16, device="cuda").to(torch.int32).to(torch.int16).view(TYPES[dtype]).view(-1, 1)
    w = torch.ones(n_out, 1, dtype=TYPES[dtype], device="cuda")
    z64 = x.double()
    for act in ("none", "relu", "gelu", "silu"):
        y = _blank(1 << 16, n_out, dtype)[0]
        with ddl.Linear(1, n_out, 1 << 16, dtype, act) as layer:
            layer.forward(x, w, y)
            layer.check()
        assert torch.equal(torch.nan_to_num(y), torch.nan_to_num(y[:, :1]).expand_as(y))
        want, got = _act(z64, act)[:, 0], y[:, 0].double()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.isinf(got), torch.isinf(want))
        ok = torch.isfinite(want)
        _within(got[ok], want[ok], 2.0 ** -20 * z64[ok, 0].abs() + U[dtype] * want[ok].abs() + TINY[dtype])


@pytest.mark.parametrize("tokens, n_in, n_out", [(3, 2240, 5568), (517, 771, 1029), (1834, 1152, 448)])
def test_binary16_gradient_of_a_bfloat16_layer(ddl, tokens, n_in, n_out):
    """Its 11 bits are not lost to a bfloat16 dz: at most the result's own rounding (2^-11 of each element) and as
    much again for the 16 bits of dz and the sum."""
    dy, x, z = _normal(1, tokens, n_out, "bf16"), _normal(2, tokens, n_in, "bf16"), _normal(4, tokens, n_out, "bf16")
    dw = _blank(n_out, n_in, "f16")[0]
    for act in ("gelu", "silu"):
        with ddl.Linear(n_in, n_out, tokens, "bf16", act) as layer:
            layer.backward(dy, x, z=z, dw=dw)
            layer.check()
        want = (dy.double() * _slope(z.double(), act)).t() @ x.double()
        assert (dw.double() - want).norm() <= 2.0 ** -10 * want.norm()


def _close_to_rounding(got, want, dtype, off):
    """In the Frobenius norm: the exact values' own rounding to the type (5 % for the sample), and `off` before it."""
    assert torch.isfinite(got.double()).all()
    rounding = (want.to(TYPES[dtype]).double() - want).norm()
    err = (got.double() - want).norm()
    assert err <= 1.05 * rounding + off, f"off by {err / want.norm():.2e}, rounding is {rounding / want.norm():.2e}"


@pytest.mark.parametrize("grad", ["f16", "f32"])
@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("scale", [1.0, 1e-4, 1e-5, 1e-6])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_dz_keeps_its_bits_in_large_calls(ddl, dtype, scale, act, grad):
    """More tiles than SMs, gradients of any size: dx and binary16 dw are off by their own rounding, not by dz's.  Before
    it: dz to 2^-21 of itself and 2^-34 (binary16) or 2^-16 (bfloat16), the slope's 2^-20 of up to 1.2 |dy|, both as if they
    added up; and a sum's additions of 16 products at 2^-22 of the result each (its partial sums grow up to it)."""
    T, K, N = 8192, 1024, 256
    dy, x = _normal(1, T, N, dtype, scale), _normal(2, T, K, dtype)
    w, z = _normal(3, N, K, dtype), _normal(4, T, N, dtype)
    dx, dw = _blank(T, K, dtype)[0], _blank(N, K, grad)[0]
    with ddl.Linear(K, N, T, dtype, act) as layer:
        layer.backward(dy, x, w, z=z, dx=dx, dw=dw)
        layer.check()
    dz = dy.double() * _slope(z.double(), act)
    kept = (2.0 ** -21 * dz.abs() + 2.0 ** -34) if dtype == "f16" else 2.0 ** -16 * dz.abs()
    kept = kept + 2.0 ** -20 * 1.2 * dy.double().abs()
    want = dz @ w.double()
    _close_to_rounding(dx, want, dtype, (kept @ w.double().abs()).norm() + (N / 16 + 16) * 2.0 ** -22 * want.norm())
    if grad == "f16":
        want = dz.t() @ x.double()
        _close_to_rounding(dw, want, grad, (kept.t() @ x.double().abs()).norm() + (T / 16 + 16) * 2.0 ** -22 * want.norm())


@pytest.mark.parametrize("grad", ["f16", "f32"])
def test_largest_gradients_in_large_calls(ddl, grad):
    """dz above binary16's largest number (65504 times a slope of 1.13) with finite dx and dw, more tiles than SMs."""
    T, K, N = 8192, 1024, 256
    dy, x, w, z = _normal(1, T, N, "f16"), _normal(2, T, K, "f16"), _normal(3, N, K, "f16", 1e-2), _normal(4, T, N, "f16")
    dy[77, 5], z[77, 5] = 65504.0, 1.5
    x[77] *= 0.01
    dx, dw = _blank(T, K, "f16")[0], _blank(N, K, grad)[0]
    with ddl.Linear(K, N, T, "f16", "gelu") as layer:
        layer.backward(dy, x, w, z=z, dx=dx, dw=dw)
        layer.check()
    dz = dy.double() * _slope(z.double(), "gelu")
    for got, want in ((dx, dz @ w.double()), (dw, dz.t() @ x.double())):
        assert torch.isfinite(got).all()
        assert (got.double() - want).norm() <= 2.0 ** -10 * want.norm()


@pytest.mark.parametrize("dtype, grad", [("f16", "f16"), ("f16", "f32"), ("bf16", "f16"), ("bf16", "f32")])
def test_fewer_tokens_need_no_more_memory(ddl, monkeypatch, dtype, grad):
    """What a handle's largest call has allocated is enough for its smaller ones (a stream capture could not allocate)."""
    K = N = 1024
    with ddl.Linear(K, N, 8192, dtype, "gelu") as layer:
        for tokens in (8192, 1024, 64, 1):
            dy, x, z = _normal(1, tokens, N, dtype), _normal(2, tokens, K, dtype), _normal(4, tokens, N, dtype)
            w, dx = _normal(3, N, K, dtype, 0.1), _blank(tokens, K, dtype)[0]
            dw, db = _blank(N, K, grad)[0], _blank(1, N, grad)[0]
            layer.backward(dy, x, w, z=z, dx=dx, dw=dw, db=db[0])
            layer.check()
            monkeypatch.setenv("DDL_INJECT_ALLOC_FAILURE", "1")
        monkeypatch.delenv("DDL_INJECT_ALLOC_FAILURE")


@pytest.mark.parametrize("tokens", [90, 3000])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_infinite_operands_of_split_products(ddl, dtype, tokens):
    """An infinity or NaN in x or w goes where the formula puts it, whatever the lower planes of dz are."""
    K, N = 136, 200
    dy, x = _normal(1, tokens, N, dtype), _normal(2, tokens, K, dtype)
    w, z = _normal(3, N, K, dtype), _normal(4, tokens, N, dtype)
    x[3, 5], x[60, 40], x[61, 41] = math.inf, -math.inf, math.nan
    w[7, 9], w[199, 135] = math.inf, -math.inf
    for act in ("gelu", "silu"):
        dz = dy.double() * _slope(z.double(), act)
        for grad in ("f32", "f16"):
            dx, dw = _blank(tokens, K, dtype)[0], _blank(N, K, grad)[0]
            with ddl.Linear(K, N, tokens, dtype, act) as layer:
                layer.backward(dy, x, w, z=z, dx=dx, dw=dw)
                layer.check()
            for got, want in ((dx, dz @ w.double()), (dw, dz.t() @ x.double())):
                assert int((~torch.isfinite(want)).sum()) >= 2 * want.shape[0]
                assert torch.equal(torch.isnan(got), torch.isnan(want))
                assert torch.equal(torch.isinf(got), torch.isinf(want))
                assert torch.equal(got[torch.isinf(got)].sign(), want[torch.isinf(want)].to(got.dtype).sign())


@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("tokens, n_in, n_out, dtype", [
    (64, 200, 136, "f16"), (128, 3759, 72, "bf16"), (256, 2624, 64, "bf16"), (384, 2944, 512, "f16"), (442, 64, 192, "f16"),
    (512, 2304, 6877, "bf16"), (562, 320, 987, "bf16"), (832, 128, 121, "bf16"), (860, 128, 256, "f16"), (1728, 122, 576, "f16"),
    (2560, 974, 64, "f16"), (5696, 79, 192, "bf16"), (8192, 1024, 1024, "bf16"), (20000, 136, 264, "f16"),
])
def test_binary32_dw_is_no_less_exact_than_binary32(ddl, tokens, n_in, n_out, dtype, act):
    """dz is exact here, so dw's error is the sum's: over several inputs no more than one and a half times what products
    in binary32 leave, and half a unit in the last place for the result."""
    own = plain = 0.0
    with ddl.Linear(n_in, n_out, tokens, dtype, act) as layer:
        for seed in range(3):
            dy, x, z = (_normal(10 * seed + k, tokens, n, dtype) for k, n in ((1, n_out), (2, n_in), (3, n_out)))
            dw = _blank(n_out, n_in, "f32")[0]
            layer.backward(dy, x, z=None if act == "none" else z, dw=dw)
            dz = dy if act == "none" else torch.where(z > 0, dy, torch.zeros_like(dy))
            want = dz.double().t() @ x.double()
            own += float((dw.double() - want).norm() / want.norm())
            plain += float((dz.float().t() @ x.float() - want).norm() / want.norm())
        layer.check()
    assert own <= 1.5 * plain + 3 * 2.0 ** -24, (own / 3, plain / 3)


def _one_sign(seed, rows, cols, dtype, top):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return ((0.5 + 0.5 * torch.rand(rows, cols, generator=gen, device="cuda")) * top).to(TYPES[dtype])


def _sums_in_64(a, b):
    """a b^T of long rows, in pieces."""
    return sum(p.double() @ q.double().t() for p, q in zip(a.split(1 << 17, 1), b.split(1 << 17, 1)))


LONG = [(3, 1 << 22, 16), (40, 1 << 21, 136), (100, 1 << 19, 136), (300, 1 << 18, 520), (2304, 20001, 2312)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows, long, cols", LONG)
def test_long_sums_of_one_sign(ddl, rows, long, cols, dtype):
    """Forward, dx and binary16 dw over the longest contractions: besides its rounding, a result may lose a quarter of half a
    unit in the last place to its sum (and a twentieth to the sums of its parts)."""
    bound = 1.3 * U[dtype]
    top = 16.0 / long  # sums of about ten
    a, b = _one_sign(1, rows, long, dtype, 1.0), _one_sign(2, cols, long, dtype, 2.0 ** 12 * top if dtype == "f16" else top)
    want = _sums_in_64(a, b)
    y, clean = _blank(rows, cols, dtype)
    z, _ = _blank(rows, cols, dtype)
    r = _one_sign(3, rows, cols, dtype, 1.0)
    with ddl.Linear(long, cols, rows, dtype, "none") as layer:
        layer.forward(a, b, y)
        layer.check()
        _within(y, want, bound * want)
        assert clean()
    with ddl.Linear(long, cols, rows, dtype, "relu") as layer:
        layer.forward(a, b, y, residual=r, z=z)
        layer.check()
        _within(z, want, bound * want)
        _within(y, want + r.double(), bound * (want + r.double()))
    # dx[rows][cols] = dy[rows][long] w[long][cols]
    w = b.t().contiguous()
    dx, clean = _blank(rows, cols, dtype)
    with ddl.Linear(cols, long, rows, dtype, "none") as layer:
        layer.backward(a, w=w, dx=dx)
        layer.check()
    _within(dx, want, bound * want)
    assert clean()
    # dw[rows][cols] = dy[long][rows]^T x[long][cols], in binary16 (bfloat16 layers too)
    dy, dw = a.t().contiguous(), _blank(rows, cols, "f16")[0]
    with ddl.Linear(cols, rows, long, dtype, "none") as layer:
        layer.backward(dy, w, dw=dw)
        layer.check()
    _within(dw, want, 1.3 * U["f16"] * want)


@pytest.mark.parametrize("n_out", [40, 37])  # rows that allow vectors, and rows that do not
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_closed_relu_units_pass_nothing_on(ddl, dtype, n_out):
    """ReLU's slope selects: whatever dy is at a unit with z <= 0, dx, dw and db are what a zero there gives."""
    T, K = 70, 64
    dy, x = _normal(1, T, n_out, dtype), _normal(2, T, K, dtype)
    w, z = _normal(3, n_out, K, dtype, 0.1), _normal(4, T, n_out, dtype)
    zeros = dy.clone()
    for t, n, g, at in ((3, 5, math.inf, -1.0), (4, 6, -math.inf, 0.0), (5, 7, math.nan, -0.0), (69, 36, math.inf, -6e4)):
        dy[t, n], zeros[t, n], z[t, n] = g, 0.0, at
    got, want = [(_blank(T, K, dtype)[0], _blank(n_out, K, "f32")[0], _blank(1, n_out, "f32")[0][0]) for _ in range(2)]
    with ddl.Linear(K, n_out, T, dtype, "relu") as layer:
        for g, (dx, dw, db) in ((dy, got), (zeros, want)):
            layer.backward(g, x, w, z=z, dx=dx, dw=dw, db=db)
        layer.check()
        for a, b in zip(got, want):
            assert bool(torch.isfinite(b).all()) and torch.equal(a, b)
        z[3, 5] = 1.0  # an open unit does pass it on
        layer.backward(dy, z=z, db=got[2])
        layer.check()
    assert float(got[2][5]) == math.inf


def test_no_tokens_and_dx_alone(ddl):
    """An empty batch's dx has no elements, and torch gives it no address."""
    with ddl.Linear(16, 8, 4, "f16", "gelu") as layer:
        e = lambda n: torch.empty(0, n, dtype=torch.float16, device="cuda")  # noqa: E731
        layer.backward(e(8), w=_normal(1, 8, 16, "f16"), z=e(8), dx=e(16))
        layer.check()


def test_residual_in_place_of_one_row(ddl):
    """A single row's stride says nothing about where its elements are."""
    x, w, r = _normal(1, 1, 64, "f16"), _normal(2, 96, 64, "f16", 0.1), _normal(3, 1, 96, "f16")
    with ddl.Linear(64, 96, 150, "f16", "silu") as layer:
        apart, _ = _blank(1, 96, "f16")
        layer.forward(x, w, apart, residual=r)
        ddl.ddl_linear_forward(layer.handle, 1, x.data_ptr(), 64, w.data_ptr(), 64, None, r.data_ptr(), 96, None, 0,
                               r.data_ptr(), 104)
        layer.check()
    assert torch.equal(apart, r)


STOPS = [dict(products=0), dict(products=1), dict(loads_even=0), dict(loads_even=3), dict(loads_odd=0), dict(loads_odd=3),
         dict(loads_even=2, loads_odd=6), dict(loads_even=7, loads_odd=4), dict(products=1, loads_even=6)]


@pytest.mark.parametrize("stop", STOPS, ids=str)
@pytest.mark.parametrize("tokens, n_in, n_out, dtype", [
    (8, 2048, 520, "f16"), (50, 2048, 264, "bf16"), (150, 1024, 136, "f16"), (150, 1024, 131, "f16"), (300, 40000, 264, "f16"),
    (2304, 1536, 2304, "bf16"), (2304, 1536, 2301, "bf16"), (2304, 20001, 2304, "f16"),
])
def test_waits_that_run_out_end_the_call(ddl, tokens, n_in, n_out, dtype, stop):
    """A role of the product kernel stops, what waits for it gives up: the call ends, the error word tells, and the calls
    after it are right.  (A stop beyond what a CTA has to do is none.)"""
    x, w = _normal(1, tokens, n_in, dtype), _normal(2, n_out, n_in, dtype, n_in ** -0.5)
    dy, r = _normal(3, tokens, n_out, dtype), _normal(4, tokens, n_out, dtype)

    def outs():
        return _blank(tokens, n_out, dtype)[0], _blank(tokens, n_in, dtype)[0], _blank(n_out, n_in, "f32")[0]
    want, void, got = outs(), outs(), outs()
    with ddl.Linear(n_in, n_out, tokens, dtype, "none") as layer:
        def forward(o):
            layer.forward(x, w, o[0], residual=r)

        def backward(o):
            layer.backward(dy, x, w, dx=o[1], dw=o[2])
        forward(want), backward(want)
        layer.check()
        for call in (forward, backward):
            ddl.ddl_linear_selftest_wait_timeout(layer.handle, 500, **stop)
            call(void)
            if stop.get("products") == 0 or stop.get("loads_even") == 0:
                with pytest.raises(ddl.DDLError) as e:
                    layer.check()
                assert e.value.status == ddl.DDL_ERR_DEVICE_CHECK
            else:
                try:
                    layer.check()
                except ddl.DDLError as e:
                    assert e.status == ddl.DDL_ERR_DEVICE_CHECK
            forward(got), backward(got)
            layer.check()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
