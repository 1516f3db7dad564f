"""Host side of the linear layers and the orthogonalised update: what the entry
points refuse, before any GPU work (no GPU is used here)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def ddl():
    from gradient_all_reduce_ddl_gb300.build import build
    build()
    from gradient_all_reduce_ddl_gb300 import ddl as mod
    return mod


def _status(ddl, fn, *args):
    try:
        fn(*args)
    except ddl.DDLError as e:
        return e.status
    return ddl.DDL_OK


@pytest.mark.parametrize("args, want", [
    ((0, 8, 8, "DDL_FP16", 0), "DDL_ERR_INVALID_ARG"),
    ((8, 0, 8, "DDL_FP16", 0), "DDL_ERR_INVALID_ARG"),
    ((8, 8, 0, "DDL_FP16", 0), "DDL_ERR_INVALID_ARG"),
    ((8, 8, 8, "DDL_FP16", 4), "DDL_ERR_INVALID_ARG"),
    ((8, 8, 8, "DDL_FP16", -1), "DDL_ERR_INVALID_ARG"),
    ((8, 8, 8, 7, 0), "DDL_ERR_INVALID_ARG"),
    ((8, 8, 8, "DDL_FP32", 0), "DDL_ERR_UNSUPPORTED"),
    ((8, (1 << 22) + 1, 8, "DDL_BF16", 0), "DDL_ERR_UNSUPPORTED"),
    ((8, 8, (1 << 22) + 1, "DDL_BF16", 0), "DDL_ERR_UNSUPPORTED"),
    (((1 << 26) + 1, 8, 8, "DDL_BF16", 0), "DDL_ERR_UNSUPPORTED"),
])
def test_linear_create_refuses(ddl, args, want):
    t, i, o, dt, act = args
    dt = getattr(ddl, dt) if isinstance(dt, str) else dt
    assert _status(ddl, ddl.ddl_linear_create, t, i, o, dt, act) == getattr(ddl, want)


def _layer(ddl, act="none"):
    return ddl.Linear(16, 24, 8, "f16", act)


# addresses that are never touched: every call below is refused first
A, B, C, D = (1 << 20, 2 << 20, 3 << 20, 4 << 20)


@pytest.mark.parametrize("change", [
    dict(tokens=9), dict(x=None), dict(w=None), dict(y=None), dict(ldx=15), dict(ldw=15), dict(ldy=23),
    dict(x=A + 1), dict(y=C + 1), dict(residual=D, ldr=23), dict(z=D, ldz=23), dict(ldx=(1 << 31) + 1),
    dict(y=A), dict(y=B + 100), dict(y=A + 15 * 2), dict(z=C, ldz=24), dict(z=A, ldz=24), dict(residual=C, ldr=25),
    dict(residual=C + 2, ldr=24), dict(bias=C), dict(residual=C, ldr=24, z=C, ldz=24),
    # column blocks of one buffer that share a column, of other pitches, or that run over the pitch
    dict(x=A, ldx=64, y=A + 15 * 2, ldy=64), dict(x=A, ldx=64, y=A + 32, ldy=65), dict(x=A, ldx=64, y=A + 41 * 2, ldy=64),
])
def test_linear_forward_refuses(ddl, change):
    a = dict(tokens=8, x=A, ldx=16, w=B, ldw=16, bias=None, residual=None, ldr=0, z=None, ldz=0, y=C, ldy=24)
    a.update(change)
    with _layer(ddl) as layer:
        assert _status(ddl, ddl.ddl_linear_forward, layer.handle, *a.values(), 0) == ddl.DDL_ERR_INVALID_ARG


def test_linear_forward_without_tokens_queues_nothing(ddl):
    with _layer(ddl) as layer:
        ddl.ddl_linear_forward(layer.handle, 0, None, 0, None, 0, None, None, 0, None, 0, None, 0, 0)


@pytest.mark.parametrize("act, change", [
    ("none", dict(tokens=9)), ("none", dict(dy=None)), ("none", dict(x=None)), ("none", dict(w=None)),
    ("gelu", dict(z=None)), ("none", dict(dx=None, dw=None, db=None)), ("none", dict(ldy=23)), ("none", dict(ldx=15)),
    ("none", dict(ldw=15)), ("relu", dict(ldz=23)), ("none", dict(lddx=15)), ("none", dict(lddw=15)),
    ("none", dict(grad=2)), ("none", dict(dw=5 * A + 2)), ("none", dict(db=6 * A + 2)), ("none", dict(dx=5 * A)),
    ("none", dict(dw=A)), ("none", dict(db=2 * A)), ("none", dict(dx=3 * A)), ("silu", dict(dx=7 * A + 2)),
    ("none", dict(dy=A + 1)),
])
def test_linear_backward_refuses(ddl, act, change):
    a = dict(tokens=8, dy=A, ldy=24, x=2 * A, ldx=16, w=3 * A, ldw=16, z=7 * A, ldz=24, dx=4 * A, lddx=16, dw=5 * A,
             lddw=16, db=6 * A, grad=ddl.DDL_FP32, accumulate=0)
    a.update(change)
    with _layer(ddl, act) as layer:
        assert _status(ddl, ddl.ddl_linear_backward, layer.handle, *a.values(), 0) == ddl.DDL_ERR_INVALID_ARG


def test_linear_calls_refuse_no_handle(ddl):
    f = ddl._lib
    assert f.ddl_linear_forward(None, 1, A, 16, B, 16, None, None, 0, None, 0, C, 24, None) == ddl.DDL_ERR_INVALID_ARG
    assert f.ddl_linear_backward(None, 1, A, 24, B, 16, C, 16, None, 0, D, 16, None, 0, None, 0, 0,
                                 None) == ddl.DDL_ERR_INVALID_ARG
    assert f.ddl_linear_check(None, None) == ddl.DDL_ERR_INVALID_ARG
    assert f.ddl_linear_create(8, 8, 8, ddl.DDL_FP16, 0, None) == ddl.DDL_ERR_INVALID_ARG
    assert f.ddl_linear_destroy(None) == ddl.DDL_OK


def test_linear_check_before_any_gpu_call(ddl):
    with _layer(ddl) as layer:
        ddl.ddl_linear_check(layer.handle, 0)


@pytest.mark.parametrize("mats, dtype, want", [
    ([], "DDL_FP32", "DDL_ERR_INVALID_ARG"),
    ([(0, 0, 4)], "DDL_FP32", "DDL_ERR_INVALID_ARG"),
    ([(0, 4, 0)], "DDL_FP32", "DDL_ERR_INVALID_ARG"),
    ([(0, 4, 4, 3)], "DDL_FP32", "DDL_ERR_INVALID_ARG"),
    ([(0, 4, 4), (15, 4, 4)], "DDL_FP32", "DDL_ERR_INVALID_ARG"),
    ([(16, 4, 4), (0, 4, 4, 5)], "DDL_FP32", "DDL_ERR_INVALID_ARG"),
    ([(0, 4, 4)], 9, "DDL_ERR_INVALID_ARG"),
    ([(1 << 61, 4, 4)], "DDL_FP32", "DDL_ERR_INVALID_ARG"),
    ([(0, 4, 4, 1 << 60)], "DDL_FP32", "DDL_ERR_INVALID_ARG"),
    ([(0, (1 << 22) + 1, 1)], "DDL_FP32", "DDL_ERR_UNSUPPORTED"),
    ([(0, 1, (1 << 22) + 1)], "DDL_FP32", "DDL_ERR_UNSUPPORTED"),
    ([(0, 4, 4), (16, 4, 4)], "DDL_FP32", "DDL_OK"),
    ([(19, 4, 4), (0, 4, 4, 5)], "DDL_FP16", "DDL_OK"),
])
def test_ortho_create_refuses(ddl, mats, dtype, want):
    dt = getattr(ddl, dtype) if isinstance(dtype, str) else dtype
    assert _status(ddl, ddl.ddl_ortho_create, mats, dt) == getattr(ddl, want)


@pytest.mark.parametrize("args", [(0, 1, 1, 1, 0), (33, 1, 1, 1, 0), (5, 1, 1, 1, -1e-7), (5, 1, 1, 1, float("nan"))])
def test_ortho_polynomial_refuses(ddl, args):
    with ddl.Ortho([(0, 4, 4)]) as o:
        assert _status(ddl, ddl.ddl_ortho_set_polynomial, o.handle, *args) == ddl.DDL_ERR_INVALID_ARG


@pytest.mark.parametrize("inp, out", [(0, A), (A, 0), (A, A + 4), (A + 2, B), (A, B + 1)])
def test_ortho_run_refuses(ddl, inp, out):
    with ddl.Ortho([(0, 4, 4)]) as o:
        assert _status(ddl, ddl.ddl_ortho_run, o.handle, inp, out, 0) == ddl.DDL_ERR_INVALID_ARG


@pytest.mark.parametrize("grad, params, mom, want", [
    (0, [A], B, "DDL_ERR_INVALID_ARG"), (C, [0], B, "DDL_ERR_INVALID_ARG"), (C, [A], 0, "DDL_ERR_INVALID_ARG"),
    (C, [], B, "DDL_ERR_INVALID_ARG"), (C, [A, A + 32], B, "DDL_ERR_INVALID_ARG"), (C, [A], A, "DDL_ERR_INVALID_ARG"),
    (C, [C], B, "DDL_ERR_INVALID_ARG"), (C, [A], C + 4, "DDL_ERR_INVALID_ARG"), (C, [A + 2], B, "DDL_ERR_INVALID_ARG"),
    (C, [A + (k << 12) for k in range(257)], B << 4, "DDL_ERR_UNSUPPORTED"),
])
def test_muon_refuses(ddl, grad, params, mom, want):
    with ddl.Ortho([(0, 4, 4)]) as o:
        assert _status(ddl, ddl.ddl_ortho_muon, o.handle, grad, params, mom, 0.1, 0.9, 0.0, True, 0) == getattr(ddl, want)


def test_muon_refuses_bfloat16_gradients(ddl):
    with ddl.Ortho([(0, 4, 4)], dtype="bf16") as o:
        assert _status(ddl, ddl.ddl_ortho_muon, o.handle, C, [A], B, 0.1, 0.9, 0.0, True, 0) == ddl.DDL_ERR_UNSUPPORTED


def test_plans_refuse_bfloat16(ddl):
    h = ctypes.c_void_p()
    topo = ddl.ddl_topology_t(ddl.DDL_RING, 1, 0, 0)
    assert ddl._lib.ddl_plan_create(4, 64, ddl.DDL_BF16, topo, 0, ctypes.byref(h)) == ddl.DDL_ERR_INVALID_ARG


def test_binding_checks_tensors(ddl):
    torch = pytest.importorskip("torch")
    cpu = torch.zeros(8, 16, dtype=torch.float16)
    with _layer(ddl) as layer:
        with pytest.raises(ValueError):
            layer.forward(cpu, cpu, cpu)
    with ddl.Ortho([(0, 4, 4)]) as o:
        with pytest.raises(ValueError):
            o.run(torch.zeros(16), torch.zeros(16))


@pytest.mark.parametrize("kind", ["linear", "ortho"])
def test_a_failing_destroy_is_not_repeated(ddl, monkeypatch, kind):
    """The handle is gone whatever destroy returns; closing again must not pass it on a second time."""
    handle = ddl.Linear(4, 4, 4) if kind == "linear" else ddl.Ortho([(0, 2, 2)])
    name, calls = f"ddl_{kind}_destroy", []
    real = getattr(ddl, name)

    def failing(h):
        calls.append(h)
        real(h)
        raise ddl.DDLError(ddl.DDL_ERR_CUDA, name)
    monkeypatch.setattr(ddl, name, failing)
    with pytest.raises(ddl.DDLError):
        handle.close()
    handle.close()
    del handle
    assert len(calls) == 1


def test_linear_backward_of_no_tokens_without_dw_and_db_queues_nothing(ddl):
    with _layer(ddl) as layer:
        ddl.ddl_linear_backward(layer.handle, 0, None, 0, None, 0, B, 16, None, 0, None, 0, None, 0, None, ddl.DDL_FP32,
                                False, 0)


@pytest.mark.parametrize("limit, want", [(0, "DDL_OK"), (2_000_000, "DDL_OK"), (2_000_001, "DDL_ERR_INVALID_ARG")])
def test_wait_selftests_refuse_longer_limits(ddl, limit, want):
    with _layer(ddl) as layer, ddl.Ortho([(0, 4, 4)]) as o:
        assert _status(ddl, ddl.ddl_linear_selftest_wait_timeout, layer.handle, limit) == getattr(ddl, want)
        assert _status(ddl, ddl.ddl_ortho_selftest_wait_timeout, o.handle, limit) == getattr(ddl, want)
    assert ddl._lib.ddl_linear_selftest_wait_timeout(None, 1, 0, 0, 0) == ddl.DDL_ERR_INVALID_ARG
    assert ddl._lib.ddl_ortho_selftest_wait_timeout(None, 1, 0, 0, 0) == ddl.DDL_ERR_INVALID_ARG
