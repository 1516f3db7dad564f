"""Host side of the AdamW step: what the entry points refuse, before any GPU work (no GPU is used here)."""
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


@pytest.mark.parametrize("tensors, dtype, bits, want", [
    ([], 0, 32, "DDL_ERR_INVALID_ARG"),
    ([(0, 0)], 0, 32, "DDL_ERR_INVALID_ARG"),
    ([(0, 4)], 0, 16, "DDL_ERR_INVALID_ARG"),
    ([(0, 4)], 3, 32, "DDL_ERR_INVALID_ARG"),
    ([(0, 4)], 2, 32, "DDL_ERR_UNSUPPORTED"),
    ([(0, 4), (3, 4)], 0, 32, "DDL_ERR_INVALID_ARG"),
    ([(8, 4), (0, 9)], 0, 8, "DDL_ERR_INVALID_ARG"),
    ([((1 << 48) + 1, 4)], 0, 32, "DDL_ERR_INVALID_ARG"),
    ([(0, (1 << 48) + 1)], 0, 32, "DDL_ERR_INVALID_ARG"),
    ([(0, 1 << 41)], 0, 8, "DDL_ERR_UNSUPPORTED"),
    ([(0, 1 << 34), (1 << 40, (1 << 34) + 1)], 0, 32, "DDL_ERR_UNSUPPORTED"),
    ([(0, 4, float("nan"))], 0, 32, "DDL_ERR_INVALID_ARG"),
    ([(0, 4, 1.0, float("inf"))], 0, 32, "DDL_ERR_INVALID_ARG"),
])
def test_create_refuses(ddl, tensors, dtype, bits, want):
    assert _status(ddl, ddl.ddl_adam_create, tensors, dtype, bits) == getattr(ddl, want)


@pytest.mark.parametrize("betas", [(-0.1, 0.9, 1e-8), (1.0, 0.9, 1e-8), (0.9, 1.0, 1e-8), (0.9, float("nan"), 1e-8),
                                   (0.9, 0.99, 0.0), (0.9, 0.99, -1.0), (0.9, 0.99, 1e-60), (0.9, 0.99, float("inf"))])
def test_constants_refuse(ddl, betas):
    with ddl.Adam([(0, 8)]) as adam:
        assert _status(ddl, ddl.ddl_adam_set_betas, adam.handle, *betas) == ddl.DDL_ERR_INVALID_ARG


def test_blocks_are_counted_by_tensor(ddl):
    with ddl.Adam([(0, 1), (1, 128), (129, 129), (300, 1000)], state="8bit") as adam:
        assert adam.n_blocks == 1 + 1 + 2 + 8


# addresses that are never touched: every call below is refused first
M = 1 << 20


@pytest.mark.parametrize("change", [
    dict(grad=None), dict(params=[]), dict(params=[2 * M, None]), dict(m=None), dict(v=None), dict(step=None),
    dict(grad=M + 2), dict(params=[2 * M + 2]), dict(m=3 * M + 1), dict(v=4 * M + 2), dict(step=5 * M + 4), dict(norm=6 * M + 2),
    dict(scales=7 * M), dict(params=[2 * M, 2 * M + 252]), dict(params=[M]), dict(m=M + 252), dict(v=3 * M), dict(step=2 * M + 248),
    dict(norm=4 * M), dict(operands=[2 * M]), dict(operands=[8 * M + 1]), dict(operands=[M]), dict(operands=[8 * M], odt=0),
    dict(params=[2 * M, 9 * M], operands=[8 * M, 8 * M + 126]), dict(params=[2 * M, 9 * M], operands=[8 * M, None]),
    dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(max_norm=float("inf")), dict(params=[(1 << 64) - 64]),
])
def test_step_refuses(ddl, change):
    a = dict(grad=M, params=[2 * M], operands=None, odt=ddl.DDL_FP16, m=3 * M, v=4 * M, scales=None, step=5 * M, max_norm=0.0,
             norm=None)
    a.update(change)
    arr = lambda ps: None if ps is None else (ctypes.c_void_p * max(1, len(ps)))(*ps)  # noqa: E731
    with ddl.Adam([(0, 64)]) as adam:
        assert ddl._lib.ddl_adam_step(adam.handle, a["grad"], len(a["params"]), arr(a["params"]), arr(a["operands"]), a["odt"],
                                      a["m"], a["v"], a["scales"], a["step"], 0.1, 0.0, 1.0, a["max_norm"], a["norm"],
                                      None) == ddl.DDL_ERR_INVALID_ARG


def test_step_refuses_too_many_copies_and_missing_scales(ddl):
    f = ddl._lib.ddl_adam_step
    ps = (ctypes.c_void_p * 257)(*[(16 + k) * M for k in range(257)])
    with ddl.Adam([(0, 64)]) as adam:
        assert f(adam.handle, M, 257, ps, None, 0, 3 * M, 4 * M, None, 5 * M, 0.1, 0.0, 1.0, 0.0, None,
                 None) == ddl.DDL_ERR_UNSUPPORTED
    with ddl.Adam([(0, 64)], state="8bit") as adam:
        assert f(adam.handle, M, 1, ps, None, 0, 3 * M, 4 * M, None, 5 * M, 0.1, 0.0, 1.0, 0.0, None,
                 None) == ddl.DDL_ERR_INVALID_ARG
        # the scales of both states: 8 bytes a block
        assert f(adam.handle, M, 1, ps, None, 0, 3 * M, 4 * M, 5 * M - 4, 5 * M, 0.1, 0.0, 1.0, 0.0, None,
                 None) == ddl.DDL_ERR_INVALID_ARG


def test_calls_refuse_no_handle(ddl):
    f = ddl._lib
    ps = (ctypes.c_void_p * 1)(2 * M)
    assert f.ddl_adam_step(None, M, 1, ps, None, 0, 3 * M, 4 * M, None, 5 * M, 0.1, 0.0, 1.0, 0.0, None,
                           None) == ddl.DDL_ERR_INVALID_ARG
    assert f.ddl_adam_blocks(None, None) == ddl.DDL_ERR_INVALID_ARG
    assert f.ddl_adam_set_betas(None, 0.9, 0.99, 1e-8) == ddl.DDL_ERR_INVALID_ARG
    assert f.ddl_adam_create(1, (ddl.ddl_tensor_t * 1)(), 0, 32, None) == ddl.DDL_ERR_INVALID_ARG
    assert f.ddl_adam_destroy(None) == ddl.DDL_OK


def test_object_checks_its_tensors(ddl):
    torch = pytest.importorskip("torch")
    host = torch.zeros(64)
    with ddl.Adam([(0, 64)]) as adam:
        with pytest.raises(ValueError):
            adam.step(host, [host], host, host, torch.zeros(1, dtype=torch.int64), 0.1)
    adam.close()  # twice is fine
