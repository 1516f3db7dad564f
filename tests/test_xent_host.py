"""Host side of the softmax cross entropy: what the entry points refuse, before any GPU work (no GPU is used here)."""
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
    ((0, 8, 8, 1, 0.0), "DDL_ERR_INVALID_ARG"),
    ((8, 0, 8, 1, 0.0), "DDL_ERR_INVALID_ARG"),
    ((8, 8, 0, 1, 0.0), "DDL_ERR_INVALID_ARG"),
    ((8, 8, 8, 7, 0.0), "DDL_ERR_INVALID_ARG"),
    ((8, 8, 8, 1, 1.0), "DDL_ERR_INVALID_ARG"),
    ((8, 8, 8, 1, -0.1), "DDL_ERR_INVALID_ARG"),
    ((8, 8, 8, 1, float("nan")), "DDL_ERR_INVALID_ARG"),
    ((8, 8, 8, 0, 0.0), "DDL_ERR_UNSUPPORTED"),
    (((1 << 20) + 1, 8, 8, 1, 0.0), "DDL_ERR_UNSUPPORTED"),
    ((8, (1 << 22) + 1, 8, 2, 0.0), "DDL_ERR_UNSUPPORTED"),
    ((8, 8, (1 << 22) + 1, 2, 0.0), "DDL_ERR_UNSUPPORTED"),
])
def test_create_refuses(ddl, args, want):
    assert _status(ddl, ddl.ddl_xent_create, *args) == getattr(ddl, want)


# addresses that are never touched: every call below is refused first
M = 1 << 20


def _head(ddl):
    return ddl.CrossEntropy(16, 24, 8, "f16")


@pytest.mark.parametrize("change", [
    dict(tokens=9), dict(x=None), dict(w=None), dict(labels=None), dict(loss=None, lse=None), dict(ldx=15), dict(ldw=15),
    dict(ldx=(1 << 31) + 1), dict(x=M + 1), dict(w=2 * M + 1), dict(bias=3 * M + 1), dict(labels=4 * M + 4), dict(loss=5 * M + 2),
    dict(lse=6 * M + 1), dict(loss=M), dict(loss=2 * M + 4), dict(lse=3 * M), dict(lse=4 * M + 60), dict(lse=5 * M + 28),
    dict(loss=(1 << 64) - 16),
])
def test_forward_refuses(ddl, change):
    a = dict(tokens=8, x=M, ldx=16, w=2 * M, ldw=16, bias=3 * M, labels=4 * M, loss=5 * M, lse=6 * M)
    a.update(change)
    with _head(ddl) as head:
        assert _status(ddl, ddl.ddl_xent_forward, head.handle, *a.values(), 0) == ddl.DDL_ERR_INVALID_ARG


def test_forward_without_tokens_queues_nothing(ddl):
    with _head(ddl) as head:
        ddl.ddl_xent_forward(head.handle, 0, None, 0, None, 0, None, None, None, None, 0)


@pytest.mark.parametrize("change", [
    dict(tokens=9), dict(x=None), dict(w=None), dict(labels=None), dict(lse=None), dict(dx=None, dw=None, db=None), dict(ldx=15),
    dict(ldw=15), dict(lddx=15), dict(lddw=15), dict(grad=2), dict(dx=8 * M + 1), dict(dw=9 * M + 2), dict(db=10 * M + 2),
    dict(lse=5 * M + 2), dict(dloss=6 * M + 1), dict(labels=4 * M + 4), dict(dx=M), dict(dw=2 * M), dict(db=3 * M), dict(dw=4 * M),
    dict(db=5 * M), dict(dx=6 * M + 2), dict(dx=9 * M + 4), dict(db=9 * M),
])
def test_backward_refuses(ddl, change):
    a = dict(tokens=8, x=M, ldx=16, w=2 * M, ldw=16, bias=3 * M, labels=4 * M, lse=5 * M, dloss=6 * M, dx=8 * M, lddx=16, dw=9 * M,
             lddw=16, db=10 * M, grad=ddl.DDL_FP32, accumulate=0)
    a.update(change)
    with _head(ddl) as head:
        assert _status(ddl, ddl.ddl_xent_backward, head.handle, *a.values(), 0) == ddl.DDL_ERR_INVALID_ARG


def test_calls_refuse_no_handle(ddl):
    f = ddl._lib
    assert f.ddl_xent_forward(None, 1, M, 16, 2 * M, 16, None, 3 * M, 4 * M, None, None) == ddl.DDL_ERR_INVALID_ARG
    assert f.ddl_xent_backward(None, 1, M, 16, 2 * M, 16, None, 3 * M, 4 * M, None, 5 * M, 16, None, 0, None, 0, 0,
                               None) == ddl.DDL_ERR_INVALID_ARG
    assert f.ddl_xent_check(None, None) == ddl.DDL_ERR_INVALID_ARG
    assert f.ddl_xent_create(8, 8, 8, ddl.DDL_FP16, 0.0, None) == ddl.DDL_ERR_INVALID_ARG
    assert f.ddl_xent_selftest_wait_timeout(None, 10, 0, 0, 0) == ddl.DDL_ERR_INVALID_ARG
    assert f.ddl_xent_destroy(None) == ddl.DDL_OK


def test_check_before_any_gpu_call(ddl):
    with _head(ddl) as head:
        ddl.ddl_xent_check(head.handle, 0)
        assert _status(ddl, ddl.ddl_xent_selftest_wait_timeout, head.handle, 2_000_001) == ddl.DDL_ERR_INVALID_ARG
    head.close()  # twice is fine


def test_no_read_only_loads_of_what_a_launch_before_may_write():
    """Kernels that start while the launch before them ends read nothing but the library's own tables as read-only memory."""
    import os
    import re

    from gradient_all_reduce_ddl_gb300.build import CSRC
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name), encoding="utf-8") as f:
            code = re.sub(r"//[^\n]*", "", f.read())
        loads = re.findall(r"__ldg\(\s*(\w+)|ld\.global\.nc", code)
        assert set(loads) <= {"tile"}, name
