"""The key/value cache calls without a GPU: exports, refusals of plans and of
arguments (nothing is launched), and the oracle's own number format."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import kv_oracle as ko

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def rc():
    from activation_residual_compression_amd import librescomp
    return librescomp


# short sequences and one block of them: never split, so no workspace and no device needed
SMALL = dict(batch=2, q_heads=4, kv_heads=2, head_dim=64, pool_blocks=8, seq_blocks=4, max_queries=4)


def test_exports_every_declared_function(rc):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "librescomp_kv.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(rc_kv_[a-z0-9_]+)\s*\(", text))
    assert names == {"rc_kv_plan_create", "rc_kv_plan_destroy", "rc_kv_store", "rc_kv_select", "rc_kv_attend",
                     "rc_kv_workspace_bytes"}
    lib = ctypes.CDLL(rc.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n


def test_header_constants_match_binding(rc):
    text = open(os.path.join(ROOT, "include", "librescomp_kv.h")).read()
    for name in ("RC_KV_BLOCK", "RC_KV_QTILE", "RC_KV_MAX_BLOCKS"):
        assert int(re.search(r"#define %s (\d+)" % name, text).group(1)) == getattr(rc, name)


@pytest.mark.parametrize("bad,status", [
    (dict(batch=0), "RC_ERR_INVALID_ARG"), (dict(q_heads=0), "RC_ERR_INVALID_ARG"),
    (dict(kv_heads=3), "RC_ERR_INVALID_ARG"), (dict(head_dim=0), "RC_ERR_INVALID_ARG"),
    (dict(head_dim=96), "RC_ERR_UNSUPPORTED"), (dict(head_dim=256), "RC_ERR_UNSUPPORTED"),
    (dict(pool_blocks=0), "RC_ERR_INVALID_ARG"), (dict(seq_blocks=0), "RC_ERR_INVALID_ARG"),
    (dict(seq_blocks=8193), "RC_ERR_UNSUPPORTED"), (dict(batch=65536), "RC_ERR_UNSUPPORTED"),
    (dict(max_queries=0), "RC_ERR_INVALID_ARG"), (dict(scale=-1.0), "RC_ERR_INVALID_ARG"),
    (dict(scale=float("nan")), "RC_ERR_INVALID_ARG"), (dict(scale=float("inf")), "RC_ERR_INVALID_ARG"),
    (dict(q_tile=64, keep_blocks=2), "RC_ERR_UNSUPPORTED"), (dict(q_tile=-1, keep_blocks=2), "RC_ERR_INVALID_ARG"),
    (dict(q_tile=1), "RC_ERR_INVALID_ARG"), (dict(keep_blocks=1), "RC_ERR_INVALID_ARG"),
    (dict(q_tile=1, keep_blocks=1025), "RC_ERR_UNSUPPORTED"),
    (dict(q_tile=128, keep_blocks=2, causal=True), "RC_ERR_INVALID_ARG"),
    (dict(dtype=7), "RC_ERR_INVALID_ARG"), (dict(max_queries=1 << 29), "RC_ERR_UNSUPPORTED"),
])
def test_plan_refusals(rc, bad, status):
    with pytest.raises(rc.RcError) as ei:
        rc.KvPlan(**{**SMALL, **bad})
    assert ei.value.status == getattr(rc, status)


def test_plan_refuses_unknown_flag_and_null(rc):
    shape = rc.rc_kv_shape_t(1, 1, 1, 64, 1, 1)
    with pytest.raises(rc.RcError) as ei:
        rc.rc_kv_plan_create(shape, "bf16", rc.rc_kv_params_t(1, 0.0, 0, 0, 2))
    assert ei.value.status == rc.RC_ERR_INVALID_ARG
    assert rc._lib.rc_kv_plan_create(shape, 0, None, ctypes.byref(ctypes.c_void_p())) == rc.RC_ERR_INVALID_ARG
    assert rc._lib.rc_kv_plan_create(shape, 0, ctypes.byref(rc.rc_kv_params_t(1, 0.0, 0, 0, 0)), None) == rc.RC_ERR_INVALID_ARG
    assert rc.rc_kv_workspace_bytes(None) == 0
    rc.rc_kv_plan_destroy(None)


def test_calls_refuse_bad_arguments_without_launching(rc):
    A, I, X = 4096, rc.RC_ERR_INVALID_ARG, rc.RC_ERR_ALIGNMENT
    cache = rc.rc_kv_cache_t(A, A, A, A, A, A)

    def view(data=A, dtype=rc.RC_BF16, b=4 * 64 * 4, t=64 * 4, h=64):
        return rc.rc_kv_view_t(data, dtype, b, t, h)

    def status(call, *args):
        try:
            call(*args)
        except rc.RcError as e:
            return e.status
        return rc.RC_OK
    with rc.KvPlan(**SMALL) as p, rc.KvPlan(**SMALL, q_tile=1, keep_blocks=2) as ps:
        h = p.handle
        for args, want in [
                ((None, 0, cache, None, A, None, 3, view(), view()), I),
                ((h, 0, rc.rc_kv_cache_t(A, 0, A, A, A, A), None, A, None, 3, view(), view()), I),
                ((h, 0, rc.rc_kv_cache_t(A, A + 8, A, A, A, A), None, A, None, 3, view(), view()), X),
                ((h, 0, cache, None, 0, None, 3, view(), view()), I),
                ((h, 0, cache, None, A + 2, None, 3, view(), view()), X),
                ((h, 0, cache, A + 1, A, None, 3, view(), view()), X),
                ((h, 0, cache, None, A, A + 2, 3, view(), view()), X),
                ((h, 0, cache, None, A, None, -1, view(), view()), I),
                ((h, 0, cache, None, A, None, 3, view(data=0), view()), I),
                ((h, 0, cache, None, A, None, 3, view(data=A + 8), view()), X),
                ((h, 0, cache, None, A, None, 3, view(dtype=5), view()), I),
                ((h, 0, cache, None, A, None, 3, view(), view(t=-8)), I),
                ((h, 0, cache, None, A, None, 3, view(), view(t=68)), X),
                ((h, 0, cache, None, A, None, 0, view(), view()), rc.RC_OK)]:
            assert status(rc.rc_kv_store, *args) == want, args
        for args, want in [
                ((h, 0, cache, None, A, 0, 5, view(), None, view(), None), I),          # over max_queries
                ((h, 0, cache, None, A, 0, -1, view(), None, view(), None), I),
                ((h, 0, cache, None, A, -1, 2, view(), None, view(), None), I),
                ((h, 0, cache, None, 0, 0, 2, view(), None, view(), None), I),
                ((h, 0, cache, None, A, 0, 2, view(dtype=rc.RC_F32), None, view(), None), I),
                ((h, 0, cache, None, A, 0, 2, view(), None, view(dtype=rc.RC_F32), None), I),
                ((h, 0, cache, None, A, 0, 2, view(), None, view(t=8), None), I),       # outputs that overlap
                ((h, 0, cache, None, A, 0, 2, view(), A, view(), None), I),             # a plan without q_tile
                ((h, 0, cache, None, A, 0, 2, view(), None, view(), A + 2), X),
                ((ps.handle, 0, cache, None, A, 0, 2, view(), A + 2, view(), None), X),
                ((h, 0, cache, None, A, 0, 0, view(), None, view(), None), rc.RC_OK)]:
            assert status(rc.rc_kv_attend, *args) == want, args
        for args, want in [
                ((h, 0, cache, None, A, 0, 2, view(), A), I),                           # a plan without q_tile
                ((ps.handle, 0, cache, None, A, 0, 2, view(), 0), I),
                ((ps.handle, 0, cache, None, A, 0, 2, view(), A + 2), X),
                ((ps.handle, 0, cache, None, A, 0, 5, view(), A), I),
                ((ps.handle, 0, cache, None, A, 0, 0, view(), A), rc.RC_OK)]:
            assert status(rc.rc_kv_select, *args) == want, args


def test_binding_refuses_host_tensors_and_wrong_shapes(rc):
    with pytest.raises(ValueError, match="device tensor"):
        rc.KvCache(torch.zeros(2, 2, 4, 64, 16, dtype=torch.uint8), torch.zeros(2, 2, 4, 64, 16, dtype=torch.uint8),
                   torch.ones(2, 2), torch.ones(2, 2), torch.zeros(2, 2, 64, dtype=torch.int8), torch.ones(2, 2))
    with pytest.raises(ValueError, match="a cache of this k has"):
        rc.KvCache(torch.zeros(2, 2, 4, 64, 16, dtype=torch.uint8), torch.zeros(2, 2, 4, 128, 16, dtype=torch.uint8),
                   torch.ones(2, 2), torch.ones(2, 2), torch.zeros(2, 2, 64, dtype=torch.int8), torch.ones(2, 2))
    with rc.KvPlan(**SMALL) as p:
        with pytest.raises(ValueError, match="device tensor"):
            p._rows(torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16), 4, "q")


def test_oracle_rounds_e4m3_to_nearest_even():
    # against torch's conversion of every midpoint between neighbours, the neighbours and values around them
    v = ko.TABLE[:127]
    mid = (v[1:] + v[:-1]) / 2
    x = np.concatenate([v, mid, np.nextafter(mid, 0), np.nextafter(mid, 500), [1e-9, 448.0]])
    x = np.concatenate([x, -x]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ko.e4m3_encode(x.astype(np.float64)) & 127, want & 127)
