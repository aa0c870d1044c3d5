"""Pages of the cache without a GPU: exports, refusals of plans and of arguments (nothing is
launched), and the oracle's own state. A plan needs device memory; the calls are refused by the
library's own checks in a child process where device memory comes from the host's."""
import ctypes
import os
import re
import subprocess
import sys

import numpy as np
import pytest
import torch

import pages_oracle as po

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 4096  # an aligned address; nothing reads it
SMALL = dict(slots=3, kv_heads=2, head_dim=64, pool_blocks=8, seq_blocks=4)
STAND_IN = """
#include <stdlib.h>
#include <string.h>
int hipMalloc(void** p, size_t n) { *p = malloc(n); return *p ? 0 : 2; }
int hipFree(void* p) { free(p); return 0; }
int hipMemset(void* p, int v, size_t n) { memset(p, v, n); return 0; }
int hipMemsetD32(void* p, int v, size_t n) { for (size_t i = 0; i < n; ++i) ((int*)p)[i] = v; return 0; }
int hipStreamSynchronize(void* s) { return 0; }
"""


@pytest.fixture(scope="module")
def rc():
    from activation_residual_compression_amd import librescomp
    return librescomp


def test_exports_every_declared_function(rc):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "librescomp_pages.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(rc_pages_[a-z0-9_]+)\s*\(", text))
    assert names == {"rc_pages_plan_create", "rc_pages_plan_destroy", "rc_pages_reserve", "rc_pages_fork",
                     "rc_pages_free", "rc_pages_compact", "rc_pages_copy", "rc_pages_workspace_bytes"}
    lib = ctypes.CDLL(rc.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n


@pytest.mark.parametrize("bad,want", [
    (dict(slots=0), "RC_ERR_INVALID_ARG"), (dict(kv_heads=0), "RC_ERR_INVALID_ARG"),
    (dict(head_dim=-64), "RC_ERR_INVALID_ARG"), (dict(head_dim=96), "RC_ERR_UNSUPPORTED"),
    (dict(pool_blocks=0), "RC_ERR_INVALID_ARG"), (dict(seq_blocks=0), "RC_ERR_INVALID_ARG"),
    (dict(slots=65536), "RC_ERR_UNSUPPORTED"), (dict(kv_heads=32768), "RC_ERR_UNSUPPORTED"),
    (dict(seq_blocks=8193), "RC_ERR_UNSUPPORTED"), (dict(pool_blocks=(1 << 28) + 1), "RC_ERR_UNSUPPORTED")])
def test_plan_refusals(rc, bad, want):
    with pytest.raises(rc.RcError) as e:
        rc.PagePlan(**{**SMALL, **bad})
    assert e.value.status == getattr(rc, want)
    assert rc._lib.rc_pages_plan_create(rc.rc_pages_shape_t(1, 1, 64, 1, 1), None) == rc.RC_ERR_INVALID_ARG
    assert rc.rc_pages_workspace_bytes(None) == 0
    rc.rc_pages_plan_destroy(None)


def refuse_calls():
    from activation_residual_compression_amd import librescomp as rc
    I, X = rc.RC_ERR_INVALID_ARG, rc.RC_ERR_ALIGNMENT
    cache, hole, off = rc.rc_kv_cache_t(A, A, A, A, A, A), rc.rc_kv_cache_t(A, 0, A, A, A, A), rc.rc_kv_cache_t(A, A, A, A + 4, A, A)

    def status(call, *args):
        try:
            call(*args)
        except rc.RcError as e:
            return e.status
        return rc.RC_OK
    plan = rc.PagePlan(**SMALL)
    assert plan.workspace_bytes > 0
    h = plan.handle
    for call, good, optional in (
            (rc.rc_pages_reserve, (h, 0, cache, A, A, A, A, None), (7,)),
            (rc.rc_pages_fork, (h, 0, A, A, A, A), ()),
            (rc.rc_pages_free, (h, 0, A, A, A), ()),
            (rc.rc_pages_compact, (h, 0, cache, A, A, None, None), (5, 6)),
            (rc.rc_pages_copy, (h, 0, cache, cache, A, A, 2), ())):
        for i, x in enumerate(good):
            def with_(y):
                return good[:i] + (y,) + good[i + 1:]
            if i == 0:
                assert status(call, *with_(None)) == I
            elif x is cache:
                assert status(call, *with_(hole)) == I
                assert status(call, *with_(off)) == X
            elif x == A or i in optional:
                assert i in optional or status(call, *with_(0)) == I, (call, i)
                assert status(call, *with_(A + 2)) == X, (call, i)
    assert status(rc.rc_pages_copy, h, 0, cache, cache, A, A, -1) == I
    assert status(rc.rc_pages_copy, h, 0, cache, cache, 0, 0, 0) == rc.RC_OK
    with pytest.raises(ValueError, match="device tensor"):
        plan.free(*plan.empty("cpu"), torch.zeros(3, dtype=torch.int32))
    plan.close()
    print("calls refused")


def test_calls_refuse_bad_arguments_without_launching(tmp_path):
    src, lib = tmp_path / "stand_in.c", tmp_path / "stand_in.so"
    src.write_text(STAND_IN)
    subprocess.run(["gcc", "-shared", "-fPIC", str(src), "-o", str(lib)], check=True)
    r = subprocess.run([sys.executable, "-c", "import sys; sys.path[:0] = ['tests', '.']; import test_pages_abi as t; t.refuse_calls()"],
                       cwd=ROOT, env=dict(os.environ, LD_PRELOAD=str(lib)), capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "calls refused" in r.stdout, r.stdout + r.stderr


def test_oracle_keeps_counts():
    rng = np.random.default_rng(0)
    o = po.Pages(6, 40, 8)
    lengths = np.zeros(6, int)
    for step in range(200):
        kind = rng.integers(4)
        if kind < 2:
            more = rng.integers(0, 100, 6) * (rng.random(6) < 0.5)
            if o.reserve(lengths, more) == 0:
                lengths = np.minimum(lengths + more, 8 * 64)
        elif kind == 2:
            source = np.where(rng.random(6) < 0.4, rng.integers(0, 6, 6), -1)
            new = np.where(source >= 0, (lengths[source] * rng.random(6)).astype(int), lengths)
            o.fork(source, new)
            lengths = new
        else:
            lengths = (lengths * rng.random(6)).astype(int)
            o.free(lengths)
            n, _ = o.compact()
            assert (o.refs[:n] > 0).all() and (o.refs[n:] == 0).all()
        assert np.array_equal(po.counts(o.table, 40), o.refs)
        assert all((o.table[s, :po.blocks_of(lengths[s])] >= 0).all() for s in range(6))
