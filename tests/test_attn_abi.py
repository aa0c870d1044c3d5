"""Attention over packed sequences and the join without a GPU: exports, refusals of plans and
of arguments (nothing is launched), and the dense reference's own masks."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import attn_dense as ad

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 4096  # an aligned address; nothing reads it


@pytest.fixture(scope="module")
def rc():
    from activation_residual_compression_amd import librescomp
    return librescomp


# short sequences: never split, so no workspace and no device needed
SMALL = dict(q_heads=4, kv_heads=2, head_dim=64, max_seqs=3, max_queries=10, max_keys=100)


def status(rc, call, *args):
    try:
        call(*args)
    except rc.RcError as e:
        return e.status
    return rc.RC_OK


def test_exports_every_declared_function(rc):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "librescomp_attn.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(rc_attn_[a-z0-9_]+)\s*\(", text))
    assert names == {"rc_attn_plan_create", "rc_attn_plan_destroy", "rc_attn_packed", "rc_attn_join",
                     "rc_attn_workspace_bytes"}
    lib = ctypes.CDLL(rc.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n
    assert re.search(r"#define RC_ATTN_MAX_PARTS (\d+)", text).group(1) == str(rc.RC_ATTN_MAX_PARTS)


@pytest.mark.parametrize("header", ["librescomp_attn.h", "librescomp_pages.h"])
def test_headers_are_c(header, tmp_path):
    src = tmp_path / "x.c"
    src.write_text('#include "%s"\nint main(void) { return 0; }\n' % header)
    subprocess.run(["gcc", "-std=c99", "-fsyntax-only", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__",
                    "-I", os.path.join(ROOT, "include"), "-I", "/opt/rocm/include", str(src)], check=True)


@pytest.mark.parametrize("bad,want", [
    (dict(q_heads=0), "RC_ERR_INVALID_ARG"), (dict(kv_heads=0), "RC_ERR_INVALID_ARG"),
    (dict(kv_heads=3), "RC_ERR_INVALID_ARG"), (dict(head_dim=0), "RC_ERR_INVALID_ARG"),
    (dict(head_dim=96), "RC_ERR_UNSUPPORTED"), (dict(head_dim=256), "RC_ERR_UNSUPPORTED"),
    (dict(max_seqs=0), "RC_ERR_INVALID_ARG"), (dict(max_seqs=65536), "RC_ERR_UNSUPPORTED"),
    (dict(max_queries=0), "RC_ERR_INVALID_ARG"), (dict(max_keys=0), "RC_ERR_INVALID_ARG"),
    (dict(max_queries=1 << 28), "RC_ERR_UNSUPPORTED"), (dict(max_keys=(1 << 30) + 1), "RC_ERR_UNSUPPORTED"),
    (dict(q_heads=65536, kv_heads=32768, max_queries=1), "RC_ERR_UNSUPPORTED"),
    (dict(scale=-1.0), "RC_ERR_INVALID_ARG"), (dict(scale=float("nan")), "RC_ERR_INVALID_ARG"),
    (dict(scale=float("inf")), "RC_ERR_INVALID_ARG"), (dict(dtype=7), "RC_ERR_INVALID_ARG")])
def test_plan_refusals(rc, bad, want):
    with pytest.raises(rc.RcError) as e:
        rc.AttnPlan(**{**SMALL, **bad})
    assert e.value.status == getattr(rc, want)


def test_plan_refuses_unknown_flag_and_null(rc):
    shape = rc.rc_attn_shape_t(1, 1, 64, 1, 1, 1)
    assert status(rc, rc.rc_attn_plan_create, shape, "bf16", rc.rc_attn_params_t(0.0, 2)) == rc.RC_ERR_INVALID_ARG
    assert rc._lib.rc_attn_plan_create(shape, 0, None, ctypes.byref(ctypes.c_void_p())) == rc.RC_ERR_INVALID_ARG
    assert rc._lib.rc_attn_plan_create(shape, 0, ctypes.byref(rc.rc_attn_params_t(0.0, 0)), None) == rc.RC_ERR_INVALID_ARG
    assert rc.rc_attn_workspace_bytes(None) == 0
    rc.rc_attn_plan_destroy(None)


def test_call_refuses_bad_arguments_without_launching(rc):
    I, X, OK = rc.RC_ERR_INVALID_ARG, rc.RC_ERR_ALIGNMENT, rc.RC_OK

    def view(data=A, dtype=rc.RC_BF16, t=4 * 64, h=64):
        return rc.rc_kv_view_t(data, dtype, 0, t, h)
    good = dict(seqs=2, qo=A, ko=A, nq=7, nk=9, mq=0, mk=0, q=view(), k=view(), v=view(), out=view(), lse=A)

    def call(plan, **kw):
        x = {**good, **kw}
        return status(rc, rc.rc_attn_packed, plan, 0, x["seqs"], x["qo"], x["ko"], x["nq"], x["nk"], x["mq"], x["mk"],
                      x["q"], x["k"], x["v"], x["out"], x["lse"])
    with rc.AttnPlan(**SMALL) as p:
        assert call(None) == I
        for kw, want in [
                (dict(qo=0), I), (dict(qo=A + 2), X), (dict(ko=A + 1), X), (dict(lse=A + 2), X),
                (dict(seqs=-1), I), (dict(seqs=4), I), (dict(nq=-1), I), (dict(nq=11), I), (dict(nk=-1), I),
                (dict(nk=101), I), (dict(mq=-1), I), (dict(mk=-1), I),
                (dict(q=view(data=0)), I), (dict(k=view(data=0)), I), (dict(v=view(data=0)), I), (dict(out=view(data=0)), I),
                (dict(q=view(data=A + 8)), X), (dict(k=view(t=-8)), I), (dict(v=view(h=68)), X), (dict(k=view(t=260)), X),
                (dict(q=view(dtype=rc.RC_F32)), I), (dict(k=view(dtype=rc.RC_F32)), I), (dict(v=view(dtype=5)), I),
                (dict(out=view(dtype=rc.RC_F32)), I),
                (dict(out=view(t=8)), I), (dict(out=view(t=0)), I), (dict(out=view(t=64, h=64)), I),   # overlapping rows
                (dict(k=view(t=1 << 40)), I),
                (dict(seqs=0), OK), (dict(nq=0, q=view(data=0), out=view(data=0)), OK)]:
            assert call(p.handle, **kw) == want, kw


def test_join_refuses_bad_arguments_without_launching(rc):
    I, X, U, OK = rc.RC_ERR_INVALID_ARG, rc.RC_ERR_ALIGNMENT, rc.RC_ERR_UNSUPPORTED, rc.RC_OK

    def view(data=A, dtype=rc.RC_BF16, b=7 * 4 * 64, t=4 * 64, h=64):
        return rc.rc_kv_view_t(data, dtype, b, t, h)
    good = dict(outs=[view(), view()], lses=[A, A], batch=2, tokens=7, heads=4, dim=64, out=view(), lse=A)

    def call(**kw):
        x = {**good, **kw}
        return status(rc, rc.rc_attn_join, 0, x["outs"], x["lses"], x["batch"], x["tokens"], x["heads"], x["dim"], x["out"],
                      x["lse"])
    for kw, want in [
            (dict(outs=[], lses=[]), I), (dict(outs=[view()] * 9, lses=[A] * 9), I),
            (dict(outs=[view(), view(dtype=rc.RC_F32)]), I), (dict(outs=[view(), view(data=0)]), I),
            (dict(lses=[A, 0]), I), (dict(lses=[A, A + 2]), X), (dict(lse=A + 1), X),
            (dict(batch=-1), I), (dict(tokens=-1), I), (dict(heads=-1), I), (dict(dim=0), I), (dict(dim=96), U),
            (dict(outs=[view(data=A + 8), view()]), X), (dict(out=view(data=A + 8)), X), (dict(out=view(dtype=9)), I),
            (dict(out=view(t=0)), I), (dict(out=view(b=64)), I), (dict(outs=[view(t=66), view()]), X),
            (dict(heads=(1 << 20) + 1, batch=1, tokens=1), U),
            (dict(batch=0), OK), (dict(tokens=0, outs=[view(data=0)] * 2, lses=[0, 0], out=view(data=0)), OK)]:
        assert call(**kw) == want, kw
    with pytest.raises(ValueError):
        rc.rc_attn_join(0, [view()], [A, A], 1, 1, 1, 64, view(), None)


def test_binding_refuses_host_tensors(rc):
    x = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    with rc.AttnPlan(**SMALL) as p:
        with pytest.raises(ValueError, match="device tensor"):
            p.attend(x, x[:, :2], x[:, :2], torch.tensor([0, 3], dtype=torch.int32), x)
    with pytest.raises(ValueError, match="device tensor"):
        rc.join_attention([x, x], [torch.zeros(3, 4)] * 2, x)
    with pytest.raises(ValueError, match="log-sum-exps"):
        rc.join_attention([x, x], [torch.zeros(3, 4)], x)


def test_dense_reference_against_rows_one_by_one():
    rng = np.random.default_rng(0)
    q, k, v = (rng.standard_normal(s) for s in ((5, 4, 64), (3, 2, 64), (3, 2, 64)))
    v[2, 0, 7] = np.inf
    out, lse, *_, strange = ad.attend(q, k, v, True, 0.125)
    assert np.isneginf(lse[:2]).all() and (out[:2] == 0).all()     # two more queries than keys
    for i in range(2, 5):
        for h in range(4):
            n = i - 1
            s = k[:n, h // 2] @ q[i, h] * 0.125
            e = np.exp(s)
            assert abs(lse[i, h] - np.log(e.sum())) < 1e-12
            assert np.abs(out[i, h, :7] - (e / e.sum()) @ v[:n, h // 2, :7]).max() < 1e-12
    assert strange.sum() == 2 and strange[4, :2, 7].all()
