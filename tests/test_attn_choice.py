"""The host's choice for a call of attention over packed sequences, without a GPU: the plan's own code, compiled for the
CPU (attn_choice.cpp), says how many blocks of threads a call gets. They have to be those that the kernels' numbering
gives rows and parts to, and what they write has to fit the workspace, also where the plan is for larger calls."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from activation_residual_compression_amd import librescomp as rc

HERE = os.path.dirname(os.path.abspath(__file__))
A = 1 << 20    # an aligned address; nothing reads it
GROUPS = 1536  # counters of the kernel for few rows


class Launch(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("kind", "grid", "waves", "u", "kg", "splits", "chunk", "direct", "part_end",
                                              "ml_end", "halves_end", "arrived")]


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("choice") / "attn_choice.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-D__HIP_PLATFORM_AMD__", "-I",
                    "/opt/rocm/include", os.path.join(HERE, "attn_choice.cpp"), "-o", out], check=True)
    lib = ctypes.CDLL(out)
    vp, i = ctypes.c_void_p, ctypes.c_int
    lib.rc_attn_plan_create.argtypes = [rc.rc_attn_shape_t, i, ctypes.POINTER(rc.rc_attn_params_t), ctypes.POINTER(vp)]
    lib.rc_attn_packed.argtypes = [vp, vp, i, vp, vp, i, i, i, i, vp, vp, vp, vp, vp]
    lib.rc_attn_join.argtypes = [vp, i, vp, ctypes.POINTER(vp), i, i, i, i, vp, vp]
    lib.rc_attn_plan_destroy.argtypes = [vp]
    lib.rc_attn_workspace_bytes.argtypes, lib.rc_attn_workspace_bytes.restype = [vp], ctypes.c_size_t
    lib.choice.restype = ctypes.POINTER(Launch)
    return lib


class Plan:
    def __init__(self, lib, q_heads, kv_heads, dim, seqs, queries, keys, f32=False, causal=False):
        self.lib, self.heads, self.f32, self.causal = lib, (q_heads, kv_heads, dim), f32, causal
        self.handle = ctypes.c_void_p()
        status = lib.rc_attn_plan_create(rc.rc_attn_shape_t(q_heads, kv_heads, dim, seqs, queries, keys),
                                         rc.RC_F32 if f32 else rc.RC_BF16,
                                         ctypes.byref(rc.rc_attn_params_t(0.0, rc.RC_ATTN_CAUSAL if causal else 0)),
                                         ctypes.byref(self.handle))
        assert status == rc.RC_OK
        self.bytes = lib.rc_attn_workspace_bytes(self.handle)

    def call(self, seqs, q_tokens, kv_tokens, max_q=0, max_kv=0):
        """(status, what was launched)."""
        qh, kh, d = self.heads
        dtype = rc.RC_F32 if self.f32 else rc.RC_BF16
        q, k = (ctypes.byref(rc.rc_kv_view_t(A, dtype, 0, h * d, d)) for h in (qh, kh))
        self.lib.choice().contents.kind = 0
        status = self.lib.rc_attn_packed(self.handle, None, seqs, A, A, q_tokens, kv_tokens, max_q, max_kv, q, k, k, q, None)
        return status, Launch.from_buffer_copy(self.lib.choice().contents)

    def close(self):
        self.lib.rc_attn_plan_destroy(self.handle)


def parts_of(keys, chunk, most):
    return np.clip(-(-keys // chunk), 1, most)


def check_call(plan, lq, lk, max_q=0, max_kv=0):
    """Every group of rows of the sequences and every part of its keys gets one block of threads. Returns whether keys
    were read in parts."""
    qh, kh, _ = plan.heads
    g = qh // kh
    lq, lk = np.array(lq), np.array(lk)
    seqs, nq, nk = len(lq), int(lq.sum()), int(lk.sum())
    status, w = plan.call(seqs, nq, nk, max_q, max_kv)
    what = (plan.heads, plan.f32, plan.causal, lq[:9], lk[:9], max_q, max_kv, {n: getattr(w, n) for n, _ in w._fields_})
    assert status == rc.RC_OK and w.kind == (1 if w.kind == 1 else 3 if plan.f32 else 2), what
    top_q, top_k = min(max_q or nq, nq), min(max_kv or nk, nk)
    assert w.part_end <= w.ml_end <= plan.bytes and w.halves_end <= plan.bytes, what
    if w.kind == 1:
        groups, most = -(-top_q * g // 16), -(-lq * g // 16)       # as all sequences may have, as each has
        counted = parts_of(lk, w.chunk, w.splits)
        if w.splits > 1:
            assert seqs * kh * groups <= GROUPS and w.waves == 4 and w.chunk % 64 == 0, what
            assert w.ml_end <= w.arrived and w.arrived + 4 * GROUPS <= plan.bytes, what
        if seqs == 1 or w.direct:
            piece = np.arange(w.grid)
            b, at = (0 * piece, piece) if seqs == 1 else (piece // groups, piece % groups)
            group, part = at // w.splits, at % w.splits
            assert w.splits == 1 or seqs == 1, what
            for s in range(seqs):
                for i in range(int(most[s])):
                    last = min(16 * i + 15, int(lq[s]) * g - 1) // g                        # the group's last query
                    seen = max(0, int(lk[s] - lq[s]) + last + 1) if plan.causal else int(lk[s])
                    have = np.sort(part[(b == s) & (group == i)])
                    want = np.arange(int(parts_of(np.array(seen), w.chunk, w.splits)))
                    assert np.array_equal(have[:len(want)], want), (what, "group", i, "of sequence", s, have, want)
        else:                                                      # pieces without gaps, in order
            assert (most * counted).sum() <= w.grid, what
    else:
        rows, per = 128 * w.u, w.grid // w.splits
        tiles = -(-lq * g // rows)
        assert w.grid % w.splits == 0 and per % kh == 0 and w.splits <= 16, what
        if w.direct:
            assert tiles.max() <= w.direct and per // kh >= w.direct * seqs, what
        else:
            assert tiles.sum() * kh <= per, what
        # a tile's parts are the longest's at most: ceil(tiles of 64 keys / chunk)
        assert w.splits == 1 or -(-(-(-top_k // 64)) // w.chunk) <= w.splits, what
    return w.splits > 1


HEADS = [(32, 8, 128), (24, 24, 128), (40, 8, 128), (64, 8, 64), (16, 4, 128), (16, 2, 64), (30, 30, 64), (12, 12, 64),
         (5, 1, 64), (20, 1, 128)]


# heads, the plan's queries and keys, the call's: the workspace limits the parts
@pytest.mark.parametrize("f32,heads,most,call", [
    (False, (32, 8, 128), (5, 8192), (5, 7168)), (False, (32, 8, 128), (16, 4000), (14, 3744)),
    (False, (24, 24, 128), (24, 2750), (22, 2494)), (False, (16, 2, 64), (16, 8250), (13, 8250)),
    (True, (12, 12, 64), (24, 5500), (21, 5244)), (False, (5, 1, 64), (13, 65536), (12, 65536))])
def test_every_part_of_one_sequence_has_a_block(lib, f32, heads, most, call):
    for causal in (False, True):
        plan = Plan(lib, *heads, 1, *most, f32, causal)
        assert check_call(plan, [call[0]], [call[1]])
        plan.close()


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("causal", [False, True])
def test_every_part_has_a_block_in_plans_larger_than_the_call(lib, f32, causal):
    rng = np.random.default_rng(2 * f32 + causal)

    def log(lo, hi):
        return int(round(np.exp(rng.uniform(np.log(lo), np.log(hi)))))
    split = 0
    for n in range(500):
        heads = HEADS[rng.integers(len(HEADS))]
        seqs = 1 if n % 2 else log(1, 80)
        queries, keys = max(log(1, 130), seqs), log(64, 70000)
        plan = Plan(lib, *heads, seqs, queries, keys, f32, causal)
        for _ in range(12):
            some = int(rng.integers(1, seqs + 1))
            lq = rng.multinomial(max(some, int(rng.integers(1, queries + 1))), np.ones(some) / some)
            lk = rng.multinomial(int(rng.integers(keys // 2, keys + 1)), rng.dirichlet(np.ones(some)))
            bounds = (int(lq.max()), int(lk.max())) if rng.random() < 0.7 else (0, 0)
            split += check_call(plan, lq, lk, *bounds)
        plan.close()
    assert split > 1000


@pytest.mark.parametrize("f32", [False, True])
def test_calls_of_more_threads_than_a_launch_can_have_are_refused(lib, f32):
    """2^32 threads: nothing is launched, neither in parts. 255 key heads of as many sequences are fewer."""
    for heads, want in ((255, rc.RC_OK), (257, rc.RC_ERR_UNSUPPORTED)):
        plan = Plan(lib, heads, heads, 64, 65535, 65535, 70000, f32)
        for nq, nk, mq, mk in ((65535, 1000, 1, 1), (100, 1000, 100, 1000), (65535, 65535, 1, 1)):
            status, w = plan.call(65535, nq, nk, mq, mk)
            assert status == want and (w.kind != 0) == (want == rc.RC_OK), (heads, nq, nk)
        plan.close()


def test_join_refuses_more_rows_than_it_can_count(lib):
    """Also where the product of batch, tokens and heads passes 64 bits and is 0 or negative there."""
    def join(batch, tokens, heads):
        view = ctypes.byref(rc.rc_kv_view_t(A, rc.RC_BF16, 1 << 39, 64 * heads, 64))
        lib.choice().contents.kind = 0
        status = lib.rc_attn_join(None, 1, view, (ctypes.c_void_p * 1)(A), batch, tokens, heads, 64, view, A)
        return status, lib.choice().contents.kind
    assert join(1, 1 << 13, 1 << 20) == (rc.RC_OK, 4)
    assert join(0, 1 << 30, 1 << 20) == (rc.RC_OK, 0)
    for shape in ((2, 1 << 13, 1 << 20), (1, 1 << 14, 1 << 20), ((1 << 31) - 1, 1 << 29, 16)):
        assert join(*shape) == (rc.RC_ERR_UNSUPPORTED, 0), shape
    for shape in ((1 << 30, 1 << 30, 16), (1 << 30, 1 << 30, 1 << 20)):     # the batches would overlap too
        assert join(*shape) == (rc.RC_ERR_INVALID_ARG, 0), shape
