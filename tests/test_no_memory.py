"""A plan for which there is no device memory is refused, and that is all: the runtime's own error of it does not stay
behind, where the caller's next launch would report it. Without a GPU, in a child process in which device memory is
refused and the runtime's last error kept as it keeps it."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STAND_IN = """
static int last;
int failures;
int hipMalloc(void** p, unsigned long n) { ++failures; return last = 2; }
int hipGetLastError(void) { const int e = last; last = 0; return e; }
int hipGetDevice(int* d) { *d = 0; return 0; }
"""


def refuse(kind):
    import ctypes
    from activation_residual_compression_amd import librescomp as rc
    make = {"attention": lambda: rc.AttnPlan(8, 2, 64, max_seqs=1, max_queries=1, max_keys=100000),
            "pages": lambda: rc.PagePlan(3, 2, 64, 8, 4),
            "cache": lambda: rc.KvPlan(batch=1, q_heads=2, kv_heads=2, head_dim=64, pool_blocks=900, seq_blocks=900, max_queries=1),
            "lowrank": lambda: rc.Plan((2, 256, 256), "f32", "lr", rank=32, iters=2),
            "blocksel": lambda: rc.Plan((1, 256, 256), "f32", "bs", grid_w=16, keep_blocks=1),
            "finite": lambda: rc.Plan((1, 256, 256), "f32", "q2", group=128, flags=rc.RC_CHECK_FINITE)}[kind]
    this = ctypes.CDLL(None)
    with pytest.raises(rc.RcError) as e:
        make()
    assert e.value.status == rc.RC_ERR_HIP and ctypes.c_int.in_dll(this, "failures").value == 1
    assert this.hipGetLastError() == 0
    print("refused")


@pytest.mark.parametrize("kind", ["attention", "pages", "cache", "lowrank", "blocksel", "finite"])
def test_a_refused_plan_leaves_no_error_behind(kind, tmp_path):
    src, lib = tmp_path / "stand_in.c", tmp_path / "stand_in.so"
    src.write_text(STAND_IN)
    subprocess.run(["gcc", "-shared", "-fPIC", str(src), "-o", str(lib)], check=True)
    r = subprocess.run([sys.executable, "-c", "import sys; sys.path[:0] = ['tests', '.']; import test_no_memory as t; t.refuse(%r)" % kind],
                       cwd=ROOT, env=dict(os.environ, LD_PRELOAD=str(lib)), capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "refused" in r.stdout, r.stdout + r.stderr
