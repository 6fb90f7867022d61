"""Layer norm's gradients at the lengths whose shared memory lies about the limit that a kernel has without being
given more: 48 KB of what is fixed and what a launch asks for together."""

import os
import subprocess
import sys
import textwrap

import pytest

import __graft_entry__

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# A kernel that has been given more keeps it for the process, so the lengths of one case are asked for from a new
# process in rising order, none of which needs more than the next.
CHILD = textwrap.dedent("""
    import sys
    sys.path[:0] = sys.argv[1:3]
    import torch
    import mx_microscaling_quantize_gb300 as mxq
    import train_ref as T
    from test_gpu_train import BF16, FP32, either, params, rows
    from test_gpu_train_edges import off_base
    for K in map(int, sys.argv[4:]):
        for M in (5, 400):
            x, dy = rows(M * K, M, K, BF16), rows(M * K + 7, M, K, BF16, 0.0)
            w, _ = params(K, K, FP32)
            if sys.argv[3] == "unaligned":
                w = off_base(w, 4)  # 16 bytes past a multiple of 32
            _, mean, rstd = mxq.mx_layer_norm(x, w, None, stats=True)
            dx, dw, db = mxq.mx_layer_norm_backward(dy, x, mean, rstd, w)
            want = T.norm_backward(T.f64(dy), T.f64(x), either(mean), T.f64(rstd), T.f64(w), True)
            T.check_values(dx, want[0], want[3], BF16, (M, K, "dx"))
            T.check_values(dw, want[1], want[4], FP32, (M, K, "dw"))
            T.check_values(db, want[2], want[5], FP32, (M, K, "db"))
    assert mxq.mx_device_errors() == 0
    print("done")
""")


# 383 columns: 16 groups of 8 x 383 bytes are 128 below 48 KB, and so on for 8, 5, 2 and 1
# groups; 8191 and 8192 need more than 48 KB alone.
@pytest.mark.parametrize("base,lengths", [
    ("aligned", [382, 383, 765, 767, 1223, 1225, 1227, 3063, 6113, 6143]), ("aligned", [767]), ("aligned", [6143, 8191]),
    ("unaligned", [384, 768, 1224, 3064, 6120, 6144]), ("unaligned", [768]), ("unaligned", [384, 8192, 768]),
])
def test_gradients_of_the_first_call_of_a_process(base, lengths):
    __graft_entry__.build()
    run = subprocess.run([sys.executable, "-c", CHILD, ROOT, os.path.join(ROOT, "tests"), base, *map(str, lengths)],
                         capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert run.returncode == 0 and run.stdout.split()[-1] == "done", run.stderr[-2000:]
