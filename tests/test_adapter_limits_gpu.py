"""The few-row adapter kernel at and above the default limit of shared memory, in a
process of its own and from several host threads."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import kronecker_sparse_matrix_b200 as ks
from tests.test_adapter_gpu import assert_forward, call, make

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# A block's dynamic shared memory is 48 KB exactly (148 SMs), the default limit with nothing
# left for what the kernel declares itself
AT_THE_LIMIT = [((2, 30, 64, 22), 49, 16), ((2, 30, 64, 22), 49, 14), ((4, 70, 160, 9), 17, 54)]


@pytest.mark.parametrize("p,n,r", AT_THE_LIMIT)
def test_a_first_call_at_the_limit(p, n, r):
    """In a fresh process: no larger call has raised the limit before."""
    code = ("import torch\nfrom tests.test_adapter_gpu import *\n"
            f"p = {p}\nq = make(p, {n}, 3, {r}, torch.float32, 'rows', 1, bias=True)\nassert_forward(call(q, p), q, p)\n")
    done = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


def test_threads_with_different_sizes():
    """Calls of one kernel with more and less shared memory at once."""
    cases = [((2, 30, c, 22), 49, 16) for c in (120, 64, 100, 72)]
    qs = [make(p, n, 3, r, torch.float32, "rows", 4) for p, n, r in cases]
    want = [call(q, p) for q, (p, _, _) in zip(qs, cases)]
    for q, y, (p, _, _) in zip(qs, want, cases):
        assert_forward(y, q, p)
    torch.cuda.synchronize()
    bad, start = [], threading.Barrier(len(cases))

    def work(q, p, w):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                for _ in range(400):
                    y = ks.adapter_matmul(q["x"], q["values"], p, q["A"], q["B"], q["ids"], q["scales"])
                torch.cuda.current_stream().synchronize()
                if not torch.equal(y, w):
                    bad.append("differs")
        except Exception as e:  # noqa: BLE001 (reported below)
            bad.append(repr(e))

    threads = [threading.Thread(target=work, args=(q, p, w)) for q, (p, _, _), w in zip(qs, cases, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    ks.sync_status()
    assert not bad, bad[:3]
