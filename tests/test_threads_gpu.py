"""Calls of one kernel with different tiles, and so different shared memory, from several host threads at once."""
import threading

import pytest
import torch

import kronecker_sparse_matrix_b200 as ks

pytestmark = pytest.mark.gpu
DEV = "cuda"


def run_together(calls, times):
    """Each call on a thread and a stream of its own, its results equal to those alone."""
    want = [call() for call in calls]
    torch.cuda.synchronize()
    bad, start = [], threading.Barrier(len(calls))

    def work(call, w):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                for _ in range(times):
                    y = call()
                torch.cuda.current_stream().synchronize()
                if not torch.equal(y, w):
                    bad.append("differs")
        except Exception as e:  # noqa: BLE001 (reported below)
            bad.append(repr(e))

    threads = [threading.Thread(target=work, args=a) for a in zip(calls, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    ks.sync_status()
    assert not bad, bad[:3]


def of(p, n, dtype):
    a, b, c, d = p
    g = torch.Generator(device=DEV).manual_seed(n)
    return (torch.randn(n, a * c * d, generator=g, device=DEV).to(dtype),
            torch.randn(a, d, b, c, generator=g, device=DEV).to(dtype), torch.randn(n, a * b * d, generator=g, device=DEV).to(dtype))


def test_tensor_core_products():
    ps = [(1, 256, 64, 16), (1, 48, 64, 16), (1, 16, 32, 16), (2, 96, 48, 32)]
    data = [of(p, 300, torch.bfloat16) for p in ps]
    run_together([lambda p=p, q=q: ks.matmul(q[0], q[1], p) for p, q in zip(ps, data)], 400)


def test_tensor_core_value_gradients():
    ps = [(1, 256, 64, 16), (1, 128, 16, 16), (1, 256, 32, 16), (2, 128, 48, 8)]
    data = [of(p, 300, torch.bfloat16) for p in ps]
    run_together([lambda p=p, q=q: ks.matmul_dv(q[2], q[0], p) for p, q in zip(ps, data)], 400)


def test_factorizations():
    mats = [torch.randn(n, n, generator=torch.Generator().manual_seed(n)).to(DEV) for n in (16, 64, 256)]
    run_together([lambda m=m: torch.cat([f.view(-1) for f in ks.butterfly_factorize(m)[0]]) for m in mats], 40)
