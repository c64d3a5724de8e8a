"""Failure paths of the adapter calls without a GPU fault: injected allocation
failures leave outputs as they were, injected timeouts of the tensor-core
pipeline are reported and the next call is right; calls from two host threads.
"""
import threading

import pytest
import torch

import kronecker_sparse_matrix_b200 as ks
from tests.test_adapter_gpu import DEV, assert_backward, assert_forward, call, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("p,dtype,n", [((1, 64, 48, 8), torch.bfloat16, 500), ((3, 20, 12, 5), torch.float32, 500),
                                       ((1, 192, 48, 8), torch.float32, 7300), ((3, 20, 12, 5), torch.bfloat16, 500)])
def test_injected_allocation_failure(monkeypatch, p, dtype, n):
    q = make(p, n, 3, 8, dtype, "segments", 1)
    args = (q["values"], p, q["A"], q["B"], q["ids"], q["scales"])
    out = torch.full((n, p[0] * p[1] * p[3]), 7.0, dtype=dtype, device=DEV)
    monkeypatch.setenv("KS_FAULT_INJECT", "alloc")
    for fn in (lambda: ks.adapter_matmul(q["x"], *args, out=out), lambda: ks.adapter_backward(q["dy"], q["x"], *args)):
        with pytest.raises(ks.KsError) as err:
            fn()
        assert err.value.status == 4 and "workspace" in str(err.value)
    ks.sync_status()
    assert (out == 7.0).all()
    monkeypatch.delenv("KS_FAULT_INJECT")
    assert_forward(call(q, p), q, p)
    assert_backward(q, p)


@pytest.mark.parametrize("p", [(1, 64, 48, 8), (2, 64, 64, 1), (2, 64, 32, 2), (1, 64, 64, 64)])
def test_injected_timeout_is_reported(monkeypatch, p):
    q = make(p, 1500, 3, 24, torch.bfloat16, "segments", 2, bias=True)
    monkeypatch.setenv("KS_FAULT_INJECT", "timeout")
    ks.adapter_matmul(q["x"], q["values"], p, q["A"], q["B"], q["ids"], q["scales"], bias=q["bias"])
    with pytest.raises(ks.KsError) as err:
        ks.sync_status()
    assert err.value.status == 6
    monkeypatch.delenv("KS_FAULT_INJECT")
    ks.sync_status()
    assert_forward(call(q, p), q, p)
    assert_backward(q, p)


def test_two_host_threads():
    p = (1, 256, 64, 16)
    qs = [make(p, n, 4, 16, torch.bfloat16, "segments", n) for n in (700, 900)]
    want = [(call(q, p), ks.adapter_backward(q["dy"], q["x"], q["values"], p, q["A"], q["B"], q["ids"], q["scales"]))
            for q in qs]
    torch.cuda.synchronize()
    bad = []

    def work(q, w):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(30):
                y = ks.adapter_matmul(q["x"], q["values"], p, q["A"], q["B"], q["ids"], q["scales"])
                g = ks.adapter_backward(q["dy"], q["x"], q["values"], p, q["A"], q["B"], q["ids"], q["scales"])
                torch.cuda.current_stream().synchronize()
                if not torch.equal(y, w[0]) or not all(torch.equal(u, v) for u, v in zip(g, w[1])):
                    bad.append(1)

    threads = [threading.Thread(target=work, args=a) for a in zip(qs, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    ks.sync_status()
    assert not bad
