"""Device-side waits are bounded: a wait on a barrier nothing signals ends with
MOE_ERR_TIMEOUT in the workspace status word, and the context stays usable.
(No trap, no fault: the kernel gives up after its limit and returns.)"""
import numpy as np
import pytest
import torch

from gpu_util import need_gpu, lib_api

pytestmark = pytest.mark.gpu


def test_wait_times_out_and_context_survives():
    need_gpu()
    M = lib_api()
    from top_softmax_router_gb300 import _lib
    ws = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    M.diag_wait_timeout(50_000_000, ws)          # 50 ms
    assert M.check_status(ws) == _lib.MOE_ERR_TIMEOUT
    assert M.check_status(ws) == 0               # cleared by the first check
    x = torch.arange(1024, device="cuda", dtype=torch.float32)
    assert float((x * 2).sum()) == float(np.arange(1024).sum() * 2)


def test_bad_expert_id_is_reported_not_faulted():
    need_gpu()
    M = lib_api()
    from top_softmax_router_gb300 import _lib
    cfg = M.Config(N=64, H=64, E=4, k=2, I=64, c=64, K_max=1)
    K, c_eff = M.chunk_plan(cfg)
    ws = torch.zeros(max(M.workspace_bytes(cfg)), dtype=torch.uint8, device="cuda")
    idx = torch.zeros(64, 2, dtype=torch.int32, device="cuda")
    idx[:, 1] = 1
    idx[5, 1] = 9                                 # out of range: the plan kernel checks and reports
    rr = torch.empty(K, 2 * c_eff, dtype=torch.int32, device="cuda")
    ro = torch.empty(64, 2, dtype=torch.int32, device="cuda")
    off = torch.empty(K, 5, dtype=torch.int32, device="cuda")
    M.plan(cfg, idx, rr, ro, off, ws)
    assert M.check_status(ws) == _lib.MOE_ERR_DEVICE_CHECK


def test_a_norm_whose_waits_may_run_out_leaves_the_context_usable():
    """A wait limit far below a copy's time: the backward either ends as ever or reports the timeout, and the next call,
    under the usual limit, gives the usual bits."""
    need_gpu()
    M = lib_api()
    from top_softmax_router_gb300 import _lib
    x, dy = (torch.randn(3000, 7168, device="cuda").bfloat16() for _ in range(2))
    ln = M.LayerNorm(M.LayerNormConfig(N=3000, H=7168))
    _, mean, rstd = ln.forward(x)
    want = ln.backward(x, None, mean, rstd, dy)
    M.set_wait_limit_ns(1000)
    try:
        ln.backward(x, None, mean, rstd, dy)
        assert M.check_status(ln.ws) in (0, _lib.MOE_ERR_TIMEOUT)
    finally:
        M.set_wait_limit_ns(0)
    assert all(torch.equal(p, q) for p, q in zip(want, ln.backward(x, None, mean, rstd, dy)))
    ln.check()


def test_a_head_whose_waits_may_run_out_leaves_the_context_usable():
    """The same for the distillation head's products."""
    need_gpu()
    M = lib_api()
    from top_softmax_router_gb300 import _lib
    N, H, V, K = 520, 2112, 5000, 4
    X, W = torch.randn(N, H, device="cuda").bfloat16(), torch.randn(V, H, device="cuda").mul(H ** -0.5).bfloat16()
    ids = torch.randint(0, V, (N, K), device="cuda", dtype=torch.int32)
    t, g = torch.randn(N, K, device="cuda"), torch.full((N,), 1 / N, device="cuda")
    kd = M.VocabDistill(M.DistillConfig(N=N, H=H, V=V, K=K))
    want = kd.forward(X, W, ids, t)
    want += kd.backward(X, W, ids, t, want[1], g)
    M.set_wait_limit_ns(1000)
    try:
        kd.forward(X, W, ids, t)
        kd.backward(X, W, ids, t, want[1], g)
        assert M.check_status(kd.ws) in (0, _lib.MOE_ERR_TIMEOUT)
    finally:
        M.set_wait_limit_ns(0)
    again = kd.forward(X, W, ids, t)
    again += kd.backward(X, W, ids, t, again[1], g)
    assert all(torch.equal(p, q) for p, q in zip(want, again))
    kd.check()
