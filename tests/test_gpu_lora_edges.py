"""Adapter gradients at the ends of what the C interface allows."""
import itertools

import pytest
import torch

import lm_head_fp32_amd as lmh

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lmh.lib()


@pytest.mark.parametrize("n", [0, 1])
@pytest.mark.parametrize("M,K,V", [(0, 64, 72), (5, 64, 72), (300, 64, 72), (5, 0, 72), (5, 64, 0)])
def test_every_choice_of_gradients_of_few_adapters(M, K, V, n):
    """Any of the three gradients, pointers to all of them or to none: a call
    without adapters has nothing to write but dX."""
    L, r = lmh.lib(), 8
    g = torch.ones((max(M, 1), max(V, 8)), device="cuda").bfloat16()
    x = torch.ones((max(M, 1), max(K, 8)), device="cuda").bfloat16()
    A = torch.ones((1, r, max(K, 8)), device="cuda").bfloat16()
    B = torch.ones((1, max(V, 8), r), device="cuda").bfloat16()
    ids = torch.zeros(max(M, 1), dtype=torch.int32, device="cuda")
    need = lmh.lmhead_lora_bwd_workspace_bytes(M, K, V, r, n)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    for which in itertools.product((False, True), repeat=3):
        for add in (0, 1):
            outs = [torch.full(s, 5.0, device="cuda") for s in (x.shape, A.shape, B.shape)]
            dX, dA, dB = (t.data_ptr() if q else None for t, q in zip(outs, which))
            rc = L.lmhead_lora_bwd(g.data_ptr(), g.stride(0), x.data_ptr(), x.stride(0), A.data_ptr(),
                                   A.stride(1), A.stride(0), B.data_ptr(), r, B.stride(0), ids.data_ptr(), None,
                                   n, r, dX, outs[0].stride(0), dA, outs[1].stride(1), outs[1].stride(0), dB, r,
                                   outs[2].stride(0), add, M, K, V, ws.data_ptr(), ws.numel(), stream)
            assert rc == 0, (which, add)
            torch.cuda.synchronize()
            # ones everywhere: t = V, u = K; without adapters the ids name none
            t, u, old = float(V), float(K), 5.0 * add
            want = [r * t + old, M * t + old, M * u + old]
            if n == 0:
                want = [float("nan"), 5.0, 5.0]
            for out, q, w, live in zip(outs, which, want, ((M, K), (r, K), (V, r))):
                ref = torch.full_like(out, 5.0)
                if q:
                    ref[..., : live[0], : live[1]] = w
                assert torch.equal(out.nan_to_num(nan=-1.0), ref.nan_to_num(nan=-1.0)), (which, add)
