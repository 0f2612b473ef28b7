"""Where the log-probability and distillation calls take memory from when they run
on a stream that is not the current one: results and workspaces belong to the
stream that the kernels run on."""
import pytest
import torch

import lm_head_fp32_amd as lmh

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lmh.lib()


def _stream_of(t):
    """The stream whose pool of the allocator holds the tensor."""
    at = t.untyped_storage().data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= at < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's")


def _calls():
    g = torch.Generator(device="cuda").manual_seed(3)
    n, V = 4, 150000
    z = torch.randn(n, V, device="cuda", generator=g)
    y = torch.tensor([1, 5, -100, 7], dtype=torch.int32, device="cuda")
    ids = torch.randint(0, V, (n, 9), device="cuda", generator=g).int()
    vals = torch.randn(n, 9, device="cuda", generator=g)
    up = torch.ones(1, device="cuda")
    st = lmh.lmhead_logprobs(z, y)[5]
    st8 = lmh.lmhead_distill_fwd(z, ids, vals)[1]
    torch.cuda.synchronize()
    return {"logprobs": (lambda **k: lmh.lmhead_logprobs(z, y, n_top=3, **k), 6),
            "logprobs_none": (lambda **k: lmh.lmhead_logprobs(z, n_top=3, entropy=False, **k), 3),
            "logprobs_bwd": (lambda **k: lmh.lmhead_logprobs_bwd(z, st, y, up, **k), 1),
            "distill_fwd": (lambda **k: lmh.lmhead_distill_fwd(z, ids, vals, **k), 2),
            "distill_bwd": (lambda **k: lmh.lmhead_distill_bwd(z, st8, ids, vals, up, **k), 1),
            "distill_fused": (lambda **k: lmh.lmhead_distill_fused(z, ids, vals, up, **k), 3)}


def _tensors(res):
    return [t for t in (res if isinstance(res, tuple) else (res,)) if t is not None]


@pytest.mark.parametrize("name", ["logprobs", "logprobs_none", "logprobs_bwd", "distill_fwd", "distill_bwd",
                                  "distill_fused"])
def test_memory_belongs_to_the_launch_stream(name, monkeypatch):
    call, count = _calls()[name]
    want = [t.clone() for t in _tensors(call())]
    assert len(want) == count
    taken = []
    inner = lmh._workspace
    monkeypatch.setattr(lmh, "_workspace", lambda *a, **k: taken.append(inner(*a, **k)) or taken[-1])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for st in (side, side.cuda_stream):
        if name.endswith("_bwd") or st is side:
            got = _tensors(call(stream=st))
        else:  # a raw handle needs a workspace
            with pytest.raises(ValueError):
                call(stream=st)
            got = _tensors(call(stream=st, workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda")))
        torch.cuda.synchronize()
        for t, w in zip(got, want):
            assert _stream_of(t) == side.cuda_stream and torch.equal(t, w)
    assert (not taken) == name.endswith("_bwd")  # these rows are worked on in parts
    if taken:
        assert _stream_of(taken[0][0]) == side.cuda_stream
    with torch.cuda.stream(side):
        for t, w in zip(_tensors(call()), want):
            assert _stream_of(t) == side.cuda_stream and torch.equal(t, w)
    torch.cuda.synchronize()


def test_results_dropped_at_once():
    """A result that is dropped while its kernels run does not hand its memory to
    the calling stream."""
    call, _ = _calls()["distill_fused"]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    for _ in range(20):
        call(stream=side)
        junk = torch.full((4, 150000), 7.0, device="cuda")
        got = call(stream=side)
        torch.cuda.synchronize()
        assert (junk == 7.0).all()
        for t, w in zip(got, want):
            assert torch.equal(t, w)
