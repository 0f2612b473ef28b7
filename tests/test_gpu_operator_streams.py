"""Where the adapter and beam calls take memory from when they run on a stream
that is not the current one: results and workspaces belong to the stream that
the kernels run on, whatever the caller keeps of them."""
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

    def rnd(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    x, W, A, B = (rnd(*s).bfloat16() for s in ((40, 64), (504, 64), (3, 8, 64), (3, 504, 8)))
    gr = rnd(40, 504).bfloat16()
    ids = (torch.arange(40, device="cuda") % 4 - 1).int()
    z, s = rnd(24, 3000), rnd(6, 4)
    n = lmh.lmhead_lora_bwd_workspace_bytes(40, 64, 504, 8, 3)
    return {
        "logits": (lambda **k: lmh.lmhead_logits_lora(x, W, A, B, ids, **k), 1,
                   lmh.lmhead_logits_lora_workspace_bytes(40, 64, 504, 8, "bf16")),
        "bwd": (lambda **k: lmh.lmhead_lora_bwd(gr, x, A, B, ids, **k), 3, n),
        "bwd_dA": (lambda **k: lmh.lmhead_lora_bwd(gr, x, A, B, ids, dX=False, dB=False, **k), 1, n),
        "select": (lambda **k: lmh.lmhead_beam_select(z, s, **k), 4,
                   lmh.lmhead_beam_select_workspace_bytes(6, 4, 3000, 4))}


def _tensors(res):
    return [t for t in (res if isinstance(res, tuple) else (res,)) if t is not None]


@pytest.mark.parametrize("name", ["logits", "bwd", "bwd_dA", "select"])
def test_memory_belongs_to_the_launch_stream(name, monkeypatch):
    call, count, need = _calls()[name]
    want = [t.clone() for t in _tensors(call())]
    assert len(want) == count
    taken = []
    inner = lmh._workspace
    monkeypatch.setattr(lmh, "_workspace", lambda *a, **k: taken.append(inner(*a, **k)) or taken[-1])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = _tensors(call(stream=side))
    torch.cuda.synchronize()
    assert len(taken) == 1
    for t in got + [taken[0][0]]:
        assert _stream_of(t) == side.cuda_stream
    for t, w in zip(got, want):
        assert torch.equal(t, w)
    # a raw handle, with the caller's workspace
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    got = _tensors(call(stream=side.cuda_stream, workspace=ws))
    torch.cuda.synchronize()
    for t, w in zip(got, want):
        assert _stream_of(t) == side.cuda_stream and torch.equal(t, w)
    with pytest.raises(ValueError):
        call(stream=side.cuda_stream)
    # without a stream: the current one's
    with torch.cuda.stream(side):
        got = _tensors(call())
    assert all(_stream_of(t) == side.cuda_stream for t in got)
    assert all(_stream_of(t) == 0 for t in _tensors(call()))
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", ["logits", "bwd", "select"])
def test_dropped_results_are_not_handed_out(name):
    """The caller keeps one result of a call that waits on its stream: the
    others' memory, and the workspace's, is not the current stream's to take."""
    call, _, _ = _calls()[name]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    res = _tensors(call(stream=side))
    sizes = [t.untyped_storage().nbytes() for t in res]
    places = {t.untyped_storage().data_ptr() for t in res}
    keep = res[-1]
    del res
    mine = [torch.full((n,), 0x5a, dtype=torch.uint8, device="cuda") for n in 4 * sizes]
    assert not places & {t.data_ptr() for t in mine}
    torch.cuda.synchronize()
    assert all(bool((t == 0x5a).all()) for t in mine)
    assert torch.equal(keep, _tensors(call())[-1])


def test_captured_on_another_stream():
    """A captured step that forks a call onto another stream and joins it."""
    call, _, _ = _calls()["select"]
    want = call()
    side = torch.cuda.Stream()
    kept = [torch.empty_like(t) for t in want]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        res = call(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        for k, t in zip(kept, res):
            k.copy_(t)
    for _ in range(3):
        for k in kept:
            k.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, w in zip(kept, want):
            assert torch.equal(k, w)
