"""Beam selection and state reordering against plain 64-bit forms.

Selected beams and tokens are whole numbers and must be equal; the scores are
FP64 values rounded once, so they are within half an FP32 step (2^-24) of the
oracle's, plus the kernel's own FP64 error (below 1e-9)."""
import numpy as np
import pytest
import torch

import lm_head_fp32_amd as lmh

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lmh.lib()


def _say(*a):
    print(*a, flush=True)


def _rows(t, pad=0):
    mult = 16 // t.element_size()
    ld = (t.shape[-1] + pad + mult - 1) // mult * mult
    buf = torch.full((t.shape[0], ld), float("nan"), dtype=t.dtype, device=t.device)
    buf[:, : t.shape[-1]] = t
    return buf[:, : t.shape[-1]]


def _oracle(logits, scores, k, finished, eos):
    """(scores, parent, token, finished) on the host in 64 bits."""
    B, W = scores.shape
    z = logits.double().cpu()
    V = z.shape[1]
    s = scores.double().cpu()
    s[torch.isposinf(s)] = float("nan")
    fin = torch.zeros(B, W, dtype=torch.bool) if finished is None else finished.bool().cpu()
    m = z.amax(1, keepdim=True)
    c = (z - (m + torch.log(torch.exp(z - m).sum(1, keepdim=True)))).reshape(B, W, V) + s[:, :, None]
    held = torch.full_like(c, -float("inf"))
    if 0 <= eos < V:
        held[:, :, eos] = s
    c = torch.where(fin[:, :, None], held, c)
    c = torch.nan_to_num(c, nan=-float("inf"), posinf=float("inf"), neginf=-float("inf"))
    c = c.reshape(B, W * V)
    order = np.stack([np.lexsort((np.arange(W * V), -row)) for row in c.numpy()])[:, :k]
    order = torch.from_numpy(order)
    parent, token = order // V, order % V
    return (torch.gather(c, 1, order), parent.int(), token.int(),
            torch.gather(fin, 1, parent) | (token == eos))


def _check(logits, scores, k, finished=None, eos=-1, **kw):
    want = _oracle(logits, scores, k, finished, eos)
    got = lmh.lmhead_beam_select(logits, scores, n_out=k, finished=finished, eos=eos, **kw)
    torch.cuda.synchronize()
    assert torch.equal(got[1].cpu(), want[1]) and torch.equal(got[2].cpu(), want[2])
    assert torch.equal(got[3].bool().cpu(), want[3])
    g, w = got[0].double().cpu(), want[0]
    assert torch.equal(torch.isneginf(g), torch.isneginf(w))
    ok = torch.isfinite(w)
    assert ((g - w).abs()[ok] <= w.abs()[ok] * 2.0 ** -24 + 1e-9).all()
    return got


def _random(B, W, V, dtype, seed, done=0.2, sigma=3.0, pad=8):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = _rows((sigma * torch.randn(B * W, V, device="cuda", generator=g)).to(dtype), pad)
    s = -20 + 2 * torch.randn(B, W, device="cuda", generator=g)
    fin = torch.rand(B, W, device="cuda", generator=g) < done
    return z, s, fin


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,W,V,k", [
    (1, 1, 1, 1), (2, 1, 5, 3), (3, 4, 3, 12), (1, 4, 32768, 4), (5, 3, 2047, 6), (5, 3, 2048, 6),
    (5, 3, 2049, 6), (2, 8, 4099, 16), (3, 5, 50001, 10), (2, 64, 3000, 64), (1, 64, 16400, 64),
    (40, 2, 700, 4), (1, 1, 300007, 64), (2, 33, 65, 33)])
def test_select_random(B, W, V, k, dtype):
    _say("beam select", B, W, V, k, dtype)
    z, s, fin = _random(B, W, V, dtype, B + W + V)
    _check(z, s, k, fin, V - 1)
    _check(z, s, k, None, 0)
    _check(z, s, k, fin.to(torch.uint8), -1)     # no token ends a beam
    _check(z, s, k, torch.ones_like(fin), V // 2)  # every beam has ended
    _check(z, s, k, fin, 2 ** 31 - 1)


@pytest.mark.parametrize("k", [1, 4, 9, 64])
def test_select_first_step(k):
    """One live beam, the others at -inf: its best tokens, in order."""
    z, s, _ = _random(3, 4, 5000, torch.float32, 1)
    s[:, 1:] = -float("inf")
    got = _check(z, s, k)
    assert not got[1].any()


def test_select_ties_go_to_the_lowest_position():
    # equal logits everywhere; a few levels only; equal beams; ties across
    # segment borders; -0 and +0
    s = torch.zeros(2, 3, device="cuda")
    _check(_rows(torch.zeros(6, 5001, device="cuda")), s, 7)
    _check(_rows(torch.zeros(6, 5001, device="cuda")), s, 64)
    z, _, _ = _random(2, 3, 9000, torch.float32, 5)
    lev = _rows(torch.round(z / 2))
    _check(lev, s, 64)
    _check(_rows(torch.round(z / 2).to(torch.bfloat16)), s, 40)
    same = _rows(z[:1].expand(6, -1).contiguous())
    _check(same, s, 12)
    edge = torch.full((6, 9000), -1.0, device="cuda")
    edge[:, 2044:2052] = 3.0
    edge[:, 8190:8194] = 3.0
    _check(_rows(edge), s, 30)
    zero = torch.zeros(6, 3000, device="cuda")
    zero[:, ::2] = -0.0
    _check(_rows(zero), s, 10)


@pytest.mark.parametrize("W,V,k", [(1, 100, 5), (2, 5000, 8), (3, 2049, 64), (32, 2100, 64)])
def test_select_logits_apart_by_less_than_a_score_resolves(W, V, k):
    # Every logit lies below 2^-60, so every score is -log V in 64 bits: the
    # logits decide within a beam, the lower beam between two.
    g = torch.Generator(device="cuda").manual_seed(V)
    z = _rows(1e-19 * torch.rand(W, V, device="cuda", generator=g).add_(1.0))
    z[:, V // 3] = z[:, V // 2]  # an equal pair
    got = lmh.lmhead_beam_select(z, torch.zeros(1, W, device="cuda"), n_out=k)
    want = np.lexsort((np.arange(V), -z[0].cpu().numpy()))[:k]
    assert not got[1].any() and got[2][0].tolist() == want.tolist()
    assert (got[0].double().cpu() + np.log(V)).abs().max() <= np.log(V) * 2.0 ** -24 + 4e-9


def test_select_of_the_largest_vocabulary():
    """Tokens up to the last that 31 bits number."""
    V = 2 ** 31 - 9
    z = torch.zeros((1, V + 1), dtype=torch.bfloat16, device="cuda")[:, :V]
    at = [V - 1, 0, 2 ** 30 + 7, V - 2049, 2047]
    for i, j in enumerate(at):
        z[0, j] = 9.0 - i
    got = lmh.lmhead_beam_select(z, torch.zeros(1, 1, device="cuda"), n_out=7, eos=V - 1)
    assert got[2][0].tolist() == at + [1, 2] and got[3][0].tolist() == [True] + 6 * [False]
    logz = np.log(V - 5 + sum(np.exp(9.0 - i) for i in range(5)))
    want = np.array([9.0, 8.0, 7.0, 6.0, 5.0, 0.0, 0.0]) - logz
    assert np.abs(got[0][0].double().cpu().numpy() - want).max() <= np.abs(want).max() * 2.0 ** -24 + 4e-9


def test_two_searches_at_once():
    """Calls on two streams, each with results and workspaces of its own."""
    z, s, fin = _random(16, 4, 40000, torch.float32, 21)
    want = lmh.lmhead_beam_select(z, s, finished=fin, eos=5)
    par = want[1]
    st = torch.randint(0, 99, (2, 64, 3, 500, 16), device="cuda", dtype=torch.int16)
    moved = lmh.lmhead_beam_reorder(st, par, out=torch.empty_like(st), beam_dim=1)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(10):
        for q in streams:
            with torch.cuda.stream(q):
                got.append((lmh.lmhead_beam_select(z, s, finished=fin, eos=5),
                            lmh.lmhead_beam_reorder(st, par, out=torch.empty_like(st), beam_dim=1)))
    torch.cuda.synchronize()
    for sel, mv in got:
        assert all(torch.equal(a, b) for a, b in zip(sel, want)) and torch.equal(mv, moved)


def test_select_eos_outside_32_bits_is_refused():
    z, s, _ = _random(1, 2, 100, torch.float32, 0)
    for eos in (2 ** 31, -2 ** 31 - 1, 2 ** 32 + 3):
        with pytest.raises(ValueError):
            lmh.lmhead_beam_select(z, s, eos=eos)


def test_select_masked_and_bad_rows():
    inf, nan = float("inf"), float("nan")
    for dtype in (torch.float32, torch.bfloat16):
        z, s, fin = _random(4, 4, 6001, dtype, 3, done=0.0)
        m = z.clone()
        m[0] = -inf                      # a beam with nothing left
        m[1, :] = -inf
        m[1, 5990:] = 1.0                # constrained to a few tokens
        m[2, 100:] = -inf
        m[3, 17] = nan                   # a broken row offers nothing
        m[4, 6000] = inf
        m[5, 2050] = -inf
        m[6] = torch.finfo(dtype).min    # masks of the type's lowest value
        m[6, 3] = 0.0
        m[7] = torch.finfo(dtype).min
        m[8:12] = -inf                   # a request with nothing at all
        m[12:16] = -inf
        m[13, 4000] = 2.0                # and one with a single token
        m = _rows(m)
        for k in (1, 4, 9, 64):
            _check(m, s, k, None, 2)
            _check(m, s, k, (torch.arange(16, device="cuda") % 3 == 0).reshape(4, 4), 6000)
        bad = s.clone()
        bad[0, 0], bad[0, 1], bad[1, 2], bad[2, 0] = nan, inf, -inf, -inf
        for k in (4, 20):
            _check(z, bad, k)
            _check(m, bad, k, torch.ones(4, 4, device="cuda", dtype=torch.bool), 5)
            _check(m, torch.full_like(s, -inf), k, None, 1)


def test_select_does_not_read_ended_rows():
    """NaN in the rows of ended and dead beams reaches nothing."""
    z, s, fin = _random(2, 4, 3000, torch.float32, 8, done=0.0)
    fin[0, 1] = True
    s[1, 2] = -float("inf")
    want = lmh.lmhead_beam_select(z, s, n_out=8, finished=fin, eos=7)
    z2 = z.clone()
    z2[1] = float("nan")
    z2[6] = float("nan")
    got = lmh.lmhead_beam_select(_rows(z2), s, n_out=8, finished=fin, eos=7)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_select_large_vocabulary_precision():
    """64 x 8 beams over 131072 tokens: every index as the 64-bit form's."""
    g = torch.Generator(device="cuda").manual_seed(12)
    B, W, V, k = 64, 8, 131072, 8
    z = 3 * torch.randn(B * W, V, device="cuda", generator=g)
    s = torch.randn(B, W, device="cuda", generator=g)
    got = lmh.lmhead_beam_select(z, s)
    lz = torch.logsumexp(z.double(), 1)
    top = torch.topk(z, k, dim=1)
    c = s.double()[:, :, None] + (top.values.double() - lz[:, None]).reshape(B, W, k)
    best = torch.topk(c.reshape(B, W * k), k, dim=1)
    torch.cuda.synchronize()
    assert torch.equal(got[1].long(), best.indices // k)
    assert torch.equal(got[2].long(), torch.gather(top.indices.reshape(B, W * k), 1, best.indices))
    assert ((got[0].double() - best.values).abs() <= best.values.abs() * 2.0 ** -24 + 1e-9).all()


def test_select_in_place_streams_and_graph():
    z, s, fin = _random(6, 4, 9000, torch.float32, 4)
    want = lmh.lmhead_beam_select(z, s, finished=fin, eos=11)
    s1, f1 = s.clone(), fin.clone()
    lmh.lmhead_beam_select(z, s1, finished=f1, eos=11, out_scores=s1, out_finished=f1)
    assert torch.equal(s1, want[0]) and torch.equal(f1, want[3])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [torch.empty_like(t) for t in want]
    for _ in range(3):
        lmh.lmhead_beam_select(z, s, finished=fin, eos=11, out_scores=got[0], out_parent=got[1],
                               out_token=got[2], out_finished=got[3], stream=side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # two steps of a search, captured in place over one workspace
    z2, _, _ = _random(6, 4, 9000, torch.float32, 40)
    hist = torch.arange(24 * 33, device="cuda", dtype=torch.int32).reshape(24, 33)
    ws = torch.empty(lmh.lmhead_beam_select_workspace_bytes(6, 4, 9000, 4), dtype=torch.uint8,
                     device="cuda")
    sc, fl, hs = s.clone(), fin.clone(), hist.clone()
    par = torch.empty((6, 4), dtype=torch.int32, device="cuda")
    tok = torch.empty_like(par)

    def search():
        for q in (z, z2):
            lmh.lmhead_beam_select(q, sc, finished=fl, eos=11, out_scores=sc, out_parent=par,
                                   out_token=tok, out_finished=fl, workspace=ws)
            lmh.lmhead_beam_reorder(hs, par)

    search()
    torch.cuda.synchronize()
    ref = [t.clone() for t in (sc, fl, hs, par, tok)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        search()
    for rep in range(3):
        sc.copy_(s), fl.copy_(fin), hs.copy_(hist)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((sc, fl, hs, par, tok), ref):
            assert torch.equal(a, b), rep


# ------------------------------------------------------------------ reordering

def _reordered(src, dst, parent, beam_dim, len_dim, lengths):
    """The plain form, on host copies."""
    B, Wo = parent.shape
    Wi = src.shape[beam_dim] // B
    out = dst.clone()
    for b in range(B):
        for i in range(Wo):
            p = int(parent[b, i])
            if not 0 <= p < Wi:
                continue
            d, s = out.select(beam_dim, b * Wo + i), src.select(beam_dim, b * Wi + p)
            if len_dim is not None and lengths is not None:
                n = min(max(int(lengths[b]), 0), src.shape[len_dim])
                d, s = d.narrow(len_dim - 1, 0, n), s.narrow(len_dim - 1, 0, n)
            d.copy_(s)
    return out


def _bits(t):
    return t.contiguous().view(torch.uint8)


CACHES = [  # shape with "R" = rows, beam_dim, len_dim, dtype
    (("R", 33), 0, None, torch.int32), (("R", 1), 0, None, torch.uint8), (("R",), 0, None, torch.float64),
    (("R", 7), 0, 1, torch.uint8), ((2, "R", 3, 19, 8), 1, 3, torch.bfloat16),
    ((3, "R", 29, 5), 1, 2, torch.float32), (("R", 2, 11, 33), 0, 2, torch.bfloat16),
    ((2, 2, "R", 40, 2, 16), 2, 3, torch.float16), (("R", 300, 3), 0, 1, torch.int8),
    (("R", 4, 1100, 64), 0, 2, torch.bfloat16)]


@pytest.mark.parametrize("shape,beam_dim,len_dim,dtype", CACHES)
@pytest.mark.parametrize("B,W", [(1, 1), (3, 4), (2, 7), (2, 13), (1, 31), (1, 64)])
def test_reorder(shape, beam_dim, len_dim, dtype, B, W):
    _say("reorder", shape, B, W, dtype)
    g = torch.Generator().manual_seed(B * W)
    sh = [B * W if d == "R" else d for d in shape]
    src = torch.randint(0, 100, sh, generator=g).to(dtype)
    other = torch.randint(0, 100, sh, generator=g).to(dtype)
    parents = [torch.randint(0, W, (B, W), generator=g), torch.arange(W).flip(0).expand(B, W),
               torch.arange(W).expand(B, W), torch.zeros(B, W, dtype=torch.int64),
               torch.randint(-2, W + 2, (B, W), generator=g), torch.full((B, W), -(2 ** 31))]
    lens = [None]
    if len_dim is not None:
        T = sh[len_dim]
        lens += [torch.randint(0, T + 1, (B,), generator=g), torch.tensor([0, T + 5, -3][:B])]
    for par in parents:
        for ln in lens:
            p32 = par.to(torch.int32).contiguous().cuda()
            l32 = None if ln is None else ln.to(torch.int32).cuda()
            d = other.cuda()
            got = lmh.lmhead_beam_reorder(src.cuda(), p32, out=d, beam_dim=beam_dim, len_dim=len_dim,
                                          lengths=l32)
            assert got is d
            assert torch.equal(_bits(d.cpu()), _bits(_reordered(src, other, par, beam_dim, len_dim, ln)))
            d = src.cuda()
            assert lmh.lmhead_beam_reorder(d, p32, beam_dim=beam_dim, len_dim=len_dim, lengths=l32) is d
            assert torch.equal(_bits(d.cpu()), _bits(_reordered(src, src, par, beam_dim, len_dim, ln)))


@pytest.mark.parametrize("off", [0, 1, 3, 5, 8])
def test_reorder_any_alignment_strides_and_beam_counts(off):
    """Views that start at any element, rows with space between them that must
    stay, and selections that change the number of beams."""
    B, Wi, Wo, T, D = 3, 2, 5, 21, 6
    g = torch.Generator().manual_seed(off)
    big_s = torch.randint(0, 100, (4, B * Wi, 3, T + 4, D), generator=g).to(torch.int16)
    big_d = torch.randint(0, 100, (4, B * Wo, 3, T + 4, D), generator=g).to(torch.int16)
    par = torch.randint(0, Wi, (B, Wo), generator=g)
    ln = torch.tensor([5, T, 0])

    def cut(t):
        return t[1:3, :, 1:, off % 4:off % 4 + T]

    want = big_d.clone()
    cut(want).copy_(_reordered(cut(big_s), cut(big_d), par, 1, 3, ln))
    s, d = big_s.cuda(), big_d.cuda()
    lmh.lmhead_beam_reorder(cut(s), par.int().cuda(), out=cut(d), beam_dim=1, len_dim=3,
                            lengths=ln.int().cuda())
    assert torch.equal(d.cpu(), want) and torch.equal(s.cpu(), big_s)
    flat_s = torch.randint(0, 100, (off + B * Wi * 37,), generator=g).to(torch.uint8)
    flat_d = torch.randint(0, 100, (off + B * Wo * 37,), generator=g).to(torch.uint8)
    want = flat_d.clone()
    want[off:] = _reordered(flat_s[off:].view(-1, 37), flat_d[off:].view(-1, 37), par, 0, None, None).view(-1)
    s, d = flat_s.cuda(), flat_d.cuda()
    lmh.lmhead_beam_reorder(s[off:].view(-1, 37), par.int().cuda(), out=d[off:].view(-1, 37))
    assert torch.equal(d.cpu(), want)
    # a source shared by every beam (stride 0), as after a prefill
    one = torch.randint(0, 100, (B, 1, 50), generator=g).to(torch.int32).cuda()
    d = torch.empty((B * Wo, 50), dtype=torch.int32, device="cuda")
    lmh.lmhead_beam_reorder(one[:, 0], torch.zeros((B, Wo), dtype=torch.int32, device="cuda"), out=d)
    assert torch.equal(d.view(B, Wo, 50), one.expand(B, Wo, 50))


def test_reorder_past_32_bit_offsets():
    """Rows beyond 2^32 bytes from the start of the state."""
    rows, T = 6, 1 << 30  # 6 GiB of bytes
    st = torch.zeros((rows, T), dtype=torch.uint8, device="cuda")
    st[:, -3:] = torch.arange(rows, device="cuda", dtype=torch.uint8)[:, None] + 1
    st[:, 7] = torch.arange(rows, device="cuda", dtype=torch.uint8)
    par = torch.tensor([[1, 0, 2], [0, 2, 0]], dtype=torch.int32, device="cuda")
    lmh.lmhead_beam_reorder(st, par)
    torch.cuda.synchronize()
    assert st[:, 7].tolist() == [1, 0, 2, 3, 5, 3]
    assert st[:, -1].tolist() == [2, 1, 3, 4, 6, 4] and st[:, T - 3].tolist() == [2, 1, 3, 4, 6, 4]
    assert not st[:, 8:1024].any()


@pytest.mark.parametrize("n_outer,B,W", [(1, 140001, 64), (3, 2 ** 22 - 1, 2)])
def test_reorder_of_many_short_rows(n_outer, B, W):
    """More rows than one launch covers."""
    g = torch.Generator(device="cuda").manual_seed(B)
    st = torch.randint(0, 256, (n_outer, B * W, 1), device="cuda", generator=g, dtype=torch.uint8)
    par = torch.randint(0, W, (B, W), device="cuda", generator=g, dtype=torch.int32)
    rows = (torch.arange(B, device="cuda")[:, None] * W + par).view(-1)
    want = st.index_select(1, rows)
    out = lmh.lmhead_beam_reorder(st, par, out=torch.zeros_like(st), beam_dim=1)
    assert torch.equal(out, want)
    lmh.lmhead_beam_reorder(st, par, beam_dim=1)
    assert torch.equal(st, want)


def test_decode_with_adapters_and_beams():
    """Several steps as a server runs them: logits of beams whose requests use
    different adapters, the next beams, their caches and histories; against
    the same steps in 64 bits."""
    B, W, K, V, r, n, steps = 3, 4, 128, 700, 8, 2, 5
    g = torch.Generator(device="cuda").manual_seed(77)
    Wt = (0.2 * torch.randn(V, K, device="cuda", generator=g)).bfloat16()
    A = (K ** -0.5 * torch.randn(n, r, K, device="cuda", generator=g)).bfloat16()
    Bm = torch.randn(n, V, r, device="cuda", generator=g).bfloat16()
    emb = torch.randn(V, K, device="cuda", generator=g)
    ids = torch.tensor([0, 1, -1], dtype=torch.int32, device="cuda").repeat_interleave(W)
    scores = torch.full((B, W), -float("inf"), device="cuda")
    scores[:, 0] = 0
    fin = torch.zeros((B, W), dtype=torch.bool, device="cuda")
    hist = torch.zeros((B * W, steps), dtype=torch.int32, device="cuda")
    cache = torch.randn(2, B * W, 3, steps, 8, device="cuda", generator=g).bfloat16()
    lens = torch.empty(B, dtype=torch.int32, device="cuda")
    x = torch.randn(B * W, K, device="cuda", generator=g).bfloat16()
    for t in range(steps):
        z = lmh.lmhead_logits_lora(x, Wt, A, Bm, ids, out_dtype="fp32")
        want = _oracle(z, scores, W, fin, 3)
        lens.fill_(t)
        href, cref = hist.cpu(), cache.cpu()
        scores, par, tok, fin = lmh.lmhead_beam_select(z, scores, finished=fin, eos=3)
        assert torch.equal(par.cpu(), want[1]) and torch.equal(tok.cpu(), want[2])
        lmh.lmhead_beam_reorder(hist, par, len_dim=1, lengths=lens)
        lmh.lmhead_beam_reorder(cache, par, beam_dim=1, len_dim=3, lengths=lens)
        assert torch.equal(hist.cpu(), _reordered(href, href, par.cpu(), 0, 1, lens.cpu()))
        assert torch.equal(_bits(cache.cpu()), _bits(_reordered(cref, cref, par.cpu(), 1, 3, lens.cpu())))
        hist[:, t] = tok.flatten()
        x = (x.float() * 0.5 + emb[tok.flatten().long()]).bfloat16()
    assert torch.isfinite(scores).all()
