"""Scores of different beams that are equal, and scores near zero.

A row's largest logit adds exactly one to the sum of exponentials about it, so
a row and the same row moved by a constant (the difference exact in FP32) give
equal scores, a token that is the only one left has the beam's score exactly,
and no candidate scores above its beam.  Error of the sum: 4e-9 relative in the
terms besides the largest ones, so log d is off by at most 4e-9 (1 - 1 / d),
and by the rounding of a few FP64 steps (1e-14)."""
import numpy as np
import pytest
import torch

import lm_head_fp32_amd as lmh

pytestmark = pytest.mark.gpu

INF = float("inf")
DTYPES = [torch.float32, torch.bfloat16]
# exact in BF16; the last ones beyond 2^28, where FP32 steps are 16 and more
LEVELS = [0.0, 1.296875, -0.25, 7.71875, 0.25, -88.5, 1.0, 10048.0, -2.0 ** 27 - 2.0 ** 20, 3.0 * 2.0 ** 26,
          2.0 ** 29 + 2.0 ** 22, 3.0e38, -2.0 ** 125]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lmh.lib()


def _rows(t):
    mult = 16 // t.element_size()
    ld = (t.shape[-1] + mult - 1) // mult * mult
    buf = torch.full((t.shape[0], ld), float("nan"), dtype=t.dtype, device="cuda")
    buf[:, : t.shape[-1]] = t
    return buf[:, : t.shape[-1]]


def _select(z, s, k, fin=None, eos=-1):
    got = lmh.lmhead_beam_select(_rows(z.cuda()), s.cuda(), n_out=k, eos=eos,
                                 finished=None if fin is None else fin.cuda())
    torch.cuda.synchronize()
    return [t.cpu() for t in got]


def _levels(dtype):
    t = torch.tensor(LEVELS)
    return t.to(dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [1, 2, 7, 2048, 2049, 5001])
@pytest.mark.parametrize("score", [0.0, -3.7])
def test_constant_rows_of_different_levels_tie(V, dtype, score):
    lv = _levels(dtype)
    W = len(lv)
    for turn in (0, 1, 5, 9):
        z = lv.roll(turn)[:, None].expand(W, V).contiguous()
        k = min(2 * V + 1, 64, W * V)
        sc, par, tok, _ = _select(z, torch.full((1, W), score), k)
        pos = np.arange(k)
        assert par[0].tolist() == (pos // V).tolist() and tok[0].tolist() == (pos % V).tolist()
        assert (sc == sc[0, 0]).all()
        c = float(torch.tensor(score)) - np.log(V)
        assert abs(float(sc[0, 0]) - c) <= abs(c) * 2.0 ** -24 + 1e-14


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [1, 300, 4100])
def test_the_only_token_left_has_the_beams_score(V, dtype):
    lv = _levels(dtype)
    W = len(lv)
    for turn in (0, 3, 8):
        z = torch.full((W, V), -INF, dtype=dtype)
        at = [(37 * w) % V for w in range(W)]
        z[range(W), at] = lv.roll(turn)
        for score in (0.0, -1.5, -40.3, -1e-30):
            s = torch.full((1, W), score)
            sc, par, tok, _ = _select(z, s, W)
            assert par[0].tolist() == list(range(W)) and tok[0].tolist() == at
            assert (sc == s).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_of_nothing_but_masks(dtype):
    """Every logit at the type's lowest value: the beam's score, not divided
    among the tokens."""
    z = torch.full((3, 2500), torch.finfo(dtype).min, dtype=dtype)
    z[1, 7] = 0.0
    s = torch.tensor([[-2.0, -2.0, -1.0]])
    sc, par, tok, _ = _select(z, s, 4)
    assert par.tolist() == [[2, 2, 2, 2]] and tok.tolist() == [[0, 1, 2, 3]] and (sc == -1.0).all()
    s[0, 2] = -INF
    sc, par, tok, _ = _select(z, s, 4)
    assert par.tolist() == [[0, 0, 0, 0]] and tok.tolist() == [[0, 1, 2, 3]] and (sc == -2.0).all()


def test_an_ended_beam_ties_with_a_forced_one():
    """Equal scores: the lower beam first, whether it has ended or not."""
    for level in LEVELS:
        for first in (True, False):
            z = torch.full((2, 50), -INF)
            z[:, 9] = level
            fin = torch.tensor([[first, not first]])
            sc, par, tok, end = _select(z, torch.full((1, 2), -2.5), 2, fin, 30)
            assert par.tolist() == [[0, 1]] and tok.tolist() == [[30, 9] if first else [9, 30]]
            assert sc.tolist() == [[-2.5, -2.5]] and end.tolist() == [[first, not first]]


@pytest.mark.parametrize("V", [5, 700, 6001])
def test_rows_moved_by_a_constant_tie(V):
    """Different multiples of 1 / 64 below 2^10, moved by multiples of 1 / 64:
    every difference is exact."""
    g = torch.Generator().manual_seed(V)
    row = (torch.randperm(V, generator=g) - V // 2) / 64.0
    moves = torch.tensor([0.0, 1.296875, -3.015625, 100.5, -777.25, 1.0 / 64])
    W, n = len(moves), min(V, 9)
    best = torch.sort(row, descending=True).indices[:n].tolist()
    for turn in range(W):
        z = row[None, :] + moves.roll(turn)[:, None]
        sc, par, tok, _ = _select(z, torch.zeros(1, W), n * W)
        assert par[0].tolist() == list(range(W)) * n
        assert tok[0].tolist() == [j for j in best for _ in range(W)]
        assert (sc.view(n, W) == sc.view(n, W)[:, :1]).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sigma", [0.01, 1.0, 8.0, 60.0])
@pytest.mark.parametrize("move", [0.0, 1.3, 4000.0])
def test_scores_near_zero(sigma, move, dtype):
    """Peaked rows under scores of zero: not above zero, and right relative to
    themselves; every index as the 64-bit form's."""
    g = torch.Generator().manual_seed(int(10 * sigma) + int(move))
    B, W, V, k = 4, 3, 4999, 8
    z = (sigma * torch.randn(B * W, V, generator=g) + move).to(dtype)
    z[0, 17] += 40.0
    z[4, 4998] += 20.0
    z[5, 0] += 12.0
    sc, par, tok, _ = _select(z, torch.zeros(B, W), k)
    assert (sc <= 0).all()
    x = z.double().numpy()
    x = x - x.max(1, keepdims=True)
    d = np.exp(x).sum(1)
    c = (x - np.log(d)[:, None]).reshape(B, W * V)
    err = 4e-9 * (1 - 1 / d) + 1e-14
    pos = np.arange(W * V)
    for b in range(B):
        order = np.lexsort((pos, -c[b]))[: k + 1]
        gaps = -np.diff(c[b][order])
        for i in range(k):
            got, w = float(sc[b, i]), int(par[b, i])
            want = c[b][order[i]]
            near = err[b * W + order[i] // V]
            assert abs(got - want) <= abs(want) * 2.0 ** -24 + near, (b, i)
            # candidates further apart than the bound stand in its order
            if gaps[i] > 1e-8 and (i == 0 or gaps[i - 1] > 1e-8):
                assert w * V + int(tok[b, i]) == order[i], (b, i)
