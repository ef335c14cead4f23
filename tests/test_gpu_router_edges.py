"""Choices of the router that 64 bits decide, at the edges of its forms: groups whose best members are NaN or lie at the end of
fp32, the first expert behind the last choice, and neighbours nearer than fp32 scores can tell in each kernel's own way of
deciding them again.

E = 96 and 100 in 8 (4) groups take the kernel with the values in shared memory, E = 64, 256 and 1024 the one that holds them in
registers (2, 8 and 32 a lane).  The choice has to be the oracle's exactly."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import gemm_uq_gb300 as uq  # noqa: E402
from oracle import router as orr  # noqa: E402

DEV = torch.device("cuda:0")
NAN, LOW = float("nan"), float("-inf")


def n(t):
    return t.double().cpu().numpy()


def _choose(x, k, score, bias=None, G=1, tg=1, gt=1):
    """The oracle's choice; the scores of a token with NaN logits are those over its other logits."""
    scores = orr.scores

    def among_numbers(v, how):
        v = np.asarray(v, np.float64)
        with np.errstate(invalid="ignore"):
            s = scores(np.where(np.isnan(v), -np.inf, v), how)
        return np.where(np.isnan(v), np.nan, s)
    orr.scores = among_numbers
    try:
        return orr.choose(n(x), k, score, None if bias is None else n(bias), G, tg, gt)
    finally:
        orr.scores = scores


def _check(x, k, score, bias=None, G=1, tg=1, gt=1, renorm=True):
    ids, w = uq.moe_route(x, k, score=score, bias=bias, groups=G, top_groups=tg, group_top=gt, renormalize=renorm)
    want = _choose(x, k, score, bias, G, tg, gt)
    bad = np.argwhere((ids.cpu().numpy() != want).any(axis=1)).reshape(-1)
    assert len(bad) == 0, f"{len(bad)} tokens, first {bad[0]}: {ids[bad[0]].tolist()}, in 64 bits {want[bad[0]].tolist()}"
    return ids, w


def _scores64(x, score):
    return orr.scores(np.asarray(x, np.float64), score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G", [(64, 8), (96, 8), (100, 4), (256, 8), (1024, 32)])
def test_groups_of_nan(E, G, score):
    """A group whose members are all NaN can be chosen, last: a token of NaN alone keeps its experts, and its weights are NaN."""
    size, g = E // G, np.random.default_rng(E)
    x = torch.from_numpy(g.normal(size=(7, E)).astype(np.float32)).to(DEV)
    x[0] = NAN
    x[1, :(G - 1) * size] = NAN                                          # numbers in the last group alone
    x[2, :G // 2 * size] = NAN
    x[3] = LOW
    x[3, size:3 * size] = NAN                                            # NaN is all that may be chosen
    x[4, ::2] = NAN
    x[5, size:2 * size] = NAN
    x[5, size + 1] = 0.3                                                 # one number beside NaN
    x[6, 1::size] = LOW
    bias = torch.from_numpy(g.normal(size=E).astype(np.float32) * 0.1).to(DEV)
    k = min(4, size)
    for b in (None, bias):
        for gt in (1, 2):
            for tg in (1, 2, G - 1):
                for renorm in (True, False):
                    ids, w = _check(x, k, score, b, G, tg, gt, renorm)
                    assert ids[0].tolist() == list(range(k)) and torch.isnan(w[0]).all()
                    assert ids[3].tolist() == list(range(size, size + k)) and torch.isnan(w[3]).all()


@pytest.mark.parametrize("E,G", [(64, 8), (96, 8), (256, 8)])
def test_groups_at_the_end_of_fp32(E, G):
    """Sums of two biases that leave fp32: the group counts, and in the order of the sums."""
    size = E // G
    x = torch.zeros(3, E, device=DEV)
    x[1, :size], x[2] = LOW, LOW
    x[2, 2 * size:3 * size] = 0.5
    for sign in (1.0, -1.0):
        bias = sign * torch.linspace(3.3e38, 2.9e38, G, device=DEV).repeat_interleave(size)
        for tg in (1, 2, 3):
            _check(x, 2, "sigmoid", bias, G, tg, 2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G", [(8, 1), (64, 8), (96, 8), (256, 1), (256, 8), (1000, 1)])
def test_nan_behind_the_lowest_numbers(E, G, score):
    """Masks of fp32's lowest value, and logits next to it, are numbers: they come in their order, and before NaN."""
    size = E // G
    low = torch.finfo(torch.float32).min
    x = torch.full((4, E), low, device=DEV)
    x[:, 0] = NAN
    x[1, 2::2] = -3.4012e38
    x[1, 3::4] = -3.4025e38
    x[2, 1:] = NAN
    x[2, size - 1] = low                                                 # one number, behind NaN
    x[3, 1:size] = LOW                                                   # the first group: NaN alone
    k = min(6, size)
    for tg in {1, max(G - 1, 1)}:
        for gt in (1, 2) if G > 1 else (1,):
            _check(x, k, score, None, G, tg, gt)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [40, 64, 200, 256, 1024])
def test_the_first_expert_behind_32_choices(E, score):
    """32 choices, the last of which and those behind it are nearer than fp32 can tell, all others far apart."""
    T, g = 64, np.random.default_rng(E)
    x = torch.from_numpy(g.normal(size=E).astype(np.float32) + g.integers(-40, 41, (T, E)).astype(np.float32) * np.float32(2.0 ** -22))
    s = _scores64(x.numpy()[:1], score)[0]
    bias = (2.0 - s).astype(np.float32)                                  # all choice values near two
    bias[g.permutation(E)[:31]] += np.arange(1, 32, dtype=np.float32)    # but for those of 31 experts
    x, bias = x.to(DEV), torch.from_numpy(bias).to(DEV)
    for k in (31, 32):
        _check(x, k, score, bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G", [(64, 8), (96, 8), (256, 8), (1024, 32)])
def test_groups_whose_best_two_cancel(E, G, score):
    """A group's best two far from one and of opposite signs: its sum has the error of the two, not one of its own size."""
    T, size, tg = 64, E // G, G // 2
    g = np.random.default_rng(E)
    x = torch.from_numpy(g.normal(size=(T, E)).astype(np.float32)).to(DEV)
    lead = 2.0 ** 20 * (1 + np.arange(G) / 64)                           # leaders far apart, so that their own order is plain
    bias = (-lead[:, None] + np.zeros((G, size))).astype(np.float32)     # the others undo the leader
    bias[:, 3] = lead
    _check(x, tg, score, torch.from_numpy(bias.reshape(-1)).to(DEV), G, tg, 2)


def _near_pairs(E, score, ranks, g):
    """Logits [64][E] and a bias whose choice values lie 2^-6 apart, but for the experts of ranks r and r + 1 (r in `ranks`), which
    are so near that fp32 does not tell, and whose order differs from token to token."""
    T = 64
    base = g.normal(size=E).astype(np.float32)
    level = (np.arange(E)[::-1] * 2.0 ** -6).astype(np.float64)
    order = g.permutation(E)                                             # order[r]: the expert of rank r
    for r in ranks:
        level[r + 1] = level[r]
    x = np.tile(base, (T, 1))
    for r in ranks:
        for e in order[r:r + 2]:
            x[:, e] += g.integers(-3, 4, T).astype(np.float32) * np.float32(2.0 ** -23)
    want = np.empty(E)
    want[order] = level
    bias = (want - _scores64(base[None], score)[0]).astype(np.float32)
    return torch.from_numpy(x).to(DEV), torch.from_numpy(bias).to(DEV)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G", [(60, 1), (64, 8), (96, 8), (256, 1), (256, 8), (1000, 1), (1024, 8)])
def test_a_few_near_pairs(E, G, score):
    """Pairs among choices that are far apart otherwise: within the choice, at its end, and behind it."""
    g = np.random.default_rng([E, G])
    k = 8
    for ranks in ((k - 1,), (1,), (0, 3, 6), (2, k - 1), (k,)):
        x, bias = _near_pairs(E, score, ranks, g)
        for gt in (1, 2) if G > 1 else (1,):
            _check(x, k, score, bias, G, G if G == 1 else 5, gt)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G", [(64, 8), (96, 8), (256, 8), (1024, 32)])
def test_near_groups(E, G, score):
    """Groups far apart but for two, the last that stays and the first that does not, whose order differs from token to token."""
    T, size, tg = 64, E // G, 3
    for gt in (1, 2):
        g = np.random.default_rng([E, gt])
        base = g.normal(size=E).astype(np.float32)
        s = _scores64(base[None], score)[0]
        total = np.arange(G)[::-1] * 0.125                               # of the groups by rank
        total[tg] = total[tg - 1]
        ranks = g.permutation(G)
        want = np.full(E, -8.0) + np.arange(E) * 2.0 ** -9               # members that do not count
        for r in range(G):
            lead = ranks[r] * size + g.permutation(size)[:2]
            want[lead[0]] = total[r] + (1.0 if gt == 2 else 0.0)
            if gt == 2:
                want[lead[1]] = -1.0
        bias = (want - s).astype(np.float32)
        x = np.tile(base, (T, 1))
        for r in (tg - 1, tg):
            x[:, ranks[r] * size:(ranks[r] + 1) * size] += g.integers(-3, 4, (T, size)).astype(np.float32) * np.float32(2.0 ** -23)
        _check(torch.from_numpy(x).to(DEV), 2, score, torch.from_numpy(bias).to(DEV), G, tg, gt)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G", [(40, 1), (64, 8), (96, 8), (256, 1), (256, 8), (480, 16), (1000, 1), (1024, 8)])
def test_equal_logits_beside_near_ones(E, G, score):
    """Few different logits, so near that fp32's scores are equal, each of many experts: an equal neighbour behind the last choice does
    not hide a higher one behind it."""
    T, g = 48, np.random.default_rng([E, G])
    if score == "sigmoid":
        steps = np.array([17.0, 18.25, 19.5, 25.5])
    else:
        steps = np.array([0.0, 1.0, 2.0, 3.0]) * 2.0 ** -23
    often = np.array([0.4, 0.4, 0.15, 0.05])
    x = torch.from_numpy(steps[g.choice(4, size=(T, E), p=often)].astype(np.float32)).to(DEV)
    x[0] = 18.25 if score == "sigmoid" else 0.0                          # all equal, as padding is
    x[1], x[1, E - 1] = x[0], x[1].max()
    bias = torch.zeros(E, device=DEV)
    for k in (1, 2, 5, 31, 32):
        for tg in {max(G // 2, -(-k // (E // G))), G}:
            for gt in (1, 2) if G > 1 else (1,):
                _check(x, min(k, E // G * tg), score, bias, G, tg, gt)
