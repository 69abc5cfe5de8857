"""The router's choice by scores (key="score"): DeepSeek-V3's node-limited choice and the general
definition written out in 64 bits, and the refusals of an unknown key."""

import ctypes

import numpy as np
import pytest
import torch

import combine_shuffling_amd as cs
import layer_ref as ref
from combine_shuffling_amd import _abi

from gpu_util import say

U = ref.U


def deepseek_v3(logits, bias, groups, kept_groups, k, scale):
    """(ids, weights, biased scores) in float64: sigmoid scores; the bias is added for the choice;
    the groups of the largest sums of their two largest; the k largest of those groups; weights of
    the unbiased scores, normalised and scaled."""
    scores = torch.sigmoid(torch.as_tensor(logits).double())
    biased = scores + torch.as_tensor(bias).double()
    by_group = biased.view(len(biased), groups, -1)
    worth = by_group.topk(2, dim=-1).values.sum(-1)
    mask = torch.zeros_like(worth).scatter_(1, worth.topk(kept_groups, dim=-1).indices, 1.0)
    allowed = mask[:, :, None].expand_as(by_group).reshape(biased.shape) > 0
    ids = biased.masked_fill(~allowed, -torch.inf).topk(k, dim=-1).indices
    w = scores.gather(1, ids)
    return ids.numpy(), (scale * w / w.sum(-1, keepdim=True)).numpy(), biased.numpy()


def scores_of(x, score):
    """float64 scores; NaN stays, -infinity has -infinity."""
    x = x.astype(np.float64)
    y = np.where(np.isnan(x), -np.inf, x)
    p = ref._shares(y) if score == "softmax" else ref.sigmoid(y)
    return np.where(np.isnan(x), np.nan, np.where(x == -np.inf, -np.inf, p))


def clear_rows(key, err, node_of, nodes, k):
    """Rows whose choice no error of each key up to its err can change."""
    node_of = np.asarray(node_of)
    ok = np.ones(len(key), dtype=bool)

    def apart(low, high, n):
        """The n of the largest low ends lie above the high ends of the others."""
        by = np.argsort(-low, kind="stable")
        return by, n >= len(by) or low[by[n - 1]] > high[by[n:]].max()

    for t in range(len(key)):
        low, high = key[t] - err[t], key[t] + err[t]
        if nodes:
            # a sum of two keys also rounds by itself
            two = lambda q, s: np.array([(1 + s * U * np.sign(v)) * v for v in (  # noqa: E731
                np.sort(q[node_of == n])[::-1][:2].sum() for n in range(node_of.max() + 1))])
            by, ok[t] = apart(two(low, -1), two(high, 1), nodes)
            kept = np.isin(node_of, by[:nodes])
            low, high = low[kept], high[kept]
        for j in range(1, k + 1):     # the j largest, for the order among them
            ok[t] &= bool(apart(low, high, j)[1])
    return ok


# ---- refusals (CPU)

@pytest.mark.parametrize("key", [2, -1])
def test_unknown_key_is_refused(key):
    p, vp, L = cs.Plan(64, 64, 8, 2, 2), ctypes.c_void_p, _abi.lib()
    c = _abi.RouterConfig(1, 1, 0, 1.0, key)
    assert L.moe_router(p._h, ctypes.byref(c), vp(16), 1, None, vp(16), vp(16),
                        None) == _abi.ERR_INVALID_ARGUMENT
    assert L.moe_router_backward(p._h, ctypes.byref(c), vp(16), 1, vp(16), vp(16), vp(16),
                                 None) == _abi.ERR_INVALID_ARGUMENT


def test_binding_refuses_an_unknown_key():
    with pytest.raises(ValueError, match="key"):
        cs.Plan(64, 64, 8, 2, 2).router(torch.zeros(64, 8), key="rank")
    with pytest.raises(ValueError, match="GPU"):
        cs.router(cs.Plan(64, 64, 8, 2, 2), torch.zeros(64, 8), key="score")


def test_the_two_keys_do_not_choose_alike():
    # Why the key matters: with logits of deviation 1.5 and a bias of 0.3, the choice by logits is
    # another one than the choice by scores.
    g = torch.Generator().manual_seed(0)
    x, b = torch.randn(256, 256, generator=g) * 1.5, torch.randn(256, generator=g) * 0.3
    ids, _, _ = deepseek_v3(x, b, 8, 4, 8, 1.0)
    by_logit = ref.router_choice(x.numpy(), b.numpy(), 8, [e // 32 for e in range(256)], 4)
    shared = np.mean([len(set(a) & set(c)) / 8 for a, c in zip(ids, by_logit)])
    assert shared < 0.5


# ---- on the GPU

@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,groups,kept,k", [(1, 256, 8, 4, 8), (300, 256, 8, 4, 8),
                                               (4500, 256, 8, 4, 8), (100, 64, 4, 2, 6),
                                               (70, 512, 16, 4, 8), (33, 1024, 64, 9, 16)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_deepseek_v3_choice(T, E, groups, kept, k, dtype, dev):
    say(f"[router key] DeepSeek-V3 T={T} E={E} groups={groups} {dtype}")
    g = torch.Generator().manual_seed(T + E)
    rows = np.arange(T) % 301
    x = (torch.randn(min(T, 301), E, generator=g) * 1.5).to(dtype)
    bias = torch.randn(E, generator=g) * 0.3
    ids, w, key = deepseek_v3(x, bias, groups, kept, k, 2.5)
    # sigmoid in float32: exp, a sum and a quotient, 8 roundings counted for them, and the bias
    err = 8 * U * torch.sigmoid(x.double()).numpy() + U * np.abs(key)
    clear = clear_rows(key, err, np.repeat(np.arange(groups), E // groups), kept, k)[rows]
    assert clear.mean() > 0.9
    plan = cs.Plan(T, 8, E, k, groups, 1)
    got, gw = plan.router(x[rows].to(dev), bias.to(dev), "sigmoid", True, 2.5, kept, key="score")
    got, gw = got.cpu().numpy(), gw.cpu().numpy().astype(np.float64)
    assert np.array_equal(got[clear], ids[rows][clear])
    want = ref.router_weights(x.double().numpy()[rows], got, "sigmoid", True, 2.5)
    assert np.abs(want[clear] - w[rows][clear]).max() < 1e-12
    # log sigmoid, its difference from the largest (|x| < 10) and exp: as for the choice by logits
    assert (np.abs(gw - want) <= (16 + k + 4 * 16) * U * want).all()


CASES = [
    # T, E, k, R, G, nodes
    (1, 1, 1, 1, 1, 0),
    (129, 64, 8, 4, 4, 0),
    (33, 100, 6, 10, 2, 3),
    (50, 30, 4, 8, 2, 2),        # nodes of 8, 8, 7, 7
    (20, 64, 1, 64, 1, 1),       # nodes of one expert
    (40, 300, 16, 6, 1, 2),
    (9, 1000, 11, 7, 1, 3),
    (4099, 64, 8, 8, 8, 0),
    (4097, 100, 6, 10, 2, 3),
    (4098, 200, 4, 20, 1, 2),
]


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,R,G,nodes", CASES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True], ids=["plain", "bias"])
def test_choice_by_score(T, E, k, R, G, nodes, score, biased, dev):
    say(f"[router key] T={T} E={E} k={k} nodes={nodes} {score} bias={biased}")
    rng = np.random.default_rng(T + E)
    few = rng.normal(size=(min(T, 301), E)).astype(np.float32) * 2
    bias = ((0.3 if score == "sigmoid" else 2.0 / E) * rng.normal(size=E)).astype(np.float32) if biased else None
    rows = np.arange(T) % 301
    lo = cs.expert_partition(E, R)
    node_of = [next(r for r in range(R) if lo[r] <= e < lo[r + 1]) // G for e in range(E)]
    p = scores_of(few, score)
    key = p + (bias.astype(np.float64) if biased else 0.0)
    # float32 scores: softmax has a sum of E terms, exp of a difference below 20
    err = (16 + E + 4 * 20 if score == "softmax" else 8) * U * p + U * np.abs(key)
    clear = clear_rows(key, err, node_of, nodes, k)[rows]
    assert clear.mean() > 0.9
    want = ref.router_choice(key, None, k, node_of, nodes)[rows]  # its float32 keys: one more rounding
    plan = cs.Plan(T, 8, E, k, R, G)
    x = torch.from_numpy(few[rows]).to(dev)
    bd = None if bias is None else torch.from_numpy(bias).to(dev)
    for renorm in (True, False):
        idx, w = cs.router(plan, x, bd, score, renorm, 1.5, nodes, key="score")
        idx = idx.cpu().numpy()
        assert np.array_equal(idx[clear], want[clear])
        assert all(len(set(r)) == k for r in idx) and idx.min() >= 0 and idx.max() < E
        ww = ref.router_weights(few[rows], idx, score, renorm, 1.5)
        assert (np.abs(w.cpu().numpy() - ww) <= (16 + E + 4 * 20) * U * ww + 2.0 ** -120).all()
    # the plan's other key is what it was
    idx, _ = cs.router(plan, x, bd, score, True, 1.5, nodes)
    assert np.array_equal(idx.cpu().numpy(), ref.router_choice(few, bias, k, node_of, nodes)[rows])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [4, 4100], ids=["wave", "lanes"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_and_equal_scores(T, score, dev):
    E, k = 64, 5
    plan = cs.Plan(T, 8, E, k, 4, 1)
    rows = torch.arange(T) % 4
    x = torch.zeros(4, E)
    x[0, :60] = -torch.inf                    # fewer than k are left
    x[1] = -torch.inf                         # nothing is left
    x[2, ::2] = float("nan")
    x[3] = 200.0 + torch.arange(E) * 0.01     # sigmoid: all round to 1
    bias = torch.zeros(E)
    bias[:60] = 5.0                           # does not bring a masked expert back
    idx, w = plan.router(x[rows].to(dev), bias.to(dev), score, True, 1.0, 0, key="score")
    idx, w = idx.cpu().reshape(T, k)[:4].tolist(), w.cpu()
    assert idx[0] == [60, 61, 62, 63, 0] and torch.equal(w[0], torch.tensor([0.25] * 4 + [0.0]))
    assert idx[1] == [0, 1, 2, 3, 4] and not w[1].any()
    assert idx[2] == [1, 3, 5, 7, 9]
    assert idx[3] == ([59, 58, 57, 56, 55] if score == "softmax" else [0, 1, 2, 3, 4])
    # limited nodes of 16 experts: the masked nodes come last
    idx, _ = plan.router(x[rows].to(dev), None, score, True, 1.0, 1, key="score")
    assert idx.cpu()[0].tolist() == [60, 61, 62, 63, 48]
