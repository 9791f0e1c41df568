"""Group-limited routing where the last chosen expert is followed by its equal: experts of
equal logit and bias on both sides of the last place, and behind them in index an expert
whose key is a little larger in 64 bits and no larger in 32.  Ids against the definition."""
import itertools

import pytest
import torch

import fp8_ref as ref
from mixture_experts_routing_router_gb300 import native as N
from test_gpu_route_grouped import SCORE, gpu_route

pytestmark = pytest.mark.gpu

F32, D = torch.float32, torch.float64

#         E    k   G  topk_groups
SIZES = [(3, 1, 1, 1), (24, 1, 1, 1), (24, 4, 1, 1), (32, 6, 4, 2), (64, 8, 1, 1), (64, 5, 4, 3), (160, 6, 8, 3),
         (256, 8, 8, 4), (256, 8, 1, 1), (48, 31, 1, 1), (33, 30, 3, 3), (1000, 16, 10, 4)]
T = 48


def rows(score, E, k, G, tg, chain, seed):
    """(logits, bias): per token some clear winners, one in each group that counts if there are
    enough of them, then `chain` equal experts that the last place falls among, then a near one."""
    g = torch.Generator().manual_seed(seed)
    n = E // G
    low = {"one": -3.0, "zero": -110.0, "softmax": -3.0}[score]
    l = low - torch.rand(T, E, generator=g)
    bias = torch.zeros(E)
    held = torch.randperm(G, generator=g)[:tg]
    for t in range(T):
        # how many of the equal ones are chosen; "one": a clear winner needs a bias, which all tokens share
        inside = 1 + (chain if score == "one" else t) % min(chain - 1, k)
        if score != "one":
            held = torch.randperm(G, generator=g)[:tg]
        clear = [int(held[j % tg]) * n + j // tg for j in range(k - inside)]
        l[t, clear] = 3.0 + 0.5 * torch.arange(len(clear), dtype=F32)
        if score == "one":
            bias[clear] = 1.0 + 0.25 * torch.arange(len(clear), dtype=F32)
        pool = sorted(e for h in held for e in range(int(h) * n, (int(h) + 1) * n) if e not in clear)
        some = sorted(torch.randperm(len(pool), generator=g)[:chain + 1].tolist())
        equal, near = [pool[i] for i in some[:-1]], pool[some[-1]]
        if score == "one":                                     # 1 + e^-x is 1 + 2^-23 for both
            l[t, equal], l[t, near] = 15.625, 16.0
        elif score == "zero":                                  # scores under FP32's normal range
            l[t, equal], l[t, near] = -100.0, -89.0
        else:                                                  # equal distances from the largest logit, rounded
            v = 0.125 + 0.125 * float(torch.rand((), generator=g))
            v = torch.tensor(v, dtype=F32)
            l[t, equal] = v
            l[t, near] = v + (2 if not clear else 1 + t % 12) * 2.0 ** -26
    return l, bias


def check(l, bias, E, k, softmax, G, tg, what):
    shape = N.make_shape(l.shape[0], 64, E, k, 64)
    for top in (1, 2):
        ids, w, st = gpu_route(shape, N.make_router(SCORE[softmax], G, tg, top, True, 2.5), l, bias)
        assert st == N.MOE_OK
        want, want_w = ref.route(l, bias, k, softmax, G, tg, top, True, 2.5)
        wrong = torch.nonzero((ids.long() != want).any(1)).flatten()
        assert len(wrong) == 0, f"{what}, group_top {top}: {len(wrong)} of {len(l)} tokens, the first {int(wrong[0])}: " \
                                f"{ids[wrong[0]].tolist()} for {want[wrong[0]].tolist()}"
        assert ((w.to(D) - want_w).abs() <= ref.W_REL * want_w + ref.W_ABS).all()


@pytest.mark.parametrize("chain", [2, 3, 9, 40])
@pytest.mark.parametrize("score", ["one", "zero", "softmax"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_equal_experts_at_the_last_place(size, score, chain):
    E, k, G, tg = size
    if chain + 1 + 2 * k > tg * (E // G) and size != (3, 1, 1, 1):
        pytest.skip("more experts than the groups hold")
    if size == (3, 1, 1, 1) and chain > 2:
        pytest.skip("more experts than there are")
    l, bias = rows(score, E, k, G, tg, chain, seed=E + chain)
    check(l, bias, E, k, score == "softmax", G, tg, (size, score, chain))
    if not bias.any():
        check(l, None, E, k, score == "softmax", G, tg, (size, score, chain))


@pytest.mark.parametrize("softmax", [False, True], ids=["sigmoid", "softmax"])
@pytest.mark.parametrize("size", [(24, 4, 1, 1), (160, 6, 8, 3), (256, 8, 1, 1), (250, 9, 10, 4)], ids=str)
def test_saturated_scores_of_coarse_logits(size, softmax):
    """BF16-valued logits of a large deviation: equal ones, and scores at 1 or 0 in FP32."""
    E, k, G, tg = size
    g = torch.Generator().manual_seed(E)
    for std in (4.0, 12.0, 40.0):
        l = (std * torch.randn(200, E, generator=g)).to(torch.bfloat16).float()
        check(l, None, E, k, softmax, G, tg, (size, std))
        check(l, 0.25 * torch.randint(-1, 2, (E,), generator=g).float(), E, k, softmax, G, tg, (size, std))


@pytest.mark.parametrize("size", [(64, 8, 1, 1), (256, 8, 1, 1), (256, 8, 8, 4), (48, 31, 1, 1)], ids=str)
def test_all_experts_equal(size):
    """Lower indices come first; with one that is a little larger, that one."""
    E, k, G, tg = size
    for softmax, v in itertools.product((False, True), (0.0, 0.2, 15.625)):
        l = torch.full((T, E), v)
        check(l, None, E, k, softmax, G, tg, (size, v))
        l[torch.arange(T), torch.arange(T) * 5 % E] = torch.tensor(v) + 2.0 ** -26 if v < 1 else 16.0
        check(l, None, E, k, softmax, G, tg, (size, v))
