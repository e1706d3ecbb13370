"""The router on the GPU near the ends of its biases' range.  Tolerances as in
test_gpu_moe_block, but where a test derives its own."""

import numpy as np
import pytest
import torch

import block_scaled_precision_x32_gb300 as mxq
from tests.test_gpu_moe_block import BF16, F32, check_route, dev, normal

pytestmark = pytest.mark.gpu

LOWEST = float(torch.finfo(F32).min)


@pytest.fixture(scope="module")
def mx():
    return mxq.library()


# ------------------------------------------------------------------ router


def grouped_logits(rng, T, E, groups):
    """Ordinary rows, and among them rows of two groups that are alike, whose order only the index decides, and rows of groups a
    few units in the last place apart."""
    x = 1.5 * normal(rng, T, E)
    size = E // groups
    for i in range(groups):
        a, b = (slice(g * size, (g + 1) * size) for g in (i, (i + 3) % groups))
        x[i::29, b] = x[i::29, a]
        x[i + 11::29, b] = x[i + 11::29, a] * (1 + np.float32(2e-7))
    return x


@pytest.mark.parametrize("T", [70, 16389])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("value", [np.inf, LOWEST, -1e38, 3e38])
@pytest.mark.parametrize("topk_groups", [1, 4])
def test_route_of_groups_with_biases_at_the_ends(mx, T, score, value, topk_groups):
    """One expert, or all of a group, always or never to be chosen by its bias, in each group in turn."""
    E, groups = 128, 8
    rng = np.random.default_rng(topk_groups)
    x = dev(grouped_logits(rng, T, E, groups))
    for ordinary, places in ((0.0, range(groups)), (0.05, range(groups))) if T < 1000 else ((0.0, (0, 3, 7)), (0.05, (4,))):
        for g in places:
            for experts in (slice(16 * g + 5, 16 * g + 6), slice(16 * g, 16 * g + 16)):
                b = (ordinary * normal(rng, E)).astype(np.float32)
                b[experts] = value
                check_route(mx, x, 8, dev(b), score=score, groups=groups, topk_groups=topk_groups, group_top=2)


@pytest.mark.parametrize("T", [70, 16389])
@pytest.mark.parametrize("group_top", [1, 2])
def test_route_of_several_groups_with_biases_at_the_ends(mx, T, group_top):
    """More groups that are always, or never, to be chosen than there are places, or than there are others; a group of the
    type's lowest value is ahead of one without any expert."""
    E, groups = 128, 8
    rng = np.random.default_rng(group_top)
    x = grouped_logits(rng, T, E, groups)
    x[3::17, 64:80] = -np.inf
    for values in ((np.inf, np.inf, np.inf, np.inf, np.inf), (LOWEST, LOWEST, LOWEST, LOWEST, LOWEST), (3e38, 3.2e38, 3e38, np.inf, 3.4e38),
                   (LOWEST, -np.inf, LOWEST, np.inf, LOWEST), (np.inf, LOWEST, -3e38, -3.2e38, 2e38)):
        b = np.zeros(E, np.float32)
        for g, v in zip((1, 2, 4, 6, 7), values):
            b[16 * g: 16 * g + 16] = v
        for score in ("softmax", "sigmoid"):
            check_route(mx, dev(x), 4, dev(b), score=score, groups=groups, topk_groups=4, group_top=group_top)


def device_us(f, n=5):
    """Device time of f's launches, the least of n replays of a captured call."""
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        f()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            f()
        times = []
        for _ in range(n):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            graph.replay()
            b.record()
            torch.cuda.synchronize()
            times.append(1e3 * a.elapsed_time(b))
    return min(times)


@pytest.mark.parametrize("value", [-1e9, -1e30, LOWEST])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_a_group_masked_by_a_finite_bias_is_no_reason_to_look_twice(mx, value, score):
    """Three of eight groups are masked: the others' scores are as far apart as they were.  A second look with 48 bits at
    every token takes six times as long and more; four times is allowed."""
    T, E = 65536, 256
    rng = np.random.default_rng(8)
    x, b = 1.5 * normal(rng, T, E), (0.05 * normal(rng, E)).astype(np.float32)
    kw = dict(score=score, groups=8, topk_groups=4, group_top=2)
    logits, plain = dev(x), dev(b)
    b[32:64] = b[128:160] = b[224:] = value
    masked = dev(b)
    check_route(mx, logits[:20001], 8, masked, **kw)
    check_route(mx, logits[:900], 8, masked, **kw)
    for n in (T, 4096):
        few = logits[:n]
        slow, usual = (device_us(lambda: mx.moe_route(few, 8, bias=v, **kw)) for v in (masked, plain))
        assert slow < 4 * usual, (n, slow, usual)


@pytest.mark.parametrize("T", [70, 16389])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_of_groups_whose_own_error_is_large(mx, T, score):
    """A dropped group, or a kept one, whose score is a difference of large numbers: it is the one that has to be looked at
    again, and not the neighbour of the border.  Biases of +-2^k leave a sum of the two best that fp32 gives to 2^(k - 23) only."""
    E, groups = 128, 8
    rng = np.random.default_rng(5)
    x = dev(1.5 * normal(rng, T, E))
    for k in (12, 18, 21, 22):
        for g in range(groups):
            b = (0.05 * normal(rng, E)).astype(np.float32)
            b[16 * g: 16 * g + 16] = -np.float32(2.0**k)
            b[16 * g + 3] = np.float32(2.0**k + (0.5 if score == "sigmoid" else 0.0))
            check_route(mx, x, 8, dev(b), score=score, groups=groups, topk_groups=3, group_top=2)


@pytest.mark.parametrize("groups,topk_groups", [(8, 2), (4, 1)])
def test_a_router_that_keeps_two_warps_worth_of_experts(mx, groups, topk_groups):
    """32 kept experts are all candidates: they do not fit the lists of the four-lane kernel, whose tokens would all be taken
    again one by one (seven times as long).  One group more is the yardstick; three times its time is allowed."""
    T, E = 65536, 128
    rng = np.random.default_rng(2)
    x, b = dev(1.5 * normal(rng, T, E)), dev(0.05 * normal(rng, E))
    kw = dict(score="sigmoid", groups=groups, group_top=2, bias=b)
    check_route(mx, x[:16400], 4, b, score="sigmoid", groups=groups, topk_groups=topk_groups, group_top=2)
    crowded, usual = (device_us(lambda: mx.moe_route(x, 4, topk_groups=n, **kw)) for n in (topk_groups, topk_groups + 1))
    assert crowded < 3 * usual, (crowded, usual)


@pytest.mark.parametrize("T", [70, 16389])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,topk,more", [(60, 4, {}), (128, 8, {}), (256, 6, dict(groups=8, topk_groups=8, group_top=2)), (512, 1, {}), (128, 32, {})])
@pytest.mark.parametrize("level", [0.0, 1024.5])
def test_route_of_ties_at_the_last_place(mx, E, topk, more, score, level, T):
    """The last place is contested by experts that are alike, and by one with a higher index that is ahead of them by less than
    24 bits tell, beside the bias: the tie among the others does not settle the place."""
    rng = np.random.default_rng(E + topk)
    x = (-4.0 + 0.1 * normal(rng, T, E)).astype(np.float32)
    for t in range(T):
        ties = 2 + t % 5 if t % 7 else 40  # more than the candidates' lists hold
        at = np.sort(rng.permutation(E)[: min(topk - 1 + ties + 1, E)])
        x[t, at[: topk - 1]] = 3.0 + np.arange(topk - 1) / 16.0
        x[t, at[topk - 1:]] = 1.0
        x[t, at[-1]] = 1.0 + 2.0**-23 if level == 0.0 else 1.0 + 2.0**-14
    bias = np.full(E, level, np.float32)
    check_route(mx, dev(x), topk, dev(bias), score=score, **more)


@pytest.mark.parametrize("T", [70, 16389])
def test_route_of_ties_among_large_biases(mx, T):
    """Few different logits beside few different biases, whose fp32 sums with a score are often equal or one step apart."""
    rng = np.random.default_rng(4)
    for E, more in ((96, {}), (256, dict(groups=8, topk_groups=3, group_top=2))):
        x = dev(np.round(4 * normal(rng, T, E)) / 4, BF16)
        bias = dev(512.0 + rng.integers(0, 3, E) / 16384.0)
        for score in ("softmax", "sigmoid"):
            check_route(mx, x, 8, bias, score=score, **more)


@pytest.mark.parametrize("seed", range(8))
def test_route_of_forms_drawn_at_random(mx, seed):
    """Any number of experts, groups and choices; ties, experts out of service, and biases of every size."""
    rng = np.random.default_rng(seed)
    for turn in range(24):
        E = int(rng.choice([32, 60, 96, 128, 160, 192, 256, 512])) if turn % 2 else int(rng.integers(1, 1025))
        groups = int(rng.choice([g for g in range(1, 33) if E % g == 0]))
        size = E // groups
        kept, top = int(rng.integers(1, groups + 1)), int(rng.integers(1, min(2, size) + 1))
        topk = int(rng.integers(1, min(9 if turn % 4 else 33, kept * size + 1)))
        T = 16384 + turn if turn in (5, 17) else int(rng.integers(1, 400))
        x = (rng.choice([1e-3, 0.1, 1.5, 4.0]) * normal(rng, T, E)).astype(np.float32)
        if turn % 3 == 0:
            x[rng.random((T, E)) < 0.3] = -np.inf
        if turn % 5 == 0:
            x = np.round(2 * x) / 2
        if turn % 7 == 0:
            x += np.float32(20.0)
        x[rng.random(T) < 0.1] = 0
        b = (rng.choice([0.0, 0.05, 0.5]) * normal(rng, E)).astype(np.float32)
        for _ in range(int(rng.integers(0, 4))):
            v = rng.choice([np.inf, -np.inf, LOWEST, -LOWEST, 0.6 * LOWEST, 1e30, -1e30, 1e9, -1e9, 1e4, -1e4, 65536.5])
            g = int(rng.integers(groups))
            b[slice(g * size, (g + 1) * size) if rng.random() < 0.5 else rng.random(E) < 0.1] = v
        check_route(mx, dev(x, BF16 if turn % 4 == 1 else F32), topk, dev(b) if turn % 6 else None, score=("softmax", "sigmoid")[turn // 2 % 2],
                    groups=groups, topk_groups=kept, group_top=top, renormalize=bool(turn // 4 % 2))
