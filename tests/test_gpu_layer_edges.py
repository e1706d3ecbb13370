"""The FP8 linear layer and the mixture-of-experts operators at the ends of their
ranges, against 64-bit references from their definitions."""

import threading

import numpy as np
import pytest
import torch

import block_scaled_precision_x32_gb300 as mxq
from tests import layer_ref as ref
from tests.test_gpu_layer import BF16, F32, bytes_dev, call, close, make_rows, make_weight, operands

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    return mxq.library()


def test_a_part_of_the_sort_that_ends_at_the_last_32_bit_row(mx):
    """One choice whose part is rounded up to 2^31 - 1 rows: every row behind it is -1, and none in front of the order or behind
    it is touched."""
    rows, edge, canary = (1 << 31) - 1, 1024, 7
    room = torch.full((rows + 2 * edge,), canary, dtype=torch.int32, device="cuda")
    source = room[edge:edge + rows]
    i32 = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    order = mxq.MoeOrder(i32(2), source, i32(1, 1))
    mx.plan_moe_sort(torch.zeros(1, 1, dtype=torch.int32, device="cuda"), 1, order, align=rows)()
    assert order.offsets.tolist() == [0, rows] and order.slots.tolist() == [[0]]
    assert int(source[0]) == 0
    assert (room[:edge] == canary).all() and (room[edge + rows:] == canary).all()
    for piece in source[1:].split(1 << 28):
        assert (piece == -1).all()


@pytest.mark.parametrize("direction", ["fwd", "dgrad"])
@pytest.mark.parametrize("E,N", [(1, 1), (2, 1), (1, 2), (3, 5)])
@pytest.mark.parametrize("K", [1, 16, 33, 100])
@pytest.mark.parametrize("M", [1, 7, 300])
def test_grouped_products_of_the_smallest_weights(mx, direction, E, N, K, M):
    """Weights of one row, whose stride no copy uses and which need not be a multiple of anything."""
    rng = np.random.default_rng(1000 * M + 10 * K + E + N)
    off = np.linspace(0, M, E + 1).astype(np.int32)
    x, xs = make_rows(rng, M, K if direction == "fwd" else N)
    w, tile = make_weight(rng, E, N, K)
    av = ref.decode_rows(x, xs)
    n = N if direction == "fwd" else K
    want, S = np.zeros((M, n)), np.zeros((M, n))
    for e in range(E):
        wd, sl = ref.decode_weight(w[e], tile[e]), slice(off[e], off[e + 1])
        want[sl], S[sl] = ref.product(av[sl], wd if direction == "fwd" else wd.T)
    for dtype in (BF16, F32):
        y = call(mx, direction)(*map(bytes_dev, (x, xs, w, tile)), offsets=bytes_dev(off), out_dtype=dtype)
        close(y, want, S, av.shape[1], dtype)


def test_sorts_of_two_host_threads(mx):
    """Sorts of 512 and of 2048 experts take different amounts of shared memory; threads that call both at once, each on a
    stream of its own, get their results."""
    rng = np.random.default_rng(41)
    failed = []

    def sorts(experts):
        try:
            ids = rng_ids[experts]
            want = ref.moe_sort(ids, experts, 1)
            with torch.cuda.stream(torch.cuda.Stream()):
                order = mxq.MoeOrder(*(torch.empty(n, dtype=torch.int32, device="cuda") for n in (experts + 1, ids.size, ids.shape)))
                plan = mx.plan_moe_sort(bytes_dev(ids), experts, order)
                ready.wait()
                for _ in range(20):
                    for _ in range(500):
                        plan()
                    torch.cuda.current_stream().synchronize()
                for got, w in zip(order, want):
                    np.testing.assert_array_equal(got.cpu().numpy(), w)
        except BaseException as e:  # a thread's failure is the test's
            failed.append((experts, e))
            ready.abort()

    rng_ids = {e: rng.integers(0, e, (1025, 1)).astype(np.int32) for e in (512, 2048)}
    ready = threading.Barrier(2)
    threads = [threading.Thread(target=sorts, args=(e,)) for e in rng_ids]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
