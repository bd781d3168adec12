"""Which kernel a call of the feed-forward block launches, and how many workgroups share its k: on the host."""
import random

import pytest

from launches import launches

torch = pytest.importorskip("torch")

P, FLOATS = 0x10000000, 2**24      # an address that is not read; a workspace's partial sums


def linear(M, N, K, ta="N", tb="T", pad=0, keep=False):
    z = (3, P, N, P, M) if keep else (1, 0, N, 0, 0)
    return "mi_linear", [ta, tb, 1, M, N, K, 1.0, P, (M if ta == "T" else K) + pad, P, (K if tb == "T" else N) + pad, 0, 0, 0, 1, 0.0, 0, 0, P, N, *z]


def gated(M, N, K, pad=0, keep=False):
    z = (P, N, P, M) * 2 if keep else (0, N, 0, 0) * 2
    return "mi_gated", [1, M, N, K, P, K + pad, P, K + pad, P, K + pad, 0, 0, 0, 2, 1, P, N, 3 if keep else 1, *z]


def plans(calls, folder, **state):
    """For each call (rows and columns of a tile, sums of a tile, tiles, workgroups to a tile), or None where no tile kernel runs."""
    out = []
    for (name, a), (rc, got) in zip(calls, launches([(name, a, state) for name, a in calls], folder)):
        assert rc == 0
        if got[-1].kernel != "lin_tile":
            out.append(None)
            continue
        BM, BN = got[-1].numbers[:2]
        cols = BN // 2 if name == "mi_gated" else BN
        M, N = a[1:3] if name == "mi_gated" else a[3:5]
        tiles = -(-M // BM) * -(-N // cols)
        assert got[-1].grid[0] % tiles == 0
        out.append((BM, cols, BM * BN, tiles, got[-1].grid[0] // tiles))
    return out


# Rows 2 bytes aligned, where the parts of as many workgroups as the card would take do not fit the workspace.
CASES = [linear(448, 4288, 16384, pad=1), linear(3128, 3184, 8192, "T", "T", pad=1), gated(228, 4432, 14603, pad=1), gated(353, 3111, 15040, pad=1)]


def test_the_plan_that_was_weighed_is_launched(tmp_path):
    for call, (_, _, floats, tiles, parts) in zip(CASES, plans(CASES, tmp_path)):
        assert parts > 1 or tiles >= 128, call
        assert tiles * parts * floats <= FLOATS


def test_long_k_is_shared_where_cus_would_stand_still(tmp_path):
    """A tile kernel on fewer than half of the 256 CUs has less than 32 blocks of 64 values of k; parts always fit."""
    rng = random.Random(7)

    def size(lo, hi):
        v = round(lo * (hi / lo) ** rng.random())
        return v // 16 * 16 if rng.random() < 0.6 and v >= 16 else v
    calls = []
    while len(calls) < 6000:
        M, N, K, pad, keep = size(1, 8192), size(16, 8192), size(16, 16384), rng.choice([0, 0, 1]), rng.random() < 0.25
        calls.append(gated(M, N, K, pad, keep) if rng.random() < 0.35 else linear(M, N, K, *rng.choice(["NT", "NT", "NN", "TN", "TT"]), pad, keep))
    shared = 0
    for (name, a), plan in zip(calls, plans(calls, tmp_path)):
        if plan is None:
            continue
        _, _, floats, tiles, parts = plan
        K = a[3] if name == "mi_gated" else a[5]
        shared += parts > 1
        assert parts > 1 or tiles >= 128 or K <= 32 * 64, (name, a)
        assert parts == 1 or tiles * parts * floats <= FLOATS, (name, a)
    assert shared > 500


@pytest.mark.parametrize("state", [{"capturing": 1}, {"no_memory": 1}])
def test_without_a_workspace_nothing_is_shared(tmp_path, state):
    calls = [*CASES, linear(70, 264, 8192, pad=1), linear(70, 264, 8192, "N", "N"), gated(70, 264, 8192, keep=True)]
    on = 0x5000     # a stream that has none yet
    calls = [(name, [*a, on]) for name, a in calls]
    got = plans(calls, tmp_path, **state)
    assert all(p is None or p[4] == 1 for p in got) and sum(p is not None for p in got) >= 6


@pytest.mark.parametrize("rows,cols", [(1000000, 64), (1000000, 128), (300000, 500), (200000, 136), (8192, 8192), (4096, 40), (70, 70), (1, 1)])
def test_backward_of_narrow_matrices_fills_the_card(tmp_path, rows, cols):
    """However few columns, rows are cut into parts for each CU: of 64 rows at least, of 512 where biases' gradients join them, which
    are no more than have room."""
    calls = [("mi_act_backward", [1, rows, cols, P, cols, 2, 1, P, cols, 0, 0, P, cols, 0, 0, 0.0, 0], {}),
             ("mi_gated_backward", [1, rows, cols, P, cols, 2, 1, P, cols, 0, 0, P, cols, 0, 0, P, cols, P, cols, 0, 0, 0.0, 0, 0], {}),
             ("mi_act_backward", [1, rows, cols, P, cols, 2, 1, P, cols, 0, 0, P, cols, 0, 0, 0.0, P], {}),
             ("mi_gated_backward", [1, rows, cols, P, cols, 2, 1, P, cols, 0, 0, P, cols, 0, 0, P, cols, P, cols, 0, 0, 0.0, P, P], {})]
    got = launches(calls, tmp_path)
    assert all(rc == 0 for rc, _ in got)
    for least, (_, each) in zip((64, 64, 512, 512), got):
        x, y, _ = each[-1].grid
        assert x == -(-cols // 128) and 1 <= y <= max(64, -(-rows // least))
        assert x * y >= min(256, x * (rows // least))
    assert all(2 * each[-1].grid[1] * cols <= FLOATS for _, each in got[2:])
