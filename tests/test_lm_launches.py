"""The launches of the language-model operators, from their host code alone (no GPU)."""
import pytest

import _launches as R

# (format, rows, labels, features, group): rows of features in LDS, many sizes per kernel
SWEEP = [(fmt, N, L, D, g) for fmt, g in ((2, 32), (3, 32), (3, 64), (3, 128)) for N in (1, 3, 7, 16, 19, 32)
         for L in (100, 5000, 70001) for D in range(256, 16385, 256)]


@pytest.fixture(scope="module")
def sweep(tmp_path_factory):
    calls = [R.w4_matvec(*c, ytype=y) for c in SWEEP for y in (0, 1)]
    return R.record(tmp_path_factory.mktemp("launches"), calls)


def test_lds_limit_does_not_depend_on_the_call(sweep):
    """A kernel's limit on dynamic LDS belongs to the process: a call that set it to its own size could
    lower it between another thread's setting and launch. It is raised once, to a constant, and every
    launch lies within it."""
    calls, (kernel, changes) = sweep
    over = 0
    for rc, launches in calls:
        assert rc == 0 and launches
        for name, grid, block, lds, limit in launches:
            assert lds <= limit <= 160 << 10, name
            over += lds > 64 << 10
    assert over > 100                        # (the sweep does reach launches that need the raised limit)
    assert changes == 1, f"the limit of {kernel} was changed {changes} times"
