"""The launches of the language-model operators, from their host code alone (no GPU)."""
import subprocess

import pytest

import _launches as R

# (format, rows, labels, features, group): rows of features in LDS, many sizes per kernel
SWEEP = [(fmt, N, L, D, g) for fmt, g in ((2, 32), (3, 32), (3, 64), (3, 128)) for N in (1, 3, 7, 16, 19, 32)
         for L in (100, 5000, 70001) for D in [*range(256, 16385, 256), 32768, 65536]]


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


def test_every_kernel_is_reached(sweep, tmp_path):
    """The library holds no kernel of these operators that no call launches."""
    calls = [R.logprobs(t, N, V, k) for t in (0, 1, 2) for N in (1, 5000) for V in (100, 100000) for k in (0, 5)]
    calls += [R.logprobs_backward(t, 3, 1000, h) for t in (0, 1, 2) for h in (False, True)]
    calls += [c for t in (0, 1, 2) for act in range(4) for c in R.ckpt8(10, 64, t, act)]
    calls += [R.ckpt8_weight_grad(T, O, D) for T in (100, 16384) for O, D in ((64, 64), (2048, 4096))]
    rest, _ = R.record(tmp_path, calls)
    assert all(rc == 0 for rc, _ in rest)
    launched = {x[0] for _, one in sweep[0] + rest for x in one}
    nm = subprocess.run(["nm", "-D", "--defined-only", R.LIB], capture_output=True, text=True, check=True).stdout
    kernels = {ln.split()[-1] for ln in nm.splitlines()}
    kernels = {k for k in kernels if any(n in k for n in ("k_w4_", "k_logprobs", "k_ckpt8_", "k_wgrad_")) and "__device_stub__" not in k}
    assert len(kernels) > 60 and kernels >= launched
    assert kernels == launched, f"no call launches {sorted(kernels - launched)}"


def test_large_tile_shapes_take_the_large_tile(tmp_path):
    """The shapes of test_gpu_ckpt8_large_tile.py run the 256 x 256 weight-gradient tile, in one segment of
    tokens and in several."""
    from test_gpu_ckpt8_large_tile import SHAPES
    calls, _ = R.record(tmp_path, [R.ckpt8_weight_grad(*s) for s in [*SHAPES, (8005, 1800, 1824)]])
    segments = set()
    for (T, O, D), (rc, launches) in zip(SHAPES, calls):
        assert rc == 0 and "k_ckpt8_wgradILi4ELi4E" in launches[0][0], (T, O, D)
        segs = launches[0][1] / (-(-O // 256) * -(-D // 256))
        assert len(launches) == (1 if segs == 1 else 2)
        segments.add(segs)
    assert 1 in segments and len(segments) >= 3
