"""What the kernels behind log probabilities from features, 8-bit integer products and dropout are built and launched
with (no GPU): registers and LDS from the compiler's report under the library's own flags, launches from the host
code alone."""
import os
import re
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

import _launches as R
from precision_label_chunk_amd import build as B

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CSRC = os.path.join(os.path.dirname(B.__file__), "csrc_lm")
SOURCES = ["linear_logprobs_kernels.hip", "i8_kernels.hip", "dropout_kernels.hip"]
NAMES = ("k_lin_", "k_i8_", "k_dropout_")
P = R.P


def forward(type, N, V, D, M=1):
    return ("elmo_linear_logprobs", "ppillillpippppzp", [P, P, type, N, V, D, D, D, P, M, P, P, P, P, 1 << 60, None])


def backward(type, N, V, D, M=1, chunk=0, dx=P, dw=P):
    return ("elmo_linear_logprobs_backward", "ppillillpipppppilpililpzp",
            [P, P, type, N, V, D, D, D, P, M, P, P, P, P, dx, 1, D, dw, 1, D, 0, chunk, P, 1 << 60, None])


def quantize(type, N, D):
    return ("elmo_i8_quantize", "pililppp", [P, type, N, D, D, P, P, None])


def matmul(type, N, L, D):
    return ("elmo_i8_matmul", "ppppllipilpzp", [P, P, P, P, N, L, D, P, type, L, P, 1 << 60, None])


def dropout(type, T, D, ld, residual):
    return ("elmo_dropout", "pilllpldllplplp", [P, type, T, D, ld, P if residual else None, ld, 0.5, 1, 2, None, 0, P, ld, None])


@pytest.fixture(scope="module")
def record(tmp_path_factory):
    def run(calls):
        with pytest.MonkeyPatch.context() as m:          # (one of these entries takes a double)
            m.setattr(R, "_CHILD", R._CHILD.replace('"z": ctypes.c_size_t', '"z": ctypes.c_size_t, "d": ctypes.c_double'))
            out, _ = R.record(tmp_path_factory.mktemp("launches"), calls)
        assert all(rc == 0 for rc, _ in out), [c for c, (rc, _) in zip(calls, out) if rc]
        return out
    return run


SIZES = [(N, V, D) for N in (1, 30, 200, 700, 5000) for V in (300, 5000, 131072) for D in (64, 768, 4096)]


def test_every_kernel_is_reached(record):
    """The library holds no kernel of these operators that no call launches, and no launch that cannot run."""
    calls = [f(t, *s) for t in (1, 2) for s in SIZES for f in (forward, backward)]
    calls += [backward(1, 20000, 300, 64), backward(1, 0, 300, 64)]
    calls += [quantize(t, 100, D) for t in (0, 1, 2) for D in (64, 4096)]
    calls += [matmul(t, N, L, D) for t in (0, 1, 2) for N in (1, 20, 33, 100, 700, 5000) for L in (300, 10000, 3000000) for D in (64, 768, 8192)
              if N * L < 1 << 31]
    calls += [matmul(0, 512, 2048, 65536)]
    calls += [dropout(t, 100, D, ld, r) for t in (0, 1, 2) for D, ld in ((64, 64), (63, 64)) for r in (False, True)]
    launched = {}
    for _, one in record(calls):
        for name, grid, block, lds, limit in one:
            assert grid >= 1 and lds == 0, name
            launched.setdefault(name, set()).add(block)
    assert all(len(b) == 1 for b in launched.values()), "a kernel launched with several block sizes"
    nm = subprocess.run(["nm", "-D", "--defined-only", R.LIB], capture_output=True, text=True, check=True).stdout
    kernels = {ln.split()[-1] for ln in nm.splitlines()}
    kernels = {k for k in kernels if any(n in k for n in NAMES) and "__device_stub__" not in k}
    assert len(kernels) >= 60
    assert kernels == set(launched), f"not launched: {sorted(kernels - set(launched))}"


def _shape(name):
    return re.search(r"TileShapeILi(\d)E", name).group(1)


def test_tile_shapes_follow_the_sizes(record):
    """Few rows and labels take small tiles, many large ones."""
    small, large = record([forward(1, 30, 1000, 256), forward(1, 4096, 131072, 768)])
    assert _shape(small[1][0][0]) == "1" and _shape(large[1][0][0]) == "4"
    one, = record([backward(1, 4096, 131072, 768)])
    assert {_shape(x[0]) for x in one[1] if "TileShape" in x[0]} == {"4"}


def test_pieces_and_gradients_asked_for(record):
    """A launch pair per piece; one that is not asked for is not computed."""
    whole, pieces, dx, dw = record([backward(1, 700, 5000, 64, chunk=5120), backward(1, 700, 5000, 64, chunk=1000),
                                    backward(1, 700, 5000, 64, dw=None), backward(1, 700, 5000, 64, dx=None)])

    def count(calls, what):
        return sum(what in x[0] for x in calls[1])
    assert count(whole, "grad_logits") == count(whole, "products") == 1
    assert count(pieces, "grad_logits") == count(pieces, "products") == 5
    assert count(dx, "k_lin_sum") == 1 and count(dw, "grad_logits") >= 1


@pytest.mark.skipif(not shutil.which(HIPCC) and not os.path.exists(HIPCC), reason="hipcc not installed")
def test_kernels_stay_in_registers(tmp_path):
    """No scratch memory, and room for the blocks that the launch rules put on a compute unit."""
    def report(src):
        cmd = [HIPCC, *B.HIPCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", os.path.join(str(tmp_path), src + ".o"),
               "-Rpass-analysis=kernel-resource-usage"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        out, name = {}, None
        for ln in r.stderr.splitlines():
            m = re.search(r"Function Name: (\S+)", ln)
            if m:
                name = m.group(1)
                out[name] = {}
            for key, pat in (("scratch", r"ScratchSize \[bytes/lane\]: (\d+)"), ("waves", r"Occupancy \[waves/SIMD\]: (\d+)"),
                             ("lds", r"LDS Size \[bytes/block\]: (\d+)")):
                m = re.search(pat, ln)
                if m and name:
                    out[name][key] = int(m.group(1))
        return out
    with ThreadPoolExecutor(len(SOURCES)) as ex:
        kernels = {k: v for rep in ex.map(report, SOURCES) for k, v in rep.items()}
    assert len(kernels) >= 60
    assert not {k: v for k, v in kernels.items() if v["scratch"]}
    need = {"4": (1, 2), "2": (2, 2), "1": (4, 4)}           # shape: blocks per compute unit, waves per SIMD
    for k, v in kernels.items():
        if "TileShape" in k:
            blocks, waves = need[_shape(k)]
            assert blocks * v["lds"] <= 160 << 10 and v["waves"] >= waves, (k, v)
