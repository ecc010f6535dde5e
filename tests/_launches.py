"""Runs the library's host code with tests/launch_recorder.c in place of the HIP runtime's launch calls
(no GPU) and gives the launches of each call: `record(tmp, calls)` in a process of its own, since the
recorder has to be loaded before the library and before the HIP runtime."""
import json
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
LIB = os.path.join(os.path.dirname(HERE), "precision_label_chunk_amd", "libelmo_xmc.so")

# what runs in the other process: pointers are addresses that nothing looks at
_CHILD = r"""
import ctypes, json, sys
so, lib, calls = sys.argv[1], sys.argv[2], json.load(sys.stdin)
R = ctypes.CDLL(so, mode=ctypes.RTLD_GLOBAL)
R.recorder_get.restype = ctypes.c_char_p
R.recorder_most_changes.restype = ctypes.c_char_p
L = ctypes.CDLL(lib)
kind = {"p": ctypes.c_void_p, "i": ctypes.c_int, "l": ctypes.c_int64, "z": ctypes.c_size_t}
out, buf = [], (ctypes.c_uint64 * 4)()
for name, sig, args in calls:
    R.recorder_clear()
    f = getattr(L, name)
    f.argtypes = [kind[c] for c in sig]
    rc = f(*args)
    one = []
    for i in range(R.recorder_count()):
        k = R.recorder_get(i, buf).decode()
        one.append([k, *buf])
    out.append([rc, one])
n = ctypes.c_int()
most = R.recorder_most_changes(ctypes.byref(n)).decode()
json.dump({"calls": out, "most": [most, n.value]}, sys.stdout)
"""


def record(tmp, calls):
    """calls: (entry, signature of "p" pointer, "i" int, "l" int64, "z" size_t, arguments). Gives
    ([(status, [(kernel, grid, block, LDS bytes, the kernel's LDS limit), ..]), ..],
    (kernel whose limit was changed most often, number of changes))."""
    if not os.path.exists(LIB):
        import __graft_entry__
        __graft_entry__.build()
    so = os.path.join(str(tmp), "launch_recorder.so")
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", "-o", so, os.path.join(HERE, "launch_recorder.c"), "-ldl"], check=True)
    r = subprocess.run([sys.executable, "-c", _CHILD, so, LIB], input=json.dumps(calls), capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    d = json.loads(r.stdout)
    return [(rc, [tuple(x) for x in one]) for rc, one in d["calls"]], tuple(d["most"])


P = 4096                                     # an aligned address that nothing looks at


def w4_matvec(fmt, N, L, D, group=32, ytype=0):
    scales = P if fmt == 3 else None
    return ("elmo_w4_matvec", "pilipppilpilp", [P, fmt, L, D, group, scales, None, P, N, D, P, ytype, L, None])


def ckpt8_weight_grad(T, O, D, accumulate=0):
    return ("elmo_ckpt8_weight_grad", "plppliipipzp", [P, O, P, P, T, O, D, P, accumulate, P, 1 << 60, None])


def logprobs(ztype, N, V, k):
    return ("elmo_logprobs", "pilllpiipppppppzp",
            [P, ztype, N, V, V, P, 1, k, P, P, P, P, P, P, P, 1 << 60, None])


def logprobs_backward(ztype, N, V, entropy):
    return ("elmo_logprobs_backward", "pilllpippppppplp",
            [P, ztype, N, V, V, P, 1, P, P, P, P, P if entropy else None, None, 2 * P, V, None])


def ckpt8(T, D, type, act):
    """The calls of one activation: saved, restored, its gradient."""
    y = 2 * P if act else None
    save = ("elmo_ckpt8_save", "pililippplp", [P, type, T, D, D, act, P, P, y, D, None])
    load = ("elmo_ckpt8_load", "pplipilp", [P, P, T, D, P, type, D, None])
    grad = ("elmo_ckpt8_act_grad", "pililippplp", [P, type, T, D, D, act, P, P, 2 * P, D, None])
    return [save, load, grad] if act else [save, load]
