"""The host side of the norms and of the linear cross entropy (argument checks,
strides at the ends of 64 bits, workspace planning) under AddressSanitizer and
UndefinedBehaviorSanitizer, host code only. Every call has made-up addresses and
is invalid by construction, so nothing is ever enqueued; the test is skipped
where a GPU is visible.
"""
import os
import subprocess
import sys
import tempfile

import pytest
import torch

from optimizer_step_layeradam_amd import build as hip_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

DRIVER = r'''
import ctypes, itertools, random, sys
sys.path.insert(0, ROOT)
import optimizer_step_layeradam_amd as la
lib = la.load(LIB)
BASE, STEP = 0x7F0000000000, 0x1000000000
FAR = (0, 1, 7, (1 << 40) - 1, 1 << 40, (1 << 63) - 1, -1, -(1 << 63))
calls = 0

def at(k):
    return BASE + k * STEP

def refused(rc):
    global calls
    calls += 1
    assert rc not in (0, 5), (rc, lib.la_last_error())   # refused on the host
    assert lib.la_last_error()

# norms: every pair of strides, over row counts up to the largest; rstd lies in x
# (forward), dbias in dweight (backward)
for outer, inner in ((1, 1), (3, 1), (1, 3), (5, 7), (1 << 30, 1), (1, 1 << 30), (1 << 15, 1 << 15)):
    for cols in (1, 40, 1 << 14):
        n = la.make_norm(la.NORM_LAYER, outer, inner, cols, la.TYPE_BF16, la.TYPE_FP32, at(10), at(11))
        need = lib.la_norm_backward_workspace_bytes(ctypes.byref(n))
        assert need > 0
        for so, si in itertools.product(FAR, FAR):
            one, rows = la.Rows(at(0), so, si), la.Rows(at(2), inner * cols, cols)
            for io in (la.NormForwardIO(one, la.Rows(), rows, la.Rows(), None, at(0)),
                       la.NormForwardIO(rows, la.Rows(), one, la.Rows(), None, at(2))):
                refused(lib.la_norm_forward(ctypes.byref(n), ctypes.byref(io), None))
            for io in (la.NormBackwardIO(one, rows, la.Rows(), la.Rows(), at(3), at(4), at(5), at(5), 2),
                       la.NormBackwardIO(rows, rows, la.Rows(), one, at(3), at(4), at(5), at(5), 2)):
                refused(lib.la_norm_backward(ctypes.byref(n), ctypes.byref(io),
                                             ctypes.c_void_p(at(6)), need, None))
for sizes in ((-1, 1, 1), (1 << 62, 1 << 62, 1), (1, 1, (1 << 63) - 1), (1 << 30, 1 << 30, 4)):
    n = la.make_norm(la.NORM_RMS, *sizes, 0, 0)
    assert lib.la_norm_backward_workspace_bytes(ctypes.byref(n)) == -1

# the loss: planning over random sizes and workspaces; its loss lies in the weight
rng = random.Random(1)
def spread(most):
    return int(round(2 ** rng.uniform(0, most)))
def desc(tokens, hidden, vocab, **kw):
    d = dict(x=at(0), weight=at(1), targets=at(2), tokens=tokens, hidden=hidden, vocab=vocab,
             type=0, target_type=0, reduction=0, loss=at(1), dx=at(4), dweight=at(5))
    d.update(kw)
    return la.make_cross_entropy(**d)
def call(d, size):
    return lib.la_linear_cross_entropy(ctypes.byref(d), ctypes.c_void_p(at(0x100)), size, None)
sizes = [(1 << 20, 1 << 20, 1 << 20), (0, 1, 1), (1, 1, 1), (1 << 20, 1, 1), (0, 1 << 20, 1 << 20)]
sizes += [(rng.choice((0, 1)) * spread(17), spread(15), spread(19)) for _ in range(300)]
for tokens, hidden, vocab in sizes:
    for kw in ({}, {"dx": 0}, {"dweight": 0}, {"dx": 0, "dweight": 0}):
        d = desc(tokens, hidden, vocab, **kw)
        need = [lib.la_linear_cross_entropy_workspace_bytes(ctypes.byref(d), c)
                for c in (1, 0, 1000, (1 << 63) - 1)]
        assert need[0] <= need[2] <= need[3] and need[0] <= need[1], (tokens, hidden, vocab, need)
        for size in (-(1 << 63), 0, need[0] - 1, *need, (need[0] + need[1]) // 2, (1 << 63) - 1):
            refused(call(d, size))
for s in FAR:
    for name in ("x_row_stride", "weight_row_stride", "dx_row_stride", "dweight_row_stride"):
        refused(call(desc(1 << 20, 64, 1 << 20, **{name: s}), 1 << 50))
for sizes in ((-1, 4, 4), (4, (1 << 63) - 1, 4), (4, 4, 0)):
    assert lib.la_linear_cross_entropy_workspace_bytes(ctypes.byref(desc(*sizes)), 0) == -1
print("refusals", calls)
'''


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up device addresses; host-only")
def test_host_code_under_asan_and_ubsan():
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    runtime = subprocess.run(["bash", "-c", f"ls {rocm}/lib/llvm/lib/clang/*/lib/linux/"
                              "libclang_rt.asan-x86_64.so | head -1"],
                             capture_output=True, text=True).stdout.strip()
    if not runtime:
        pytest.skip("clang ASan runtime not found")
    with tempfile.TemporaryDirectory() as d:
        lib = os.path.join(d, "liblayeradam_san.so")
        sanitize = ["-Xarch_host", "-fsanitize=address",
                    "-Xarch_host", "-fsanitize=undefined",
                    "-Xarch_host", "-fno-sanitize-recover=undefined",
                    "-Xarch_host", "-fno-omit-frame-pointer"]
        hip_build.build(out=lib, extra=["-O1", "-g"] + sanitize)
        script = os.path.join(d, "driver.py")
        with open(script, "w") as f:
            f.write(f"ROOT = {ROOT!r}\nLIB = {lib!r}\n" + DRIVER)
        env = dict(os.environ, LD_PRELOAD=runtime,
                   ASAN_OPTIONS="detect_leaks=0:detect_odr_violation=0")
        r = subprocess.run([sys.executable, script], env=env, capture_output=True, text=True,
                           timeout=300)
        assert r.returncode == 0 and "refusals" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]
