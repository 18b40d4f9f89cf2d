"""GPU: device bounds checks of the checked build (libflowloop_checked.so, -DFR_DEVICE_CHECKS).

In a child process that loads the checked build: the loop runs with no check firing and matches the
oracle; then a buffer is declared smaller than it is (fr_debug_limit_extent), so that the stores
past the declared extent are refused without any access leaving the real allocation.  The call
reports FR_ERR_DEVICE with the store site's where-code, and with the real extents restored the next
call gives the first result bit for bit.  Both executions are covered: the CUDA graph (GEMM residual
epilogue, 0x9001; attention output, 0x9010) and the persistent kernel (in-proj, 0xa021; attention
output, 0xa010).
"""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CHECKED = os.path.join(ROOT, "flow_matching_action_loop_b200", "libflowloop_checked.so")

CHILD = r'''
import numpy as np, torch
from flow_matching_action_loop_b200 import (FR_ERR_DEVICE, FR_EXEC_GRAPH, FR_EXEC_PERSISTENT, FR_PATH_TENSOR,
                                            FrError, fr_device_checks)
from oracle import oracle as O
from tests import _common as C
assert fr_device_checks()
cfg = C.get_config("b1_ragged_bf16")
inp = C.inputs("b1_ragged_bf16")
want = O.denoise(cfg, inp["weights"], inp["prefix_k"], inp["prefix_v"], inp["x0"])
for mode, cases in ((FR_EXEC_GRAPH, (("h", 64, "00009001"), ("obuf", 256, "00009010"))),
                    (FR_EXEC_PERSISTENT, (("h", 64, "0000a021"), ("obuf", 256, "0000a010")))):
    got, loop = C.run_library(cfg, inp, path=FR_PATH_TENSOR, exec_mode=mode)
    rel, cos = C.chunk_metrics(got, want)
    assert np.all(rel <= C.TOL_BF16_REL_L2) and np.all(cos >= C.TOL_BF16_COS), (mode, rel, cos)
    pk, pv, x0 = C.to_device(inp, cfg, torch)
    for buf, limit, where in cases:
        loop.limit_extent(buf, limit)
        loop.denoise(x0)
        try:
            loop.sync_status()
            raise AssertionError(f"{buf}: no bounds check fired")
        except FrError as e:
            assert e.code == FR_ERR_DEVICE, (buf, e)
            assert where in str(e), (buf, where, str(e))
        assert loop.sync_status() == 0            # read and cleared
        loop.limit_extent(buf, 0)
        again = loop.denoise(x0).cpu().numpy()
        assert loop.sync_status() == 0
        assert np.array_equal(again, got), buf
    loop.close()
print("CHECKS_OK")
'''


def _checked_library():
    if not os.path.exists(CHECKED):
        r = subprocess.run([sys.executable, os.path.join(ROOT, "flow_matching_action_loop_b200", "build.py"), "--checked"],
                           capture_output=True, text=True, timeout=1200)
        assert r.returncode == 0, r.stdout + r.stderr
    return CHECKED


def test_bounds_checks_fire_on_declared_extents_and_clear():
    env = dict(os.environ, FR_LIBRARY=_checked_library(), PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0 and "CHECKS_OK" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]


# The cache ops: for each buffer that an op stores into, half of its extent is declared.  What lies below it is as in
# an unlimited call, what lies at or past it stays as it was, and the status word has the store's where-code.
CHILD_CACHE = r'''
import torch
import flow_matching_action_loop_b200 as fr
from tests import test_cache_ops_gpu as T
assert fr.fr_device_checks()
ptr, s = T.ptr, T.stream()


def tree(spec):
    c = T.Case(*spec).device()
    def call():
        c.o.fill_(T.MARK), c.lse.fill_(T.MARK), c.scratch.fill_(0xFF)
        c.run()
        return {"o": c.o.clone(), "lse": c.lse.clone()}
    return {"o": torch.full_like(c.o, T.MARK), "lse": torch.full_like(c.lse, T.MARK)}, call, c


def weights():
    _, call, c = tree((3, 8, 2, 128, 40, 900, [800, 500, 3], "tree"))
    lse, acc0 = call()["lse"], torch.rand(c.B, c.Hkv, c.S).cuda()
    def run():
        acc = acc0.clone()
        fr.fr_attention_weights(ptr(c.dq), ptr(c.dk), ptr(lse), ptr(c.dlens), ptr(c.dwords), 0, ptr(acc), c.B, c.Hq, c.Hkv, c.N, c.S,
                                c.dh, s)
        return {"acc": acc}
    return {"acc": acc0}, run


B, Hkv, S, dh, N, keep = 6, 2, 300, 64, 20, 150
state = dict(k=torch.randn(B, Hkv, S, dh).cuda(), acc=torch.rand(B, Hkv, S).cuda(),
             pos=torch.stack([torch.stack([torch.randperm(S) for _ in range(Hkv)]) for _ in range(B)]).int().cuda())
state["v"] = -state["k"]
lens = torch.tensor([280, 270, 200, 160, 279, 280], dtype=torch.int32).cuda()
path = torch.arange(1, N + 1, dtype=torch.int32).repeat(B, 1).cuda()
npath = torch.full((B,), N - 1, dtype=torch.int32).cuda()


def commit():
    init = dict(state, lens=torch.full_like(lens, -7))
    def run():
        t = {n: x.clone() for n, x in init.items()}
        fr.fr_cache_commit(ptr(t["k"]), ptr(t["v"]), ptr(t["acc"]), ptr(t["pos"]), ptr(lens), ptr(path), ptr(npath), ptr(t["lens"]), B, Hkv,
                           N, S, dh, fr.FR_DTYPE_F32, s)
        return t
    return init, run


def evict():
    init = dict(k=state["k"], v=state["v"], acc=torch.full_like(state["acc"], -7.0), pos=torch.full_like(state["pos"], -7),
                src=torch.full((B, Hkv, keep), -7, dtype=torch.int32).cuda(), lens=torch.full_like(lens, -7))
    def run():
        t = {n: x.clone() for n, x in init.items()}
        fr.fr_cache_evict(ptr(t["k"]), ptr(t["v"]), ptr(state["acc"]), ptr(state["pos"]), ptr(lens), ptr(t["acc"]), ptr(t["pos"]),
                          ptr(t["lens"]), ptr(t["src"]), B, Hkv, S, dh, fr.FR_DTYPE_F32, keep, 20, s)
        return t
    return init, run


def check(what, init, run, buffers):
    full = run()
    assert fr.fr_ops_sync_status(s) == 0, what
    for buffer, names, unit, where in buffers:   # unit: the tensor's elements per element of the extent
        half = init[names[0]].numel() // unit // 2
        fr.fr_debug_limit_op_extent(buffer, half)
        got = run()
        try:
            fr.fr_ops_sync_status(s)
            raise AssertionError(f"{what} {buffer}: no check fired")
        except fr.FrError as e:
            assert e.code == fr.FR_ERR_DEVICE and where in str(e), (what, buffer, str(e))
        for n in got:
            g, f, i = got[n].flatten(), full[n].flatten(), init[n].flatten()
            at = half * unit if n in names else f.numel()
            assert torch.equal(g[:at], f[:at]) and torch.equal(g[at:], i[at:]), (what, buffer, n)
            assert n not in names or not torch.equal(f[at:], i[at:])
        fr.fr_debug_limit_op_extent(buffer, 0)
        again = run()
        assert fr.fr_ops_sync_status(s) == 0 and all(torch.equal(again[n], full[n]) for n in full), (what, buffer)


both = (("o", ("o",), 1, "00009020"), ("lse", ("lse",), 1, "00009021"))
for spec in ((40, 8, 8, 64, 1, 200, [150 + b for b in range(40)], "chain"),              # units whole
             (24, 32, 8, 128, 1, 4200, [4190 - 97 * b for b in range(24)], "chain"),     # cut: the merge stores
             (2, 16, 16, 64, 128, 4300, [4095, 3900], "chain")):                         # a cluster per unit
    init, run, c = tree(spec)
    check("tree", init, run, both)
init, run, c = tree((24, 32, 8, 128, 1, 4200, [4190 - 97 * b for b in range(24)], "chain"))
want = run()
fr.fr_debug_limit_op_extent("scratch", 16)
got = run()
try:
    fr.fr_ops_sync_status(s)
    raise AssertionError("scratch: no check fired")
except fr.FrError as e:
    assert e.code == fr.FR_ERR_DEVICE and "00009022" in str(e), str(e)
assert torch.all(c.scratch[64:] == 0xFF)
# rows whose parts were not written (0xFF: NaN) are left alone
assert bool(((got["o"] == want["o"]) | (got["o"] == T.MARK)).all()) and bool((got["o"] == T.MARK).any())
fr.fr_debug_limit_op_extent("scratch", 0)
check("weights", *weights(), (("acc", ("acc",), 1, "00009030"),))
check("commit", *commit(), (("rows", ("k", "v"), 4, "00009040"), ("acc", ("acc",), 1, "00009041"), ("pos", ("pos",), 1, "00009041"),
                            ("lens", ("lens",), 1, "00009042")))
check("evict", *evict(), (("rows", ("k", "v"), 4, "00009050"), ("acc", ("acc",), 1, "00009051"), ("pos", ("pos",), 1, "00009051"),
                          ("src", ("src",), 1, "00009052"), ("lens", ("lens",), 1, "00009053")))
print("CHECKS_OK")
'''


def test_bounds_checks_of_the_cache_ops():
    env = dict(os.environ, FR_LIBRARY=_checked_library(), PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", CHILD_CACHE], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "CHECKS_OK" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]


def test_cache_ops_under_the_checks():
    """The cache ops' own tests on the checked build: no check fires, and the results are the same."""
    env = dict(os.environ, FR_LIBRARY=_checked_library(), PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-m", "pytest", "tests/test_cache_ops_gpu.py", "-m", "gpu", "-x", "-q", "-p", "no:cacheprovider"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-1000:]
