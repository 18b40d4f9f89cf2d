"""The stand-alone ops' host code on a CUDA runtime that does nothing (tests/c/fake_cuda.cpp): the calls that set the
ops up fail one at a time, in a child process each."""
import glob
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    """The library's own objects, linked with the fake runtime in place of CUDA's."""
    from flow_matching_action_loop_b200 import build
    build.build()
    out = str(tmp_path_factory.mktemp("fake") / "libflowloop_fake.so")
    fake = os.path.join(ROOT, "tests", "c", "fake_cuda.cpp")
    obj = out + ".o"
    cuda = os.path.join(os.path.dirname(os.path.dirname(build.NVCC)), "include")
    for cmd in (["g++", "-std=c++17", "-O1", "-fPIC", "-I", cuda, "-c", fake, "-o", obj],
                ["g++", "-shared", "-o", out, obj] + sorted(glob.glob(os.path.join(build.BUILD, "*.o")))):
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
    return out


PRELUDE = r'''
import ctypes
import flow_matching_action_loop_b200 as fr
from flow_matching_action_loop_b200 import _abi
lib, A = _abi.load_library(), 4096
lib.fake_fail.argtypes, lib.fake_fail.restype = [ctypes.c_char_p, ctypes.c_int], None


def code(call):
    try:
        call()
    except fr.FrError as e:
        return e.code, str(e)
    return 0, ""


attention = lambda: code(lambda: fr.fr_attention(A, A, A, A, 1, 8, 1, 8, 64, 64))
cache_ops = {
    "tree": lambda: code(lambda: fr.fr_attention_tree(A, A, A, A, A, A, A, 1, 8, 1, 4, 100, 128)),
    "weights": lambda: code(lambda: fr.fr_attention_weights(A, A, A, A, A, A, A, 1, 8, 1, 4, 100, 128)),
    "commit": lambda: code(lambda: fr.fr_cache_commit(A, A, A, A, A, A, A, 2 * A, 1, 1, 4, 100, 128, 1)),
    "evict": lambda: code(lambda: fr.fr_cache_evict(A, A, A, A, A, 2 * A, 2 * A, 2 * A, A, 1, 1, 100, 128, 1, 10, 2)),
}
'''


def child(library, body):
    r = subprocess.run([sys.executable, "-c", PRELUDE + body + '\nprint("CHILD_OK")'], cwd=ROOT, capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, FR_LIBRARY=library, PYTHONPATH=ROOT))
    assert r.returncode == 0 and "CHILD_OK" in r.stdout, r.stdout[-2000:] + r.stderr[-3000:]


def test_every_op_launches(library):
    child(library, r'''
assert attention()[0] == 0 and lib.fake_launches() == 1
for name, op in cache_ops.items():
    before = lib.fake_launches()
    assert op() == (0, ""), (name, op())
    assert lib.fake_launches() > before
assert fr.fr_ops_sync_status() == 0
''')


@pytest.mark.parametrize("call", ["cudaOccupancyMaxActiveClusters"])
def test_a_failure_of_the_cache_ops_set_up_is_theirs_alone(library, call):
    """Clusters cannot be queried: the cache ops report it, on every call; attention and the status word work."""
    child(library, f'''
lib.fake_fail(b"{call}", 1)
assert attention()[0] == 0
for name, op in cache_ops.items():
    rc, text = op()
    assert rc == fr.FR_ERR_CUDA and "fake" in text, (name, rc, text)
assert lib.fake_launches() == 1
assert fr.fr_ops_sync_status() == 0 and attention()[0] == 0
''')


@pytest.mark.parametrize("registers", [160, 176])
def test_attention_tree_refuses_a_build_whose_registers_do_not_add_up(library, registers):
    """Its kernel moves registers between warpgroups and would wait for good; nothing is launched."""
    child(library, f'''
lib.fake_registers({registers})
for _ in range(2):
    rc, text = cache_ops["tree"]()
    assert rc == fr.FR_ERR_UNSUPPORTED and "{registers} registers" in text, (rc, text)
assert lib.fake_launches() == 0
assert cache_ops["weights"]()[0] == 0 and cache_ops["commit"]()[0] == 0 and cache_ops["evict"]()[0] == 0
''')


def test_attention_tree_takes_a_cluster_per_unit_only_for_few_tiles(library):
    """Lengths are device data: a cluster's CTAs would run the tiles of one long sample alone while the others idle,
    however short the others are.  (units, tiles of 128 slots) -> CTAs of a cluster, with 148 / c of them resident."""
    child(library, r'''
for units, tiles, want in ((1, 7, 7), (8, 17, 9), (9, 65, 13), (16, 65, 9), (74, 9, 2), (74, 33, 2), (74, 35, 1), (74, 258, 1), (72, 258, 1),
                           (37, 65, 4), (37, 69, 1), (49, 51, 3), (49, 52, 1), (1, 129, 1), (200, 9, 1)):
    rc, text = code(lambda: fr.fr_attention_tree(A, A, A, A, A, A, A, units, 8, 1, 1, tiles * 128, 128, A, 40 << 20))
    assert rc == 0 and lib.fake_cluster() == want, (units, tiles, lib.fake_cluster(), text)
''')
