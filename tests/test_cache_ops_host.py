"""The cache ops' argument checks and host utilities (no GPU): refused before any device work."""
import numpy as np
import pytest

from tests import _cache as R


@pytest.fixture(scope="module")
def abi():
    from flow_matching_action_loop_b200 import _abi
    _abi.load_library()
    return _abi


A = 4096   # an aligned address that nothing reads


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 64, 65, 256])
def test_tree_mask_is_the_ancestors(abi, n):
    rng = np.random.default_rng(n)
    parents = [int(rng.integers(-1, i)) if i else -1 for i in range(n)]
    want = np.zeros((n, n), bool)
    for i in range(n):
        j = i
        while j >= 0:
            want[i, j] = True
            j = parents[j]
    got = abi.fr_tree_mask(parents)
    assert got.shape == (n, -(-n // 32)) and np.array_equal(got, R.words_of(want))
    assert np.array_equal(R.sees(got, n), want)


def test_tree_mask_refusals(abi):
    for parents, code in (([0], abi.FR_ERR_ARG), ([-1, 1], abi.FR_ERR_ARG), ([-1, -2], abi.FR_ERR_ARG), ([], abi.FR_ERR_UNSUPPORTED),
                          ([-1] * 257, abi.FR_ERR_UNSUPPORTED)):
        with pytest.raises(abi.FrError) as e:
            abi.fr_tree_mask(parents)
        assert e.value.code == code


# B, Hq, Hkv, N, S_max, dh
SIZES = [((0, 8, 1, 4, 100, 128), "ARG"), ((1, 0, 1, 4, 100, 128), "ARG"), ((1, 8, 0, 4, 100, 128), "ARG"), ((1, 8, 1, 0, 100, 128), "ARG"),
         ((1, 8, 1, 4, 0, 128), "ARG"), ((1, 8, 1, 4, 100, -1), "ARG"), ((1, 8, 3, 4, 100, 128), "UNSUPPORTED"),
         ((1, 8, 1, 4, 100, 96), "UNSUPPORTED"), ((1, 8, 1, 257, 1000, 128), "UNSUPPORTED"), ((1, 8, 1, 4, (1 << 24) + 1, 128), "UNSUPPORTED"),
         ((4097, 8, 1, 4, 100, 128), "UNSUPPORTED"), ((1, 1025, 1, 4, 100, 128), "UNSUPPORTED"), ((1, 8, 1, 4, 3, 128), "SHAPE"),
         # 4096 samples x 2048 row tiles x 257 key tiles: more than an int counts
         ((4096, 1024, 1, 256, 257 * 128, 64), "UNSUPPORTED"), ((4096, 1024, 1, 256, 1 << 24, 64), "UNSUPPORTED")]


@pytest.mark.parametrize("sizes,code", SIZES)
def test_attention_sizes_refused(abi, sizes, code):
    lib, want = abi.load_library(), getattr(abi, "FR_ERR_" + code)
    assert lib.fr_attention_tree(A, A, A, A, A, A, A, *sizes, A, 1 << 30, None) == want, abi.fr_last_error()
    assert lib.fr_attention_weights(A, A, A, A, A, A, A, *sizes, None) == want, abi.fr_last_error()
    assert abi.fr_attention_tree_scratch_bytes(*sizes) == 0


def test_attention_pointers_refused(abi):
    lib, sizes = abi.load_library(), (1, 8, 1, 4, 100, 128)
    for i in (0, 1, 2, 3, 5):   # mask and lse may be NULL
        for bad in (None, A + 2):
            args = [A] * 7
            args[i] = bad
            assert lib.fr_attention_tree(*args, *sizes, A, 1 << 30, None) == abi.FR_ERR_ARG
    for i in (0, 1, 2, 3, 6):
        for bad in (None, A + 2):
            args = [A] * 7
            args[i] = bad
            assert lib.fr_attention_weights(*args, *sizes, None) == abi.FR_ERR_ARG
    for i, bad in ((4, A + 1), (6, A + 1), (5, A + 16), (0, A + 8)):   # o is stored 32 bytes at a time
        args = [A] * 7
        args[i] = bad
        assert lib.fr_attention_tree(*args, *sizes, A, 1 << 30, None) == abi.FR_ERR_ARG


# B, Hkv, N, S_max, dh, dtype
MOVES = [((0, 1, 4, 100, 128, 1), "ARG"), ((1, 0, 4, 100, 128, 1), "ARG"), ((1, 1, 0, 100, 128, 1), "ARG"), ((1, 1, 4, 0, 128, 1), "ARG"),
         ((1, 1, 4, 100, 0, 1), "ARG"), ((1, 1, 4, 100, 128, 2), "ARG"), ((1, 1, 4, 100, 520, 1), "UNSUPPORTED"),
         ((1, 1, 4, 100, 12, 1), "UNSUPPORTED"), ((1, 1, 257, 1000, 128, 1), "UNSUPPORTED"), ((4097, 1, 4, 100, 128, 1), "UNSUPPORTED"),
         ((1, 1025, 4, 100, 128, 1), "UNSUPPORTED"), ((1, 1, 4, (1 << 24) + 1, 128, 1), "UNSUPPORTED"), ((1, 1, 5, 4, 128, 1), "SHAPE")]


@pytest.mark.parametrize("sizes,code", MOVES)
def test_commit_sizes_refused(abi, sizes, code):
    lib = abi.load_library()
    ptrs = [A * (i + 1) for i in range(8)]
    assert lib.fr_cache_commit(*ptrs, *sizes, None) == getattr(abi, "FR_ERR_" + code), abi.fr_last_error()


def test_move_pointers_refused(abi):
    lib = abi.load_library()
    for i in (0, 1, 4, 5, 6, 7):
        for bad in (None, A + 2):
            ptrs = [A * (j + 1) for j in range(8)]
            ptrs[i] = bad
            assert lib.fr_cache_commit(*ptrs, 1, 1, 4, 100, 128, 1, None) == abi.FR_ERR_ARG
    ptrs = [A * (j + 1) for j in range(8)]
    ptrs[7] = ptrs[4]   # lens_out is lens
    assert lib.fr_cache_commit(*ptrs, 1, 1, 4, 100, 128, 1, None) == abi.FR_ERR_ARG
    for i in range(9):
        for bad in (None, A + 2):
            ptrs = [A * (j + 1) for j in range(9)]
            ptrs[i] = bad
            assert lib.fr_cache_evict(*ptrs, 1, 1, 100, 128, 1, 10, 2, None) == abi.FR_ERR_ARG
    for i, j in ((5, 2), (6, 3), (7, 4)):   # an output that is its input
        ptrs = [A * (n + 1) for n in range(9)]
        ptrs[i] = ptrs[j]
        assert lib.fr_cache_evict(*ptrs, 1, 1, 100, 128, 1, 10, 2, None) == abi.FR_ERR_ARG


# B, Hkv, S_max, dh, dtype, keep, recent
EVICTS = [((0, 1, 100, 128, 1, 10, 2), "ARG"), ((1, 1, 100, 128, 3, 10, 2), "ARG"), ((1, 1, 100, 128, 1, 0, 0), "ARG"),
          ((1, 1, 100, 128, 1, 10, -1), "ARG"), ((1, 1, 100, 128, 1, 101, 2), "SHAPE"), ((1, 1, 100, 128, 1, 10, 11), "SHAPE"),
          ((1, 1, (1 << 19) + 1, 128, 1, 10, 2), "UNSUPPORTED"), ((1, 1, 100, 4, 1, 10, 2), "UNSUPPORTED")]


@pytest.mark.parametrize("sizes,code", EVICTS)
def test_evict_sizes_refused(abi, sizes, code):
    lib = abi.load_library()
    ptrs = [A * (i + 1) for i in range(9)]
    assert lib.fr_cache_evict(*ptrs, *sizes, None) == getattr(abi, "FR_ERR_" + code), abi.fr_last_error()


def test_attention_scratch(abi):
    """40 MiB cover every size; what one tile holds needs none."""
    most = 0
    for dh in (64, 128, 256):
        assert abi.fr_attention_tree_scratch_bytes(2, 8, 1, 16, 128, dh) == 0
        for sizes in ((1, 8, 1, 1, 1 << 24), (4096, 1024, 1, 256, 1 << 20), (64, 32, 8, 64, 4096), (1, 128, 1, 256, 999)):
            B, Hq, Hkv, N, S = sizes
            n = abi.fr_attention_tree_scratch_bytes(B, Hq, Hkv, N, S, dh)
            assert n % 16 == 0
            most = max(most, n)
    assert most <= 40 << 20
    lib = abi.load_library()
    n = abi.fr_attention_tree_scratch_bytes(1, 8, 1, 4, 1000, 128)
    if n:
        for scratch, size in ((None, n), (A, n - 1)):
            assert lib.fr_attention_tree(A, A, A, A, A, A, A, 1, 8, 1, 4, 1000, 128, scratch, size, None) == abi.FR_ERR_SHAPE


def test_wait_limit_refused(abi):
    with pytest.raises(abi.FrError) as e:
        abi.fr_ops_set_wait_limit(10 ** 10 + 1)
    assert e.value.code == abi.FR_ERR_ARG
    abi.fr_ops_set_wait_limit(0)


def test_declared_extents_need_the_checked_build(abi):
    for name, code in (("o", abi.FR_ERR_UNSUPPORTED), ("rows", abi.FR_ERR_UNSUPPORTED)):
        with pytest.raises(abi.FrError) as e:
            abi.fr_debug_limit_op_extent(name, 10)
        assert e.value.code == code


@pytest.mark.parametrize("sizes", [(1, 8, 1, 4, 1000, 128), (1, 8, 1, 1, 513, 64), (4, 16, 2, 24, 2148, 256)])
def test_attention_scratch_too_small_is_refused(abi, sizes):
    lib, n = abi.load_library(), abi.fr_attention_tree_scratch_bytes(*sizes)
    assert n > 0
    for scratch, size in ((None, n), (A, n - 1), (A, 0)):
        assert lib.fr_attention_tree(A, A, A, A, A, A, A, *sizes, scratch, size, None) == abi.FR_ERR_SHAPE, abi.fr_last_error()
