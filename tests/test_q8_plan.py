"""The INT8 product's choice of form (coda_matmul_q8_plan), checked on the CPU: it plans no cluster
that does not fit the device, and its tiles keep to the kernel's limits."""

import random

import pytest


@pytest.fixture(scope="module")
def B():
    import __graft_entry__ as g

    g.build()
    from gemm_epilogue_fusion_gemm0_gb300 import binding

    return binding


WHOLE = (76, 36, 16)  # clusters of 2, 4 and 8 blocks that a whole device holds, about


def shapes(n):
    rng = random.Random(7)
    for _ in range(n):
        e = lambda lo, hi, step: max(step, int(2 ** rng.uniform(lo, hi)) // step * step)  # noqa: E731
        yield e(0, 14, 1), e(4, 16, 16), e(4, 16, 16)


def test_the_forms(B):
    for M, K, N, form in ((1, 4096, 28672, 1), (8, 8192, 8192, 1), (32, 4096, 4096, 1), (33, 4096, 4096, 2),
                          (24, 4096, 28672, 2), (1024, 4096, 14336, 2), (8192, 4096, 28672, 3)):
        assert B.coda_matmul_q8_plan(M, K, N, 152, 76, WHOLE)[0] == form


def test_limits(B):
    for M, K, N in shapes(2000):
        form, split, tokens, narrow = B.coda_matmul_q8_plan(M, K, N, 152, 76, WHOLE)
        assert form in (1, 2, 3)
        assert (form == 3) <= (M > 1024) and (form == 1) <= (M <= 32)
        assert split in ((1, 2, 4, 8) if form == 1 else (1, 2, 4) if form == 2 else (1,))
        if form == 2:
            # 256 columns and more go in two instructions of a multiple of 16 tokens
            assert 0 < tokens <= 384 and tokens % (32 if tokens > 256 else 16) == 0
            assert tokens <= 128 or not narrow
            # every part of a tile along K has work
            assert split <= -(-K // 64)
        else:
            assert tokens == 0 and not narrow


@pytest.mark.parametrize("clusters", [(76, 36, 0), (20, 0, 0), (1, 1, 1), (3, 1, 0)])
def test_clusters_that_do_not_fit_are_not_planned(B, clusters):
    for M, K, N in shapes(1000):
        form, split, _, _ = B.coda_matmul_q8_plan(M, K, N, 40, 18, clusters)
        assert form in (1, 2, 3)
        if split > 1:
            blocks = split if form == 1 else 2 * split
            assert clusters[{2: 0, 4: 1, 8: 2}[blocks]] > 0


def test_a_device_without_room_for_a_pair(B):
    """The other two forms need none; only a call that has no other form is refused."""
    for M, K, N in shapes(1000):
        form, split, _, _ = B.coda_matmul_q8_plan(M, K, N, 2, 0, (0, 0, 0))
        few = M <= 8 or (M <= 32 and B.coda_matmul_q8_plan(M, K, N, 152, 76, WHOLE)[0] == 1)
        assert form == (1 if few else 3 if M > 1024 else 0) and split == 1


def test_bad_arguments(B):
    for bad in ((0, 64, 64, 152, 76, WHOLE), (-1, 64, 64, 152, 76, WHOLE), (4, 24, 64, 152, 76, WHOLE),
                (4, 64, 64, 0, 76, WHOLE), (4, 64, 64, 152, -1, WHOLE), (4, 64, 64, 152, 76, (1, -1, 0))):
        with pytest.raises(ValueError):
            B.coda_matmul_q8_plan(*bad)
    assert B.raw().coda_matmul_q8_plan(4, 64, 64, 152, 76, None, None) == -1
