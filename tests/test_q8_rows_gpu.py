"""The row kernels' forms: rows of more than 16384 columns that blocks walk through a ring (from 4
rows per SM on), either side of its limits, and the norm's calls with h and without, which the
binding does not make, in every form.  Definitions and tolerances as in test_q8_gpu.py."""

import os
import subprocess
import sys

import pytest
import torch

from test_q8_gpu import U, bf, check_codes, clean, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    import __graft_entry__ as g

    g.build()
    from gemm_epilogue_fusion_gemm0_gb300 import binding

    torch.cuda.set_device(0)
    return binding


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# Ring: (rows, columns); rows of a block in and out of step with the ring, its phases several times
# over (at 16392 columns the quantiser's ring holds 6 rows, the norm's 6 or 2), ragged last vectors.
RING = [(1300, 16392), (2501, 16392), (1301, 20008), (700, 28672), (1999, 28680), (611, 32760), (997, 32768)]
# Either side of the ring's limits in rows and columns, and rows too long for two of them (with z).
BESIDE = [(1300, 16384), (-1, 16392), (0, 16392), (1, 16392), (620, 32776)]


def shape(M, d):
    return (M if M > 1 else 4 * sms() + M), d


@pytest.mark.parametrize("M,n", RING + BESIDE)
def test_quant(B, M, n):
    M, n = shape(M, n)
    x = bf(randn(M + n, M, n, std=3.0))
    x[1] = 0
    x[M - 1] = 0
    q, s = B.coda_quant_q8(x)
    for rows in (slice(0, 320), slice(M - 320, M)):
        check_codes(q[rows], s[rows], x[rows].double(), 0)
    at = torch.arange(0, M, 37, device="cuda")
    check_codes(q[at], s[at], x[at].double(), 0)
    # every row against the quantiser in blocks, by its own definition of the row's largest value
    assert torch.equal(s, (x.abs().amax(1).double() / 127.0).float())
    assert torch.equal(q.abs().amax(1) == 127, x.abs().amax(1) > 0)
    clean(B)


@pytest.mark.parametrize("with_z", [False, True])
@pytest.mark.parametrize("M,d", RING + BESIDE)
def test_norm(B, M, d, with_z):
    M, d = shape(M, d)
    eps = 1e-5
    x, z = bf(randn(M + d, M, d, std=2.0)), (bf(randn(M + d + 1, M, d)) if with_z else None)
    gamma = bf(randn(d, d, std=0.3, mean=1.0))
    x[2] = 0
    if with_z:
        z[2] = 0
    h, q, s = B.coda_add_rmsnorm_q8(x, gamma, eps, z=z)
    if with_z:
        for at in range(0, M, 500):
            assert torch.equal(h[at:at + 500], bf(x[at:at + 500].float() + z[at:at + 500].float()))
    # a row at a time in fp64 costs 8 bytes a value: all rows, in pieces
    terms = 42 if d <= 32768 else d / 1024 + 10
    for at in range(0, M, 250):
        rows = slice(at, min(at + 250, M))
        v = x[rows].double() + (z[rows].double() if with_z else 0.0)
        check_codes(q[rows], s[rows], v * gamma.double(), 0,
                    scale_factor=1.0 / torch.sqrt((v * v).mean(1) + eps), rel=(terms / 2 + 12) * U)
    assert not q[2].any() and s[2] == 0
    clean(B)


FORMS = [(300, 264), (257, 1024), (100, 4104), (5, 32776), (700, 16392)]


@pytest.mark.parametrize("M,d", FORMS)
def test_norm_with_h_and_without(B, M, d):
    """z with h not wanted, and h without z (a copy of x): the same codes and scales, and nothing but
    the outputs written."""
    x, z, gamma = bf(randn(1, M, d)), bf(randn(2, M, d)), bf(randn(3, d, std=0.3, mean=1.0))
    for res in (None, z):
        _, q, s = B.coda_add_rmsnorm_q8(x, gamma, 1e-5, z=res)
        q2, s2 = torch.zeros_like(q), torch.zeros_like(s)
        h = None if res is not None else torch.full((M + 2, d), -7.0, device="cuda", dtype=torch.bfloat16)
        p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        rc = B.raw().coda_add_rmsnorm_q8(x.data_ptr(), p(res), gamma.data_ptr(), 1e-5, M, d,
                                         None if h is None else h[1:].data_ptr(), q2.data_ptr(), s2.data_ptr(),
                                         torch.cuda.current_stream().cuda_stream)
        assert rc == B.CODA_OK
        assert torch.equal(q, q2) and torch.equal(s, s2)
        if h is not None:
            assert torch.equal(h[1:-1], x) and (h[[0, -1]] == -7).all()
    clean(B)


def test_ring_writes_its_rows_alone(B):
    M, n = 1301, 16392
    x = bf(randn(1, M, n))
    want_q, want_s = B.coda_quant_q8(x)
    q = torch.full((M * n + 64,), 77, device="cuda", dtype=torch.int8)
    s = torch.full((M + 8,), -3.0, device="cuda")
    B.coda_quant_q8(x, q=q[32:32 + M * n].view(M, n), s=s[4:4 + M])
    assert torch.equal(q[32:32 + M * n].view(M, n), want_q) and torch.equal(s[4:4 + M], want_s)
    assert (q[:32] == 77).all() and (q[32 + M * n:] == 77).all() and (s[:4] == -3).all() and (s[4 + M:] == -3).all()


def test_ring_rows_of_extreme_values(B):
    """Rows of one block in turn: the smallest values, the largest, an infinity, a NaN, zeros; none
    reaches its neighbours in the ring."""
    M, n = 1220, 16400
    x = bf(randn(1, M, n))
    b = sms()  # the stride of a block's rows
    rows = {k: 3 + k * b for k in range(6)}
    x[rows[0]] = 2.0 ** -133
    x[rows[1]] = 3.0e38
    x[rows[2], 16399] = float("inf")
    x[rows[3], 0] = float("nan")
    x[rows[4]] = 0
    q, s = B.coda_quant_q8(x)
    assert (q[rows[0]] == 127).all() and (q[rows[1]] == 127).all()
    assert torch.isnan(s[[rows[2], rows[3]]]).all() and s[rows[4]] == 0 and not q[rows[4]].any()
    fine = torch.ones(M, dtype=torch.bool, device="cuda")
    fine[[rows[2], rows[3]]] = False
    assert torch.isfinite(s[fine]).all()
    check_codes(q[rows[5]][None], s[rows[5]][None], x[rows[5]][None].double(), 0)
    clean(B)


def test_ring_on_two_streams_and_from_graphs(B):
    M, d = 1000, 16424
    x = [bf(randn(i, M, d)) for i in (1, 2)]
    gamma = bf(randn(3, d, std=0.3, mean=1.0))
    want = [(*B.coda_quant_q8(t), *B.coda_add_rmsnorm_q8(t, gamma, 1e-5, z=x[0])) for t in x]
    streams = [torch.cuda.Stream() for _ in x]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [(*B.coda_quant_q8(t, stream=st), *B.coda_add_rmsnorm_q8(t, gamma, 1e-5, z=x[0], stream=st))
               for t, st in zip(x, streams)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for t in x:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append((*B.coda_quant_q8(t), *B.coda_add_rmsnorm_q8(t, gamma, 1e-5, z=x[0])))
        graphs.append(g)
    for g in graphs + graphs:
        g.replay()
    torch.cuda.synchronize()
    for w, a, b in zip(want, got, outs):
        for i, j, k in zip(w, a, b):
            assert torch.equal(i, j) and torch.equal(i, k)
    clean(B)


@pytest.mark.skipif(os.environ.get("CODA_CHECKED_BUILD") == "1", reason="is the child")
def test_rows_in_the_checked_build():
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.join(here, "test_q8_rows_gpu.py"), "-m", "gpu", "-x",
                        "-q", "-k", "not checked"], env=dict(os.environ, CODA_CHECKED_BUILD="1"),
                       capture_output=True, text=True, timeout=600, cwd=os.path.dirname(here))
    assert r.returncode == 0 and " passed" in r.stdout, (r.stdout + r.stderr)[-4000:]
