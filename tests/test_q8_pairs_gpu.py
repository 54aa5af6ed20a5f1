"""The INT8 product's form with two blocks per SM beside kernels that take tensor memory one block at a
time: the pair's blocks get the same columns (status word clean, nothing NaN) and the results stay."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    import __graft_entry__ as g

    g.build()
    from gemm_epilogue_fusion_gemm0_gb300 import binding

    torch.cuda.set_device(0)
    return binding


def test_pairs_beside_single_blocks(B):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    code = lambda *s: torch.randint(-128, 128, s, device="cuda", dtype=torch.int8, generator=g)  # noqa: E731
    bf = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    M, K, N = 40, 512, 24576  # 96 tiles: more than one wave of pairs, so two blocks per SM
    p = (code(M, K), torch.rand(M, device="cuda", generator=g), code(K, N), torch.rand(N, device="cuda", generator=g))
    want = B.coda_matmul_q8(*p)
    # sums of products below 2^14 * 512 = 2^23 are exact; then two fp32 roundings and one to bf16
    ref = (p[0].double() @ p[2].double()) * p[1].double()[:, None] * p[3].double()
    assert ((want.double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -22) * ref.abs()).all()
    f = (bf(130, 512), bf(512, 512), bf(130, 512), bf(512), bf(512, 1024))
    ys = [torch.empty_like(want) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    mode = B.coda_get_mma_mode()
    B.coda_set_mma_mode(0)  # single-CTA tiles
    try:
        want_f = B.coda_fwd(*f, 1e-5)
        outs = [torch.empty_like(t) for t in want_f]
        ws = B.workspace(B.coda_fwd_workspace_bytes(130, 512, 1024), "cuda")
        torch.cuda.synchronize()
        for _ in range(40):
            for y, st in zip(ys, streams):
                B.coda_matmul_q8(*p, y=y, stream=st)
            B.coda_fwd(*f, 1e-5, h=outs[0], r=outs[1], y=outs[2], ws=ws, stream=streams[2])
        torch.cuda.synchronize()
    finally:
        B.coda_set_mma_mode(mode)
    for y in ys:
        assert torch.equal(y, want)
    for a, b in zip(outs, want_f):
        assert torch.equal(a, b)
    st, detail = B.coda_get_device_status()
    assert st == B.CODA_OK, hex(detail)
