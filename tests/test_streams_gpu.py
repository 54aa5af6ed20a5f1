"""Calls on a stream other than the current one whose outputs and workspaces the binding allocates."""

import pytest
import torch

pytestmark = pytest.mark.gpu

BLOCK = 128


@pytest.fixture(scope="module")
def B():
    import __graft_entry__ as g

    g.build()
    from gemm_epilogue_fusion_gemm0_gb300 import binding

    torch.cuda.set_device(0)
    return binding


def inputs():
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    bf = torch.bfloat16
    rn = lambda *s, std=1.0: (torch.randn(*s, device="cuda", generator=g) * std).to(bf)  # noqa: E731
    M, d, N1, Dout = 200, 256, 512, 128
    t = {"x": rn(M, d), "z": rn(M, d), "W0": rn(d, d, std=d ** -0.5), "W1": rn(d, N1, std=d ** -0.5),
         "gamma": rn(d), "W2": rn(N1 // 2, Dout, std=0.1), "dout": rn(M, Dout), "dy": rn(M, N1), "y": rn(M, N1),
         "h": rn(M, d), "r": torch.rand(M, device="cuda", generator=g) + 0.5}
    code = lambda *s: torch.randint(-127, 128, s, device="cuda", dtype=torch.int8, generator=g)  # noqa: E731
    t["a_q"], t["W_q"] = code(1100, d), code(d, N1)
    t["a_s"], t["w_s"] = torch.rand(1100, device="cuda", generator=g), torch.rand(N1, device="cuda", generator=g)
    t["y_q"], t["y_s"] = code(M, N1), torch.rand(M, N1 // BLOCK, device="cuda", generator=g) * 0.02
    return t


CALLS = {
    "quant": lambda B, t, st: B.coda_quant_q8(t["x"], block=BLOCK, stream=st),
    "dequant": lambda B, t, st: (B.coda_dequant_q8(t["y_q"], t["y_s"], block=BLOCK, stream=st),),
    "norm": lambda B, t, st: B.coda_add_rmsnorm_q8(t["x"], t["gamma"], 1e-5, z=t["z"], stream=st),
    "product": lambda B, t, st: (B.coda_matmul_q8(t["a_q"], t["a_s"], t["W_q"], t["w_s"], stream=st),),
    "bwd_q8": lambda B, t, st: B.coda_bwd_swiglu_dgrad_q8(t["dout"], t["W2"], t["y_q"], t["y_s"], t["W1"], t["h"],
                                                          t["r"], t["gamma"], want_a=True, stream=st),
    "fwd": lambda B, t, st: B.coda_fwd(t["x"], t["W0"], t["z"], t["gamma"], t["W1"], 1e-5, stream=st),
    "fwd_swiglu": lambda B, t, st: B.coda_fwd_swiglu(t["x"], t["W0"], t["z"], t["gamma"], t["W1"], 1e-5,
                                                     want_y=True, stream=st),
    "dgrad": lambda B, t, st: (B.coda_bwd_dgrad(t["dy"], t["W1"], t["h"], t["r"], t["gamma"], stream=st),),
    "swiglu_dgrad": lambda B, t, st: B.coda_bwd_swiglu_dgrad(t["dout"], t["W2"], t["y"], t["W1"], t["h"], t["r"],
                                                             t["gamma"], stream=st),
    "bwd": lambda B, t, st: tuple(B.coda_bwd(t["dy"], t["x"], t["W0"], t["W1"], t["h"], t["r"], t["gamma"],
                                             stream=st).values()),
}


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("name", CALLS)
def test_memory_still_in_use_on_the_current_stream_is_not_taken(B, name, raw):
    """Blocks freed on the current stream whose reads and writes there are still to come: the
    call's outputs and workspace, of the same sizes, must not lie in them."""
    t = inputs()
    side = torch.cuda.Stream()
    want = [o.clone() for o in CALLS[name](B, t, None)]
    sizes = [o.numel() * o.element_size() for o in want]
    sizes += [1 << k for k in range(12, 24)]  # whatever the workspace's size, a block it would fit
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = [torch.full((n,), 7, device="cuda", dtype=torch.uint8) for n in sizes for _ in range(2)]
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)  # some 25 ms
    copies = []
    for i, h in enumerate(held):
        if i % 2:
            h.fill_(9)  # a write to come
        else:
            copies.append(h.clone())  # a read to come
    del held, h
    got = CALLS[name](B, t, side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert all((c == 7).all() for c in copies)
    st, detail = B.coda_get_device_status()
    assert st == B.CODA_OK, hex(detail)


@pytest.mark.parametrize("name", CALLS)
def test_outputs_are_kept_for_the_current_stream(B, name):
    """An output freed while the current stream still has to read it is not handed to the
    other stream's next call."""
    t = inputs()
    side = torch.cuda.Stream()
    want = [o.clone() for o in CALLS[name](B, t, None)]
    torch.cuda.synchronize()
    got = CALLS[name](B, t, side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(50_000_000)
    late = [o.clone() for o in got]
    del got
    zero = {k: torch.zeros_like(v) for k, v in t.items()}  # another call, other values, the same sizes
    side.synchronize()
    CALLS[name](B, zero, side)
    torch.cuda.synchronize()
    for a, b in zip(late, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", CALLS)
def test_captured_on_a_forked_stream(B, name):
    t = inputs()
    want = [o.clone() for o in CALLS[name](B, t, None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        got = CALLS[name](B, t, side)
        main.wait_stream(side)
        out = [o + 0 for o in got]
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, want):
        assert torch.equal(a, b)


def test_the_current_stream_by_its_own_name(B):
    """stream= naming the current stream is the plain call, by object or by handle; 1 is CUDA's
    handle of the legacy default stream."""
    t = inputs()
    want = CALLS["norm"](B, t, None)
    cur = torch.cuda.current_stream()
    for st in (cur, cur.cuda_stream, 0, 1):
        for a, b in zip(CALLS["norm"](B, t, st), want):
            assert torch.equal(a, b)
    with torch.cuda.stream(torch.cuda.Stream()) as _:
        torch.cuda.current_stream().wait_stream(cur)
        got = CALLS["norm"](B, t, torch.cuda.current_stream())
        torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_a_stream_of_another_library(B):
    """Any object that names its handle and its device."""

    class Stream:
        device = torch.device("cuda", 0)

        def __init__(self, handle):
            self.cuda_stream = handle

    t = inputs()
    side = torch.cuda.Stream()
    for name in ("norm", "fwd"):
        want = CALLS[name](B, t, None)
        torch.cuda.synchronize()
        got = CALLS[name](B, t, Stream(side.cuda_stream))
        side.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
