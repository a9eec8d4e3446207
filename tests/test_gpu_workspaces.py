"""What calls on one stream share: a workspace, counters, and graphs that hold their addresses."""
import numpy as np
import pytest
import torch

import kda_inputs as KI
import prefill_kda_chunk_gb300 as K
from test_gpu_cache import F32, I32, built, cache_case, i32, make  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------- calls that write to the workspace

def heads_gradient():
    r = make(1)
    x, dy, w = r(700, 5, 128), r(700, 5, 128), 1 + 0.1 * r(128, dtype=F32)
    return lambda: K.qk_norm_rope_backward(x, None, dy, None, w)


def attention():
    case = cache_case([9000, 77], 16, 2, 128, 64)
    return lambda: K.paged_decode_fp8(*case)


def plan():
    B = 5000   # more slots than one launch takes
    lens = torch.arange(B, dtype=I32, device="cuda") % 40
    table = torch.arange(4 * B, dtype=I32, device="cuda").view(B, 4)
    free = torch.arange(4 * B, 6 * B, dtype=I32, device="cuda")
    new, count = i32([3] * B), i32([2 * B])
    return lambda: K.page_plan(table, lens, new, free, count, 16, 3 * B)


def convolution_gradient():
    r = make(2)
    x, dy, w = r(600, 256), r(600, 256), r(256, 4, dtype=F32)
    return lambda: K.short_conv_backward(x, w, dy)


class Prefill:
    """The same prefill on the path `impl`."""

    def __init__(self, impl, seqlens=(300, 130, 0, 700), H=3, seed=5):
        self.impl, self.d = impl, KI.make_case(list(seqlens), H=H, seed=seed, init_state=True)
        self.x = {n: self.d[n].cuda().contiguous() for n in ("q", "k", "v", "g", "beta", "initial_state", "cu_seqlens")}

    def __call__(self):
        assert K.kda_set_recurrent_impl(self.impl) == 0
        try:
            x = self.x
            return K.chunk_prefill(x["q"], x["k"], x["v"], x["g"], x["beta"], initial_state=x["initial_state"],
                                   cu_seqlens=x["cu_seqlens"], scale=self.d["scale"])
        finally:
            K.kda_set_recurrent_impl(1)

    def check(self, got):
        """As near to the 64-bit oracle as the prefill's parity tests ask."""
        import oracle
        d = self.d
        ref = oracle.recurrent(d["q"], d["k"], d["v"], d["g"], d["beta"], initial_state=d["initial_state"],
                               cu_seqlens=d["cu_seqlens"], scale=d["scale"])
        for g, r in zip(got, ref):
            g = g.double().cpu().numpy()
            assert np.linalg.norm(g - r) <= 1e-2 * np.linalg.norm(r)
            assert np.max(np.abs(g - r)) <= 2e-2 * np.max(np.abs(r))


WRITERS = {"gradient of the norms": heads_gradient, "attention": attention, "plan": plan,
           "gradient of the convolution": convolution_gradient, "prefill": lambda: Prefill(1)}


def captured(call, stream):
    call()   # (its workspace)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        held = call()
    return graph, held


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("writer", WRITERS)
def test_replays_between_calls_of_the_fused_prefill(writer):
    """The ring counters of the 64-token chunks in one launch are zero at every call, whatever a graph
    has written to the stream's workspace since the call before."""
    fused, call = Prefill(4), WRITERS[writer]()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        fused()   # the larger of the workspaces is there
        graph, _ = captured(call, stream)
        ref = fused()
        for _ in range(2):
            graph.replay()
            got = fused()
            stream.synchronize()
            assert same(got, ref)
    K.check_device_error(stream.cuda_stream)
    fused.check(ref)


@pytest.mark.parametrize("writer", WRITERS)
def test_calls_between_replays_of_the_fused_prefill(writer):
    """Likewise where the prefill is what the graph holds."""
    fused, call = Prefill(4), WRITERS[writer]()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call()
        ref = fused()
        graph, held = captured(fused, stream)
        for _ in range(2):
            for t in held:
                t.zero_()
            call()
            graph.replay()
            stream.synchronize()
            assert same(held, ref)
    K.check_device_error(stream.cuda_stream)
    fused.check(ref)


def test_counters_are_shared_in_turns():
    """The attention's arrival counters and the ring counters lie in one buffer; each leaves it zero."""
    few, many, call = Prefill(4), Prefill(4, (150, 64), H=40, seed=6), attention()
    ref = [few(), call(), many()]
    for _ in range(2):
        assert all(same(f(), r) for f, r in zip((few, call, many), ref))
        assert all(same(f(), r) for f, r in zip((many, few, call), (ref[2], ref[0], ref[1])))
    K.check_device_error()
    many.check(ref[2])


def used():
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    free, total = torch.cuda.mem_get_info()
    return total - free


def test_growing_keeps_what_graphs_hold_and_no_more():
    """A call is captured, then ever larger ones follow on its stream: of their workspaces (86 to 345 MB) the
    last one stays, and the graph's own (11 MB), with which a replay is still right."""
    H, r = 32, make(7)

    def gradient(T):
        x = [r(T, H, 128) for _ in range(4)]
        g, beta = -r(T, H, 128, dtype=F32).abs(), r(T, H, dtype=F32).sigmoid()
        return lambda: K.chunk_prefill_backward(x[0], x[1], x[2], g, beta, x[3])

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        assert K.kda_workspace_release() == 0
        first = gradient(64)
        ref = first()
        graph, held = captured(first, stream)
        before, sizes = used(), (512, 1024, 1536, 2048)
        for T in sizes:
            gradient(T)()
        stream.synchronize()
        grown = used() - before
        for t in held:
            if t is not None:
                t.zero_()
        graph.replay()
        stream.synchronize()
        assert all(a is None and b is None or torch.equal(a, b) for a, b in zip(held, ref))
    K.check_device_error(stream.cuda_stream)
    last = K.kda_backward_workspace_bytes(1, sizes[-1], H, 1, False)
    assert last > 300 << 20 and grown < last + (64 << 20), f"{grown >> 20} MB more for {last >> 20}"
    del graph, held
    assert K.kda_workspace_release() == 0
    assert used() <= before + (64 << 20)
