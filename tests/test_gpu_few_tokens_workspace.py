"""The few-token products' workspaces (a column order and more than GEMV_GATHERS values of x, or a mixture): on another
stream than the caller's, and in captured graphs."""
import numpy as np
import pytest

import few_ref as fr
import post_weight_quantization_21_amd as gq
from gpu_util import cuda, torch_mod
from test_gpu_few_tokens import _acts, _dev, _experts

pytestmark = pytest.mark.gpu
D, M, E, FF, K = 1024, 5, 4, 160, 2


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = torch_mod()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gq.load_library()


@pytest.fixture(scope="module")
def layers(oracle_mod):
    """(name, call(x, ws, stream), bytes of its workspace) of each product, with a column order that is prepared."""
    rng = np.random.default_rng(31)
    w = _dev(fr.make_packed(rng, oracle_mod, D, D, 4, 64, True))
    _, dw = _experts(rng, oracle_mod, E, D, FF, 4, 32, True)
    R = cuda(rng.standard_normal((E, D)).astype(np.float32))
    assert M * D > gq.GEMV_GATHERS
    one, many = gq.workspace_bytes(gq.OP_GEMV, D, D, M), gq.moe_workspace_bytes(M, D, FF, E, K)
    assert one > 0 and many > 0
    return [("gemv", lambda x, ws=None, stream=None: gq.gemv(x, w, ws=ws, stream=stream), one),
            ("gemv_gated", lambda x, ws=None, stream=None: gq.gemv_gated(x, w, w, ws=ws, stream=stream), one),
            ("moe_layer", lambda x, ws=None, stream=None: gq.moe_layer(x, *dw, router=R, top_k=K, ws=ws, stream=stream)[0], many)]


def test_memory_of_another_stream(layers):
    """A call on a stream that is busy takes its workspace and its result from that stream's memory: what the caller
    allocates and fills meanwhile is apart from both."""
    torch = torch_mod()
    x = _acts(np.random.default_rng(32), M, D, "bf16")[0]
    want = [call(x) for _, call, _ in layers]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for (name, call, size), expect in zip(layers, want):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        y = call(x, stream=side)
        junk = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda") for n in 8 * [size] + 8 * [M * D * 2]]
        torch.cuda.synchronize()
        assert torch.equal(y, expect) and all(bool((j == 0x55).all()) for j in junk), name


def test_given_workspace_on_another_stream(layers):
    torch = torch_mod()
    x = _acts(np.random.default_rng(33), M, D, "bf16")[0]
    side = torch.cuda.Stream()
    for name, call, size in layers:
        expect = call(x)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            ws = torch.full((size + 256,), 0xAA, dtype=torch.uint8, device="cuda")
        y = call(x, ws=ws[:size], stream=side)
        side.synchronize()
        assert torch.equal(y, expect) and bool((ws[size:] == 0xAA).all()), name


@pytest.mark.parametrize("given", [False, True])
def test_two_graphs(layers, given):
    """Two graphs, captured one after the other and replayed in turn with new inputs and eager calls in between, each
    with workspaces of its own (of its pool, or given)."""
    torch = torch_mod()
    rng = np.random.default_rng(34)
    inputs = [_acts(rng, M, D, "bf16")[0] for _ in range(4)]
    for name, call, size in layers:
        want = [call(x) for x in inputs]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call(inputs[0])
        torch.cuda.synchronize()
        graphs = []
        for _ in range(2):
            buf, ws = inputs[0].clone(), torch.empty(size, dtype=torch.uint8, device="cuda") if given else None
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                out = call(buf, ws=ws)
            graphs.append((g, buf, ws, out))
        for i, j in ((0, 1), (2, 3), (3, 3), (1, 0), (2, 1)):
            for (g, buf, _, _), k in zip(graphs, (i, j)):
                buf.copy_(inputs[k])
                g.replay()
            eager = call(inputs[(i + 1) % 4])
            torch.cuda.synchronize()
            assert torch.equal(graphs[0][3], want[i]) and torch.equal(graphs[1][3], want[j]), name
            assert torch.equal(eager, want[(i + 1) % 4]), name


def test_inputs_dropped_on_return(layers):
    """What a call on another, busy stream reads may be dropped at once: its memory is not handed out again before."""
    torch = torch_mod()
    x = _acts(np.random.default_rng(35), M, D, "bf16")[0]
    for name, call, size in layers:
        expect = call(x)
        side = torch.cuda.Stream()
        x_copy, ws = x.clone(), torch.empty(size, dtype=torch.uint8, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        y = call(x_copy, ws=ws, stream=side)
        at = {x_copy.data_ptr(), ws.data_ptr()}
        del x_copy, ws
        junk = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda") for n in 4 * [size] + 4 * [M * D * 2]]
        assert not at & {j.data_ptr() for j in junk}, name
        torch.cuda.synchronize()
        assert torch.equal(y, expect), name


def test_stream_named_inside_a_capture(layers):
    """A captured call that names the capturing stream, its input dropped inside the capture."""
    torch = torch_mod()
    rng = np.random.default_rng(36)
    inputs = [_acts(rng, M, D, "bf16")[0] for _ in range(3)]
    for name, call, size in layers:
        want = [call(x * 2) for x in inputs]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        buf = inputs[0].clone()
        call(buf, stream=side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            x = buf * 2
            out = call(x, stream=side)
            del x
        for i in (0, 2, 1, 1):
            buf.copy_(inputs[i])
            g.replay()
            eager = call(inputs[i] * 2)
            torch.cuda.synchronize()
            assert torch.equal(out, want[i]) and torch.equal(eager, want[i]), name
