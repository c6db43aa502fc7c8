"""Attention and the norm's gradient in captured graphs: workspaces that the
graph keeps, whatever the stream does afterwards."""
import pytest
import torch

import attention_reference as ref
from test_gpu_attention import DEV, DT, _inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sp():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    import submanifold_sparse_convolution_device_amd as m
    m.lib()
    return m


def _step(sp, seed, nq, nk, dtype="bf16"):
    """A step that needs workspaces: single queries over long keys, their
    gradient, and the norm's gradient; and the tensors that it reads."""
    cu_q, cu_k = ref.offsets(nq).to(DEV), ref.offsets(nk).to(DEV)
    _, (q, k, v), grad = _inputs(seed, sum(nq), sum(nk), 4, 2, 32, dtype)
    grad = grad.to(DEV)
    w = torch.ones(32, dtype=DT[dtype], device=DEV)
    h = dict(causal=True)

    def step():
        out, lse = sp.attention(q, k, v, cu_q, cu_k, return_lse=True, **h)
        grads = sp.attention_backward(grad, q, k, v, out, lse, cu_q, cu_k, **h)
        return (out, lse, *grads, *sp.norm_rotary_backward(grads[1], grads[2], k, v, w, w))

    return step, (q, k, v)


def _capture(step, stream):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = step()
    return graph, got


def _check_replays(graph, got, step, inputs, between):
    for i in range(4):
        for t in inputs:
            t.copy_(torch.randn(t.shape, device=DEV))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        between()
        want = step()
        torch.cuda.synchronize()
        for n, (a, b) in enumerate(zip(kept, want)):
            assert torch.equal(a, b), (i, n)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_streams_first_call_is_captured(sp, dtype):
    """Nothing is allocated for the stream before the capture."""
    step, inputs = _step(sp, 1, [1, 2, 1], [900, 40, 3000], dtype)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph, got = _capture(step, side)
    _check_replays(graph, got, step, inputs, lambda: None)


def test_the_streams_workspace_grows_after_the_capture(sp):
    """Later calls on the stream need far more, and what they free is taken by
    others: the replays still write into memory of their own."""
    step, inputs = _step(sp, 2, [1, 2, 1], [900, 40, 3000])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        step()
        side.synchronize()
        graph, got = _capture(step, side)
        factor = [1]

        def grow():
            factor[0] *= 2
            larger, _ = _step(sp, 3, [1] * (4 * factor[0]), [5000] * (4 * factor[0]))
            larger()
            coords = torch.stack(torch.meshgrid(*(torch.arange(n) for n in (1, 20, 20, 20)), indexing="ij"), -1).reshape(-1, 4)
            sp.build_map(coords.int().to(DEV), 3).free()

        _check_replays(graph, got, step, inputs, grow)


def test_two_graphs_of_one_stream_run_beside_each_other(sp):
    steps = [_step(sp, 4 + i, [1] * 8, [6000 - 700 * i] * 8) for i in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = [_capture(s, side) for s, _ in steps]
    want = [s() for s, _ in steps]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for stream, (graph, _) in zip(streams, graphs):
            with torch.cuda.stream(stream):
                graph.replay()
                graph.replay()
        torch.cuda.synchronize()
        for w, (_, got) in zip(want, graphs):
            for a, b in zip(w, got):
                assert torch.equal(a, b)


def test_captured_calls_without_a_workspace_are_refused(sp):
    """The plain entry points, called from C or ctypes under capture: an error
    before anything is enqueued, and the capture goes on."""
    cu = torch.tensor([0, 5], dtype=torch.int32, device=DEV)
    x = torch.randn(5, 2, 32, device=DEV).bfloat16()
    out, lse = sp.attention(x, x, x, cu, return_lse=True)
    grads = [torch.empty_like(x) for _ in range(3)]
    a = sp._attention_args(x, x, x, cu, None, False, (-1, -1), None)
    g = sp._PACK_ATTENTION_GRADIENTS.pack(*sp._heads_tensor("g", x), *(v for t in grads for v in sp._heads_tensor("g", t)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    y = torch.zeros(4, device=DEV)
    with torch.cuda.graph(graph, stream=side):
        rc = sp.lib().spconv_attention_backward(a, out.data_ptr(), lse.data_ptr(), g, torch.cuda.current_stream().cuda_stream)
        y.add_(1)
    assert sp.STATUS[rc] == "SPCONV_ERR_INVALID_ARG" and "workspace" in sp.lib().spconv_last_error().decode()
    graph.replay()
    torch.cuda.synchronize()
    assert bool((y == 1).all())
