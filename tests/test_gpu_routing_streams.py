"""Routing, dispatch and the loss over a head matrix on other streams, in captured graphs, and two calls at once.

Outputs on a stream that is not PyTorch's current one must not take a block
that the current stream's queued work still reads (its allocator hands a freed
block to the next request of the stream that it was made for), so each test
frees blocks of exactly the outputs' sizes with queued work that reads them.
"""

import pytest
import torch

from tests._util import require_gpu

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def mk():
    return require_gpu()


def inputs(seed, T=300):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*shape, dt=BF, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)

    E, k, H, V = 40, 4, 136, 1003
    logits = n(T, E, dt=torch.float32)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k, dim=1).indices
    ids[torch.rand(T, k, generator=g, device="cuda") < 0.1] = -1
    key = torch.where(ids < 0, E, ids).flatten()
    place = torch.empty_like(key)
    place[torch.sort(key, stable=True).indices] = torch.arange(T * k, device="cuda")
    place = torch.where(key < E, place, -1 - place).view(T, k)
    return {"logits": logits, "bias": n(E, dt=torch.float32, std=0.1), "ids": ids, "place": place, "x": n(T, H),
            "dw": n(T, k, dt=torch.float32), "y": n(T * k, H), "w": n(T, k, dt=torch.float32), "dout": n(T, H),
            "head": n(V, H, std=H ** -0.5), "t": torch.randint(-1, V, (T,), generator=g, device="cuda"),
            "lse": n(T, dt=torch.float32) + 7, "dloss": n(T, dt=torch.float32), "dlse": n(T, dt=torch.float32), "E": E}


CALLS = {
    "route": lambda mk, d, s: mk.muon_route(d["logits"], 4, bias=d["bias"], stream=s),
    "route_backward": lambda mk, d, s: (mk.muon_route_backward(d["dw"], d["logits"], d["ids"], stream=s),),
    "dispatch": lambda mk, d, s: mk.muon_dispatch(d["x"], d["ids"], d["E"], stream=s),
    "dispatch_backward": lambda mk, d, s: (mk.muon_dispatch_backward(d["y"], d["place"], stream=s),),
    "combine": lambda mk, d, s: (mk.muon_combine(d["y"], d["place"], d["w"], stream=s),),
    "combine_backward": lambda mk, d, s: mk.muon_combine_backward(d["dout"], d["y"], d["place"], d["w"], stream=s),
    "head_loss": lambda mk, d, s: mk.muon_head_loss(d["x"], d["head"], d["t"], stream=s),
    "head_loss_backward": lambda mk, d, s: mk.muon_head_loss_backward(
        d["dloss"], d["x"], d["head"], d["t"], d["lse"], dlse=d["dlse"], stream=s),
}


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", CALLS)
def test_outputs_belong_to_the_stream_that_writes_them(mk, name, raw):
    call, d, other = CALLS[name], inputs(1), inputs(2)
    want = [t.clone() for t in call(mk, other, None)]
    first = list(call(mk, d, None))
    values = [t.clone() for t in first]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    addresses = {t.data_ptr() for t in first}
    torch.cuda._sleep(50_000_000)            # about 25 ms of queued work on the current stream,
    read = [t.clone() for t in first]        # then reads of blocks that are free from here on
    addresses -= {t.data_ptr() for t in read}
    del first
    got = call(mk, other, side.cuda_stream if raw else side)
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    assert not addresses & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(read, values))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


class Elsewhere:
    """A stream of another device."""
    def __init__(self):
        self.cuda_stream = torch.cuda.current_stream().cuda_stream
        self.device_index = torch.cuda.current_device() + 1


@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_another_device_than_the_streams_are_refused(mk, name):
    with pytest.raises(ValueError, match="cuda:0, the call's stream on cuda:1"):
        CALLS[name](mk, inputs(4), Elsewhere())


@pytest.mark.parametrize("T", [40, 3000])    # dispatch sorts in one launch and in two
@pytest.mark.parametrize("name", CALLS)
def test_captured_and_replayed_on_new_inputs(mk, name, T):
    call, d, other = CALLS[name], inputs(5, T), inputs(6, T)
    want = [t.clone() for t in call(mk, other, None)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(mk, d, None)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = call(mk, d, None)
    for k, v in d.items():
        if isinstance(v, torch.Tensor):
            v.copy_(other[k])
    for _ in range(2):                       # a replay leaves nothing behind for the next
        for t in got:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert mk.muon_get_device_status() == 0


def test_two_graphs_with_workspaces_of_their_own_run_at_once(mk):
    a, b = inputs(7, 700), inputs(8, 700)
    n = mk.muon_head_loss_backward_workspace_bytes(700, 1003, 136)
    made = []
    for d in (a, b):
        want = [t.clone() for t in CALLS["head_loss_backward"](mk, d, None)]
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            got = mk.muon_head_loss_backward(d["dloss"], d["x"], d["head"], d["t"], d["lse"], dlse=d["dlse"],
                                             workspace=ws)
        made.append((graph, side, got, want, ws))
    for _ in range(5):
        for graph, side, *_ in made:
            with torch.cuda.stream(side):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, got, want, _ in made:
        assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("name", CALLS)
def test_equal_calls_give_equal_bits(mk, name):
    d = inputs(9, 2500)
    first = [t.clone() for t in CALLS[name](mk, d, None)]
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, CALLS[name](mk, d, None)))


@pytest.mark.parametrize("name", CALLS)
def test_inputs_are_left_as_they_were(mk, name):
    d = inputs(10)
    before = {k: v.clone() for k, v in d.items() if isinstance(v, torch.Tensor)}
    CALLS[name](mk, d, None)
    assert all(torch.equal(d[k], v) for k, v in before.items())
