"""The operators on a stream that is not PyTorch's current one: whose memory the outputs take.

PyTorch's allocator gives a freed block to the next request of the stream that
it was made for, whatever work of that stream is still queued on it.  So a call
on another stream must not be given such a block: each test frees blocks of
exactly the outputs' sizes on the current stream, with queued work that still
reads them, calls the operator on a second stream, and looks at the addresses
and at what the queued work read.
"""

import pytest
import torch

from tests._util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mk():
    return require_gpu()


def inputs(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*shape, dt=torch.bfloat16, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)

    T, H, F, V = 96, 256, 136, 3000
    return {"x": n(T, H), "w1": n(2, H, F, std=H ** -0.5), "w3": n(2, H, F, std=H ** -0.5),
            "w2": n(2, F, H, std=F ** -0.5), "off": torch.tensor([0, 40, T], device="cuda"), "gate": n(T, F),
            "up": n(T, F), "dy": n(T, H), "r": n(T, H, dt=torch.float32), "w": n(H), "g": n(T, H),
            "rstd": n(T, dt=torch.float32).abs() + 0.5, "logits": n(T, V),
            "tokens": torch.randint(0, V, (T,), generator=g, device="cuda"), "lse": n(T, dt=torch.float32) + 9,
            "entropy": n(T, dt=torch.float32) + 7, "dl": n(T, dt=torch.float32), "de": n(T, dt=torch.float32)}


CALLS = {
    "gated_ffn": lambda mk, d, s: mk.muon_gated_ffn(d["x"], d["w1"], d["w3"], d["w2"], d["off"], keep=True, stream=s),
    "gated_ffn_backward": lambda mk, d, s: mk.muon_gated_ffn_backward(
        d["dy"], d["x"], d["gate"], d["up"], d["w1"], d["w3"], d["w2"], d["off"], stream=s),
    "block_norm": lambda mk, d, s: mk.muon_block_norm(d["r"], d["x"], w_post=d["w"], gate=d["g"], w_pre=d["w"],
                                                      stream=s),
    "block_norm_backward": lambda mk, d, s: mk.muon_block_norm_backward(
        d["r"], d["dy"], d["r"], d["x"], d["rstd"], d["rstd"], w_post=d["w"], gate=d["g"], w_pre=d["w"], stream=s),
    "token_logprobs": lambda mk, d, s: mk.muon_token_logprobs(d["logits"], d["tokens"], top=4, stream=s),
    "token_logprobs_backward": lambda mk, d, s: (mk.muon_token_logprobs_backward(
        d["logits"], d["tokens"], d["lse"], d["entropy"], d["dl"], d["de"], stream=s),),
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
    # a dropped output's block goes to the next call of that stream, and to no request of the current one
    freed = {t.data_ptr() for t in got}
    shapes = [(t.shape, t.dtype) for t in got]
    del got
    assert not freed & {torch.empty(s, dtype=dt, device="cuda").data_ptr() for s, dt in shapes}
    again = call(mk, other, side)
    assert {t.data_ptr() for t in again} == freed
    torch.cuda.synchronize()


def test_outputs_given_by_the_caller_are_left_where_they_are(mk):
    d, side = inputs(3), torch.cuda.Stream()
    want = mk.muon_gated_ffn(d["x"], d["w1"], d["w3"], d["w2"], d["off"])
    out = torch.zeros_like(want)
    side.wait_stream(torch.cuda.current_stream())
    assert mk.muon_gated_ffn(d["x"], d["w1"], d["w3"], d["w2"], d["off"], out=out, stream=side) is out
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)


class Elsewhere:
    """A stream of another device."""
    def __init__(self):
        self.cuda_stream = torch.cuda.current_stream().cuda_stream
        self.device_index = torch.cuda.current_device() + 1


@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_another_device_than_the_streams_are_refused(mk, name, monkeypatch):
    d = inputs(4)
    with pytest.raises(ValueError, match="cuda:0, the call's stream on cuda:1"):
        CALLS[name](mk, d, Elsewhere())
    # the current stream of a current device that is not the tensors'
    elsewhere = (torch.cuda.current_stream().cuda_stream, torch.cuda.current_device() + 1, True)
    monkeypatch.setattr(mk, "_raw_stream", lambda stream: elsewhere)
    with pytest.raises(ValueError, match="cuda:0, the call's stream on cuda:1"):
        CALLS[name](mk, d, None)
