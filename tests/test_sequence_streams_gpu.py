"""The sequence operators on a stream that is not torch's current one: what they allocate belongs to that stream."""

import pytest
import torch

import token_level_head_block_gb300 as mhla

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
B, N, H, D = 3, 6007, 12, 64


def tensors():
    gen = torch.Generator(device=DEV).manual_seed(1)
    normal = lambda *s: torch.randn(*s, generator=gen, device=DEV)
    x = {n: normal(B, N, H, D).bfloat16() for n in ("q", "k", "v", "dout")}
    x["g"] = torch.nn.functional.logsigmoid(normal(B, N, H) + 3).bfloat16()
    x["w"] = 1 + 0.1 * normal(D)
    x["state"] = normal(B, H, D, D)
    return x


def calls(x):
    args = (x["q"], x["k"], x["v"], x["g"])
    one = [t[:, :1] for t in args]
    return {
        "gated_forward": lambda **kw: mhla.gated_forward(*args, scale=0.125, state=x["state"], **kw),
        "gated_backward": lambda **kw: mhla.gated_backward(*args, x["dout"], scale=0.125, state=x["state"], **kw),
        "gated_step": lambda **kw: (mhla.gated_step(*one, x["state"].clone(), scale=0.125, **kw),),
        "qk_norm": lambda **kw: mhla.qk_norm(x["q"], x["k"], x["w"], x["w"], **kw),
        "qk_norm_backward": lambda **kw: mhla.qk_norm_backward(x["q"], x["k"], x["dout"], x["v"], x["w"], x["w"], **kw),
    }


@pytest.mark.parametrize("name", ["gated_forward", "gated_backward", "qk_norm", "qk_norm_backward"])
@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
def test_memory_is_not_handed_to_another_stream(name, handle):
    """An output dropped while its stream may still write it: the current stream gets other memory."""
    x = tensors()
    run = calls(x)[name]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    got = run(stream=s.cuda_stream if handle else s)
    places = [(t.data_ptr(), t.numel() * t.element_size(), t.shape, t.dtype) for t in got]
    del got
    for at, size, shape, dtype in places:
        if size < 1 << 20:      # small blocks come from shared segments: their addresses say nothing
            continue
        other = [torch.empty(shape, dtype=dtype, device=DEV) for _ in range(3)]
        assert all(t.data_ptr() != at for t in other)
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", ["gated_forward", "gated_backward", "gated_step", "qk_norm", "qk_norm_backward"])
def test_the_same_bits_as_on_the_current_stream(name):
    x = tensors()
    run = calls(x)[name]
    want = run()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream, 0, torch.cuda.default_stream()):
        torch.cuda.synchronize()
        got = run(stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):                                            # current and given alike
        got = run(stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_work_queued_on_both_streams():
    """A chain on its own stream while the current one allocates, writes and frees memory of the same sizes."""
    x = tensors()
    run = calls(x)["gated_forward"]
    want = run()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        out, state = run(stream=s)
        junk = [torch.full_like(x["q"], float("nan")) for _ in range(2)]
        del junk
        s.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(state, want[1])
        del out, state


def test_stream_of_another_device_is_refused():
    if torch.cuda.device_count() < 2:
        class Elsewhere(torch.cuda.Stream):
            device = torch.device("cuda:1")
        s = Elsewhere()
    else:
        s = torch.cuda.Stream(device="cuda:1")
    x = tensors()
    with pytest.raises(ValueError):
        calls(x)["gated_forward"](stream=s)
