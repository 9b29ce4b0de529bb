"""Weights made on a stream of their own while the current stream is busy."""
from types import SimpleNamespace

import pytest
import torch

import mx4_reference as ref
from mixture_experts_layer_29_b200 import mx4

pytestmark = pytest.mark.gpu


def busy():
    torch.cuda._sleep(1_000_000_000)        # some half a second on the current stream


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_weights_on_another_stream_do_not_wait_for_the_current_one(cuda_device, fmt, handle):
    """A weight that is not contiguous is copied on the way; the copy and the memory are the stream's."""
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.randn(3, 384, 200, device="cuda", generator=g).transpose(1, 2)       # [3, 200, 384]
    code, byte, _ = ref.quantize(w, fmt)
    codes = ref.pack(code).contiguous()
    want = mx4.quantize_weight(w.contiguous(), fmt)
    at = ref.scale_index([200 * i for i in range(4)], 384, fmt, "cuda")
    st = torch.cuda.Stream()
    for _ in range(2):                      # kernels loaded, memory at hand: neither waits for the device below
        mx4.quantize_weight(w, fmt, stream=st), mx4.from_checkpoint(fmt, codes, byte, stream=st)
    junk = [torch.full((3 * 200 * 384,), 7.0, device="cuda") for i in range(3)]
    del junk
    torch.cuda.synchronize()
    start, done = torch.cuda.Event(), torch.cuda.Event()
    busy()
    start.record()
    s = st.cuda_stream if handle else st
    a = mx4.quantize_weight(w, fmt, stream=s)
    b = mx4.from_checkpoint(fmt, codes, byte, stream=s)
    # memory that a copy leaves behind is used again on the current stream only once it is the stream's no more
    junk = [torch.full((3 * 200 * 384,), 7.0, device="cuda") for _ in range(3)]
    done.record(st)
    done.synchronize()
    assert not start.query()                # the current stream is still busy
    with torch.cuda.stream(st):
        same = [torch.equal(a.codes, want.codes), torch.equal(a.scales[at], want.scales[at]),
                torch.equal(b.scales[at], byte.flatten(0, 1))]
    torch.cuda.synchronize()
    assert all(same) and junk


@pytest.mark.parametrize("kind", ["default handle", "object"])
def test_weights_on_streams_that_are_not_torchs(cuda_device, kind):
    """The legacy default stream by its handle, and any object that has a handle."""
    w = torch.randn(2, 128, 256, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    want = mx4.quantize_weight(w, "mxfp4")
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = mx4.quantize_weight(w, "mxfp4", stream=0 if kind == "default handle" else SimpleNamespace(cuda_stream=st.cuda_stream))
    torch.cuda.synchronize()
    assert torch.equal(got.codes, want.codes)
