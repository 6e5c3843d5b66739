"""Calls on a stream of their own: `stream=` as a torch stream or as its handle.

Nothing here waits for the whole device between the work of the current stream
and the call, so memory that one stream hands to the other too early shows as
a wrong value.  The order is forced: the stream that must not be overtaken
sleeps first.
"""
import pytest
import torch

from tiled_attention_blackwell_b200 import attn, build
from tiled_attention_blackwell_b200.workloads import make_tensors

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HANDLES = [lambda s: s, lambda s: s.cuda_stream]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    build.build()
    attn.lib()
    yield
    assert attn.device_status() == attn.ATTN_OK


def sleep():
    """About a tenth of a second of the current stream's time."""
    torch.cuda._sleep(200_000_000)


def on_device(t):
    return {n: x.to(DEV) if torch.is_tensor(x) else x for n, x in t.items()}


def decode_arguments(g, *, Hq=8, Hkv=2, D=128, page=16, lens=(700, 64, 300)):
    need = [-(-n // page) for n in lens]
    table = torch.zeros(len(lens), max(need), dtype=torch.int32)
    for b, n in enumerate(need):
        table[b, :n] = sum(need[:b]) + torch.arange(n, dtype=torch.int32)
    kc, vc = (torch.randn(sum(need), page, Hkv, D, generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(len(lens), Hq, D, generator=g).to(torch.bfloat16)
    return [x.to(DEV) for x in (q, kc, vc, table, torch.tensor(lens, dtype=torch.int32))]


@pytest.mark.parametrize("handle", HANDLES, ids=["stream", "handle"])
def test_slopes_from_the_host_on_a_side_stream(handle):
    """ALiBi slopes as a list, brought to the device by the call."""
    slopes = [0.5, 0.25, 0.125, 0.0625]
    t = on_device(make_tensors(1, 4, 2, 200, 200, 64, 1, with_dout=True))
    window = dict(causal=True, window=(60, 0), sinks=3)
    x = decode_arguments(torch.Generator().manual_seed(2), Hq=4)

    def every(s, stream=None):
        out = []
        for kw in (dict(causal=True), window):
            o, lse = attn.attention(t["q"], t["k"], t["v"], alibi_slopes=s, stream=stream, **kw)
            out += [o, lse, *attn.attention_backward(t["q"], t["k"], t["v"], o, lse, t["dout"], alibi_slopes=s,
                                                     stream=stream, **kw)]
        return out + list(attn.decode_paged(*x, alibi_slopes=s, stream=stream))

    want = every(torch.tensor(slopes, device=DEV))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = every(slopes, handle(side))
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
