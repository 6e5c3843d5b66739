"""Calls on a stream of their own: `stream=` as a torch stream or as its handle.

Nothing here waits for the whole device between the work of the current stream
and the call, so memory that one stream hands to the other too early shows as
a wrong value.  The order is forced: the stream that must not be overtaken
sleeps first.
"""
import pytest
import torch

from tiled_attention_blackwell_b200 import attn, build
from tiled_attention_blackwell_b200.workloads import make_tensors, make_tensors_fp4, make_tensors_fp8

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


@pytest.mark.parametrize("handle", HANDLES, ids=["stream", "handle"])
def test_slopes_from_the_host_do_not_wait_for_the_stream(handle):
    """The call returns while its stream has work of its own to do, and what
    holds the slopes is not given away till then."""
    t = on_device(make_tensors(1, 4, 2, 200, 200, 64, 1))
    x = decode_arguments(torch.Generator().manual_seed(2), Hq=4)
    kw = dict(alibi_slopes=[0.5, 0.25, 0.125, 0.0625])

    def both(**more):
        return attn.attention(t["q"], t["k"], t["v"], causal=True, window=(60, 0), sinks=3, **kw, **more) + \
            attn.decode_paged(*x, **kw, **more)

    want = both()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        sleep()
    got = both(stream=handle(side))
    assert not side.query()
    small = [torch.zeros(4, device=DEV) for _ in range(4)]
    torch.cuda.synchronize()
    check(got, want)
    check_value(small, 0)


def calls():
    """Every call that allocates: its name and a function of the stream."""
    t = on_device(make_tensors(1, 4, 2, 300, 300, 128, 3, with_dout=True))
    q, k, v, dout = (t[n] for n in ("q", "k", "v", "dout"))
    plain, docs = dict(causal=True), dict(causal=True, doc_offsets=[0, 70, 201, 300])
    window = dict(causal=True, window=(140, 0), sinks=4)
    saved = {n: attn.attention(q, k, v, **kw) for n, kw in (("docs", docs), ("window", window))}
    f8, f4 = on_device(make_tensors_fp8(1, 4, 2, 300, 300, 128, 4)), on_device(make_tensors_fp4(1, 4, 2, 300, 300, 128, 5))
    names = [f"{x}_{y}" for x in "qkv" for y in ("codes", "scales", "global")]
    long = on_device(make_tensors(1, 4, 2, 200, 1500, 128, 6))
    g = torch.Generator().manual_seed(7)
    qkv = torch.randn(60, 12 * 128, generator=g).to(torch.bfloat16).to(DEV)
    nq, nk, nv = (x.unflatten(-1, (-1, 128)) for x in qkv.split([8 * 128, 2 * 128, 2 * 128], -1))
    w, (cos, sin) = torch.ones(128, device=DEV), attn.rope_table(60, 128, device=DEV)
    pos = torch.arange(60, dtype=torch.int32, device=DEV)
    norm = (nq, nk, w, w, cos, sin, pos)
    grads = [torch.randn(60, h, 128, generator=g).to(DEV) for h in (8, 2)]
    caches = [torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    token = decode_arguments(g)
    return {
        "attention": lambda s: attn.attention(q, k, v, stream=s, **plain),
        "attention docs": lambda s: attn.attention(q, k, v, stream=s, **docs),
        "attention_backward docs": lambda s: attn.attention_backward(q, k, v, *saved["docs"], dout, stream=s, **docs),
        "attention_fp8": lambda s: attn.attention_fp8(*(f8[n] for n in "qkv"), stream=s, **docs,
                                                      **{n: f8[n] for n in ("q_descale", "k_descale", "v_descale")}),
        "attention_fp4": lambda s: attn.attention_fp4(*(f4[n] for n in names), stream=s, **docs),
        "window": lambda s: attn.attention(q, k, v, stream=s, **window),
        "window in parts": lambda s: attn.attention(long["q"], long["k"], long["v"], stream=s, causal=True,
                                                    window=(900, 0), sinks=4),
        "window backward": lambda s: attn.attention_backward(q, k, v, *saved["window"], dout, stream=s, **window),
        "qk_norm_rope": lambda s: attn.qk_norm_rope(*norm, stream=s),
        "qk_norm_rope_backward": lambda s: attn.qk_norm_rope_backward(*grads, *norm, stream=s),
        "qk_norm_rope_cache": lambda s: (attn.qk_norm_rope_cache(nq, nk, nv, w, w, cos, sin, pos, pos, *caches,
                                                                 stream=s),),
        "decode_paged": lambda s: attn.decode_paged(*token, stream=s),
    }


NAMES = ["attention", "attention docs", "attention_backward docs", "attention_fp8", "attention_fp4", "window",
         "window in parts", "window backward", "qk_norm_rope", "qk_norm_rope_backward", "qk_norm_rope_cache",
         "decode_paged"]
FROM_HOST = ("attention docs", "attention_backward docs", "attention_fp8", "attention_fp4")  # document offsets as a list


@pytest.fixture(scope="module")
def every():
    x = calls()
    assert list(x) == NAMES
    return x


def check(got, want):
    same = [torch.equal(a, b) for a, b in zip(got, want)]
    assert all(same), same


def check_value(blocks, value):
    """Blocks that hold what their stream wrote."""
    kept = [bool((x == value).all()) for x in blocks]
    assert all(kept), kept


def fill_free_blocks(want, value):
    """Writes `value` to blocks of the results' sizes, queued on the current
    stream, and gives them back to its pool before they are written."""
    blocks = [torch.empty_like(x) for x in want for _ in range(2)]
    for x in blocks:
        x.fill_(value)


@pytest.mark.parametrize("handle", HANDLES, ids=["stream", "handle"])
@pytest.mark.parametrize("name", NAMES)
def test_memory_that_the_current_stream_still_writes_is_not_taken(every, name, handle):
    """Blocks that the current stream freed, but has yet to write, are no place
    for the results (or workspaces) of a call on another stream."""
    call = every[name]
    want = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    sleep()
    fill_free_blocks(want, 7)
    got = call(handle(side))
    torch.cuda.synchronize()
    check(got, want)


@pytest.mark.parametrize("name", NAMES)
def test_memory_of_a_call_stays_its_own_until_it_has_run(every, name):
    """Results that are dropped at once, and what the call allocates for itself,
    are not handed to the current stream while the call has yet to run there."""
    call = every[name]
    want = call(None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        sleep()
    call(side)  # dropped
    assert not side.query()  # nor has it waited for the stream
    mine = [torch.full_like(x, 7) for x in want for _ in range(3)]
    kept = call(side)
    small = [torch.zeros(4, dtype=torch.int32, device=DEV) for _ in range(3)]
    torch.cuda.synchronize()
    check_value(mine, 7)
    check_value(small, 0)
    check(kept, want)


@pytest.mark.parametrize("name", NAMES)
def test_results_in_use_on_the_current_stream_are_not_taken_by_the_next_call(every, name):
    """Results of a side stream's call that the current stream reads late, after
    they were dropped, while the side stream's next call allocates."""
    call = every[name]
    want = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    got = call(side)
    torch.cuda.current_stream().wait_stream(side)
    sleep()
    read = [x.clone() for x in got]
    del got
    with torch.cuda.stream(side):
        mine = [torch.full_like(x, 7) for x in want for _ in range(3)]
    torch.cuda.synchronize()
    check(read, want)
    check_value(mine, 7)


@pytest.mark.parametrize("name", [n for n in NAMES if n not in FROM_HOST])
def test_captured_on_a_stream_beside_the_capturing_one(every, name):
    call = every[name]
    want = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = call(side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        for x in got:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        check(got, want)


def test_the_default_stream_by_its_handle(every):
    """Handle 0 is the default stream, also where another one is current."""
    want = every["window"](None)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    with torch.cuda.stream(other):
        got = every["window"](0)
        other.wait_stream(torch.cuda.default_stream())
        read = [x.clone() for x in got]
    torch.cuda.synchronize()
    check(read, want)
