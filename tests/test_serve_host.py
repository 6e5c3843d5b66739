"""Host-side checks of the head norms, the cache write and the decode (no GPU
needed): bad arguments are refused before any CUDA call."""
import ctypes

import pytest
import torch

from tiled_attention_blackwell_b200 import attn, build

P = 0x10000  # a fake, aligned device address: never dereferenced


@pytest.fixture(scope="module")
def L():
    build.build()
    return attn.lib()


NORM = dict(q=P, k=P, qo=P, ko=P, qs=512, ks=256, qos=512, kos=256, qw=P, kw=P, wf=0, cos=P, sin=P, pos=P, tokens=4,
            Hq=4, Hkv=2, D=128, rot=64, maxpos=100, eps=1e-6, inter=0)


def call_norm(L, **kw):
    a = {**NORM, **kw}
    return L.attn_qk_norm_rope(a["q"], a["k"], a["qo"], a["ko"], a["qs"], a["ks"], a["qos"], a["kos"], a["qw"],
                               a["kw"], a["wf"], a["cos"], a["sin"], a["pos"], a["tokens"], a["Hq"], a["Hkv"],
                               a["D"], a["rot"], a["maxpos"], a["eps"], a["inter"], None)


def call_norm_cache(L, **kw):
    a = {**NORM, **dict(v=P, vs=256, slots=P, kc=P, vc=P, kv=0, kd=1.0, vd=1.0, n=64), **kw}
    return L.attn_qk_norm_rope_cache(a["q"], a["k"], a["v"], a["qo"], a["qs"], a["ks"], a["vs"], a["qos"], a["qw"],
                                     a["kw"], a["wf"], a["cos"], a["sin"], a["pos"], a["slots"], a["kc"], a["vc"],
                                     a["kv"], a["kd"], a["vd"], a["n"], a["tokens"], a["Hq"], a["Hkv"], a["D"],
                                     a["rot"], a["maxpos"], a["eps"], a["inter"], None)


def call_norm_bwd(L, **kw):
    a = {**NORM, **dict(dq=P, dk=P, dqf=1, dkf=0, dqw=P, dkw=P, dqs=512, dks=256, ws=P, wsb=1 << 22), **kw}
    return L.attn_qk_norm_rope_bwd(a["dq"], a["dk"], a["dqf"], a["dkf"], a["q"], a["k"], a["qo"], a["ko"], a["dqw"],
                                   a["dkw"], a["dqs"], a["dks"], a["qs"], a["ks"], a["qos"], a["kos"], a["qw"],
                                   a["kw"], a["wf"], a["cos"], a["sin"], a["pos"], a["tokens"], a["Hq"], a["Hkv"],
                                   a["D"], a["rot"], a["maxpos"], a["eps"], a["inter"], a["ws"], a["wsb"], None)


INV, UNS, MIS = attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED, attn.ATTN_ERR_MISALIGNED
COMMON = [(dict(q=0), INV), (dict(k=0), INV), (dict(qw=0), INV), (dict(cos=0), INV), (dict(pos=0), INV),
          (dict(tokens=0), INV), (dict(tokens=-1), INV), (dict(Hq=0), INV), (dict(D=96), UNS), (dict(rot=0), INV),
          (dict(rot=24), INV), (dict(rot=144), INV), (dict(maxpos=0), INV), (dict(eps=-1.0), INV),
          (dict(eps=float("nan")), INV), (dict(inter=2), INV), (dict(wf=-1), INV), (dict(q=P + 8), MIS),
          (dict(qw=P + 8), MIS), (dict(sin=P + 4), MIS), (dict(pos=P + 2), MIS), (dict(qs=511), INV),
          (dict(qs=504), INV), (dict(ks=260), INV), (dict(tokens=1 << 40), UNS)]


@pytest.mark.parametrize("call", [call_norm, call_norm_cache, call_norm_bwd])
@pytest.mark.parametrize("kw,status", COMMON)
def test_norm_refusals(L, call, kw, status):
    assert call(L, **kw) == status
    assert L.attn_last_error_detail().decode() != ""


@pytest.mark.parametrize("kw,status", [
    (dict(v=0), INV), (dict(vs=128), INV), (dict(slots=0), INV), (dict(slots=P + 1), MIS), (dict(kc=0), INV),
    (dict(vc=P + 4), MIS), (dict(kv=2), INV), (dict(n=0), INV), (dict(kd=0.5), INV), (dict(kv=1, kd=0.0), INV), (dict(kv=1, kd=1e-39), INV),
    (dict(kv=1, vd=float("inf")), INV), (dict(kv=1, kd=1e-39), INV)])
def test_norm_cache_refusals(L, kw, status):
    assert call_norm_cache(L, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dq=0), INV), (dict(dqs=256), INV), (dict(dqf=2), INV), (dict(dqw=0), INV), (dict(dkw=P + 2), MIS),
    (dict(ws=0), INV), (dict(ws=P + 8), MIS), (dict(wsb=100), INV), (dict(qo=P + 4), MIS)])
def test_norm_bwd_refusals(L, kw, status):
    assert call_norm_bwd(L, **kw) == status


def call_decode(L, **kw):
    a = dict(q=P, kc=P, vc=P, kv=0, kd=1.0, vd=1.0, table=P, lens=P, o=2 * P, lse=P, B=2, Hq=4, Hkv=2, D=128, pages=8,
             page=16, width=4, scale=0.1, wl=-1, sinks=0, cap=0.0, slopes=None, ws=P, wsb=1 << 24)
    a.update(kw)
    return L.attn_decode_paged(a["q"], a["kc"], a["vc"], a["kv"], a["kd"], a["vd"], a["table"], a["lens"], a["o"],
                               a["lse"], a["B"], a["Hq"], a["Hkv"], a["D"], a["pages"], a["page"], a["width"],
                               a["scale"], a["wl"], a["sinks"], a["cap"], a["slopes"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=0), INV), (dict(kc=0), INV), (dict(table=0), INV), (dict(lens=0), INV), (dict(lse=0), INV),
    (dict(ws=0), INV), (dict(wsb=100), INV), (dict(q=P + 8), MIS), (dict(vc=P + 4), MIS), (dict(table=P + 2), MIS),
    (dict(o=P), INV), (dict(slopes=P + 2), MIS), (dict(B=0), INV), (dict(Hq=3), INV), (dict(pages=0), INV), (dict(width=0), INV),
    (dict(D=96), UNS), (dict(page=8), UNS), (dict(page=24), UNS), (dict(page=0), UNS), (dict(kv=3), INV),
    (dict(kd=2.0), INV), (dict(kv=1, vd=-1.0), INV), (dict(scale=0.0), INV), (dict(scale=float("nan")), INV),
    (dict(wl=-2), INV), (dict(sinks=-1), INV), (dict(cap=-1.0), INV), (dict(cap=float("inf")), INV),
    (dict(page=1 << 20, width=1 << 12), UNS), (dict(Hq=1 << 16, Hkv=1 << 16, width=1 << 20), UNS)])
def test_decode_refusals(L, kw, status):
    assert call_decode(L, **kw) == status
    assert L.attn_last_error_detail().decode() != ""


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU path only")
def test_valid_calls_without_gpu_report_cuda_error(L):
    for call in (call_norm, call_norm_cache, call_norm_bwd, call_decode):
        assert call(L) == attn.ATTN_ERR_CUDA
    assert call_decode(L, kv=1, kd=0.1, vd=3.0, wl=0, sinks=4, cap=30.0, slopes=P) == attn.ATTN_ERR_CUDA


def test_workspace_sizes(L):
    assert attn.decode_workspace_size(128) >= 296 * 2 * 16 * 128 * 4 and attn.decode_workspace_size(0) == 0
    assert L.attn_qk_norm_rope_bwd_workspace_size(64) >= 2 * 148 * 2 * 64 * 4


class _CudaStandIn(torch.Tensor):
    """A CPU tensor that reports itself as a CUDA tensor (see test_boundary)."""

    @property
    def is_cuda(self):
        return True


def stand_in(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(_CudaStandIn)


# The native binding looks at types and shapes before it looks at the device,
# so CPU tensors reach each of its checks; a call whose tensors are all right
# ends at the device.

F32, I32, F8 = torch.float32, torch.int32, torch.float8_e4m3fn


def cpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def norm_tensors(**other):
    return {**dict(q=cpu(5, 4, 128), k=cpu(5, 2, 128), q_weight=cpu(128), k_weight=cpu(128), cos=cpu(9, 32, dtype=F32),
                   sin=cpu(9, 32, dtype=F32), positions=cpu(5, dtype=I32)), **other}


def norm_calls(t):
    dq, dk = torch.zeros(t["q"].shape) if torch.is_tensor(t["q"]) else cpu(5, 4, 128), cpu(5, 2, 128)
    yield lambda **kw: attn.qk_norm_rope(*t.values(), **kw)
    yield lambda **kw: attn.qk_norm_rope_backward(dq, dk, *t.values(), **kw)
    yield lambda **kw: attn.qk_norm_rope_cache(t["q"], t["k"], cpu(5, 2, 128), *list(t.values())[2:],
                                               cpu(5, dtype=I32), cpu(3, 16, 2, 128), cpu(3, 16, 2, 128), **kw)


@pytest.mark.parametrize("name,bad", [
    ("q", 3), ("q", cpu(5, 4, 128, dtype=torch.float16)), ("q", cpu(4, 128)), ("k", cpu(6, 2, 128)),
    ("k", cpu(5, 2, 64)), ("k", cpu(1, 5, 2, 128)), ("q_weight", cpu(64)), ("q_weight", cpu(128, dtype=torch.float16)),
    ("k_weight", cpu(128, dtype=F32)), ("k_weight", cpu(256)[::2]), ("cos", cpu(9, 32)), ("cos", cpu(9, 1, 32, dtype=F32)),
    ("sin", cpu(8, 32, dtype=F32)), ("sin", cpu(32, 9, dtype=F32).T), ("positions", cpu(5, dtype=torch.int64)),
    ("positions", cpu(4, dtype=I32)), ("positions", cpu(10, dtype=I32)[::2])])
def test_norm_binding_refuses(L, name, bad):
    for call in norm_calls(norm_tensors(**{name: bad})):
        with pytest.raises(TypeError, match=name):
            call()


def test_bindings_refuse_cpu_tensors(L):
    for call in norm_calls(norm_tensors()):
        with pytest.raises(TypeError, match="q must be a CUDA tensor"):
            call()
        with pytest.raises(TypeError):
            call(eps="x")
    t = norm_tensors()
    with pytest.raises(TypeError, match="dq must be a bf16 or fp32"):
        attn.qk_norm_rope_backward(cpu(5, 4, 64), cpu(5, 2, 128), *t.values())
    with pytest.raises(TypeError, match="dk must be a bf16 or fp32"):
        attn.qk_norm_rope_backward(cpu(5, 4, 128), cpu(5, 2, 128, dtype=torch.float16), *t.values())


@pytest.mark.parametrize("name,bad", [
    ("v", cpu(5, 4, 128)), ("v", cpu(5, 2, 128, dtype=F32)), ("slots", cpu(5, dtype=torch.int64)),
    ("slots", cpu(1, 5, dtype=I32)), ("k_cache", cpu(3, 16, 2, 128, dtype=F32)), ("k_cache", cpu(48, 2, 128)),
    ("k_cache", cpu(3, 2, 16, 128).transpose(1, 2)), ("k_cache", cpu(3, 16, 4, 128)),
    ("v_cache", cpu(3, 16, 4, 128)), ("v_cache", cpu(4, 16, 2, 128)), ("v_cache", cpu(3, 16, 2, 128, dtype=F8))])
def test_cache_binding_refuses(L, name, bad):
    t = norm_tensors()
    x = dict(v=cpu(5, 2, 128), slots=cpu(5, dtype=I32), k_cache=cpu(3, 16, 2, 128), v_cache=cpu(3, 16, 2, 128))
    x[name] = bad
    if name == "k_cache" and bad.shape == (3, 16, 4, 128):
        x["v_cache"] = bad
    with pytest.raises(TypeError, match=name):
        attn.qk_norm_rope_cache(t["q"], t["k"], x["v"], *list(t.values())[2:], x["slots"], x["k_cache"], x["v_cache"])


@pytest.mark.parametrize("name,bad", [
    ("q", cpu(2, 4, 128, dtype=torch.float16)), ("q", cpu(2, 1, 4, 128)), ("q", cpu(4, 2, 128).transpose(0, 1)),
    ("page_table", cpu(3, 4, dtype=I32)), ("page_table", cpu(2, 4, dtype=torch.int64)), ("page_table", cpu(8, dtype=I32)),
    ("seq_lens", cpu(2)), ("seq_lens", cpu(2, 1, dtype=I32)), ("k_cache", cpu(8, 16, 2, 64)),
    ("v_cache", cpu(8, 16, 2, 128, dtype=F8)), ("k_cache", None)])
def test_decode_binding_refuses(L, name, bad):
    t = dict(q=cpu(2, 4, 128), k_cache=cpu(8, 16, 2, 128), v_cache=cpu(8, 16, 2, 128), page_table=cpu(2, 4, dtype=I32),
             seq_lens=cpu(2, dtype=I32))
    with pytest.raises(TypeError, match="q must be a CUDA tensor"):
        attn.decode_paged(*t.values())
    t[name] = bad
    if name == "k_cache" and bad is not None:
        t["v_cache"] = bad
    with pytest.raises(TypeError, match=name):
        attn.decode_paged(*t.values())
    with pytest.raises(ValueError):
        attn.decode_paged(cpu(2, 4, 128), *list(t.values())[1:], window=(3, -2))


class _OnOther(torch.Tensor):
    """A CPU tensor that says it is on a second GPU."""

    @property
    def device(self):
        return torch.device("cuda", 1)


def test_a_stream_of_another_device_is_refused(L, monkeypatch):
    """Calls run on the device's current stream: one that another device's stream
    was given to would run elsewhere than asked."""
    class Stream:
        device, cuda_stream = torch.device("cuda", 0), 0x100
    monkeypatch.setattr(attn, "_torch_stream", lambda stream, device: Stream())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: Stream())
    t = norm_tensors(q=cpu(5, 4, 128).as_subclass(_OnOther))
    x = cpu(1, 16, 2, 64).as_subclass(_OnOther)
    calls = [lambda: attn.attention(x, x, x, stream=7), lambda: attn.attention(x, x, x, window=(3, 0), sinks=1, stream=7),
             lambda: attn.decode_paged(t["q"], x, x, None, None, stream=7)]
    for call in calls + [lambda call=call: call(stream=7) for call in norm_calls(t)]:
        with pytest.raises(TypeError, match="stream is of cuda:0"):
            call()


# ------------------------------------------------- windows with first tokens

def call_fwd_sinks(L, **kw):
    a = dict(q=P, k=P, v=P, o=P, lse=P, B=1, Hq=2, Hkv=2, Sq=16, Sk=16, D=128, scale=0.1, causal=1, wl=7, wr=-1,
             sinks=4, ws=None, wsb=0, opts=None)
    a.update(kw)
    return L.attn_fwd_sinks(a["q"], a["k"], a["v"], a["o"], a["lse"], a["B"], a["Hq"], a["Hkv"], a["Sq"], a["Sk"],
                            a["D"], a["scale"], a["causal"], a["wl"], a["wr"], a["sinks"], a["ws"], a["wsb"],
                            None if a["opts"] is None else ctypes.byref(a["opts"]), None)


def call_bwd_sinks(L, **kw):
    a = dict(q=P, k=P, v=P, o=P, lse=P, dout=P, dq=P, dk=P, dv=P, B=1, Hq=2, Hkv=2, Sq=16, Sk=16, D=128, scale=0.1,
             causal=1, wl=7, wr=-1, sinks=4, ws=P, wsb=1 << 24, opts=None)
    a.update(kw)
    return L.attn_bwd_sinks(*[a[n] for n in ("q", "k", "v", "o", "lse", "dout", "dq", "dk", "dv", "B", "Hq", "Hkv",
                                             "Sq", "Sk", "D", "scale", "causal", "wl", "wr", "sinks", "ws", "wsb")],
                            None if a["opts"] is None else ctypes.byref(a["opts"]), None)


@pytest.mark.parametrize("call", [call_fwd_sinks, call_bwd_sinks])
@pytest.mark.parametrize("kw,status", [
    (dict(sinks=-1), INV), (dict(q=0), INV), (dict(lse=0), INV), (dict(B=0), INV), (dict(Hq=3, Hkv=2), INV),
    (dict(D=96), UNS), (dict(scale=0.0), INV), (dict(wl=-2), INV), (dict(wr=-2), INV), (dict(v=P + 8), MIS)])
def test_sinks_refusals(L, call, kw, status):
    assert call(L, **kw) == status
    assert L.attn_last_error_detail().decode() != ""


def test_sinks_forward_workspace(L):
    # 777 queries of 8 heads are 4 x 8 items of 256 rows: 4 parts of two blocks or more each fill 148 SMs
    need = attn.sinks_workspace_size(1, 8, 2, 777, 2345, 64, True, (500, 0), 130)
    assert need == 4 * 777 * 8 * 65 * 4  # (500 + 255) / 128 + 1 steps of the window, 2 of first keys: 8, in 4 parts
    assert attn.sinks_workspace_size(1, 8, 2, 777, 2345, 64, True, (5000, 0), 130) == 4 * 777 * 8 * 65 * 4
    assert attn.sinks_workspace_size(2, 16, 16, 8192, 8192, 128, True, (1023, 0), 4) == 0  # fills the device
    assert attn.sinks_workspace_size(1, 2, 2, 100, 200, 128, True, (10, 0), 4) == 0  # one block
    assert attn.sinks_workspace_size(1, 8, 2, 777, 2345, 64, True, (-1, 0), 4) == 0
    assert attn.sinks_workspace_size(1, 8, 2, 777, 2345, 64, True, (500, 0), 0) == 0
    kw = dict(Hq=8, Sq=777, Sk=2345, D=64, wl=500, sinks=130, wsb=need)
    assert call_fwd_sinks(L, **{**kw, "ws": P, "wsb": need - 1}) == INV
    assert call_fwd_sinks(L, **{**kw, "ws": P + 4}) == MIS


def test_sinks_workspace(L):
    size = attn.bwd_workspace_size(2, 16, 16, 4096, 4096, 128, 4)
    # D_i, and for the one block with first keys four parts of 8 of the 32 query blocks: fp32 dK and dV
    assert size == 2 * 16 * 4096 * 4 + 4 * 1 * 2 * 16 * 2 * 128 * 128 * 4
    assert attn.bwd_workspace_size(2, 16, 16, 4096, 4096, 128, 0) == 2 * 16 * 4096 * 4
    assert L.attn_bwd_sinks_workspace_size(2, 16, 0, 4096, 4096, 128, 4) == 2 * 16 * 4096 * 4
    assert L.attn_bwd_sinks_workspace_size(0, 16, 16, 4096, 4096, 128, 4) == 0
    # one key head and 8 key blocks: the other 7 are cut too, into at most 148 / 8 parts
    size = attn.bwd_workspace_size(1, 32, 1, 1000, 1000, 64, 4)
    assert size == 32 * 1000 * 4 + (32 * 8 // 8 + 18 * 7) * 2 * 128 * 64 * 4
    # more first keys than keys; at most 64 parts
    assert attn.bwd_workspace_size(1, 8, 1, 1 << 16, 130, 64, 10 ** 6) == 8 * (1 << 16) * 4 + 64 * 2 * 2 * 128 * 64 * 4
    need = attn.bwd_workspace_size(1, 2, 2, 16, 16, 128, 4)
    assert call_bwd_sinks(L, wsb=need - 1) == INV


@pytest.mark.parametrize("name,bad", [
    ("q", cpu(1, 16, 2, 64, dtype=F32)), ("q", cpu(16, 2, 64)), ("q", cpu(1, 2, 16, 64).transpose(1, 2)),
    ("k", cpu(2, 16, 2, 64)), ("k", cpu(1, 16, 2, 128)), ("k", None), ("v", cpu(1, 17, 2, 64)),
    ("v", cpu(1, 16, 2, 64, dtype=F32)), ("o", cpu(1, 16, 1, 64)), ("lse", cpu(1, 2, 16)), ("lse", cpu(1, 16, 2, dtype=F32)),
    ("dout", cpu(1, 16, 2, 64, dtype=F32))])
def test_sinks_bindings_refuse(L, name, bad):
    x = cpu(1, 16, 2, 64)
    t = dict(q=x, k=x, v=x, o=x, lse=cpu(1, 2, 16, dtype=F32), dout=x)
    kw = dict(causal=True, window=(4, 0), sinks=2)
    for call in (lambda: attn.attention(t["q"], t["k"], t["v"], **kw), lambda: attn.attention_backward(*t.values(), **kw)):
        with pytest.raises(TypeError, match="q must be a CUDA tensor"):
            call()
    t[name] = bad
    if name in "qkv":
        with pytest.raises(TypeError, match=name):
            attn.attention(t["q"], t["k"], t["v"], **kw)
    with pytest.raises(TypeError, match=name):
        attn.attention_backward(*t.values(), **kw)
    with pytest.raises(attn.AttnError) as e:
        attn.attention(x, x, x, doc_offsets=[0, 16], **kw)
    assert e.value.status == attn.ATTN_ERR_UNSUPPORTED
    with pytest.raises(TypeError):
        attn.attention(x, x, x, causal=True, window=(4, 0), sinks="2")


def test_sinks_beside_documents_are_refused(L):
    q, lse = stand_in(1, 16, 2, 64), stand_in(1, 2, 16, dtype=torch.float32)
    docs = stand_in(2, dtype=torch.int32)
    with pytest.raises(attn.AttnError) as e:
        attn.attn_fwd(q, q, q, q, lse, scale=0.1, causal=True, window=(4, 0), doc_offsets=docs, sinks=2, stream=0)
    assert e.value.status == attn.ATTN_ERR_UNSUPPORTED
    dq = stand_in(1, 16, 2, 64, dtype=torch.float32)
    with pytest.raises(attn.AttnError):
        attn.attn_bwd(q, q, q, q, lse, q, dq, q, q, stand_in(1 << 20, dtype=torch.uint8), scale=0.1, window=(4, 0),
                      doc_offsets=docs, sinks=2, stream=0)
    with pytest.raises(TypeError):
        attn.attn_fwd(q, stand_in(1, 16, 4, 64), q, q, lse, scale=0.1, window=(4, 0), sinks=2, stream=0)
    with pytest.raises(attn.AttnError) as e:
        attn.attn_fwd(q, q, q, q, lse, scale=0.1, window=(4, 0), sinks=-2, stream=0)
    assert e.value.status == attn.ATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("sinks", [0, 2])
def test_a_key_that_is_no_tensor_is_refused_by_name(L, sinks):
    q, lse, dq = stand_in(1, 16, 2, 64), stand_in(1, 2, 16, dtype=F32), stand_in(1, 16, 2, 64, dtype=F32)
    for k in (None, [1.0], 3):
        with pytest.raises(TypeError, match="k must be"):
            attn.attn_bwd(q, k, q, q, lse, q, dq, q, q, stand_in(1 << 20, dtype=torch.uint8), scale=0.1, window=(4, 0),
                          sinks=sinks, stream=0)


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU path only")
def test_valid_sinks_calls_without_gpu_report_cuda_error(L):
    for sinks in (0, 4, 1000):
        assert call_fwd_sinks(L, sinks=sinks) == attn.ATTN_ERR_CUDA
        assert call_bwd_sinks(L, sinks=sinks) == attn.ATTN_ERR_CUDA
