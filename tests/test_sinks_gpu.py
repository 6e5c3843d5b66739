"""GPU parity of attention with a sliding window and first tokens that stay
visible (forward and backward) against plain 64-bit arithmetic.

Tolerances, from the roundings alone.  Forward: as in the decode's tests, with
d = 2^-8 for the weights' rounding to bf16 and 2^-13 for the cubic that stands
in for some exponentials (7.5e-5 of the value).  Backward, element by element:
P and dS are rounded to bf16 (2^-8) after an exponential within 2^-13, and dS
= P (dP - D) carries the fp32 errors of dP and D (D values of the head summed:
D 2^-23 of their terms' sizes); the results sum these over the keys or rows,
and dK, dV are rounded once more.
"""
import math

import pytest
import torch

from tiled_attention_blackwell_b200 import attn, build
from tiled_attention_blackwell_b200.workloads import make_tensors

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    build.build()
    attn.lib()
    yield
    assert attn.device_status() == attn.ATTN_OK


def visible(Sq, Sk, causal, window, sinks):
    i = torch.arange(Sq)[:, None] + (Sk - Sq)
    j = torch.arange(Sk)[None, :]
    see = torch.ones(Sq, Sk, dtype=torch.bool)
    if causal:
        see &= j <= i
    if window[1] >= 0:
        see &= j <= i + window[1]
    if window[0] >= 0:
        see &= (j >= i - window[0]) | (j < sinks)
    return see


def scores(q, k, b, h, G, scale, see, softcap, slopes):
    """(masked scores, their derivative by the scaled product, sizes of their terms) of one head."""
    qh, kh = q[b, :, h], k[b, :, h // G]
    s = scale * qh @ kh.T
    size = scale * qh.abs() @ kh.abs().T
    ds = torch.ones_like(s)
    if softcap:
        ds = 1 - torch.tanh(s / softcap) ** 2
        s = softcap * torch.tanh(s / softcap)
        size = size + 2 * softcap
    if slopes is not None:
        Sq, Sk = s.shape
        dist = (torch.arange(Sq)[:, None] + (Sk - Sq) - torch.arange(Sk)[None, :]).abs().double()
        s = s - float(slopes[h]) * dist
        size = size + float(slopes[h]) * dist
    return s.masked_fill(~see, -math.inf), ds, size


def check_forward(t, o, lse, scale, see, softcap=0.0, slopes=None):
    q, k, v = (t[n].double() for n in ("q", "k", "v"))
    D, G = q.shape[-1], q.shape[2] // k.shape[2]
    o, lse = o.double().cpu(), lse.double().cpu()
    assert not torch.isnan(o).any()
    some = see.any(-1)
    for b in range(q.shape[0]):
        for h in range(q.shape[2]):
            s, _, size = scores(q, k, b, h, G, scale, see, softcap, slopes)
            want = torch.logsumexp(s, -1)
            p = torch.where(see, (s - want[:, None]).exp(), 0.0)
            vh = v[b, :, h // G]
            ref = p @ vh
            e = D * 2.0 ** -23 * float(size.max())
            d = 2.0 ** -8 + 2.0 ** -13 + e
            bound = 2 * d * (p @ vh.abs()) + 2.0 ** -8 * ref.abs()
            assert ((o[b, :, h] - ref).abs() <= bound).all(), float(((o[b, :, h] - ref).abs() - bound).max())
            assert torch.isneginf(lse[b, h][~some]).all() and (o[b, :, h][~some] == 0).all()
            err = (lse[b, h] - want).abs()[some]
            assert (err <= e + 2.0 ** -13 + 2.0 ** -22 * want[some].abs()).all(), float(err.max())


def check_backward(t, o, lse, grads, scale, see, softcap=0.0, slopes=None):
    q, k, v, do = (t[n].double() for n in ("q", "k", "v", "dout"))
    D, G = q.shape[-1], q.shape[2] // k.shape[2]
    o, lse = o.double().cpu(), lse.double().cpu()
    want = [torch.zeros_like(x) for x in (q, k, v)]
    bound = [torch.zeros_like(x) for x in (q, k, v)]
    for b in range(q.shape[0]):
        for h in range(q.shape[2]):
            s, f, size = scores(q, k, b, h, G, scale, see, softcap, slopes)
            p = torch.where(see, (s - lse[b, h][:, None]).exp(), 0.0)
            qh, kh, vh, dh = q[b, :, h], k[b, :, h // G], v[b, :, h // G], do[b, :, h]
            delta = (dh * o[b, :, h]).sum(-1, keepdim=True)
            ds = p * f * (dh @ vh.T - delta)
            e = D * 2.0 ** -23
            fp32 = p * (dh.abs() @ vh.abs().T + (dh * o[b, :, h]).abs().sum(-1, keepdim=True)) * e
            rel = 2.0 ** -8 + 2.0 ** -12 + e * float(size.max())
            # the cap's derivative comes from the same exponential: off by 2^-20 of one
            eds = rel * ds.abs() + fp32 + (2.0 ** -18 * p * (dh @ vh.T - delta).abs() if softcap else 0.0)
            ep = rel * p
            want[0][b, :, h] = scale * ds @ kh
            bound[0][b, :, h] = scale * eds @ kh.abs() + 2.0 ** -20 * scale * ds.abs() @ kh.abs()
            want[1][b, :, h // G] += scale * ds.T @ qh
            bound[1][b, :, h // G] += scale * eds.T @ qh.abs() + 2.0 ** -18 * scale * ds.T.abs() @ qh.abs()
            want[2][b, :, h // G] += p.T @ dh
            bound[2][b, :, h // G] += ep.T @ dh.abs() + 2.0 ** -18 * p.T @ dh.abs()
    for i, (got, name) in enumerate(zip(grads, ("dq", "dk", "dv"))):
        got = got.double().cpu()
        b = bound[i] + (0.0 if i == 0 else 2.0 ** -8 * want[i].abs())
        assert not torch.isnan(got).any(), name
        assert ((got - want[i]).abs() <= b + 1e-30).all(), (name, float(((got - want[i]).abs() - b).max()))


def case(B, Hq, Hkv, Sq, Sk, D, seed, *, causal=True, window=(100, 0), sinks=4, softcap=None, slopes=None, std=1.0):
    t = make_tensors(B, Hq, Hkv, Sq, Sk, D, seed, with_dout=True, qk_std=std)
    g = {n: x.to(DEV) for n, x in t.items()}
    kw = dict(scale=D ** -0.5, causal=causal, window=window, sinks=sinks, softcap=softcap,
              alibi_slopes=None if slopes is None else slopes.to(DEV))
    o, lse = attn.attention(g["q"], g["k"], g["v"], **kw)
    grads = attn.attention_backward(g["q"], g["k"], g["v"], o, lse, g["dout"], **kw)
    see = visible(Sq, Sk, causal, window, sinks)
    check_forward(t, o, lse, D ** -0.5, see, softcap or 0.0, slopes)
    check_backward(t, o, lse, grads, D ** -0.5, see, softcap or 0.0, slopes)
    return g, kw, o, lse, grads


@pytest.mark.parametrize("S", [1, 2, 127, 128, 129, 255, 256, 257, 400, 900])
@pytest.mark.parametrize("D", [64, 128])
def test_lengths(S, D):
    case(1, 2, 2, S, S, D, seed=S, window=(100, 0), sinks=4)


@pytest.mark.parametrize("window,sinks", [((0, 0), 1), ((0, 0), 128), ((1, 0), 129), ((127, 0), 4), ((128, 0), 127),
                                          ((129, 0), 130), ((200, 0), 256), ((300, 0), 257), ((63, 0), 500),
                                          ((100, 0), 699), ((100, 0), 700), ((10, 0), 5000), ((699, 0), 4),
                                          ((100, -1), 5), ((50, 70), 9)])
def test_windows_and_sinks(window, sinks):
    case(1, 2, 1, 700, 700, 128, seed=sinks, window=window, sinks=sinks)
    case(1, 1, 1, 450, 450, 64, seed=sinks, window=window, sinks=sinks)


@pytest.mark.parametrize("causal,window", [(False, (60, 30)), (False, (0, 0)), (False, (40, -1)), (False, (300, 200))])
@pytest.mark.parametrize("sinks", [3, 140])
def test_without_causal(causal, window, sinks):
    case(1, 2, 2, 600, 600, 64, seed=5, causal=causal, window=window, sinks=sinks)
    case(1, 2, 2, 300, 500, 128, seed=6, causal=causal, window=window, sinks=sinks)


@pytest.mark.parametrize("Sq,Sk", [(1, 700), (129, 1000), (700, 1), (700, 130), (500, 300), (33, 64), (777, 1345)])
@pytest.mark.parametrize("sinks", [2, 200])
def test_queries_and_keys_of_unequal_length(Sq, Sk, sinks):
    case(1, 2, 1, Sq, Sk, 128, seed=Sq, window=(150, 0), sinks=sinks)
    case(1, 2, 1, Sq, Sk, 64, seed=Sq, window=(150, 0), sinks=sinks, causal=False)


@pytest.mark.parametrize("heads", [(4, 1), (6, 3), (12, 2)])
def test_grouped_heads_and_batches(heads):
    case(2, *heads, 520, 520, 128, seed=heads[0], window=(130, 0), sinks=4)
    case(3, *heads, 260, 260, 64, seed=heads[0], window=(20, 0), sinks=150)


@pytest.mark.parametrize("heads", [(8, 1), (32, 1), (6, 2)])
@pytest.mark.parametrize("sinks", [3, 200])
def test_few_key_heads_whose_query_heads_are_cut_into_parts(heads, sinks):
    case(1, *heads, 600, 600, 64, seed=sinks, window=(150, 0), sinks=sinks)
    case(1, *heads, 130, 700, 128, seed=sinks, window=(70, 40), sinks=sinks, causal=False)


@pytest.mark.parametrize("softcap,with_slopes", [(15.0, False), (None, True), (4.0, True)])
def test_score_modifiers(softcap, with_slopes):
    slopes = 2.0 ** -torch.arange(2, 6).float() if with_slopes else None
    for D in (64, 128):
        case(1, 4, 2, 420, 420, D, seed=D, window=(90, 0), sinks=6, softcap=softcap, slopes=slopes, std=1.5)


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_exponential_modes_and_thresholds(mode):
    t = make_tensors(1, 2, 2, 600, 600, 128, 3, qk_std=1.5)
    g = {n: x.to(DEV) for n, x in t.items()}
    for tau in (0.0, 8.0):
        o, lse = attn.attention(g["q"], g["k"], g["v"], causal=True, window=(120, 0), sinks=4,
                                options=attn.default_options(exp2_mode=mode, rescale_threshold=tau))
        check_forward(t, o, lse, 128 ** -0.5, visible(600, 600, True, (120, 0), 4))


@pytest.mark.parametrize("D", [64, 128])
def test_a_window_over_everything_is_plain_attention(D):
    t = make_tensors(1, 4, 2, 500, 500, D, 9, with_dout=True)
    g = {n: x.to(DEV) for n, x in t.items()}
    o, lse = attn.attention(g["q"], g["k"], g["v"], causal=True)
    # Without a lower end the first keys change nothing: the same kernel runs.
    o2, lse2 = attn.attention(g["q"], g["k"], g["v"], causal=True, window=(-1, 0), sinks=4)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    # A window of 500 keys over 500 rows hides nothing, but not bit for bit: a block on the diagonal is summed by
    # groups of 32 keys, with every exponential on MUFU, where the plain kernel sums by pairs of a half.  Both
    # hold the forward's bound.
    o2, lse2 = attn.attention(g["q"], g["k"], g["v"], causal=True, window=(500, 0), sinks=4)
    for out, stat in ((o, lse), (o2, lse2)):
        check_forward(t, out, stat, D ** -0.5, visible(500, 500, True, (500, 0), 4))
    # sinks = 0 is the window alone
    o, lse = attn.attention(g["q"], g["k"], g["v"], causal=True, window=(70, 0))
    want = attn.attention_backward(g["q"], g["k"], g["v"], o, lse, g["dout"], causal=True, window=(70, 0))
    o2, _ = attn.attention(g["q"], g["k"], g["v"], causal=True, window=(70, 0), sinks=0)
    got = attn.attention_backward(g["q"], g["k"], g["v"], o, lse, g["dout"], causal=True, window=(70, 0), sinks=0)
    assert torch.equal(o, o2) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_many_parts_deterministic_captured_and_on_a_side_stream():
    g, kw, o, lse, grads = case(1, 6, 1, 1300, 1300, 128, seed=12, window=(200, 0), sinks=20)
    args = [g[n] for n in ("q", "k", "v")] + [o, lse, g["dout"]]
    assert all(torch.equal(a, b) for a, b in zip(attn.attention_backward(*args, **kw), grads))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = attn.attention_backward(*args, stream=side, **kw)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, grads))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o2, lse2 = attn.attention(*args[:3], **kw)
        got = attn.attention_backward(args[0], args[1], args[2], o2, lse2, g["dout"], **kw)
    for _ in range(2):
        for x in got:
            x.zero_()
        graph.replay()
        assert torch.equal(o, o2) and all(torch.equal(a, b) for a, b in zip(got, grads))


def test_the_decode_sees_what_the_forward_sees():
    """The last row of the forward under a window with sinks is the decode's."""
    Hq, Hkv, D, S, page = 8, 2, 128, 700, 16
    t = make_tensors(1, Hq, Hkv, S, S, D, 14)
    g = {n: x.to(DEV) for n, x in t.items()}
    pages = -(-S // page)
    kc, vc = (torch.nn.functional.pad(g[n][0], (0, 0, 0, 0, 0, pages * page - S)).view(pages, page, Hkv, D)
              for n in ("k", "v"))
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    for n in (S, 300, 1):
        lens = torch.tensor([n], dtype=torch.int32, device=DEV)
        o, lse = attn.decode_paged(g["q"][:, n - 1].contiguous(), kc, vc, table, lens, window=(99, 0), sinks=5)
        see = visible(S, S, True, (99, 0), 5)[n - 1:n, :n]
        one = {"q": t["q"][:, n - 1:n], "k": t["k"][:, :n], "v": t["v"][:, :n]}
        check_forward(one, o.unsqueeze(1), lse.unsqueeze(-1), D ** -0.5, see)
        of, lf = attn.attention(g["q"], g["k"], g["v"], causal=True, window=(99, 0), sinks=5)
        check_forward(one, of[:, n - 1:n], lf[..., n - 1:n], D ** -0.5, see)


def test_a_training_step_of_the_whole_path():
    """Norm and rotation, attention with sinks, and back to the gradients of the
    projection's output and the head weights: against the same path in 64 bits
    by torch's own differentiation.  The intermediate tensors are bf16, so the
    gradients agree to a few times their roundings (in the norm of each)."""
    B, S, Hq, Hkv, D = 2, 300, 4, 2, 64
    gen = torch.Generator().manual_seed(15)
    qkv = torch.randn(B, S, (Hq + 2 * Hkv) * D, generator=gen).to(torch.bfloat16)
    qw, kw = (1 + 0.1 * torch.randn(2, D, generator=gen)).unbind(0)
    do = torch.randn(B, S, Hq, D, generator=gen).to(torch.bfloat16)
    cos, sin = attn.rope_table(S, D, device=DEV)
    pos = torch.arange(S, dtype=torch.int32).repeat(B, 1)

    def parts(x):
        return (y.unflatten(-1, (-1, D)) for y in x.split([Hq * D, Hkv * D, Hkv * D], -1))

    x = qkv.to(DEV)
    q, k, v = parts(x)
    args = (q, k, qw.to(DEV), kw.to(DEV), cos, sin, pos.to(DEV))
    qn, kn = attn.qk_norm_rope(*args)
    mask = dict(causal=True, window=(60, 0), sinks=4)
    v = v.contiguous()
    o, lse = attn.attention(qn, kn, v, **mask)
    dqn, dkn, dv = attn.attention_backward(qn, kn, v, o, lse, do.to(DEV), **mask)
    grad = torch.empty_like(x)
    gq, gk, gv = parts(grad)
    _, _, dqw, dkw = attn.qk_norm_rope_backward(dqn, dkn, *args, dq_in=gq, dk_in=gk)
    gv.copy_(dv)

    xd, qwd, kwd = qkv.double().requires_grad_(), qw.double().requires_grad_(), kw.double().requires_grad_()
    q, k, v = parts(xd)
    c, s = (a.double().cpu()[None, :, None] for a in (cos, sin))

    def norm_rope(y, w):
        y = w * y * (y.pow(2).mean(-1, keepdim=True) + 1e-6).rsqrt()
        a, b = y.chunk(2, -1)
        return torch.cat((a * c - b * s, b * c + a * s), -1)

    q, k = norm_rope(q, qwd).transpose(1, 2), norm_rope(k, kwd).transpose(1, 2).repeat_interleave(2, 1)
    see = visible(S, S, True, (60, 0), 4)
    p = torch.softmax((q @ k.transpose(-1, -2) * D ** -0.5).masked_fill(~see, -math.inf), -1)
    out = (p @ v.transpose(1, 2).repeat_interleave(2, 1)).transpose(1, 2)
    out.backward(do.double())
    for got, want in ((o, out), (grad, xd.grad), (dqw, qwd.grad), (dkw, kwd.grad)):
        got, want = got.double().cpu(), want.detach()
        assert float((got - want).norm() / want.norm()) <= 4 * 2.0 ** -8


@pytest.mark.parametrize("shape", [(1, 2, 1, 1, 700, 128), (1, 8, 2, 777, 2345, 64), (1, 2, 2, 300, 2000, 128), (2, 3, 1, 130, 900, 64),
                                   (1, 4, 4, 260, 100, 128)])
@pytest.mark.parametrize("window,sinks,causal", [((900, 0), 4, True), ((260, 0), 300, True), ((100, 50), 130, False),
                                                 ((400, -1), 7, False)])
def test_parts_of_a_call_of_few_rows(shape, window, sinks, causal):
    """With a workspace the keys are cut into parts; without, they are not:
    both hold the forward's bound (a part's output is normalised in fp32 and
    weighted by exp of its LSE less the row's, within 2^-18 in all)."""
    B, Hq, Hkv, Sq, Sk, D = shape
    t = make_tensors(B, Hq, Hkv, Sq, Sk, D, Sq + sinks)
    g = {n: x.to(DEV) for n, x in t.items()}
    see = visible(Sq, Sk, causal, window, sinks)
    size = attn.sinks_workspace_size(B, Hq, Hkv, Sq, Sk, D, causal, window, min(sinks, Sk))
    o, lse = torch.empty_like(g["q"]), torch.empty(B, Hq, Sq, device=DEV)
    for ws in (None, torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)) if size else (None,):
        for out in (o, lse):
            out.fill_(float("nan"))
        attn.attn_fwd(g["q"], g["k"], g["v"], o, lse, scale=D ** -0.5, causal=causal, window=window, sinks=sinks,
                      workspace=ws)
        check_forward(t, o, lse, D ** -0.5, see)
    again = attn.attention(g["q"], g["k"], g["v"], causal=causal, window=window, sinks=sinks)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)


def test_parts_with_score_modifiers_and_captured():
    slopes = 2.0 ** -torch.arange(2, 6).float()
    t = make_tensors(1, 4, 2, 200, 1500, 128, 31, qk_std=1.5)
    g = {n: x.to(DEV) for n, x in t.items()}
    kw = dict(causal=True, window=(1000, 0), sinks=20, softcap=8.0, alibi_slopes=slopes.to(DEV))
    assert attn.sinks_workspace_size(1, 4, 2, 200, 1500, 128, True, (1000, 0), 20) > 0
    o, lse = attn.attention(g["q"], g["k"], g["v"], **kw)
    check_forward(t, o, lse, 128 ** -0.5, visible(200, 1500, True, (1000, 0), 20), 8.0, slopes)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = attn.attention(g["q"], g["k"], g["v"], **kw)
    for _ in range(2):
        for x in got:
            x.zero_()
        graph.replay()
        assert torch.equal(got[0], o) and torch.equal(got[1], lse)


def test_nan_and_infinity_stay_in_their_rows():
    """A NaN in a query row, and in a key of the window, reaches the rows that
    see it and no other, in one piece and in parts alike."""
    shape, window, sinks = (1, 2, 1, 200, 1500, 128), (900, 0), 4
    t = make_tensors(*shape, 33)
    t["q"][0, 140, 1, 7] = float("nan")
    t["q"][0, 190, 0, 3] = float("inf")
    t["k"][0, 450, 0, 9] = float("nan")
    see = visible(200, 1500, True, window, sinks)
    g = {n: x.to(DEV) for n, x in t.items()}
    bad = see[:, 450].repeat(2, 1)
    bad[1, 140] = bad[0, 190] = True
    assert 0 < int(bad.sum()) < bad.numel() // 2
    size = attn.sinks_workspace_size(*shape, True, window, sinks)
    assert size > 0
    for ws in (None, torch.empty(size, dtype=torch.uint8, device=DEV)):
        o, lse = torch.empty_like(g["q"]), torch.empty(1, 2, 200, device=DEV)
        attn.attn_fwd(g["q"], g["k"], g["v"], o, lse, scale=128 ** -0.5, causal=True, window=window, sinks=sinks,
                      workspace=ws)
        assert torch.equal(torch.isnan(o[0]).all(-1).T.cpu(), bad)
        assert torch.isfinite(o[0].transpose(0, 1)[~bad.to(DEV)]).all()
        assert torch.isfinite(lse[0][~bad.to(DEV)]).all()


def test_first_keys_that_fill_the_device_are_not_cut():
    """Many first keys of many heads: the workspace holds no parts, or few."""
    rows = attn.bwd_workspace_size(2, 16, 16, 2048, 2048, 64)
    assert attn.bwd_workspace_size(2, 16, 16, 2048, 2048, 64, sinks=2048) == \
        attn.bwd_workspace_size(2, 16, 16, 2048, 2048, 64, sinks=2 ** 40)
    assert attn.bwd_workspace_size(40, 16, 16, 2048, 2048, 64, sinks=4) == \
        attn.bwd_workspace_size(40, 16, 16, 2048, 2048, 64)
    assert attn.bwd_workspace_size(2, 16, 16, 2048, 2048, 64, sinks=4) > rows
    # 9 blocks of 66 heads: whole, where each would have two parts; of 40 heads: two parts for three.
    case(1, 66, 66, 1100, 1100, 64, seed=34, window=(100, 0), sinks=1090)
    case(1, 80, 40, 1100, 1100, 64, seed=35, window=(100, 0), sinks=1090)


def test_two_streams_at_once():
    """Two calls in flight together, each with its own allocations."""
    a, b = (make_tensors(1, 4, 2, 300, 1500, 128, s, with_dout=True) for s in (36, 37))
    kw = dict(causal=True, window=(700, 0), sinks=4)
    ga, gb = ({n: x.to(DEV) for n, x in t.items()} for t in (a, b))

    def both(g, stream=None):
        o, lse = attn.attention(g["q"], g["k"], g["v"], stream=stream, **kw)
        return (o, lse, *attn.attention_backward(g["q"], g["k"], g["v"], o, lse, g["dout"], stream=stream, **kw))

    want = [both(ga), both(gb)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for handle in (lambda s: s, lambda s: s.cuda_stream):
        got = [both(g, handle(s)) for _ in range(4) for g, s in zip((ga, gb), streams)]
        torch.cuda.synchronize()
        for i, res in enumerate(got):
            assert all(torch.equal(x, y) for x, y in zip(res, want[i % 2]))


@pytest.mark.parametrize("Sq", [1000, 200])
@pytest.mark.parametrize("parts", [False, True])
def test_a_wait_that_runs_out_is_reported(Sq, parts):
    """As for the plain forward: the first CTA withholds a key copy (nothing
    faults), in one piece (without a workspace) and in parts; the next call is
    right again."""
    shape, mask = (1, 4, 2, Sq, 1500, 128), dict(causal=True, window=(900, 0), sinks=4)
    t = make_tensors(*shape, 38)
    g = {n: x.to(DEV) for n, x in t.items()}
    opts = attn.default_options(wait_timeout_us=20000, debug_withhold_kv=1)
    size = attn.sinks_workspace_size(*shape, True, (900, 0), 4)
    assert size > 0
    ws = torch.zeros(size, dtype=torch.uint8, device=DEV) if parts else None
    o, lse = torch.empty_like(g["q"]), torch.empty(1, 4, Sq, device=DEV)
    attn.attn_fwd(g["q"], g["k"], g["v"], o, lse, scale=128 ** -0.5, options=opts, workspace=ws, **mask)
    assert attn.device_status() == attn.ATTN_ERR_DEVICE_TIMEOUT
    assert attn.device_status() == attn.ATTN_OK
    attn.attn_fwd(g["q"], g["k"], g["v"], o, lse, scale=128 ** -0.5, workspace=ws, **mask)
    check_forward(t, o, lse, 128 ** -0.5, visible(Sq, 1500, True, (900, 0), 4))


def test_tiles_at_the_ends_of_rows_and_groups():
    """Last tiles of one row, heads that do not fill the last schedule group, and
    rows before the first key beside rows behind it."""
    for heads in ((9, 9), (20, 2)):
        case(1, *heads, 257, 257, 64, seed=39, window=(60, 0), sinks=3)
        case(3, *heads, 129, 100, 64, seed=40, window=(60, 0), sinks=3)
    case(1, 2, 2, 513, 300, 128, seed=41, window=(130, 0), sinks=200)
    case(1, 2, 2, 640, 200, 128, seed=42, causal=False, window=(130, 100), sinks=20)


def test_the_output_may_be_a_view_aligned_to_16_bytes():
    t = make_tensors(1, 2, 2, 300, 300, 64, 43)
    g = {n: x.to(DEV) for n, x in t.items()}
    kw = dict(scale=0.125, causal=True, window=(80, 0), sinks=4)
    want, _ = attn.attention(g["q"], g["k"], g["v"], **kw)
    buf = torch.full((300 * 2 * 64 + 24,), 7.0, dtype=torch.bfloat16, device=DEV)
    o, lse = buf[8:8 + 300 * 2 * 64].view(1, 300, 2, 64), torch.empty(1, 2, 300, device=DEV)
    attn.attn_fwd(g["q"], g["k"], g["v"], o, lse, **kw)
    assert torch.equal(o, want) and (buf[:8] == 7).all() and (buf[-16:] == 7).all()
