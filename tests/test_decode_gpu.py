"""GPU parity of the decode over a paged cache against plain 64-bit arithmetic.

Tolerances, from the roundings alone.  The output is sum w_j v_j / sum w_j
with the same rounded weights above and below, each within
d = 2^-8 (bf16 weights; 2^-11 for the f16 ones of an 8-bit cache) of the
exact one, so it is off by at most 2 d sum p_j |v_j| before its own rounding
to bf16 (2^-8 |o|); f16 weights below 2^-14 of the largest are off by up to
2^-25 instead.  A score is off by D 2^-23 of the sizes of its terms (fp32
sums in the tensor cores), which moves a weight by as much again, and the
LSE by that, the rounding of ex2 and log2 (2^-20) and its own (2^-23 |LSE|).
"""
import math

import pytest
import torch

from tiled_attention_blackwell_b200 import attn, build

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    build.build()
    attn.lib()
    yield
    assert attn.device_status() == attn.ATTN_OK


def problem(lens, Hq, Hkv, D, page, dtype, seed, *, spare=2, q_std=1.0, garbage=True):
    """Caches whose hidden places hold NaN, a shuffled page table whose
    unused entries are out of range, and the rest of a call's arguments."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    width = max(max(need), 1) + 1
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), width), 2 ** 30, dtype=torch.int32)
    at = 0
    kc, vc = (torch.full((pages, page, Hkv, D), float("nan") if garbage else 0.0) for _ in range(2))
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        j = torch.arange(n)
        kc[table[b].long()[j // page], j % page] = torch.randn(n, Hkv, D, generator=g)
        vc[table[b].long()[j // page], j % page] = torch.randn(n, Hkv, D, generator=g)
    kd, vd = (1.0, 1.0) if dtype != FP8 else (1 / 60, 1 / 33)
    kc, vc = ((x / d).to(dtype) for x, d in ((kc, kd), (vc, vd)))
    q = (q_std * torch.randn(len(lens), Hq, D, generator=g)).to(torch.bfloat16)
    return dict(q=q, kc=kc, vc=vc, table=table, lens=torch.tensor(lens, dtype=torch.int32), kd=kd, vd=vd)


def reference(t, *, scale, window=-1, sinks=0, softcap=0.0, slopes=None):
    """(o, its bound, lse, its bound), in 64 bits on the CPU."""
    q, kc, vc, table = t["q"].double(), t["kc"], t["vc"], t["table"].long()
    B, Hq, D = q.shape
    page, Hkv = kc.shape[1:3]
    G = Hq // Hkv
    o, ob = torch.zeros(B, Hq, D, dtype=torch.float64), torch.zeros(B, Hq, D, dtype=torch.float64)
    lse, lb = torch.full((B, Hq), -math.inf, dtype=torch.float64), torch.zeros(B, Hq, dtype=torch.float64)
    f8 = kc.dtype == FP8
    for b, n in enumerate(t["lens"].tolist()):
        if n == 0:
            continue
        j = torch.arange(n)
        if window >= 0:
            j = j[(j >= n - 1 - window) | (j < sinks)]
        k, v = (c[table[b][j // page], j % page].double() * d for c, d in ((kc, t["kd"]), (vc, t["vd"])))
        for h in range(Hq):
            s = scale * (k[:, h // G] @ q[b, h])
            size = scale * (k[:, h // G].abs() @ q[b, h].abs())
            if softcap:
                s = softcap * torch.tanh(s / softcap)
                size = size + softcap * 2.0  # softcap (1 - 2 r): its terms' sizes
            if slopes is not None:
                s = s - float(slopes[h]) * (n - 1 - j).double()
                size = size + float(slopes[h]) * (n - 1 - j).double()
            lse[b, h] = torch.logsumexp(s, 0)
            p = torch.softmax(s, 0)
            e = D * 2.0 ** -23 * float(size.max())
            d = (2.0 ** -11 if f8 else 2.0 ** -8) + e + 2.0 ** -18
            o[b, h] = p @ v[:, h // G]
            ob[b, h] = 2 * d * (p @ v[:, h // G].abs()) + 2.0 ** -8 * o[b, h].abs()
            if f8:
                ob[b, h] += 2.0 ** -25 * p.max() * v[:, h // G].abs().sum(0) * 2
            lb[b, h] = e + 2.0 ** -18 + 2.0 ** -22 * lse[b, h].abs()
    return o, ob, lse, lb


def run(t, **kw):
    g = {n: x.to(DEV) if torch.is_tensor(x) else x for n, x in t.items()}
    return attn.decode_paged(g["q"], g["kc"], g["vc"], g["table"], g["lens"], k_descale=g["kd"],
                             v_descale=g["vd"], **kw)


def check(t, got, **kw):
    o, lse = (x.double().cpu() for x in got)
    want, ob, want_lse, lb = reference(t, **kw)
    assert not torch.isnan(o).any() and not torch.isnan(lse).any()
    assert ((o - want).abs() <= ob).all(), float(((o - want).abs() - ob).max())
    none = torch.isneginf(want_lse)
    assert torch.equal(torch.isneginf(lse), none)
    assert ((lse - want_lse)[~none].abs() <= lb[~none]).all(), float(((lse - want_lse)[~none].abs() - lb[~none]).max())
    assert (o[none] == 0).all()


LENS = [[1], [0], [16], [17, 0, 1], [1000], [33, 512, 0, 7, 300, 129, 15, 64], [2500, 31], list(range(0, 70))]


@pytest.mark.parametrize("lens", LENS, ids=lambda x: "x".join(map(str, x[:4])))
@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8])
@pytest.mark.parametrize("D", [64, 128])
def test_lengths(lens, dtype, D):
    t = problem(lens, 8, 2, D, 16, dtype, seed=len(lens) + D)
    check(t, run(t), scale=D ** -0.5)


@pytest.mark.parametrize("heads", [(1, 1), (5, 1), (16, 16), (16, 1), (17, 1), (40, 1), (64, 2), (6, 3)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8])
def test_heads(heads, dtype):
    t = problem([130, 700, 3], *heads, 128, 32, dtype, seed=heads[0])
    check(t, run(t), scale=128 ** -0.5)


@pytest.mark.parametrize("page", [16, 48, 64, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8])
def test_page_sizes(page, dtype):
    for D in (64, 128):
        t = problem([1, 255, 256, 257, 1023], 4, 2, D, page, dtype, seed=page)
        check(t, run(t), scale=D ** -0.5)


@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 1), (15, 0), (16, 16), (100, 4), (100, 17), (100, 130),
                                          (600, 40), (5000, 4), (-1, 9), (37, 5000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8])
def test_windows_and_sinks(window, sinks, dtype):
    t = problem([1, 5, 16, 101, 117, 118, 700, 1500], 8, 2, 128, 16, dtype, seed=window + sinks + 3)
    check(t, run(t, window=None if window < 0 else (window, 0), sinks=sinks), scale=128 ** -0.5, window=window,
          sinks=sinks)
    t = problem([700, 129], 4, 4, 64, 32, dtype, seed=1)
    check(t, run(t, window=(window, -1), sinks=sinks), scale=0.125, window=window, sinks=sinks)


def test_more_first_keys_than_fit_an_int_are_all_of_them():
    t = problem([200, 33], 4, 2, 64, 16, torch.bfloat16, seed=74)
    want = run(t, window=(20, 0), sinks=200)
    for sinks in (201, 2 ** 31 - 1, 2 ** 31, 2 ** 40, 10 ** 30):
        got = run(t, window=(20, 0), sinks=sinks)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for sinks in (-1, -2 ** 40):
        with pytest.raises(attn.AttnError) as e:
            run(t, window=(20, 0), sinks=sinks)
        assert e.value.status == attn.ATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8])
@pytest.mark.parametrize("D", [64, 128])
def test_pages_outside_a_window_may_be_given_away(dtype, D):
    """Entries of pages without a visible key are out of range: unused and not
    reported; the pages' old places hold NaN."""
    for heads in ((4, 1), (8, 4)):
        lens, window, sinks, page = [1000, 330, 95, 16, 47], 70, 18, 16
        t = problem(lens, *heads, D, page, dtype, seed=D)
        for b, n in enumerate(lens):
            for i in range(-(-n // page)):
                if i * page >= sinks and i * page + page <= n - 1 - window:
                    old = int(t["table"][b, i])
                    for c in ("kc", "vc"):
                        t[c][old] = torch.full_like(t[c][old].float(), float("nan")).to(dtype)
                    t["table"][b, i] = -1 - i
        got = run(t, window=(window, 0), sinks=sinks)
        assert attn.device_status() == attn.ATTN_OK
        t["table"] = t["table"].clamp_min(0)  # (the reference never looks at those keys)
        check(t, got, scale=D ** -0.5, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8])
def test_score_modifiers_and_scale(dtype):
    slopes = 2.0 ** -torch.arange(1, 9).float()
    t = problem([1, 300, 77], 8, 2, 128, 16, dtype, seed=40, q_std=3.0)
    check(t, run(t, scale=0.3, softcap=20.0), scale=0.3, softcap=20.0)
    check(t, run(t, scale=0.3, alibi_slopes=slopes.to(DEV)), scale=0.3, slopes=slopes)
    check(t, run(t, softcap=5.0, alibi_slopes=slopes.tolist(), window=(90, 0), sinks=3), scale=128 ** -0.5,
          softcap=5.0, slopes=slopes, window=90, sinks=3)


@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8])
def test_rising_scores_and_one_dominating_key(dtype):
    """Scores that grow along the cache (the maximum moves all the time) and a
    key far above the others."""
    t = problem([900], 4, 1, 128, 16, dtype, seed=50)
    ramp = torch.linspace(0, 3, 900)
    tab = t["table"][0].long()
    j = torch.arange(900)
    k = torch.sign(t["q"][0, 0].float()) * ramp[:, None]
    k[450] = 6 * torch.sign(t["q"][0, 0].float())
    t["kc"][tab[j // 16], j % 16, 0] = (k / t["kd"]).to(dtype)
    check(t, run(t), scale=128 ** -0.5)


@pytest.mark.parametrize("heads,n", [((8, 2), 1000), ((8, 8), 77), ((32, 2), 3000), ((6, 3), 20), ((40, 1), 300)])
@pytest.mark.parametrize("D", [64, 128])
def test_weights_of_a_bf16_cache_keep_their_bits(heads, n, D):
    """Beside the output's own rounding (2^-8 of it) only fp32's: weights in two
    bf16 words are off by 2^-17."""
    t = problem([n, 2 * n], *heads, D, 16, torch.bfloat16, seed=n + D, q_std=0.3)
    o, _ = (x.double().cpu() for x in run(t))
    want, bound, _, _ = reference(t, scale=D ** -0.5)
    # the bound holds 2 * 2^-8 sum p |v| for the weights: 2 * 2^-17 in its place
    G = heads[0] // heads[1]
    for b, m in enumerate((n, 2 * n)):
        j = torch.arange(m)
        k, v = (c[t["table"].long()[b][j // 16], j % 16].double() for c in (t["kc"], t["vc"]))
        for h in range(heads[0]):
            p = torch.softmax(k[:, h // G] @ t["q"][b, h].double() * D ** -0.5, 0)
            bound[b, h] -= 2 * (2.0 ** -8 - 2.0 ** -17) * (p @ v[:, h // G].abs())
    assert ((o - want).abs() <= bound).all(), float(((o - want).abs() / bound).max())


@pytest.mark.parametrize("gap", [17.5, 21.0])
@pytest.mark.parametrize("heads", [(8, 8, 128), (12, 3, 128), (8, 8, 64), (20, 1, 64)])
def test_small_weights_beside_a_dominating_key_of_an_8_bit_cache(gap, heads):
    """A first token `gap` nats above n others: all of the output is theirs (its
    V is 0, theirs 1), at weights of 2^-25 and 2^-30 of the largest.  Enough
    sequences, on the same pages, that blocks hold whole pairs.

    f16 weights, 2^7 times the exact ones, are off by half of 2^-24 at most where
    they are subnormal: 2^-32 of the largest weight each."""
    Hq, Hkv, D = heads
    n, page, B = 70000, 80, 600 // Hkv
    pages = n // page
    kc, vc = (torch.zeros(pages, page, Hkv, D, dtype=torch.float32) for _ in range(2))
    kc[0, 0], vc[:] = 1.0, 1.0
    vc[0, 0] = 0.0
    kc, vc = (x.to(FP8).to(DEV) for x in (kc, vc))
    table = torch.arange(pages, dtype=torch.int32, device=DEV).repeat(B, 1)
    lens = torch.full((B,), n, dtype=torch.int32, device=DEV)
    q = torch.ones(B, Hq, D, dtype=torch.bfloat16, device=DEV)
    o, lse = (x.double().cpu() for x in attn.decode_paged(q, kc, vc, table, lens, scale=gap / D))
    total = 1 + (n - 1) * math.exp(-gap)
    want = (n - 1) * math.exp(-gap) / total
    e = D * 2.0 ** -23 * gap
    bound = (2 * (2.0 ** -11 + e + 2.0 ** -18) + 2.0 ** -8) * want + 2.0 ** -32 * (n - 1)
    assert (o - want).abs().max() <= bound, (float(o.min()), float(o.max()), want)
    want = gap + math.log(total)
    assert (lse - want).abs().max() <= e + 2.0 ** -18 + 2.0 ** -22 * want


def test_tiny_and_huge_queries_against_an_8_bit_cache():
    for std in (1e-20, 1e-3, 300.0):
        t = problem([200, 31], 4, 2, 128, 16, FP8, seed=60, q_std=std)
        scale = 128 ** -0.5 / max(std, 1.0)
        check(t, run(t, scale=scale), scale=scale)
    t["q"][0, 1] = 0.0
    t["q"][1, 2, 5] = float("inf")
    o, lse = run(t, scale=scale)
    assert torch.isfinite(o[0]).all() and torch.isnan(o[1, 2]).all() and torch.isfinite(o[1, 3]).all()


def test_many_blocks_share_one_sequence():
    """Long enough that every block takes a part of each pair; also for a
    single key head, whose pair all blocks share."""
    for heads, n in (((8, 1), 9000), ((4, 4), 5000)):
        t = problem([n, 0, 40], *heads, 128, 16, torch.bfloat16, seed=n)
        check(t, run(t), scale=128 ** -0.5)


def test_bit_identical_again_and_with_dirty_workspace():
    t = problem([700, 1300, 64, 1], 16, 2, 128, 16, torch.bfloat16, seed=70)
    want = run(t)
    ws = torch.full((attn.decode_workspace_size(128),), 0xFF, dtype=torch.uint8, device=DEV)
    for _ in range(3):
        got = run(t, workspace=ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_replayed_with_other_lengths_and_two_graphs_of_one_workspace():
    t = problem([700, 1300, 64, 1], 8, 2, 64, 16, torch.bfloat16, seed=71)
    g = {n: x.to(DEV) if torch.is_tensor(x) else x for n, x in t.items()}
    ws = torch.empty(attn.decode_workspace_size(64), dtype=torch.uint8, device=DEV)
    graphs = []
    torch.cuda.synchronize()
    for window in (None, (50, 0)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = attn.decode_paged(g["q"], g["kc"], g["vc"], g["table"], g["lens"], window=window, sinks=4,
                                    workspace=ws)
        graphs.append((graph, got, window))
    for lens in ([700, 1300, 64, 1], [1, 0, 63, 1], [699, 4, 0, 0]):
        g["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        t["lens"] = torch.tensor(lens, dtype=torch.int32)
        for graph, got, window in graphs:
            graph.replay()
            check(t, got, scale=0.125, window=-1 if window is None else window[0], sinks=4)


def test_on_a_side_stream():
    t = problem([700, 64], 8, 2, 128, 16, torch.bfloat16, seed=72)
    want = run(t)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = run(t, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_bad_pages_and_lengths_are_reported_and_stay_in_bounds():
    t = problem([40, 50, 33], 4, 2, 64, 16, torch.bfloat16, seed=73)
    good = reference(t, scale=0.125)
    t["table"][1, 1] = -7
    t["table"][1, 2] = 2 ** 31 - 1
    o, lse = run(t)
    assert attn.device_status() == attn.ATTN_ERR_RANGE
    for b in (0, 2):  # the other sequences are untouched by it
        assert ((o[b].double().cpu() - good[0][b]).abs() <= good[1][b]).all()
    t = problem([40, 50, 33], 4, 2, 64, 16, torch.bfloat16, seed=73)
    t["lens"][0] = -3
    got = run(t)
    assert attn.device_status() == attn.ATTN_ERR_RANGE
    t["lens"][0] = 0
    check(t, got, scale=0.125)
    t["table"] = t["table"][:, :3].contiguous()  # room for 48 keys
    t["lens"][:] = torch.tensor([40, 48, 49])
    t["table"][2, 2] = t["table"][2, 0]
    got = run(t)
    assert attn.device_status() == attn.ATTN_ERR_RANGE
    assert attn.device_status() == attn.ATTN_OK


def test_a_serving_run():
    """Prefill chunks and single tokens through the norm, rotation and cache
    write, then the decode, for two sequences of one 8-bit and one bf16 cache;
    the new token's attention as the definition gives it."""
    Hq, Hkv, D, page, rot = 8, 2, 128, 16, 64
    g = torch.Generator().manual_seed(80)
    cos, sin = attn.rope_table(256, rot, device=DEV)
    qw, kw = ((1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16).to(DEV) for _ in range(2))
    for dtype, d in ((torch.bfloat16, 1.0), (FP8, 1 / 64)):
        kc, vc = (torch.full((12, page, Hkv, D), float("nan")).to(dtype).to(DEV) for _ in range(2))
        table = torch.randperm(12, generator=g).to(torch.int32).view(2, 6)
        lens = [0, 0]
        steps = [(37, 0), (1, 50), (1, 1), (0, 1), (20, 3), (1, 1)]
        for new in steps:
            rows = [(b, lens[b] + i) for b in (0, 1) for i in range(new[b])]
            pad = 3  # tokens behind the last sequence
            pos = torch.tensor([p for _, p in rows] + [0] * pad, dtype=torch.int32)
            slots = torch.tensor([int(table[b, p // page]) * page + p % page for b, p in rows] + [-1] * pad,
                                 dtype=torch.int32)
            qkv = torch.randn(len(rows) + pad, (Hq + 2 * Hkv) * D, generator=g).to(torch.bfloat16).to(DEV)
            q, k, v = (x.unflatten(-1, (-1, D)) for x in qkv.split([Hq * D, Hkv * D, Hkv * D], -1))
            qn = attn.qk_norm_rope_cache(q, k, v, qw, kw, cos, sin, pos.to(DEV), slots.to(DEV), kc, vc,
                                         k_descale=d, v_descale=d)
            lens = [lens[b] + new[b] for b in (0, 1)]
            # the last new token of each sequence (a sequence without one: its old keys, an arbitrary query)
            last = [max([i for i, r in enumerate(rows) if r[0] == b], default=0) for b in (0, 1)]
            t = dict(q=qn[last].cpu(), kc=kc.cpu(), vc=vc.cpu(), table=table,
                     lens=torch.tensor(lens, dtype=torch.int32), kd=d, vd=d)
            check(t, run(t, window=(30, 0), sinks=4), scale=D ** -0.5, window=30, sinks=4)


def test_two_streams_at_once():
    a, b = (problem([700, 64, 2000], 8, 2, 128, 16, d, seed=90) for d in (torch.bfloat16, FP8))
    want = [run(a), run(b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    ga, gb = ({n: x.to(DEV) if torch.is_tensor(x) else x for n, x in t.items()} for t in (a, b))
    torch.cuda.synchronize()
    for handle in (lambda s: s, lambda s: s.cuda_stream):
        got = [run(g, stream=handle(s)) for _ in range(8) for g, s in zip((ga, gb), streams)]
        torch.cuda.synchronize()
        for i, res in enumerate(got):
            assert all(torch.equal(x, y) for x, y in zip(res, want[i % 2]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8])
def test_a_cache_of_more_than_32_bits(dtype):
    """Values, bytes and pages past 2^32: tokens written at the far end and in
    the middle of a large cache, and read back through the decode."""
    Hq, Hkv, D, page = 8, 8, 128, 16
    pages = 2 ** 32 // (page * Hkv * D) + 300
    d = 1.0 if dtype == torch.bfloat16 else 1 / 32
    kc, vc = (torch.zeros(pages, page, Hkv, D, dtype=dtype, device=DEV) for _ in range(2))
    n = 100
    place = torch.tensor([pages - 1, 2 ** 31 // (page * Hkv * D), pages - 299, 1, pages // 2, pages - 7, 0],
                         dtype=torch.int32)
    g = torch.Generator().manual_seed(91)
    q, k, v = (torch.randn(n, h, D, generator=g).to(torch.bfloat16).to(DEV) for h in (Hq, Hkv, Hkv))
    w = torch.ones(D, dtype=torch.bfloat16, device=DEV)
    cos, sin = attn.rope_table(n, D, device=DEV)
    j = torch.arange(n, dtype=torch.int32)
    slots = place[j.long() // page] * page + j % page
    qn = attn.qk_norm_rope_cache(q, k, v, w, w, cos, sin, j.to(DEV), slots.to(DEV), kc, vc, k_descale=d, v_descale=d)
    # The same in a small cache: the same values, so the same results.
    small_k, small_v = (torch.zeros(7, page, Hkv, D, dtype=dtype, device=DEV) for _ in range(2))
    qs = attn.qk_norm_rope_cache(q, k, v, w, w, cos, sin, j.to(DEV), j.to(DEV), small_k, small_v, k_descale=d,
                                 v_descale=d)
    assert torch.equal(qn, qs)
    for big, small in ((kc, small_k), (vc, small_v)):
        assert torch.equal(big[place.long().to(DEV)].view(torch.uint8), small.view(torch.uint8))
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    got, want = (attn.decode_paged(qn[-1:], a, b, t.to(DEV)[None], lens, k_descale=d, v_descale=d)
                 for a, b, t in ((kc, vc, place), (small_k, small_v, torch.arange(7, dtype=torch.int32))))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    t = dict(q=qn[-1:].cpu(), kc=small_k.cpu(), vc=small_v.cpu(), table=torch.arange(7, dtype=torch.int32)[None],
             lens=torch.tensor([n], dtype=torch.int32), kd=d, vd=d)
    check(t, got, scale=D ** -0.5)
