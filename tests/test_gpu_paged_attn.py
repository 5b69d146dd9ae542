"""Attention of new tokens over the paged cache against the fp64 definition (bounds: attn_util)."""
import numpy as np
import pytest
import torch

import oracle.attn as oa
from attn_util import Cache, attn_excess, attn_reference, attn_within, f64

pytestmark = pytest.mark.gpu


def lib():
    import gated_delta_rule_105_b200 as g
    return g


def queries(c, hq, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return (size * torch.randn(c.n_tok, hq, c.d, generator=g)).bfloat16()


def call(c, q, dev=None, cu=True, **kw):
    g = lib()
    dev = c.cuda() if dev is None else dev
    o, lse = g.paged_attn_fwd(q if q.is_cuda else q.cuda(), dev["kc"], dev["vc"], dev["table"], dev["lens"],
                              dev["cu"] if cu else None, dev["ks"], dev["vs"], return_lse=True, **kw)
    g.check_error()
    return o, lse


def check(c, hq, seed, window=0, o_dtype=torch.bfloat16, scale=None, size=1.0, **kw):
    q = queries(c, hq, seed, size)
    scale = c.d ** -0.5 if scale is None else scale
    o, lse = call(c, q, window=window, o_dtype=o_dtype, scale=scale, **kw)
    ref = attn_reference(c, f64(q), scale, window)
    eo, el = attn_excess(o, lse, ref, c, window, o_dtype)
    assert eo <= 1.0 and el <= 1.0, (eo, el)
    return o, lse, ref


# (positions, new tokens), query heads, KV heads, channels, page, window: single tokens, chunks, mixes, empty and odd
CASES = [
    ([1], [1], 1, 1, 64, 16, 0), ([1], [1], 16, 1, 128, 128, 0), ([17], [1], 3, 1, 128, 16, 0), ([128], [1], 4, 2, 64, 32, 0),
    ([129, 1, 255, 256, 257], [1] * 5, 8, 2, 128, 64, 0), ([1000, 3, 513], [1, 1, 1], 10, 2, 64, 16, 0),
    ([1000, 3, 513], [1, 1, 1], 10, 2, 128, 16, 100), ([300, 40], [4, 4], 12, 4, 128, 32, 0), ([33, 70], [33, 7], 2, 2, 64, 16, 0),
    ([200, 64, 5], [200, 1, 5], 4, 2, 128, 64, 0), ([150, 300, 90], [0, 40, 0], 6, 2, 64, 32, 0),
    ([260, 90], [130, 90], 8, 1, 128, 16, 0), ([260, 90, 31], [130, 90, 2], 8, 4, 64, 128, 50), ([400], [300], 4, 4, 128, 64, 129),
    ([140, 20], [140, 20], 5, 1, 64, 16, 1), ([520], [260], 2, 1, 128, 128, 0), ([90, 1400], [90, 3], 20, 1, 64, 64, 0)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("total,new,hq,hkv,d,page,window", CASES)
def test_matches_the_definition(kind, total, new, hq, hkv, d, page, window):
    c = Cache(total, new, hkv, d, page, kind, seed=sum(total) + hq).fill()
    check(c, hq, 3, window)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [1, 70])
def test_fp32_output_and_other_scales(kind, d, new):
    c = Cache([200, 90], [new, new], 2, d, 32, kind, seed=new + d).fill(kscale=3.0, vscale=50.0)
    check(c, 6, 5, 0, torch.float32, scale=0.5, size=2.0)
    check(c, 6, 5, 0, torch.float32, scale=0.0)
    check(c, 6, 5, 40, torch.float32, scale=-0.1)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 4, 100])
def test_growing_scores(kind, new):
    """Keys whose scores rise along the sequence by far more than fp32's exponent of 2 holds: the running maximum moves
    in every block, and the sums so far have to be scaled down each time."""
    L = 700
    c = Cache([L], [new], 1, 64, 16, kind, seed=1).fill()
    for pos in range(L):
        x = c.rng.standard_normal((1, 64)) * 0.1
        x[0, 0] = 0.5 * pos
        c.put("k", c.table[0, pos // 16], pos % 16, x)
    q = queries(c, 2, 1)
    q[:, :, 0] = 8.0
    o, lse = call(c, q)
    ref = attn_reference(c, f64(q), 64 ** -0.5, 0)
    eo, el = attn_excess(o, lse, ref, c, 0, torch.bfloat16)
    assert eo <= 1.0 and el <= 1.0
    q[:, :, 0] = -8.0  # and falling ones
    o, lse = call(c, q)
    eo, el = attn_excess(o, lse, attn_reference(c, f64(q), 64 ** -0.5, 0), c, 0, torch.bfloat16)
    assert eo <= 1.0 and el <= 1.0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,hq,window", [(1, 4, 0), (3, 4, 30), (60, 4, 0), (60, 4, 25), (200, 2, 90)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_what_a_token_does_not_see_does_not_reach_it(kind, new, hq, window, value):
    """NaN or infinity in the keys and values of one new token: earlier tokens, and later ones whose window has passed
    it, come out as without it; the tokens that see it are not finite."""
    L = 230
    c = Cache([L, 40], [new, 1], 2, 64, 16, kind, seed=new).fill()
    q = queries(c, hq, 2)
    clean, clean_lse = call(c, q, window=window)
    bad = new // 2
    pos = L - new + bad
    x = np.zeros((2, 64))
    x[:, 5] = value
    pg, r = c.table[0, pos // 16], pos % 16
    for which in ("v", "k"):
        c.put(which, pg, r, x)
        o, lse = call(c, q, window=window)
        for t in range(new):
            seen = t >= bad and (not window or t < bad + window)
            if seen:
                assert not torch.isfinite(o[t]).all()
            else:
                assert torch.equal(o[t], clean[t]) and torch.equal(lse[t], clean_lse[t]), (which, t)
        assert torch.equal(o[new:], clean[new:])


@pytest.mark.parametrize("new", [1, 5, 90])
@pytest.mark.parametrize("d,hq,hkv,page,window", [(64, 4, 2, 16, 0), (128, 8, 1, 64, 77)])
def test_8_bit_cache_is_its_read_back(new, d, hq, hkv, page, window):
    """Dequantised rows are exact in bf16, so attention over the 8-bit cache is that over the read-back rows in a bf16
    cache; P is rounded with V's power of two in it, which shifts nothing but the exponent."""
    g = lib()
    total = [333, 90, 150]
    c = Cache(total, [min(new, t) for t in total], hkv, d, page, "e4m3", seed=d + new).fill(kscale=4.0, vscale=0.3)
    q = queries(c, hq, 4)
    dev = c.cuda()
    o8, l8 = call(c, q, dev, window=window)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(total)]), dtype=torch.int32, device="cuda")
    k, v = g.kv_read(dev["kc"], dev["vc"], dev["table"], cu, sum(total), dev["ks"], dev["vs"])
    kc = torch.full(dev["kc"].shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    lens = torch.tensor(total, dtype=torch.int32, device="cuda")
    g.kv_append(k, v, kc, vc, dev["table"], lens, cu)
    o16, l16 = call(c, q, {**dev, "kc": kc, "vc": vc, "ks": None, "vs": None}, window=window)
    # same products and weights, added in other orders: twice the sums' share of the bound
    ref = attn_reference(c, f64(q), d ** -0.5, window)
    assert np.all(np.abs(f64(o8) - f64(o16)) <= 2.0 ** -7 * np.abs(ref[0]) + ref[2] * (2.0 ** -7 + 2.0 ** -12))
    assert np.all(np.abs(f64(l8) - f64(l16)) <= 1e-4)


def test_uniform_tokens_without_cu_seqlens_and_strided_queries():
    c = Cache([100, 64, 31, 250], [3] * 4, 2, 128, 16, "bf16", 21).fill()
    q = queries(c, 8, 8)
    a, la = call(c, q)
    b, lb = call(c, q, cu=False)
    assert torch.equal(a, b) and torch.equal(la, lb)
    fused = torch.full((12, 8 * 128 + 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    fused[:, :1024] = q.cuda().view(12, 1024)
    s, ls = call(c, fused[:, :1024].view(12, 8, 128))
    assert torch.equal(a, s) and torch.equal(la, ls)


def test_rows_behind_the_last_sequence_stay_as_they_were():
    c = Cache([100, 64], [40, 1], 2, 64, 16, "e4m3", 22).fill()
    dev = c.cuda()
    q = torch.randn(50, 4, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    o = torch.full((50, 4, 64), 77.0, dtype=torch.bfloat16, device="cuda")
    got = lib().paged_attn_fwd(q, dev["kc"], dev["vc"], dev["table"], dev["lens"], dev["cu"], dev["ks"], dev["vs"], o=o)
    lib().check_error()
    assert got.data_ptr() == o.data_ptr() and (o[41:] == 77).all()
    ref = attn_reference(c, f64(q[:41]), 0.125, 0)
    assert np.all(np.abs(f64(o[:41]) - ref[0]) <= 2.0 ** -7 * (ref[2] + np.abs(ref[0])))


def test_repeats_to_the_bit_and_two_streams_with_their_own_workspaces():
    g = lib()
    cs = [Cache([3000, 500, 1], [1, 1, 1], 2, 128, 64, "bf16", 31).fill(), Cache([900, 300], [200, 1], 2, 128, 64, "bf16", 32).fill()]
    qs = [queries(c, 8, 9).cuda() for c in cs]
    devs = [c.cuda() for c in cs]
    want = [call(c, q, dev) for c, q, dev in zip(cs, qs, devs)]
    ws = [torch.empty(g.paged_attn_workspace_bytes(c.n_tok, len(c.total), 8, 2, 128), dtype=torch.uint8, device="cuda") for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    got = [[] for _ in cs]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                d = devs[i]
                got[i].append(g.paged_attn_fwd(qs[i], d["kc"], d["vc"], d["table"], d["lens"], d["cu"], return_lse=True, workspace=ws[i]))
    torch.cuda.synchronize()
    for w, all_ in zip(want, got):
        for o, lse in all_:
            assert torch.equal(o, w[0]) and torch.equal(lse, w[1])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_captured_step_replays_with_new_lengths(kind):
    """A decode step -- append, attend -- captured once and replayed as the sequences grow, pages being added."""
    g = lib()
    n, hkv, hq, d, page = 3, 2, 8, 64, 16
    c = Cache([60, 5, 130], [1] * n, hkv, d, page, kind, 41, spare=8, extra_cols=4).fill(upto_new=False)
    dev = c.cuda()
    free = [p for p in range(c.n_pages) if p not in set(c.table[c.table >= 0].tolist())]
    k, v, q = (torch.zeros(n, h, d, dtype=torch.bfloat16, device="cuda") for h in (hkv, hkv, hq))
    ws = torch.empty(g.paged_attn_workspace_bytes(n, n, hq, hkv, d), dtype=torch.uint8, device="cuda")
    o = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")

    def step():
        g.kv_append(k, v, dev["kc"], dev["vc"], dev["table"], dev["lens"], dev["cu"], dev["ks"], dev["vs"])
        return g.paged_attn_fwd(q, dev["kc"], dev["vc"], dev["table"], dev["lens"], dev["cu"], dev["ks"], dev["vs"],
                                o=o, return_lse=True, workspace=ws)[1]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lse = step()
    gen = torch.Generator().manual_seed(5)
    for it in range(20):
        new = [torch.randn(n, h, d, generator=gen).bfloat16() for h in (hkv, hkv, hq)]
        for t, x in zip((k, v, q), new):
            t.copy_(x)
        if it:
            for i in range(n):
                c.total[i] += 1
                if (c.total[i] - 1) % page == 0:
                    c.table[i, (c.total[i] - 1) // page] = free.pop()
            dev["table"].copy_(torch.from_numpy(c.table))
            dev["lens"].copy_(torch.tensor(c.total, dtype=torch.int32))
        for i in range(n):
            pos = c.total[i] - 1
            for which, x in zip(("k", "v"), new):
                c.put(which, c.table[i, pos // page], pos % page, f64(x[i]))
        graph.replay()
        g.check_error()
        eo, el = attn_excess(o, lse, attn_reference(c, f64(new[2]), d ** -0.5, 0), c, 0, torch.bfloat16)
        assert eo <= 1.0 and el <= 1.0, it


def test_many_sequences_and_a_long_one():
    rng = np.random.default_rng(3)
    total = [int(x) for x in rng.integers(1, 40, 400)] + [6000]
    new = [int(min(t, x)) for t, x in zip(total, rng.integers(0, 3, 401))]
    c = Cache(total, new, 1, 64, 32, "bf16", 51).fill()
    check(c, 4, 1)


@pytest.mark.parametrize("what", ["page", "len_long", "len_short", "cu_order"])
@pytest.mark.parametrize("new", [2, 60])
def test_bad_device_arguments_are_reported(what, new):
    g = lib()
    c = Cache([100, 100, 100], [new] * 3, 2, 64, 16, "bf16", 61).fill()
    q = queries(c, 4, 1).cuda()
    good, _ = call(c, q)
    dev = c.cuda()
    if what == "page":
        dev["table"][1, 2] = 1 << 30
    elif what == "len_long":
        dev["lens"][1] = 1 << 30
    elif what == "len_short":
        dev["lens"][1] = new - 1
    else:
        dev["cu"][2] = 0
    o = torch.full_like(good, 5.0)
    g.paged_attn_fwd(q, dev["kc"], dev["vc"], dev["table"], dev["lens"], dev["cu"], o=o)
    with pytest.raises(g.GdnError) as e:
        g.check_error()
    assert e.value.status == 5
    g.check_error()
    if what != "cu_order":  # a later sequence then claims the same rows
        assert torch.equal(o[:new], good[:new]) and torch.equal(o[2 * new:], good[2 * new:])
        if what != "page":
            assert (o[new:2 * new] == 5).all()


def test_an_attention_layer_beside_a_mixer_layer():
    """One decode step of a hybrid block as a server runs it: residual norm with 8-bit output, projections, cache write,
    attention over it, the next residual norm, then the mixer's own decode step; against the same in fp64."""
    g = lib()
    n, hq, hkv, d, dm = 4, 8, 2, 128, 512
    c = Cache([300, 17, 64, 129], [1] * n, hkv, d, 64, "e4m3", 71).fill(upto_new=False)
    gen = torch.Generator().manual_seed(6)
    x, r = torch.randn(n, dm, generator=gen).bfloat16(), torch.randn(n, dm, generator=gen).bfloat16()
    w = 1 + 0.1 * torch.randn(dm, generator=gen)
    W = torch.randn(dm, (hq + 2 * hkv) * d, generator=gen) / dm ** 0.5
    dev = c.cuda()
    norm = g.add_rmsnorm_fwd(x.cuda(), w.cuda(), r.cuda(), out_dtype=torch.float8_e4m3fn, group=128)
    y = (norm["y"].float().view(n, -1, 128) * norm["scale"][..., None]).view(n, dm)
    qkv = (y @ W.cuda()).bfloat16()
    q, k, v = (qkv[:, a:b].view(n, -1, d) for a, b in ((0, hq * d), (hq * d, (hq + hkv) * d), ((hq + hkv) * d, (hq + 2 * hkv) * d)))
    g.kv_append(k, v, dev["kc"], dev["vc"], dev["table"], dev["lens"], None, dev["ks"], dev["vs"])
    o, lse = g.paged_attn_fwd(q, dev["kc"], dev["vc"], dev["table"], dev["lens"], None, dev["ks"], dev["vs"], window=128,
                              return_lse=True)
    g.check_error()
    for i in range(n):
        pos = c.total[i] - 1
        for which, t in (("k", k), ("v", v)):
            c.put(which, c.table[i, pos // 64], pos % 64, f64(t[i]))
    eo, el = attn_excess(o, lse, attn_reference(c, f64(q), d ** -0.5, 128), c, 128, torch.bfloat16)
    assert eo <= 1.0 and el <= 1.0
    h = 4
    state = torch.zeros(n, h, 128, 256, device="cuda")
    qq, kk = (o.reshape(n, 8, 128)[:, a:a + h].contiguous() for a in (0, 4))
    vv = torch.cat([qq, kk], -1).contiguous()
    gate, beta = -torch.ones(n, h, device="cuda"), torch.full((n, h), 0.5, device="cuda")
    out = g.decode_fwd(qq, kk, vv, gate, beta, state)
    # from a zero state: o = scale beta (k . q) v
    want = 128 ** -0.5 * 0.5 * (qq.double() * kk.double()).sum(-1, keepdim=True) * vv.double()
    assert torch.allclose(out.double(), want, rtol=2.0 ** -6, atol=1e-6)
    tail = g.add_rmsnorm_fwd(out.reshape(n, -1)[:, :dm].contiguous(), w.cuda(), norm["s"])
    assert torch.isfinite(tail["y"].float()).all() and tail["s"].shape == (n, dm)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,d,window", [(24, 1, 64, 0), (33, 1, 128, 0), (96, 2, 64, 40), (256, 1, 128, 0)])
def test_many_heads_share_a_kv_head(kind, hq, hkv, d, window):
    """One token a sequence with more query rows per KV head than the decode kernel takes at a time, or at all."""
    c = Cache([300, 1, 129], [1] * 3, hkv, d, 32, kind, hq).fill()
    o, lse, _ = check(c, hq, 4, window)
    for i in range(3):  # the batch's other sequences do not matter
        one = Cache([c.total[i]], [1], hkv, d, 32, kind, hq)
        one.kc, one.vc, one.ks, one.vs, one.table, one.n_pages = c.kc, c.vc, c.ks, c.vs, c.table[i:i + 1], c.n_pages
        q = queries(c, hq, 4)[i:i + 1]
        a, la = call(one, q, window=window, scale=d ** -0.5)
        eo, el = attn_excess(a, la, attn_reference(one, f64(q), d ** -0.5, window), one, window, torch.bfloat16)
        assert eo <= 1.0 and el <= 1.0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("total,new,hq,d,window", [([5000], [20], 16, 128, 0), ([5000], [35], 8, 64, 1000),
                                                   ([2600, 7, 2000], [90, 1, 1], 4, 128, 0)])
def test_short_chunks_over_long_contexts(kind, total, new, hq, d, window):
    """Few items of many parts: every CTA has a tile or two, and the parts outnumber the items by far."""
    c = Cache(total, new, 1, d, 64, kind, sum(new)).fill()
    check(c, hq, 6, window)
    check(c, hq, 6, window, torch.float32)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_captured_chunks_replay_with_other_sequences(kind):
    """A mixed call captured once; replayed with other lengths and another share of the rows among the sequences."""
    g = lib()
    c = Cache([900, 700, 40], [200, 1, 39], 2, 64, 16, kind, 43).fill()
    dev = c.cuda()
    q = queries(c, 4, 2)
    qd = q.cuda()
    ws = torch.empty(g.paged_attn_workspace_bytes(240, 3, 4, 2, 64), dtype=torch.uint8, device="cuda")
    o = torch.empty(240, 4, 64, dtype=torch.bfloat16, device="cuda")

    def step():
        return g.paged_attn_fwd(qd, dev["kc"], dev["vc"], dev["table"], dev["lens"], dev["cu"], dev["ks"], dev["vs"],
                                o=o, return_lse=True, workspace=ws)[1]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lse = step()
    for total, new in (([900, 700, 40], [200, 1, 39]), ([300, 700, 5], [1, 238, 1]), ([900, 0, 1], [239, 0, 1]), ([7, 7, 9], [1, 2, 3])):
        c.total, c.new, n = total, new, sum(new)
        c.cu = torch.tensor([0, *np.cumsum(new)], dtype=torch.int32)
        dev["cu"].copy_(c.cu)
        dev["lens"].copy_(torch.tensor(total, dtype=torch.int32))
        o.fill_(55)
        graph.replay()
        g.check_error()
        eo, el = attn_excess(o[:n], lse[:n], attn_reference(c, f64(q), 0.125, 0), c, 0, torch.bfloat16)
        assert eo <= 1.0 and el <= 1.0 and (o[n:] == 55).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_work_far_apart_among_the_sequences(kind):
    """Chunks with scores of decoding sequences between them, and decoding ones among many without a new token."""
    total, new = [150] + [3] * 90 + [200] + [2] * 40 + [130, 260], [150] + [1] * 90 + [60] + [0] * 40 + [40, 1]
    check(Cache(total, new, 2, 64, 32, kind, 61).fill(), 4, 3)
    total, new = [5] + [1] * 100 + [300, 9] + [4] * 70 + [33], [1] + [0] * 100 + [1, 1] + [0] * 70 + [1]
    check(Cache(total, new, 1, 128, 16, kind, 62).fill(), 4, 3)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float8_e4m3fn])
def test_pages_behind_the_first_4_gb(kind):
    """Pages at the end of a pool whose byte and element offsets pass 32 bits, against the same pages in a small pool."""
    g = lib()
    hkv, page, d, far = 2, 64, 128, (1 << 32) // (2 * 64 * 128) + 40  # pages: 2^32 elements and more
    lens, new = [700, 130, 65], [1, 130, 40]
    gen = torch.Generator().manual_seed(71)
    k, v = (torch.randn(sum(lens), hkv, d, generator=gen).bfloat16().cuda() for _ in range(2))
    q = torch.randn(sum(new), 8, d, generator=gen).bfloat16().cuda()
    total = torch.tensor(lens, dtype=torch.int32, device="cuda")
    all_, cu = (torch.tensor([0, *np.cumsum(x)], dtype=torch.int32, device="cuda") for x in (lens, new))
    near = torch.randperm(36, generator=gen).view(3, 12).to(torch.int32).cuda()
    got = []
    for pages, shift in ((36, 0), (far, far - 36)):
        kc, vc = (torch.empty(pages, hkv, page, d, dtype=kind, device="cuda") for _ in range(2))
        ks, vs = (None if kind is torch.bfloat16 else torch.empty(pages, hkv, page, dtype=torch.uint8, device="cuda") for _ in range(2))
        for t in (kc, vc, ks, vs):  # nothing is left to chance in the places that no token takes
            if t is not None:
                t[shift:].view(torch.uint8).zero_()
        table = near + shift
        g.kv_append(k, v, kc, vc, table, total, all_, ks, vs)
        got.append([*g.paged_attn_fwd(q, kc, vc, table, total, cu, ks, vs, return_lse=True),
                    g.paged_attn_fwd(q[:3], kc, vc, table, total, None, ks, vs),
                    *g.kv_read(kc, vc, table, all_, sum(lens), ks, vs)])
        g.check_error()
        del kc, vc, ks, vs
    for a, b in zip(*got):
        assert torch.equal(a, b)
    if kind is torch.bfloat16:
        assert torch.equal(got[1][3], k) and torch.equal(got[1][4], v)
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 40])
def test_sequences_share_the_pages_of_a_prefix(kind, new):
    c = Cache([200, 200, 150], [new] * 3, 2, 64, 32, kind, 81).fill()
    for i in (1, 2):
        c.table[i, :4] = c.table[0, :4]
    check(c, 4, 2)
    check(c, 4, 2, 70)


def test_calls_without_tokens():
    g = lib()
    c = Cache([40, 9], [1, 1], 2, 64, 16, "e4m3", 82).fill()
    dev = c.cuda()
    before = {k: dev[k].view(torch.uint8).clone() for k in ("kc", "vc", "ks", "vs")}
    none = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    for by in (cu, None):
        g.kv_append(none, none, dev["kc"], dev["vc"], dev["table"], dev["lens"], by, dev["ks"], dev["vs"])
        o, lse = g.paged_attn_fwd(none, dev["kc"], dev["vc"], dev["table"], dev["lens"], by, dev["ks"], dev["vs"], return_lse=True)
        assert o.shape == (0, 2, 64) and lse.shape == (0, 2)
    assert g.kv_read(dev["kc"], dev["vc"], dev["table"], cu, 0, dev["ks"], dev["vs"])[0].shape == (0, 2, 64)
    # rows, but none that belongs to a sequence
    q = torch.ones(5, 4, 64, dtype=torch.bfloat16, device="cuda")
    o = torch.full((5, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    g.paged_attn_fwd(q, dev["kc"], dev["vc"], dev["table"], dev["lens"], cu, dev["ks"], dev["vs"], o=o)
    g.kv_append(q[:, :2].contiguous(), q[:, :2].contiguous(), dev["kc"], dev["vc"], dev["table"], dev["lens"], cu, dev["ks"], dev["vs"])
    g.check_error()
    assert (o == 3).all()
    for k, t in before.items():
        assert torch.equal(dev[k].view(torch.uint8), t)
    n = g.add_rmsnorm_fwd(torch.zeros(0, 128, dtype=torch.bfloat16, device="cuda"), torch.ones(128, device="cuda"))
    assert n["y"].shape == (0, 128) and n["rstd"].shape == (0,)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("new,hq,d,window", [(1, 4, 64, 1), (1, 4, 128, 100), (3, 12, 64, 129), (2, 20, 128, 250), (90, 4, 128, 100),
                                             (300, 2, 64, 65), (150, 6, 128, 1)])
def test_pages_that_the_window_has_passed_may_be_gone(kind, page, new, hq, d, window):
    """Block-table entries of pages that no token of the call sees: freed (any number), nothing is reported, and the
    results are those of the full table to the bit."""
    total = [900, 45 + new, 301 + new, 2 * new]
    c = Cache(total, [new] * 4, 2, d, page, kind, page + new).fill()
    q = queries(c, hq, 3)
    want = call(c, q, window=window)
    ref = attn_reference(c, f64(q), d ** -0.5, window)
    assert attn_within(*want, ref, c, window, torch.bfloat16)
    gone = 0
    for i, (t, a) in enumerate(zip(c.total, c.new)):
        first = max(0, t - a + 1 - window) // page
        c.table[i, :first] = np.resize([-1, 1 << 30, -2 ** 31], first)
        gone += first
    assert gone > 0
    dev = c.cuda()
    for cu in (True, False):
        o, lse = call(c, q, dev, cu=cu, window=window)  # (raises if the error word is set)
        if cu:
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        else:
            assert attn_within(o, lse, ref, c, window, torch.bfloat16)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,hq,d,window", [(1, 4, 64, 0), (1, 4, 128, 300), (3, 12, 64, 0), (4, 8, 128, 300), (90, 4, 128, 0),
                                             (90, 4, 64, 300), (300, 2, 128, 0), (150, 6, 64, 333)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_bad_value_reaches_its_own_channel_only(kind, new, hq, d, window, value):
    """A NaN or an infinity in one channel of a value: in the tokens that see it that channel is not finite (over 8 bits, where
    the row is NaN throughout, every channel); other channels, other tokens and every lse are as without it, to the bit,
    wherever the key lies -- in a tile that all rows of a chunk see, in one that some see, at the window's edge."""
    L = 650
    c = Cache([L, 40], [new, min(new, 40)], 2, d, 16, kind, seed=new).fill()
    q = queries(c, hq, 2)
    clean, clean_lse = call(c, q, window=window)
    assert torch.isfinite(clean).all() and torch.isfinite(clean_lse).all()
    first = max(0, L - new + 1 - window) if window else 0
    for pos in sorted({first, first + 5, max(first, L - new - 200), max(first, L - new - 1), L - new + new // 2, L - 1}):
        pg, r = c.table[0, pos // 16], pos % 16
        if kind == "bf16":
            was = c.vc[pg, :, r, 5].clone()
            c.vc[pg, :, r, 5] = value
        else:
            was = c.vc.view(torch.uint8)[pg, :, r].clone(), c.vs[pg, :, r].clone()
            c.put("v", pg, r, np.full((2, d), value))
        o, lse = call(c, q, window=window)
        assert torch.equal(lse, clean_lse), pos
        for t in range(new):
            own = L - new + t
            if not (pos <= own and (not window or pos > own - window)):
                assert torch.equal(o[t], clean[t]), (pos, t)
            elif kind == "e4m3":
                assert torch.isnan(o[t]).all(), (pos, t)
            else:
                assert torch.isnan(o[t, :, 5]).all() if np.isnan(value) else (o[t, :, 5] == value).all(), (pos, t)
                assert torch.equal(o[t, :, :5], clean[t, :, :5]) and torch.equal(o[t, :, 6:], clean[t, :, 6:]), (pos, t)
        assert torch.equal(o[new:], clean[new:])
        if kind == "bf16":
            c.vc[pg, :, r, 5] = was
        else:
            c.vc.view(torch.uint8)[pg, :, r], c.vs[pg, :, r] = was


@pytest.mark.parametrize("new", [1, 60])
@pytest.mark.parametrize("window", [0, 100])
def test_opposite_infinities_among_the_values(new, window):
    """+inf and -inf in one channel: NaN for the tokens that see both, an infinity for those that see one."""
    L, hq, d = 400, 4, 64
    c = Cache([L], [new], 1, d, 32, "bf16", 7).fill()
    q = queries(c, hq, 3)
    at = {L - new - 50: float("inf"), L - new // 2 - 1: -float("inf")}
    for pos, value in at.items():
        c.vc[c.table[0, pos // 32], :, pos % 32, 9] = value
    o, lse = call(c, q, window=window)
    assert torch.isfinite(lse).all()
    for t in range(new):
        own = L - new + t
        want = sum(v for pos, v in at.items() if pos <= own and (not window or pos > own - window))
        got = o[t, :, 9]
        assert torch.isfinite(got).all() if want == 0 else torch.isnan(got).all() if np.isnan(want) else (got == want).all(), t
        assert torch.isfinite(o[t, :, :9]).all() and torch.isfinite(o[t, :, 10:]).all()


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,packed", [(1, True), (6, False), (40, True)])
def test_large_values_under_rising_scores(kind, d, new, packed):
    """Values close to fp32's largest number, and a key far along whose score is above the first one's by less than the running
    maximum's lag (2^7.2): the weighted mean is finite.  Enough (sequence, head) items that CTAs walk along whole ones, and
    a distance (768) that every unit of keys divides, so that one warp meets both keys."""
    g = lib()
    n, hkv, G, L, page = 8, 64, 2, 900, 64
    gen = torch.Generator().manual_seed(d + new)
    k = torch.zeros(L, hkv, d)
    k[:, :, 0] = -40.0
    k[3, :, 0], k[771, :, 0] = 0.0, 5.0
    v = (1 + 0.8 * torch.rand(L, hkv, d, generator=gen)) * torch.sign(torch.randn(L, hkv, d, generator=gen)) * 2.0 ** 126
    q = torch.zeros(n * new, hkv * G, d)
    q[:, :, 0] = d ** 0.5 * (0.95 + 0.05 * torch.rand(n * new, hkv * G, generator=gen))
    pages = -(-L // page)
    kc, vc = (torch.zeros(pages, hkv, page, d, dtype=kind, device="cuda") for _ in range(2))
    ks, vs = (None if kind is torch.bfloat16 else torch.zeros(pages, hkv, page, dtype=torch.uint8, device="cuda") for _ in range(2))
    table = torch.randperm(pages, generator=gen).to(torch.int32).repeat(n, 1).cuda()
    lens = torch.full((n,), L, dtype=torch.int32, device="cuda")
    g.kv_append(k.bfloat16().cuda(), v.bfloat16().cuda(), kc, vc, table[:1].contiguous(), lens[:1], None, ks, vs)
    q = q.bfloat16().cuda()
    cu = torch.arange(0, n * new + 1, new, dtype=torch.int32, device="cuda") if packed else None
    o, lse = g.paged_attn_fwd(q, kc, vc, table, lens, cu, ks, vs, o_dtype=torch.float32, return_lse=True)
    kk, vv = g.kv_read(kc, vc, table[:1].contiguous(), torch.tensor([0, L], dtype=torch.int32, device="cuda"), L, ks, vs, torch.float32)
    g.check_error()
    # every new token lies behind both keys; the others' weights are below e^-38
    s = torch.einsum("thgd,lhd->thgl", q.double().view(-1, hkv, G, d), kk.double()) * d ** -0.5
    pos = (L - new + torch.arange(new, device="cuda")).repeat(n)
    s.masked_fill_((torch.arange(L, device="cuda") > pos[:, None])[:, None, None], -float("inf"))
    w = torch.softmax(s, -1)
    want = torch.einsum("thgl,lhd->thgd", w, vv.double()).reshape(o.shape)
    size = torch.einsum("thgl,lhd->thgd", w, vv.double().abs()).reshape(o.shape)
    es = 40 * (d * 2.0 ** -23 + 4 * 2.0 ** -24)
    assert torch.isfinite(o).all()
    assert ((o.double() - want).abs() <= size * (2.0 ** -8 + 2 * es + 2.0 ** -21 + (2 * L + 64) * 2.0 ** -23) + 2.0 ** -24 * want.abs()).all()
    assert ((lse.double() - torch.logsumexp(s, -1).reshape(lse.shape)).abs() <= es + 2.0 ** -22 + (L + 64) * 2.0 ** -23 + 40 * 2.0 ** -22).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,chunks", [(257, {0: 40, 255: 150, 256: 60}), (300, {256: 40, 299: 90}), (700, {10: 33, 300: 140, 511: 50, 512: 50, 699: 70}),
                                      (700, {690: 300}), (1030, {1024: 40, 1029: 9})])
def test_chunks_far_along_many_sequences(kind, n, chunks):
    """More sequences than either kernel looks over at a time, some of them with chunks, also in the last look only; one
    token or none in the others."""
    rng = np.random.default_rng(n)
    new = [int(x) for x in rng.integers(0, 2, n)]
    total = [int(x) for x in rng.integers(1, 6, n)]
    if n == 700 and len(chunks) == 1:
        new = [0] * n
    for i, a in chunks.items():
        new[i], total[i] = a, a + int(rng.integers(0, 200))
    c = Cache(total, new, 2, 64, 16, kind, n).fill()
    check(c, 8, 4)
    check(c, 8, 4, 37)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,G,d,window", [(2, 5, 64, 0), (2, 8, 128, 0), (3, 4, 64, 50), (3, 3, 128, 0), (4, 8, 64, 0), (4, 3, 128, 90),
                                            (2, 16, 64, 0), (4, 4, 128, 0), (4, 7, 64, 200)])
def test_several_tokens_a_sequence_packed_and_not(kind, new, G, d, window):
    """2 to 4 tokens of each sequence, 9 to 32 query rows per KV head: with cu_seqlens and without, several passes over the keys
    or one."""
    c = Cache([400, 129, new, 250, 61], [new] * 5, 2, d, 32, kind, new + G).fill()
    q = queries(c, 2 * G, 5)
    ref = attn_reference(c, f64(q), d ** -0.5, window)
    for cu in (True, False):
        for o_dtype in (torch.bfloat16, torch.float32):
            o, lse = call(c, q, cu=cu, window=window, o_dtype=o_dtype)
            assert attn_within(o, lse, ref, c, window, o_dtype), (cu, o_dtype)


@pytest.mark.parametrize("variant,dv", [("gdn", 128), ("gdn", 256), ("gdn2", 128)])
def test_chunks_beside_a_mixer_on_another_stream(variant, dv):
    """The chunk kernel takes all of an SM's tensor memory, the mixer's kernels parts of it: calls of both on two streams
    at once give what they give alone, to the bit."""
    from gated_delta_rule_105_b200.inputs import generate
    from parity_util import run_cuda
    g = lib()
    inp = generate(2, 1024, 8, 128, dv, "bf16", seed=5, variant=variant)
    c = Cache([700, 300, 129], [130, 1, 60], 2, 128, 64, "bf16", 91).fill()
    dev, q = c.cuda(), queries(c, 8, 2).cuda()
    args = q, dev["kc"], dev["vc"], dev["table"], dev["lens"], dev["cu"]
    ws = torch.empty(g.paged_attn_workspace_bytes(c.n_tok, 3, 8, 2, 128), dtype=torch.uint8, device="cuda")
    want_mixer = run_cuda(inp, variant)
    assert g.last_kernel() == "tc"
    want = g.paged_attn_fwd(*args, return_lse=True)
    g.check_error()
    dev_inp = {k: v.cuda() if torch.is_tensor(v) else v for k, v in inp.items()}
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    mixer, attn = [], []
    for _ in range(20):
        with torch.cuda.stream(one):
            mixer.append(run_cuda(dev_inp, variant))
        with torch.cuda.stream(two):
            for _ in range(4):
                attn.append(g.paged_attn_fwd(*args, return_lse=True, workspace=ws))
    torch.cuda.synchronize()
    g.check_error()
    for o, hT in mixer:
        assert torch.equal(o, want_mixer[0]) and torch.equal(hT, want_mixer[1])
    for o, lse in attn:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
