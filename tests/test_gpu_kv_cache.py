"""Writing new tokens into the paged cache and reading it back, against the fp64 definition, to the bit."""
import numpy as np
import pytest
import torch

import oracle.attn as oa
from attn_util import Cache, f64

pytestmark = pytest.mark.gpu


def lib():
    import gated_delta_rule_105_b200 as g
    return g


def raw(t):
    return t.cpu().view(torch.uint8).numpy()


def expected_after(c, k, v):
    """The cache (as bytes, and scales) after the new tokens' rows went in one by one."""
    out = {}
    for name, x in (("k", k), ("v", v)):
        cache = (c.kc if name == "k" else c.vc).clone()
        scale = None if c.kind == "bf16" else (c.ks if name == "k" else c.vs).clone()
        xs = x.to(torch.float64).numpy()
        for i, (t, a) in enumerate(zip(c.total, c.new)):
            for j in range(a):
                pos, row = t - a + j, int(c.cu[i]) + j
                pg, r = c.table[i, pos // c.page], pos % c.page
                if c.kind == "bf16":
                    cache[pg, :, r] = x[row].to(torch.bfloat16)
                else:
                    for h in range(c.hkv):
                        code, byte = oa.quantise_row(xs[row, h])
                        cache.view(torch.uint8)[pg, h, r] = torch.from_numpy(code)
                        scale[pg, h, r] = byte
        out[name] = (raw(cache), None if scale is None else scale.numpy())
    return out


def check_append(c, k, v, kd=None, vd=None, cu=True):
    g, dev = lib(), c.cuda()
    want = expected_after(c, k, v)
    g.kv_append(k.cuda() if kd is None else kd, v.cuda() if vd is None else vd, dev["kc"], dev["vc"], dev["table"],
                dev["lens"], dev["cu"] if cu else None, dev["ks"], dev["vs"])
    g.check_error()
    for name in ("k", "v"):
        got = raw(dev[name + "c"])
        w = want[name][0]
        if c.kind == "bf16":  # NaN payloads of unused places count too: nothing else may be touched
            assert np.array_equal(got, w)
        else:
            assert np.array_equal(got, w)
            assert np.array_equal(dev[name + "s"].cpu().numpy(), want[name][1])
    return dev


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("total,new,hkv,d,page", [
    ([1], [1], 1, 64, 16), ([7, 40, 33], [7, 1, 33], 2, 128, 16), ([130, 5, 64], [66, 0, 64], 3, 64, 32),
    ([129], [2], 16, 128, 128), ([300, 17, 1, 64, 90], [45, 17, 1, 3, 0], 5, 128, 64), ([20] * 37, [1] * 37, 2, 64, 16)])
def test_append_to_the_bit(kind, dtype, total, new, hkv, d, page):
    c = Cache(total, new, hkv, d, page, kind, seed=len(total) + d).fill(upto_new=False)
    x = [torch.from_numpy(c.rng.standard_normal((c.n_tok, hkv, d)) * np.exp(c.rng.standard_normal((c.n_tok, hkv, 1)) * 3)).to(dtype)
         for _ in range(2)]
    check_append(c, *x)


def test_append_without_cu_seqlens_and_from_a_fused_projection():
    c = Cache([40, 19, 3], [3, 3, 3], 2, 128, 16, "e4m3", 5).fill(upto_new=False)
    fused = torch.randn(9, 8 * 128 + 2 * 256, generator=torch.Generator().manual_seed(2)).bfloat16()
    k, v = fused[:, 1024:1280].view(9, 2, 128), fused[:, 1280:].view(9, 2, 128)
    fd = fused.cuda()
    check_append(c, k, v, fd[:, 1024:1280].view(9, 2, 128), fd[:, 1280:].view(9, 2, 128), cu=False)


def test_append_special_values():
    """Zeros, the smallest and largest numbers, exact borders of the scale, ties of the code, NaN and infinities."""
    vals = [0.0, -0.0, 2.0 ** -133, 2.0 ** -126, 3.3895e38, -3.3895e38, 448.0, 7.0, 7.03125, 14.0, 1.0, 17 / 16, 19 / 16,
            2.0 ** -109, 448 * 2.0 ** -117, 1e30]
    T = len(vals) + 3
    c = Cache([T], [T], 2, 64, 16, "e4m3", 9)
    k = torch.zeros(T, 2, 64, dtype=torch.float64)
    rng = np.random.default_rng(1)
    for i, a in enumerate(vals):
        k[i, 0] = torch.from_numpy(rng.uniform(-1, 1, 64)) * abs(a)
        k[i, 0, 3] = a
        k[i, 1, i] = a
    k[-3, 0, 5], k[-2, 0, 6], k[-1, 1, 7] = float("nan"), float("inf"), -float("inf")
    # the inputs as the kernel sees them
    for dt in (torch.bfloat16, torch.float32):
        x = k.to(dt)
        check_append(c, x, x.flip(1).contiguous())


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("total,hkv,d,page", [([1], 1, 64, 16), ([7, 0, 40, 33], 2, 128, 16), ([130, 64], 9, 64, 128),
                                               ([300, 17, 1], 16, 128, 32), ([5] * 40, 1, 128, 16)])
def test_read_back_is_exact(kind, dtype, total, hkv, d, page):
    g = lib()
    c = Cache(total, total, hkv, d, page, kind, seed=d + page).fill(kscale=30.0, vscale=0.01)
    dev = c.cuda()
    n_rows = c.n_tok + 3
    out = [torch.full((n_rows, hkv, d), 12352.0, dtype=dtype, device="cuda") for _ in range(2)]
    k, v = g.kv_read(dev["kc"], dev["vc"], dev["table"], dev["cu"], n_rows, dev["ks"], dev["vs"], dtype=dtype, k=out[0],
                     v=out[1])
    g.check_error()
    for name, got in (("k", k), ("v", v)):
        want = np.concatenate([c.dense(name, i) for i in range(len(total))])
        assert np.array_equal(f64(got)[:c.n_tok], want)
        assert (f64(got)[c.n_tok:] == 12352.0).all()  # rows behind the last sequence stay as they were


def test_read_back_of_nan_rows():
    g = lib()
    c = Cache([3], [3], 1, 64, 16, "e4m3", 3).fill()
    c.ks[c.table[0, 0], 0, 1] = 255
    dev = c.cuda()
    k, v = g.kv_read(dev["kc"], dev["vc"], dev["table"], dev["cu"], 3, dev["ks"], dev["vs"])
    assert torch.isnan(k[1]).all() and torch.isfinite(k[[0, 2]]).all() and torch.isfinite(v).all()


@pytest.mark.parametrize("what", ["page", "page_neg", "len_long", "len_short", "cu_order"])
def test_bad_device_arguments_are_reported_and_skipped(what):
    g = lib()
    c = Cache([40, 40, 40], [2, 2, 2], 2, 64, 16, "bf16", 11).fill()
    x = torch.ones(6, 2, 64, dtype=torch.bfloat16)
    dev = c.cuda()
    before = {n: dev[n].clone() for n in ("kc", "vc")}
    if what == "page":
        dev["table"][1, 2] = c.n_pages
    elif what == "page_neg":
        dev["table"][1, 2] = -1
    elif what == "len_long":
        dev["lens"][1] = c.table.shape[1] * 16 + 1
    elif what == "len_short":
        dev["lens"][1] = 1
    else:
        dev["cu"][1] = 5
        dev["cu"][2] = 2
    g.kv_append(x.cuda(), x.cuda(), dev["kc"], dev["vc"], dev["table"], dev["lens"], dev["cu"])
    with pytest.raises(g.GdnError) as e:
        g.check_error()
    assert e.value.status == 5
    g.check_error()  # cleared
    if what != "cu_order":  # the other sequences are written, the bad one is not
        for i in (0, 2):
            pg, r = c.table[i, 39 // 16], 39 % 16
            assert (dev["kc"][int(pg), :, r] == 1).all()
        pg = int(c.table[1, 2])
        assert torch.equal(dev["kc"][pg].view(torch.int16), before["kc"][pg].view(torch.int16))
    if what.startswith("page"):
        n_rows = 120
        cu = torch.tensor([0, 40, 80, 120], dtype=torch.int32, device="cuda")
        g.kv_read(dev["kc"], dev["vc"], dev["table"], cu, n_rows)
        with pytest.raises(g.GdnError):
            g.check_error()


def many(hkv, d, kind, lens, page=32, seed=0):
    """A cache of random rows for sequences of the given lengths, on the device, and its block table."""
    gen = torch.Generator().manual_seed(seed)
    per = [-(-n // page) for n in lens]
    pages = sum(per) + 1
    table = torch.full((len(lens), max(per)), -1, dtype=torch.int32)
    order, at = torch.randperm(pages, generator=gen).to(torch.int32), 0
    for i, n in enumerate(per):
        table[i, :n] = order[at:at + n]
        at += n
    shape = (pages, hkv, page, d)
    if kind == "bf16":
        c = [torch.randn(shape, generator=gen).bfloat16().cuda() for _ in range(2)] + [None, None]
    else:
        c = [torch.randint(0, 0x7f, shape, generator=gen, dtype=torch.uint8).view(torch.float8_e4m3fn).cuda() for _ in range(2)]
        c += [torch.randint(120, 130, shape[:3], generator=gen, dtype=torch.uint8).cuda() for _ in range(2)]
    return c, table.cuda(), torch.tensor([0, *np.cumsum(lens)], dtype=torch.int32).cuda()


# heads and channels that put one, two and four tokens into a warp; lengths that end inside a warp's tokens, and none
@pytest.mark.parametrize("hkv,d", [(1, 64), (3, 128), (4, 128), (5, 64), (16, 128)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_long_calls_read_what_is_there(hkv, d, kind):
    g = lib()
    lens = [0, 1501, 2, 0, 1000, 3, 1, 700]
    (kc, vc, ks, vs), table, cu = many(hkv, d, kind, lens)
    n, page = sum(lens), 32
    out = [torch.full((n + 6, hkv, d), 9.0, device="cuda") for _ in range(2)]
    g.kv_read(kc, vc, table, cu, n + 6, ks, vs, torch.float32, *out)
    g.check_error()
    for cache, scale, got in ((kc, ks, out[0]), (vc, vs, out[1])):
        x = cache.float() if scale is None else cache.float() * torch.exp2(scale.float() - 127)[..., None]
        for i, m in enumerate(lens):
            pos = torch.arange(m, device="cuda")
            want = x[table[i].long()[pos // page], :, pos % page]
            assert torch.equal(got[int(cu[i]):int(cu[i]) + m], want), i
        assert (got[n:] == 9).all()


@pytest.mark.parametrize("hkv,d", [(1, 64), (3, 128), (4, 128), (5, 64), (16, 128)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_long_calls_write_what_short_ones_do(hkv, d, kind, dtype):
    """Several tokens a warp against calls of few tokens, which the tests above hold against the definition."""
    g = lib()
    lens, new = [1501, 2, 40, 1003, 3, 1, 700], [1501, 0, 7, 999, 3, 1, 699]
    a, table, _ = many(hkv, d, kind, lens)
    b = [None if t is None else t.clone() for t in a]
    cu = torch.tensor([0, *np.cumsum(new)], dtype=torch.int32)
    n = int(cu[-1])
    gen = torch.Generator().manual_seed(1)
    k, v = (torch.randn(n + 5, hkv, d, generator=gen).to(dtype).cuda() for _ in range(2))
    total = torch.tensor(lens, dtype=torch.int32).cuda()
    g.kv_append(k, v, a[0], a[1], table, total, cu.cuda(), a[2], a[3])
    for i, m in enumerate(new):
        for lo in range(0, m, 500):  # the sequence's tokens in pieces
            hi, at = min(m, lo + 500), int(cu[i])
            g.kv_append(k[at + lo:at + hi], v[at + lo:at + hi], b[0], b[1], table[i:i + 1].clone(), total[i:i + 1] - (m - hi), None, b[2], b[3])
    g.check_error()
    for x, y in zip(a, b):
        assert x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_long_uniform_call_and_bad_arguments_in_one():
    g = lib()
    lens = [800] * 4
    a, table, cu = many(2, 64, "e4m3", lens)
    b = [t.clone() for t in a]
    gen = torch.Generator().manual_seed(2)
    k, v = (torch.randn(2800, 2, 64, generator=gen).cuda() for _ in range(2))
    total = torch.tensor(lens, dtype=torch.int32).cuda()
    by = torch.arange(5, dtype=torch.int32, device="cuda") * 700
    g.kv_append(k, v, a[0], a[1], table, total, None, a[2], a[3])
    g.kv_append(k, v, b[0], b[1], table, total, by, b[2], b[3])
    g.check_error()
    for x, y in zip(a, b):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    # a page outside the pool and a length below its tokens: those rows are skipped, the others written
    bad, short = table.clone(), total.clone()
    bad[1, 10], short[2] = 10 ** 6, 699
    c = [torch.zeros_like(t) for t in a]
    g.kv_append(k, v, c[0], c[1], bad, short, None, c[2], c[3])
    with pytest.raises(g.GdnError):
        g.check_error()
    out = [torch.full((3200, 2, 64), 5.0, device="cuda") for _ in range(2)]
    g.kv_read(c[0], c[1], bad, cu, 3200, c[2], c[3], torch.float32, *out)
    with pytest.raises(g.GdnError):
        g.check_error()
    full = g.kv_read(a[0], a[1], table, cu, 3200, a[2], a[3], torch.float32)
    g.check_error()
    for got, want in zip(out, full):
        for i in range(4):
            s = slice(800 * i + 100, 800 * (i + 1))
            if i == 2:
                assert (got[s] == 0).all()
            elif i == 1:
                hole = slice(1120, 1152)  # page 10
                assert (got[hole] == 5).all() and torch.equal(got[900:1120], want[900:1120]) and torch.equal(got[1152:1600], want[1152:1600])
            else:
                assert torch.equal(got[s], want[s])
