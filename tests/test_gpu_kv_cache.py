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
