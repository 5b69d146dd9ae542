"""Arguments that the attention layer's entry points refuse: on the host, before any launch (CPU, no device)."""
import ctypes

import pytest
import torch

from gated_delta_rule_105_b200 import binding as bd

A = 0x10000  # a 16-byte aligned fake device address; never dereferenced by the host checks
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_105_b200 import build
    build.build()
    return bd.load_library()


def append(lib, **kw):
    a = dict(k=A, v=A, ks=256, vs=256, kc=A, vc=A, ksc=A, vsc=A, bt=A, sl=A, cu=A, n_tok=4, n_seqs=2, n_pages=8,
             max_pages=4, page=16, hkv=2, d=128, dt=1, cdt=2)
    a.update(kw)
    return lib.gdn_kv_append(*[a[x] for x in ("k", "v", "ks", "vs", "kc", "vc", "ksc", "vsc", "bt", "sl", "cu", "n_tok",
                                              "n_seqs", "n_pages", "max_pages", "page", "hkv", "d", "dt", "cdt")], None)


def read(lib, **kw):
    a = dict(kc=A, vc=A, ksc=A, vsc=A, bt=A, cu=A, k=A, v=A, n_rows=4, n_seqs=2, n_pages=8, max_pages=4, page=16, hkv=2,
             d=128, cdt=2, dt=1)
    a.update(kw)
    return lib.gdn_kv_read(*[a[x] for x in ("kc", "vc", "ksc", "vsc", "bt", "cu", "k", "v", "n_rows", "n_seqs", "n_pages",
                                            "max_pages", "page", "hkv", "d", "cdt", "dt")], None)


def attn(lib, **kw):
    a = dict(q=A, qs=512, kc=A, vc=A, ksc=A, vsc=A, bt=A, sl=A, cu=A, scale=0.1, window=0, o=A, lse=A, n_tok=4, n_seqs=2,
             n_pages=8, max_pages=4, page=16, hq=4, hkv=2, d=128, cdt=2, odt=1, ws=A, wsb=1 << 40)
    a.update(kw)
    return lib.gdn_paged_attn_fwd(*[a[x] for x in ("q", "qs", "kc", "vc", "ksc", "vsc", "bt", "sl", "cu", "scale", "window",
                                                   "o", "lse", "n_tok", "n_seqs", "n_pages", "max_pages", "page", "hq",
                                                   "hkv", "d", "cdt", "odt", "ws", "wsb")], None)


CACHE = [(dict(kc=None), 1), (dict(vc=A + 8), 1), (dict(bt=None), 1), (dict(bt=A + 4), 1), (dict(ksc=None), 1),
         (dict(vsc=A + 1), 1), (dict(n_seqs=0), 1), (dict(n_seqs=65536), 1), (dict(n_pages=0), 1), (dict(max_pages=0), 1),
         (dict(page=8), 2), (dict(page=48), 2), (dict(page=256), 2), (dict(hkv=0), 1), (dict(d=96), 2), (dict(d=256), 2),
         (dict(cdt=0), 2), (dict(cdt=7), 2), (dict(cdt=1), 1), (dict(n_pages=1 << 26), 2),
         (dict(max_pages=1 << 27), 2), (dict(cu=A + 4), 1)]


@pytest.mark.parametrize("kw,status", CACHE + [
    (dict(k=None), 1), (dict(v=A + 2), 1), (dict(sl=None), 1), (dict(ks=255), 1), (dict(vs=260), 1), (dict(ks=128), 1),
    (dict(n_tok=-1), 1), (dict(n_tok=3, cu=None), 1), (dict(dt=2), 2), (dict(dt=0, ks=258), 1)])
def test_append_refusals(lib, kw, status):
    assert append(lib, **kw) == status
    assert lib.gdn_last_error().decode() != ""


@pytest.mark.parametrize("kw,status", CACHE + [(dict(cu=None), 1), (dict(k=None), 1), (dict(v=A + 8), 1),
                                               (dict(n_rows=-1), 1), (dict(dt=2), 2)])
def test_read_refusals(lib, kw, status):
    assert read(lib, **kw) == status
    assert lib.gdn_last_error().decode() != ""


@pytest.mark.parametrize("kw,status", CACHE + [
    (dict(q=None), 1), (dict(q=A + 8), 1), (dict(o=None), 1), (dict(lse=A + 4), 1), (dict(sl=None), 1), (dict(qs=511), 1),
    (dict(qs=516), 1), (dict(hq=3), 1), (dict(hq=1), 1), (dict(hq=2 * 257), 1), (dict(odt=2), 2), (dict(scale=NAN), 1),
    (dict(scale=INF), 1), (dict(window=-1), 1), (dict(n_tok=-2), 1), (dict(n_tok=3, cu=None), 1), (dict(ws=None), 1),
    (dict(wsb=64), 1), (dict(n_tok=1 << 30), 2)])
def test_attention_refusals(lib, kw, status):
    assert attn(lib, **kw) == status
    assert lib.gdn_last_error().decode() != ""


def test_no_tokens_is_no_work(lib):
    assert append(lib, n_tok=0, k=None, v=None) == 0
    assert read(lib, n_rows=0, k=None, v=None) == 0
    assert attn(lib, n_tok=0, q=None, o=None, ws=None, wsb=0) == 0
    assert norm(lib, rows=0, x=None, y=None) == 0


def norm(lib, **kw):
    a = dict(x=A, res=A, w=A, s=A, y=A, ysc=A, rstd=A, rows=4, d=256, dt=1, ydt=2, group=128, eps=1e-5)
    a.update(kw)
    return lib.gdn_add_rmsnorm_fwd(*[a[x] for x in ("x", "res", "w", "s", "y", "ysc", "rstd", "rows", "d", "dt", "ydt",
                                                    "group", "eps")], None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(w=None), 1), (dict(y=None), 1), (dict(ysc=None), 1), (dict(res=A + 2), 1), (dict(s=A + 8), 1),
    (dict(rows=-1), 1), (dict(rows=1 << 31), 1), (dict(d=12), 2), (dict(d=0), 2), (dict(d=16392), 2), (dict(dt=2), 2),
    (dict(ydt=0), 2), (dict(group=64), 2), (dict(d=192), 2), (dict(ydt=1), 1), (dict(ydt=1, group=0), 1), (dict(eps=-1.0), 1),
    (dict(eps=NAN), 1)])
def test_norm_refusals(lib, kw, status):
    assert norm(lib, **kw) == status
    assert lib.gdn_last_error().decode() != ""


def norm_bwd(lib, **kw):
    a = dict(dy=A, s=A, w=A, rstd=A, ds=A, dx=A, dw=A, rows=4, d=256, dt=1, ws=A, wsb=1 << 40)
    a.update(kw)
    return lib.gdn_add_rmsnorm_bwd(*[a[x] for x in ("dy", "s", "w", "rstd", "ds", "dx", "dw", "rows", "d", "dt", "ws", "wsb")],
                                   None)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), 1), (dict(s=None), 1), (dict(w=None), 1), (dict(rstd=None), 1), (dict(dx=None), 1), (dict(dw=None), 1),
    (dict(ds=A + 2), 1), (dict(d=20), 2), (dict(dt=2), 2), (dict(rows=-1), 1), (dict(ws=None), 1), (dict(wsb=16), 1)])
def test_norm_backward_refusals(lib, kw, status):
    assert norm_bwd(lib, **kw) == status
    assert lib.gdn_last_error().decode() != ""


def test_workspace_sizes(lib):
    assert bd.paged_attn_workspace_bytes(0, 1, 8, 2, 128) == 0
    assert bd.paged_attn_workspace_bytes(1, 1, 8, 3, 128) == 0
    assert bd.paged_attn_workspace_bytes(1, 1, 8, 2, 96) == 0
    assert bd.paged_attn_workspace_bytes(4096, 2, 8, 2, 128) > 0
    assert bd.add_rmsnorm_bwd_workspace_bytes(0, 64) == 0 and bd.add_rmsnorm_bwd_workspace_bytes(7, 64) > 0


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    kc = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    bt, sl = torch.zeros(1, 4, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    k, q = torch.zeros(1, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    e8 = kc.view(torch.uint8).view(torch.float8_e4m3fn)[..., :64].contiguous()
    sc = torch.zeros(4, 2, 16, dtype=torch.uint8)
    for call in (lambda: bd.kv_append(k, k, kc, kc, bt, sl), lambda: bd.paged_attn_fwd(q, kc, kc, bt, sl),
                 lambda: bd.kv_read(kc, kc, bt, torch.zeros(2, dtype=torch.int32), 1),
                 lambda: bd.add_rmsnorm_fwd(k, torch.ones(64)), lambda: bd.add_rmsnorm_bwd(k, k, torch.ones(64), sl.float()),
                 lambda: bd.kv_append(k, k, e8, e8, bt, sl), lambda: bd.kv_append(k, k, kc, kc, bt, sl, None, sc, sc),
                 lambda: bd.kv_append(k[:, :1], k[:, :1], kc, kc, bt, sl), lambda: bd.kv_append(k.half(), k.half(), kc, kc, bt, sl),
                 lambda: bd.kv_append(k, k, kc, kc, bt.long(), sl), lambda: bd.kv_append(k, k, kc, kc, bt, sl.long()),
                 lambda: bd.kv_append(k, k, kc, kc, bt, torch.ones(2, dtype=torch.int32)),
                 lambda: bd.kv_append(k.transpose(1, 2), k.transpose(1, 2), kc, kc, bt, sl),
                 lambda: bd.paged_attn_fwd(q.float(), kc, kc, bt, sl), lambda: bd.paged_attn_fwd(q, kc, kc[:3], bt, sl),
                 lambda: bd.paged_attn_fwd(q, kc.half(), kc.half(), bt, sl),
                 lambda: bd.paged_attn_fwd(q, kc, kc, bt, sl, o_dtype=torch.float16),
                 lambda: bd.add_rmsnorm_fwd(k, torch.ones(64), group=64), lambda: bd.add_rmsnorm_fwd(k.half(), torch.ones(64)),
                 lambda: bd.add_rmsnorm_fwd(k, torch.ones(64), out_dtype=torch.float16)):
        with pytest.raises(ValueError):
            call()


def test_scales_and_windows_out_of_range(lib):
    assert attn(lib, scale=3e38) == 1  # times log2(e): no fp32 number
    kc = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    bt, sl = torch.zeros(1, 4, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    for window in (-1, 1 << 31, (1 << 32) + 5):
        with pytest.raises(ValueError, match="window"):
            bd.paged_attn_fwd(q, kc, kc, bt, sl, window=window)


@pytest.mark.parametrize("page", [16, 128])
def test_block_tables_whose_positions_would_pass_32_bits(lib, page):
    """What the kernels add to a position before they clamp it must stay below 2^31."""
    most = ((1 << 31) - 4096) // page
    for call in (append, read, attn):
        assert call(lib, page=page, max_pages=most + 1) == 2
        assert "2^31 - 4096" in lib.gdn_last_error().decode()


def test_workspaces_whose_bytes_are_not_their_own(lib):
    """numel() of an expanded or strided tensor is not what may be written from its address on."""
    kc = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    bt, sl = torch.zeros(1, 4, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    s, w, rstd = torch.zeros(3, 64), torch.ones(64), torch.ones(3)
    good = torch.empty(1 << 24, dtype=torch.uint8)
    for bad in (torch.empty(1, dtype=torch.uint8).expand(1 << 24), good[::2], good.view(4096, 4096).T, good.view(torch.int8),
                good.view(torch.float32)):
        with pytest.raises(ValueError, match="contiguous uint8"):
            bd.paged_attn_fwd(q, kc, kc, bt, sl, workspace=bad)
        with pytest.raises(ValueError, match="contiguous uint8"):
            bd.add_rmsnorm_bwd(s, s, w, rstd, workspace=bad)
    with pytest.raises(ValueError, match="CUDA"):  # past this check, and refused for the tensors' device
        bd.paged_attn_fwd(q, kc, kc, bt, sl, workspace=good)
