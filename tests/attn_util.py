"""Inputs and error bounds of the attention layer's tests.

Bounds are per element and follow from the arithmetic.  u(t) below is half a step of type t relative to the value
(bf16 2^-8, fp32 2^-24).
Attention, with weights p_j, o = sum p_j v_j / sum p_j:
  * a score is a sum of d products in fp32: off by at most d 2^-23 sum_c |q_c k_c| scale (twice u per addition, since
    the tensor cores may cut instead of round), plus 4 u(fp32) |score| for the scaling by log2(e) and the subtraction
    of the maximum; |score| <= the same sum.  Call it e_s.  A weight is then off by 2 e_s relative (its own and its
    share in the denominator) and by 2^-21 for ex2.approx (2^-22, in both);
  * the weights are rounded to bf16 for the product with V: u(bf16) relative;
  * n additions in fp32 in numerator and denominator: n 2^-23 each; joining parts adds less than 64 2^-23.
  |o - o_ref| <= mean_p(|v|) (u(bf16) + 2 e_s + 2^-21 + (2 n + 64) 2^-23) + u(type of o) |o_ref|.
  |lse - lse_ref| <= e_s + 2^-22 + (n + 64) 2^-23 + 4 u(fp32) |lse_ref|.
"""
import numpy as np
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


class Cache:
    """A paged cache and the sequences in it.  ``total`` positions per sequence, of which the last ``new`` are new;
    every place that belongs to no sequence holds NaN (bf16) or the NaN scale (8 bits)."""

    def __init__(self, total, new, hkv, d, page, kind, seed, spare=2, extra_cols=1):
        rng = np.random.default_rng(seed)
        self.rng, self.total, self.new, self.hkv, self.d, self.page, self.kind = rng, total, new, hkv, d, page, kind
        per = [-(-t // page) for t in total]
        self.n_pages = sum(per) + spare
        order = rng.permutation(self.n_pages)
        self.table = np.full((len(total), max(1, max(per)) + extra_cols), -7, np.int32)
        at = 0
        for i, c in enumerate(per):
            self.table[i, :c] = order[at:at + c]
            at += c
        shape = (self.n_pages, hkv, page, d)
        if kind == "bf16":
            self.kc, self.vc = (torch.full(shape, float("nan"), dtype=torch.bfloat16) for _ in range(2))
            self.ks = self.vs = None
        else:
            self.kc, self.vc = (torch.full(shape, 0x7e, dtype=torch.uint8).view(torch.float8_e4m3fn) for _ in range(2))
            self.ks, self.vs = (torch.full(shape[:3], 255, dtype=torch.uint8) for _ in range(2))
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
        self.lens = torch.tensor(total, dtype=torch.int32)
        self.n_tok = int(sum(new))

    def fill(self, upto_new=True, kscale=1.0, vscale=1.0):
        """Random rows at every position (without ``upto_new`` not at the new tokens' own)."""
        for i, (t, a) in enumerate(zip(self.total, self.new)):
            for pos in range(t if upto_new else t - a):
                pg, r = self.table[i, pos // self.page], pos % self.page
                for which, sc in (("k", kscale), ("v", vscale)):
                    self.put(which, pg, r, self.rng.standard_normal((self.hkv, self.d)) * sc)
        return self

    def put(self, which, pg, r, x):
        import oracle.attn as oa
        cache = self.kc if which == "k" else self.vc
        if self.kind == "bf16":
            cache[pg, :, r] = torch.from_numpy(np.asarray(x)).to(torch.bfloat16)
        else:
            scale = self.ks if which == "k" else self.vs
            for h in range(self.hkv):
                code, byte = oa.quantise_row(np.asarray(x)[h])
                cache.view(torch.uint8)[pg, h, r] = torch.from_numpy(code)
                scale[pg, h, r] = byte

    def dense(self, which, i, lo=0, hi=None):
        import oracle.attn as oa
        cache, scale = (self.kc, self.ks) if which == "k" else (self.vc, self.vs)
        raw = f64(cache) if self.kind == "bf16" else cache.view(torch.uint8).numpy()
        return oa.cache_rows(raw, None if scale is None else scale.numpy(), self.table[i], self.page, lo,
                             self.total[i] if hi is None else hi)

    def cuda(self):
        dev = {k: getattr(self, k) for k in ("kc", "vc", "ks", "vs", "cu", "lens")}
        out = {k: None if v is None else v.cuda() for k, v in dev.items()}
        out["table"] = torch.from_numpy(self.table).cuda()
        return out


def attn_reference(c, q, scale, window):
    """fp64 attention of q [n_tok, Hq, d] (fp64): o, lse and the bounds' ingredients, packed like q."""
    import oracle.attn as oa
    parts = []
    for i, a in enumerate(c.new):
        at = int(c.cu[i])
        if a:
            parts.append(oa.attention(q[at:at + a], c.dense("k", i), c.dense("v", i), scale, window))
    return [np.concatenate([p[j] for p in parts]) for j in range(4)]


def attn_excess(o, lse, ref, c, window, o_dtype):
    """(largest |o - ref| / bound, largest |lse - ref| / bound): at most 1 each."""
    ro, rl, absv, mass = ref
    d, n = ro.shape[-1], max(c.total)
    if window:
        n = min(n, window)
    es = mass * (d * 2.0 ** -23 + 4 * 2.0 ** -24)
    bo = absv * (2.0 ** -8 + 2 * es[..., None] + 2.0 ** -21 + (2 * n + 64) * 2.0 ** -23) + U[o_dtype] * np.abs(ro)
    bl = es + 2.0 ** -22 + (n + 64) * 2.0 ** -23 + 4 * 2.0 ** -24 * np.abs(rl)
    return float(np.max(np.abs(f64(o) - ro) / bo)), float(np.max(np.abs(f64(lse) - rl) / bl))


def attn_within(o, lse, ref, c, window, o_dtype):
    """Every element within :func:`attn_excess`'s bound, without its quotients: a token that sees one key whose value has the
    8-bit code 0 has output 0 and bound 0."""
    ro, rl, absv, mass = ref
    d, n = ro.shape[-1], min(max(c.total), window or max(c.total))
    es = mass * (d * 2.0 ** -23 + 4 * 2.0 ** -24)
    bo = absv * (2.0 ** -8 + 2 * es[..., None] + 2.0 ** -21 + (2 * n + 64) * 2.0 ** -23) + U[o_dtype] * np.abs(ro)
    bl = es + 2.0 ** -22 + (n + 64) * 2.0 ** -23 + 4 * 2.0 ** -24 * np.abs(rl)
    return bool(np.all(np.abs(f64(o) - ro) <= bo) and np.all(np.abs(f64(lse) - rl) <= bl))
