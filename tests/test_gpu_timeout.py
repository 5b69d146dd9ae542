"""The device time-out path of the tensor-core kernel, made to run without any GPU fault.

``gdn_debug_stall`` makes the chunk kernel wait on a barrier that nothing arrives on, with a ~1 ms limit: the
wait runs out, the kernel sets the device error word and every warp leaves through its own bounded waits after
draining what it issued.  The host then reads GDN_ERR_TIMEOUT, the context stays usable, and the next ordinary
call is parity-green against the fp64 oracle.
"""
import pytest
import torch

from gated_delta_rule_105_b200 import binding as bd
from gated_delta_rule_105_b200.inputs import generate
from parity_util import TOL, f64, o_excess, relerr, run_cuda, run_oracle

pytestmark = pytest.mark.gpu


def test_stalled_wait_reports_timeout_and_the_next_call_is_correct():
    inp = generate(1, 130, 2, 128, 128, "bf16", seed=55, h0_std=0.05)
    bd.set_kernel("tc")
    try:
        bd.debug_stall(True)
        try:
            run_cuda(inp, "gdn")
        finally:
            bd.debug_stall(False)
        with pytest.raises(bd.GdnError) as ei:
            bd.check_error()
        assert ei.value.status == bd.GDN_ERR_TIMEOUT
        bd.check_error()  # the word was cleared and the context is still usable
        o, hT = run_cuda(inp, "gdn")
        bd.check_error()
        assert bd.last_kernel() == "tc"
    finally:
        bd.set_kernel("auto")
    ro, rh = run_oracle(inp, "gdn")
    assert o_excess(f64(o), ro, "bf16", "f32") <= 1.0
    assert relerr(f64(hT), rh) <= TOL["bf16"]


def test_stall_does_not_touch_the_simt_kernel():
    inp = generate(1, 70, 2, 64, 64, "f32", seed=56)
    bd.debug_stall(True)
    try:
        o, hT = run_cuda(inp, "gdn")
        bd.check_error()
    finally:
        bd.debug_stall(False)
    assert bd.last_kernel() == "simt"
    ro, rh = run_oracle(inp, "gdn")
    assert o_excess(f64(o), ro, "f32", "f32") <= 1.0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
def test_stalled_attention_chunks_report_timeout_and_the_next_call_is_correct(kind, d):
    """The same of the attention layer's chunk kernel, with more key tiles than its rings hold, so that copies, products and
    softmax steps of the row tile that is not held up are in flight when the wait runs out."""
    import gated_delta_rule_105_b200 as g
    from attn_util import Cache, attn_excess, attn_reference
    c = Cache([1500, 40, 700], [150, 1, 90], 2, d, 64, kind, 5).fill()
    dev = c.cuda()
    q = torch.randn(c.n_tok, 8, d, generator=torch.Generator().manual_seed(1)).bfloat16()

    def call():
        return g.paged_attn_fwd(q.cuda(), dev["kc"], dev["vc"], dev["table"], dev["lens"], dev["cu"], dev["ks"], dev["vs"],
                                return_lse=True)

    want = call()
    bd.check_error()
    for _ in range(2):
        bd.debug_stall(True)
        try:
            call()
        finally:
            bd.debug_stall(False)
        with pytest.raises(bd.GdnError) as ei:
            bd.check_error()
        assert ei.value.status == bd.GDN_ERR_TIMEOUT
        bd.check_error()
        got = call()
        bd.check_error()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    eo, el = attn_excess(*want, attn_reference(c, f64(q), d ** -0.5, 0), c, 0, torch.bfloat16)
    assert eo <= 1.0 and el <= 1.0


def test_stall_does_not_touch_decoding():
    import gated_delta_rule_105_b200 as g
    from attn_util import Cache
    c = Cache([300, 40], [1, 1], 2, 64, 16, "bf16", 6).fill()
    dev = c.cuda()
    q = torch.randn(2, 8, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    args = q, dev["kc"], dev["vc"], dev["table"], dev["lens"]
    want = g.paged_attn_fwd(*args)
    bd.debug_stall(True)
    try:
        got = g.paged_attn_fwd(*args)
        bd.check_error()
    finally:
        bd.debug_stall(False)
    assert torch.equal(got, want)
