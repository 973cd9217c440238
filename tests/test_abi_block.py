"""Refusals of the norm and router entry points, on the host: every bad argument is answered
before a launch, through the C ABI and through the binding."""

import ctypes

import pytest
import torch

from microscaling_precision_quantization_amd import binding as B

P = 0x10000
MIS = 0x10004
NAN = float("nan")
BF, F32 = B.OUT_BF16, B.OUT_F32


def test_rmsnorm_quantize_validation():
    def f(fmt=B.MXFP8, x=P, xd=BF, rows=4, cols=64, ld=64, w=P, eps=1e-6, n=P, q=P, s=P, t=None, rstd=P):
        return B.lib().rmsnorm_quantize(fmt, x, xd, rows, cols, ld, w, eps, n, q, s, t, rstd, None)

    assert f(rows=-1) == 2 and f(cols=-1) == 2
    assert f(rows=0) == 0 and f(rows=0, x=None) == 0
    assert f(fmt=9) == 4 and f(fmt=B.BF16_NVFP4T) == 4 and f(xd=2) == 4
    assert f(eps=0.0) == 4 and f(eps=-1.0) == 4 and f(eps=NAN) == 4 and f(eps=float("inf")) == 4
    assert f(x=None) == 1 and f(q=None) == 1 and f(s=None) == 1 and f(fmt=B.NVFP4) == 1
    assert f(fmt=B.BF16, n=None) == 1
    assert f(cols=48, ld=48) == 2 and f(fmt=B.MXFP4, cols=48, ld=48) == 2
    assert f(fmt=B.NVFP4, cols=40, ld=40, t=P) == 2 and f(fmt=B.BF16, cols=12, ld=12) == 2
    assert f(ld=32) == 2 and f(cols=16416, ld=16416) == 2
    assert f(ld=68) == 3 and f(xd=F32, ld=66) == 3
    assert f(x=MIS) == 3 and f(w=MIS) == 3 and f(n=MIS) == 3 and f(q=MIS) == 3 and f(rstd=P + 2) == 3
    assert f(fmt=B.NVFP4, t=P + 2) == 3


def test_rmsnorm_backward_validation():
    def f(dn=P, dn2=None, dd=F32, x=P, xd=BF, rstd=P, w=P, res=None, rows=4, cols=64, dx=P, dw=P, ws=P, wsn=1 << 20):
        return B.lib().rmsnorm_backward(dn, dn2, dd, x, xd, rstd, w, res, 1.0, rows, cols, dx, dw, ws, wsn, None)

    need = B.lib().mxq_workspace_bytes(B.OP_NORM_BACKWARD, 4, 64, 0)
    assert need > 0 and B.lib().mxq_workspace_bytes(B.OP_NORM_BACKWARD, 0, 64, 0) == 0
    assert f(rows=-1) == 2 and f(cols=60) == 2 and f(cols=16392) == 2
    assert f(dd=2) == 4 and f(xd=2) == 4 and f(w=None) == 4               # dw without a weight
    assert f(dn=None) == 1 and f(x=None) == 1 and f(rstd=None) == 1 and f(dx=None) == 1
    assert f(ws=None) == 5 and f(wsn=need - 1) == 5
    assert f(dn=MIS) == 3 and f(dn2=MIS) == 3 and f(res=MIS) == 3 and f(dx=MIS) == 3 and f(dw=MIS) == 3
    assert f(ws=MIS) == 3
    assert f(rows=0, dw=None, dn=None) == 0 and f(cols=0) == 0


def test_gate_residual_validation():
    def f(x=P, xd=BF, y=P, yd=F32, w=P, gate=P, mode=1, eps=1e-6, rows=4, cols=64, out=P, rstd=P):
        return B.lib().rmsnorm_gate_residual(x, xd, y, yd, w, gate, mode, eps, 1.0, 1.0, rows, cols, out, rstd, None)

    assert f(rows=-1) == 2 and f(cols=60) == 2 and f(cols=16392) == 2
    assert f(mode=4) == 4 and f(mode=-1) == 4 and f(eps=0.0) == 4 and f(xd=3) == 4 and f(yd=3) == 4
    assert f(gate=None) == 1 and f(gate=None, mode=2) == 1 and f(x=None) == 1 and f(y=None) == 1 and f(out=None) == 1
    assert f(gate=P + 2) == 3 and f(gate=MIS, mode=2) == 3 and f(gate=MIS, mode=3) == 3 and f(x=MIS) == 3 and f(y=MIS) == 3 and f(out=MIS) == 3 and f(w=MIS) == 3
    assert f(rows=0) == 0 and f(cols=0) == 0

    def g(d=P, dd=BF, y=P, yd=F32, rstd=P, w=P, gate=P, mode=2, rows=4, cols=64, dy=P, dw=P, dg=P, ws=P, wsn=1 << 20):
        return B.lib().rmsnorm_gate_residual_backward(d, dd, y, yd, rstd, w, gate, mode, 1.0, rows, cols, dy, dw, dg,
                                                      ws, wsn, None)

    assert g(rows=-1) == 2 and g(cols=60) == 2 and g(mode=5) == 4 and g(w=None) == 4
    assert g(mode=0) == 4                                                   # dgate without a gate
    assert g(d=None) == 1 and g(y=None) == 1 and g(rstd=None) == 1 and g(dy=None) == 1 and g(gate=None) == 1
    assert g(ws=None) == 5 and g(ws=None, dw=None) == 5 and g(wsn=16) == 5
    assert g(d=MIS) == 3 and g(dg=MIS) == 3 and g(ws=MIS) == 3
    assert g(rows=0, dw=None, dg=None) == 0


def test_route_validation():
    def f(z=P, valid=None, T=4, G=8, ld=8, k=2, pad=4, total=32, idx=P, w=P, counts=P, off=P, row=P, slot=P, loss=P,
          ws=P, wsn=1 << 20):
        return B.lib().moe_route(z, valid, T, G, ld, k, pad, total, 0.1, idx, w, counts, off, row, slot, loss, ws, wsn,
                                 None)

    assert B.route_slots(4, 8, 2, 4) == 32
    assert f(total=28) == 2 and f(total=34) == 2                            # below the worst case; no multiple of pad
    assert f(k=0) == 2 and f(k=9) == 2 and f(G=0) == 2 and f(G=2000, ld=2000, total=1 << 20) == 2
    assert f(pad=0) == 2 and f(T=-1) == 2 and f(ld=7) == 2 and f(total=1 << 31) == 2
    assert f(T=(1 << 22) + 1, total=1 << 24) == 2                           # tokens beyond 2^22
    assert f(G=64, ld=64, k=33, total=1 << 12) == 2                         # topk beyond 32
    for name in ("z", "idx", "w", "counts", "off", "row", "slot"):
        assert f(**{name: None}) == 1, name
    assert f(ws=None) == 5 and f(wsn=8) == 5
    assert f(z=P + 2) == 3 and f(off=MIS) == 3 and f(slot=MIS) == 3 and f(ws=MIS) == 3
    assert B.lib().mxq_route_slots(4, 8, 0, 1) == -1 and B.lib().mxq_route_slots(-1, 8, 1, 1) == -1
    with pytest.raises(ValueError, match="no routing"):
        B.route_slots(4, 8, 40, 1)

    def g(z=P, T=4, G=8, ld=8, k=2, idx=P, w=P, dw=P, counts=P, dl=P, out=P, od=F32):
        return B.lib().moe_route_backward(z, T, G, ld, k, idx, w, dw, counts, dl, 0.1, out, od, None)

    assert g(k=9) == 2 and g(ld=4) == 2 and g(T=-1) == 2 and g(G=1025, ld=1025) == 2
    assert g(z=None) == 1 and g(idx=None) == 1 and g(out=None) == 1 and g(w=None) == 1 and g(counts=None) == 1
    assert g(out=P + 2) == 3 and g(od=2) == 4 and g(T=0) == 0


def test_combine_backward_validation():
    def f(dy=P, dd=F32, o=P, S=8, T=4, k=2, H=64, slot=P, w=P, row=P, d_o=P, dw=P):
        return B.lib().moe_combine_backward(dy, dd, o, S, T, k, H, slot, w, row, d_o, dw, None)

    assert f(H=60) == 2 and f(H=16392) == 2 and f(k=33) == 2 and f(S=-1) == 2 and f(T=-1) == 2 and f(dd=2) == 4
    for name in ("dy", "o", "slot", "w", "row", "d_o", "dw"):
        assert f(**{name: None}) == 1, name
    assert f(dy=MIS) == 3 and f(o=MIS) == 3 and f(d_o=MIS) == 3 and f(slot=MIS) == 3
    assert f(T=0, S=0) == 0


def test_binding_refuses_wrong_buffers():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    f32 = lambda *s: torch.zeros(s, dtype=torch.float32)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    x, y = bf(4, 64), f32(4, 64)
    with pytest.raises(ValueError, match="x: expected a bfloat16 or float32"):
        B.rmsnorm_quantize(x.half())
    with pytest.raises(ValueError, match="2-D"):
        B.rmsnorm_quantize(bf(64))
    with pytest.raises(ValueError, match="unknown format"):
        B.rmsnorm_quantize(x, fmt=77)
    with pytest.raises(ValueError, match="weight: shape"):
        B.rmsnorm_quantize(x, f32(32))
    with pytest.raises(ValueError, match="weight: dtype"):
        B.rmsnorm_quantize(x, bf(64))
    with pytest.raises(ValueError, match="innermost"):
        B.rmsnorm_quantize(bf(64, 4).t())
    with pytest.raises(ValueError, match="row stride"):
        B.rmsnorm_quantize(bf(1, 64).expand(4, 64))
    with pytest.raises(ValueError, match="GPU tensor"):
        B.rmsnorm_quantize(x)
    with pytest.raises(ValueError, match="dn2: dtype"):
        B.rmsnorm_backward(y, x, f32(4), dn2=x)
    with pytest.raises(ValueError, match="rstd: shape"):
        B.rmsnorm_backward(y, x, f32(3))
    with pytest.raises(ValueError, match="d_res: dtype"):
        B.rmsnorm_backward(y, x, f32(4), d_res=y)
    with pytest.raises(ValueError, match="gate_mode"):
        B.rmsnorm_gate_residual(x, y, gate=f32(4), gate_mode="row")
    with pytest.raises(ValueError, match="gate_mode is 'none'"):
        B.rmsnorm_gate_residual(x, y, gate=f32(4))
    with pytest.raises(ValueError, match="gate: shape"):
        B.rmsnorm_gate_residual(x, y, gate=f32(4), gate_mode="channel")
    with pytest.raises(ValueError, match="gate: expected a tensor"):
        B.rmsnorm_gate_residual(x, y, gate_mode="token")
    with pytest.raises(ValueError, match="contiguous"):
        B.rmsnorm_gate_residual(bf(4, 128)[:, :64], y)
    with pytest.raises(ValueError, match="dgate: shape"):
        B.rmsnorm_gate_residual_backward(x, y, f32(4), gate=f32(4), gate_mode="token", out=(f32(4, 64), None, f32(64)))
    with pytest.raises(ValueError, match="logits: dtype"):
        B.moe_route(bf(4, 8), 2)
    with pytest.raises(ValueError, match="valid: shape"):
        B.moe_route(f32(4, 8), 2, valid=torch.ones(3, dtype=torch.bool))
    with pytest.raises(ValueError, match="no routing"):
        B.moe_route(f32(4, 8), 0)
    plan = B.RoutePlan(4, 8, 2, dev="cpu")
    assert plan.slots == 8 and plan.loss is None
    with pytest.raises(ValueError, match="other sizes"):
        B.moe_route(f32(5, 8), 2, out=plan)
    with pytest.raises(ValueError, match="without a loss"):
        B.moe_route(f32(4, 8), 2, out=plan, balance_coef=0.1)
    with pytest.raises(ValueError, match="total"):
        B.RoutePlan(4, 8, 2, pad=4, total=28, dev="cpu")
    with pytest.raises(ValueError, match="GPU tensor"):
        B.moe_route(f32(4, 8), 2, out=plan)
    with pytest.raises(ValueError, match="counts: shape"):
        B.moe_route_backward(f32(4, 8), i32(4, 2), f32(4, 2), i32(8))
    with pytest.raises(ValueError, match="row_index: shape"):
        B.moe_combine_backward(y, f32(8, 64), torch.zeros((4, 2), dtype=torch.int64), f32(4, 2), i32(7))


@pytest.mark.parametrize("name,index", [("cuda", 3), ("cuda:1", 1), (2, 2), (torch.device("cuda"), 3),
                                        (torch.device("cuda", 1), 1)])
def test_streams_of_devices_named_in_any_way(monkeypatch, name, index):
    """A device may be a torch.device, a string or an index, as for torch's own calls; without an
    index it is the current one."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i, raising=False)
    assert B._stream(name) == 100 + index


def test_a_plan_keeps_no_loss_of_another_call():
    """A plan with a loss is refused where the call would leave that loss as it was."""
    plan = B.RoutePlan(4, 8, 2, loss=True, dev="cpu")
    with pytest.raises(ValueError, match="a plan with a loss"):
        B.moe_route(torch.zeros(4, 8), 2, out=plan)
    with pytest.raises(ValueError, match="GPU tensor"):      # with a coefficient, even zero, it is written
        B.moe_route(torch.zeros(4, 8), 2, out=plan, balance_coef=0.0)


def test_backward_refuses_slots_that_its_weight_gradients_would_leave_out():
    """The weight gradients' GEMMs reduce over slots that begin at multiples of 8; at any other offset
    they write nothing, so such a block, or such a routing from the host, is refused when it is made."""
    from types import SimpleNamespace

    import numpy as np

    from microscaling_precision_quantization_amd import inputs, pipeline
    make = lambda T=192, G=16, pad=32: pipeline.MoeBlockNvfp4(T, 64, G, 32, 3, "cpu", pad=pad, backward=True)
    for kw in (dict(pad=1), dict(pad=4), dict(pad=12), dict(T=190), dict(G=24)):
        with pytest.raises(ValueError, match="expected multiples of 8, 8 and 16"):
            make(**kw)
    logits = np.random.default_rng(0).standard_normal((64, 16)).astype(np.float32)
    fwd = lambda r: SimpleNamespace(r=r, dev="cpu", G=16, H=64, I=32, S=r.slots)
    for pad in (1, 4, 12):                                   # 12: some offset is no multiple of 8
        r = pipeline.MoeRoutingDevice(inputs.route_topk(logits, 3, pad=pad), "cpu")
        assert any(int(v) % 8 for v in r.offsets)
        with pytest.raises(ValueError, match="multiple of 8"):
            pipeline.MoeDequantBackward(fwd(r))
        with pytest.raises(ValueError, match="multiple of 8"):
            pipeline.MoeDequantBackward(fwd(B.RoutePlan(64, 16, 3, pad, dev="cpu")))
    for pad in (8, 32):
        r = pipeline.MoeRoutingDevice(inputs.route_topk(logits, 3, pad=pad), "cpu")
        assert pipeline.MoeDequantBackward(fwd(r)).dw_d.shape == (16, 64, 32)
        assert make(pad=pad).bwd.dw_gu.shape == (16, 64, 64)
    assert pipeline.MoeBlockNvfp4(5, 64, 3, 32, 2, "cpu").plan.pad == 1           # forward only: any sizes


def test_combine_backward_without_choices_or_slots():
    """topk = 0 takes no dy, slot_of or weights, whatever the tokens; the slots' own buffers are
    still required."""
    f = lambda S, o=P, row=P, d_o=P, T=4: B.lib().moe_combine_backward(None, F32, o, S, T, 0, 64, None, None, row, d_o,
                                                                       None, None)
    assert f(0) == 0 and f(0, T=0) == 0
    assert f(8, o=None) == 1 and f(8, row=None) == 1 and f(8, d_o=None) == 1


def test_combine_backward_of_rows_without_elements():
    """hidden = 0 takes no slot buffers, and without tokens there is nothing to launch."""
    f = lambda T, k, dy=P: B.lib().moe_combine_backward(dy, F32, None, 8, T, k, 0, P, P, None, None, P, None)
    assert f(0, 2) == 0 and f(4, 0) == 0
    assert f(4, 2, dy=None) == 1


def test_route_slots_of_sizes_that_the_router_refuses():
    """-1 for every size that moe_route answers with a shape error, whatever total it is given, and a
    plan of such a size is not made."""
    f = B.lib().mxq_route_slots
    for T, G, k, pad in ((4, 8, 9, 1), (10, 4, 8, 1), (4, 8, 0, 1), (4, 0, 1, 1), (4, 2000, 2, 1), (-1, 8, 2, 1),
                         (4, 8, 2, 0), ((1 << 22) + 1, 8, 2, 1), (4, 64, 33, 1),
                         (1 << 20, 1024, 2, 1 << 21), (8, 8, 1, 1 << 30)):    # the last two: 2^31 slots and more
        assert f(T, G, k, pad) == -1, (T, G, k, pad)
        total = (1 << 31) - 1 - ((1 << 31) - 1) % max(pad, 1)
        assert B.lib().moe_route(P, None, T, G, max(G, 1), k, pad, total, 0.1, P, P, P, P, P, P, P, P, 1 << 40, None) == 2
        with pytest.raises(ValueError, match="no routing"):
            B.RoutePlan(T, G, k, pad, dev="cpu")
    assert f(4, 8, 8, 1) == 32 and f(0, 8, 8, 4) == 0 and f(1, 1, 1, 0x7FFFFFFF) == 0x7FFFFFFF


def test_rows_without_elements_are_refused():
    """They have no mean: no statistic, and no gradient of a token's gate, is handed back for them."""
    x, y, one = torch.zeros((4, 0), dtype=torch.bfloat16), torch.zeros((4, 0)), torch.zeros(4)
    empty = torch.zeros(0)
    for call in (lambda: B.rmsnorm_quantize(x, fmt=B.BF16), lambda: B.rmsnorm_backward(y, x, one, empty),
                 lambda: B.rmsnorm_gate_residual(x, y), lambda: B.rmsnorm_gate_residual_backward(x, y, one, None, one, "token"),
                 lambda: B.moe_combine_backward(y, y, torch.zeros((4, 1), dtype=torch.int64), torch.zeros((4, 1)),
                                                torch.zeros(4, dtype=torch.int32))):
        with pytest.raises(ValueError, match="rows without elements"):
            call()


def test_eps_that_would_leave_the_binary32_range():
    """Below 2^-252 the statistic of a row of zeros passes the binary32 range: refused wherever it is
    held in binary32."""
    for eps, status in ((2.0 ** -253, 4), (1e-80, 4), (5e-324, 4), (2.0 ** -252, 1), (1e-30, 1)):     # 1: x is null
        assert B.lib().rmsnorm_quantize(B.BF16, None, BF, 4, 64, 64, P, eps, P, None, None, None, P, None) == status
        assert B.lib().rmsnorm_gate_residual(None, BF, P, F32, P, None, 0, eps, 1.0, 1.0, 4, 64, P, P, None) == status
    assert B.lib().rmsnorm_quantize(B.BF16, None, BF, 4, 64, 64, P, 1e-80, P, None, None, None, None, None) == 1


def test_every_call_runs_on_the_device_of_its_tensors(monkeypatch):
    """A kernel is launched on the device that is current, so a call makes its tensors' device the
    current one around the launch and hands in that device's stream; every call of the library that
    takes a stream goes this way."""
    import inspect
    import re

    from microscaling_precision_quantization_amd import pipeline
    current, seen = [0], []

    class Device:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            self.before, current[0] = current[0], self.dev.index

        def __exit__(self, *exc):
            current[0] = self.before

    class Lib:
        def moe_combine(self, *args):
            seen.append((current[0], args))
            return 0

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i, raising=False)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(B, "lib", lambda: Lib())
    for index in (0, 1):
        B._call("moe_combine", torch.device("cuda", index), 7)
    assert seen == [(0, (7, 100)), (1, (7, 101))] and current == [0]
    source = inspect.getsource(B) + inspect.getsource(pipeline)
    assert len(re.findall(r"_stream\(", source)) == 3        # its definition and _call's two
    assert len(re.findall(r"_check\(", source)) == 3
    takes_stream = {n for n in B._SIGS if not n.startswith("mxq_")}
    assert takes_stream - {"quantize_mxfp8_multi", "quantize_mxfp4_multi"} <= set(re.findall(r'_call\(\s*"(\w+)"', source))
