"""Refusals of the gated feed-forward block and of the 4-bit matrix-vector products, on the host: every
bad argument is answered before a launch, through the C ABI and through the binding."""

import pytest
import torch

from microscaling_precision_quantization_amd import binding as B

P = 0x10000
MIS = 0x10004
BF, F32 = B.OUT_BF16, B.OUT_F32
ROW, TENSOR, GROUP = 0, 1, 2
BIG = 1 << 31


def test_gemm_swiglu_validation():
    def f(fmt=B.BF16, M=4, I=16, K=64, A=P, sA=P, tA=P, ta=ROW, W=P, sB=P, tB=P, tb=TENSOR, h=P, gu=P, ws=P,
          wsn=1 << 30):
        return B.lib().gemm_swiglu(fmt, M, I, K, A, sA, tA, ta, W, sB, tB, tb, h, gu, ws, wsn, None)

    need = B.lib().mxq_workspace_bytes(B.OP_GEMM_SWIGLU, 4, 32, 4096)
    assert need == 8 * 4 * 32 * 4 and B.lib().mxq_workspace_bytes(B.OP_GEMM_SWIGLU, 4, 32, 512) == 0
    assert B.lib().mxq_workspace_bytes(B.OP_GEMM_SWIGLU, 0, 32, 4096) == 0
    assert B.lib().mxq_workspace_bytes(B.OP_GEMM_SWIGLU, 16384, 4096, 7168) == 0
    assert f(K=4096, ws=None) == 5 and f(K=4096, wsn=need - 1) == 5 and f(K=4096, ws=MIS) == 3

    assert f(M=-1) == 2 and f(I=-8) == 2 and f(K=-8) == 2
    for fmt in (0, B.MXFP4, B.BF16_NVFP4T, 9):
        assert f(fmt=fmt) == 4
    assert f(M=0) == 0 and f(I=0) == 0 and f(M=0, A=None, h=None) == 0
    assert f(A=None) == 1 and f(W=None) == 1 and f(h=None) == 1
    for fmt in (B.MXFP8, B.NVFP4):
        assert f(fmt=fmt, sA=None) == 1 and f(fmt=fmt, sB=None) == 1
        assert f(fmt=fmt, K=40) == 2 and f(fmt=fmt, sA=MIS) == 3 and f(fmt=fmt, sB=MIS) == 3
    assert f(fmt=B.NVFP4, tA=None) == 1 and f(fmt=B.NVFP4, tB=None) == 1
    assert f(fmt=B.NVFP4, ta=GROUP) == 4 and f(fmt=B.NVFP4, tb=GROUP) == 4
    assert f(fmt=B.NVFP4, tA=P + 2) == 3 and f(fmt=B.NVFP4, tB=P + 2) == 3
    assert f(I=12) == 2 and f(K=12) == 2 and f(K=(1 << 22) + 8) == 2
    assert f(I=1 << 23, K=64) == 2                                          # 2 inter rows of B: 2^31 bytes
    assert f(M=1 << 40) == 2 and f(M=1 << 31, I=1 << 12) == 2               # more tiles than a grid holds
    assert f(A=MIS) == 3 and f(W=MIS) == 3 and f(h=MIS) == 3 and f(gu=MIS) == 3


def test_gemm_swiglu_backward_validation():
    def f(fmt=B.BF16, M=4, I=16, K=64, A=P, sA=P, W=P, sB=P, gu=P, gd=BF, d=P, h=P, ws=P, wsn=1 << 30):
        return B.lib().gemm_swiglu_backward(fmt, M, I, K, A, sA, W, sB, gu, gd, d, h, ws, wsn, None)

    need = B.lib().mxq_workspace_bytes(B.OP_GEMM_SWIGLU, 4, 16, 4096)
    assert f(K=4096, ws=None) == 5 and f(K=4096, wsn=need - 1) == 5 and f(K=4096, ws=MIS) == 3

    assert f(M=-1) == 2 and f(I=-8) == 2 and f(K=-8) == 2
    for fmt in (B.NVFP4, B.MXFP4, B.BF16_NVFP4T, 0):
        assert f(fmt=fmt) == 4
    assert f(gd=2) == 4 and f(gd=-1) == 4
    assert f(M=0) == 0 and f(I=0, d=None) == 0
    assert f(A=None) == 1 and f(W=None) == 1 and f(gu=None) == 1 and f(d=None) == 1
    assert f(fmt=B.MXFP8, sA=None) == 1 and f(fmt=B.MXFP8, sB=None) == 1
    assert f(I=12) == 2 and f(K=12) == 2 and f(fmt=B.MXFP8, K=40) == 2
    assert f(I=1 << 24, K=64) == 2 and f(M=1 << 40) == 2
    assert f(A=MIS) == 3 and f(W=MIS) == 3 and f(gu=MIS) == 3 and f(d=MIS) == 3 and f(h=MIS) == 3
    assert f(fmt=B.MXFP8, sA=MIS) == 3 and f(fmt=B.MXFP8, sB=MIS) == 3


def test_grouped_gemm_swiglu_validation():
    need = B.lib().mxq_workspace_bytes(B.OP_GROUPED_SWIGLU, 257, 0, 0)
    assert need > 0 and B.lib().mxq_workspace_bytes(B.OP_GROUPED_SWIGLU, 256, 0, 0) == 0

    def f(fmt=B.NVFP4, G=3, off=P, total=8, I=16, K=64, idx=P, rows=8, A=P, sA=P, tA=P, ta=ROW, W=P, sB=P, tB=P, tb=GROUP,
          h=P, gu=P, ws=P, wsn=need):
        return B.lib().grouped_gemm_swiglu(fmt, G, off, total, I, K, idx, rows, A, sA, tA, ta, W, sB, tB, tb, h, gu, ws,
                                           wsn, None)

    assert f(G=-1) == 2 and f(total=-1) == 2 and f(I=-8) == 2 and f(K=-1) == 2 and f(rows=-1) == 2
    for fmt in (B.MXFP8, B.MXFP4, B.BF16_NVFP4T, 0):
        assert f(fmt=fmt) == 4
    assert f(G=0) == 0 and f(total=0) == 0 and f(I=0) == 0
    assert f(off=None) == 1 and f(A=None) == 1 and f(W=None) == 1 and f(h=None) == 1
    assert f(sA=None) == 1 and f(sB=None) == 1 and f(tA=None) == 1 and f(tB=None) == 1
    assert f(ta=GROUP) == 4 and f(tb=TENSOR) == 4
    assert f(I=12) == 2 and f(K=40) == 2 and f(fmt=B.BF16, K=12) == 2
    assert f(rows=BIG // 32) == 2 and f(fmt=B.BF16, rows=BIG // 128) == 2   # the gathered operand: 2^31 bytes
    assert f(I=1 << 25) == 2 and f(total=1 << 40) == 2 and f(G=1 << 40) == 2
    assert f(off=P + 4) == 3 and f(idx=P + 2) == 3 and f(h=MIS) == 3 and f(gu=MIS) == 3 and f(A=MIS) == 3 and f(W=MIS) == 3
    assert f(G=257, ws=None) == 5 and f(G=257, wsn=need - 1) == 5 and f(G=257, ws=MIS) == 3


def test_grouped_gemm_swiglu_backward_validation():
    need = B.lib().mxq_workspace_bytes(B.OP_GROUPED_SWIGLU, 257, 0, 0)
    assert need > 0 and B.lib().mxq_workspace_bytes(B.OP_GROUPED_SWIGLU, 256, 0, 0) == 0

    def f(fmt=B.BF16_NVFP4T, G=3, off=P, total=8, I=16, K=64, A=P, W=P, sB=P, tB=P, gu=P, gd=F32, d=P, h=P, ws=P,
          wsn=need):
        return B.lib().grouped_gemm_swiglu_backward(fmt, G, off, total, I, K, A, W, sB, tB, gu, gd, d, h, ws, wsn, None)

    assert f(G=-1) == 2 and f(total=-1) == 2 and f(I=-8) == 2 and f(K=-8) == 2
    for fmt in (B.NVFP4, B.MXFP8, B.MXFP4, 0):
        assert f(fmt=fmt) == 4
    assert f(gd=2) == 4
    assert f(G=0) == 0 and f(total=0) == 0 and f(I=0) == 0
    assert f(off=None) == 1 and f(A=None) == 1 and f(W=None) == 1 and f(gu=None) == 1 and f(d=None) == 1
    assert f(sB=None) == 1 and f(tB=None) == 1
    assert f(I=24) == 2 and f(K=12) == 2 and f(I=1 << 20, K=1 << 12) == 2
    assert f(fmt=B.BF16, I=1 << 24) == 2 and f(total=1 << 40) == 2
    assert f(off=P + 4) == 3 and f(gu=MIS) == 3 and f(d=MIS) == 3 and f(h=MIS) == 3 and f(A=MIS) == 3 and f(tB=P + 2) == 3
    assert f(G=257, ws=None) == 5 and f(G=257, wsn=need - 1) == 5 and f(G=257, ws=MIS) == 3


def test_gemv_validation():
    def f(fmt=B.NVFP4, rows=4, N=16, K=64, x=P, ld=64, W=P, s=P, t=P, sc=TENSOR, y=P, yd=F32, ldy=16):
        return B.lib().gemv_block_scaled(fmt, rows, N, K, x, ld, W, s, t, sc, y, yd, ldy, None)

    def g(fmt=B.NVFP4, rows=4, N=16, K=64, x=P, ld=64, W=P, s=P, t=P, sc=TENSOR, y=P, ldy=16):
        return B.lib().gemv_swiglu(fmt, rows, N, K, x, ld, W, s, t, sc, y, ldy, None)

    assert g(N=1 << 20, K=1 << 12, ld=1 << 12, ldy=1 << 20) == 2            # gate and up rows: 2^32 bytes
    assert f(yd=2) == 4 and f(y=P + 2) == 3 and f(y=P + 1, yd=BF) == 3
    for q in (f, g):
        assert q(rows=-1) == 2 and q(rows=65) == 2 and q(N=-1) == 2
        for fmt in (B.MXFP8, B.BF16, B.BF16_NVFP4T, 0):
            assert q(fmt=fmt) == 4
        assert q(rows=0) == 0 and q(N=0) == 0 and q(rows=0, x=None, y=None) == 0
        assert q(x=None) == 1 and q(W=None) == 1 and q(s=None) == 1 and q(t=None) == 1 and q(y=None) == 1
        assert q(sc=GROUP) == 4
        assert q(K=0, ld=64) == 2 and q(K=48) == 2 and q(ld=32) == 2 and q(ldy=8) == 2 and q(K=1 << 23, ld=1 << 23) == 2
        assert q(N=1 << 40, ldy=1 << 40) == 2 and q(ld=1 << 29) == 2
        assert q(x=MIS) == 3 and q(W=MIS) == 3 and q(s=P + 1) == 3 and q(t=P + 2) == 3 and q(ld=68) == 3 and q(y=P + 1) == 3


def test_moe_decode_validation():
    def f(fmt=B.MXFP4, T=4, k=2, E=8, n=16, K=64, x=P, ld=64, idx=P, W=P, s=P, t=None, sc=GROUP, h=P):
        return B.lib().moe_decode_gate_up(fmt, T, k, E, n, K, x, ld, idx, W, s, t, sc, h, None)

    need = B.lib().mxq_workspace_bytes(B.OP_DECODE_DOWN, 4, 16, 2)
    assert need == 4 * 2 * 16 * 4
    assert B.lib().mxq_workspace_bytes(B.OP_DECODE_DOWN, 0, 16, 2) == 0

    def g(fmt=B.MXFP4, T=4, k=2, E=8, n=16, K=64, x=P, idx=P, w=P, W=P, s=P, t=None, sc=GROUP, h=P, yd=F32, ws=P, wsn=need):
        return B.lib().moe_decode_down(fmt, T, k, E, n, K, x, idx, w, W, s, t, sc, h, yd, ws, wsn, None)

    assert g(ws=None) == 5 and g(wsn=need - 1) == 5 and g(ws=P + 2) == 3
    assert g(T=64, k=32, E=64, K=1 << 20, wsn=1 << 20) == 2                 # h of 2^32 bytes

    for q in (f, g):
        assert q(T=-1) == 2 and q(T=65) == 2 and q(k=-1) == 2 and q(k=33) == 2 and q(E=-1) == 2 and q(E=1025) == 2
        assert q(n=-1) == 2 and q(E=0) == 2 and q(n=1 << 40) == 2
        for fmt in (B.MXFP8, B.BF16, 0):
            assert q(fmt=fmt) == 4
        assert q(T=0) == 0 and q(n=0) == 0
        assert q(x=None) == 1 and q(idx=None) == 1 and q(W=None) == 1 and q(s=None) == 1 and q(h=None) == 1
        assert q(fmt=B.NVFP4) == 1 and q(fmt=B.NVFP4, t=P, sc=TENSOR) == 4
        assert q(K=48) == 2 and q(K=0) == 2
        assert q(x=MIS) == 3 and q(W=MIS) == 3 and q(idx=P + 2) == 3 and q(h=P + 1) == 3
    assert f(k=0) == 0 and g(k=0) == 2                      # nothing to write; a sum of nothing is refused
    assert f(ld=32) == 2 and f(ld=68) == 3
    assert g(w=None) == 1 and g(w=P + 2) == 3 and g(yd=2) == 4 and g(h=P + 2) == 3


def test_binding_refuses_what_does_not_fit():
    bf, u8, f32, i32 = torch.bfloat16, torch.uint8, torch.float32, torch.int32
    e = lambda *s, dt=bf: torch.empty(s, dtype=dt)
    bad = lambda fn, *a, **kw: pytest.raises(ValueError, fn, *a, **kw)
    x, w = e(4, 64), e(32, 64)
    bad(B.gemm_swiglu, B.MXFP4, x, None, w, None)
    bad(B.gemm_swiglu, B.BF16, x, None, e(31, 64), None)                    # odd rows
    bad(B.gemm_swiglu, B.BF16, x, None, e(32, 72), None)
    bad(B.gemm_swiglu, B.BF16, x.float(), None, w, None)
    bad(B.gemm_swiglu, B.BF16, e(4, 1, 64), None, w, None)
    bad(B.gemm_swiglu, B.BF16, x, None, w, None)                            # not on a GPU
    bad(B.gemm_swiglu, B.MXFP8, e(4, 64, dt=u8), None, e(32, 64, dt=u8), e(32, 2, dt=u8))
    bad(B.gemm_swiglu_backward, B.NVFP4, x, None, w, None, e(4, 64))
    bad(B.gemm_swiglu_backward, B.BF16, x, None, w, None, e(4, 64, dt=torch.float16))
    bad(B.gemm_swiglu_backward, B.BF16, x, None, w, None, e(4, 32))
    off = torch.tensor([0, 2, 4])
    bad(B.grouped_gemm_swiglu, B.MXFP8, off, x, e(2, 32, 64), inter=16, K=64)
    bad(B.grouped_gemm_swiglu, B.BF16, off, x, e(2, 32, 64), inter=24, K=64)
    bad(B.grouped_gemm_swiglu, B.BF16, off, e(5, 64), e(2, 32, 64), inter=16, K=64)
    bad(B.grouped_gemm_swiglu_backward, B.NVFP4, off, x, e(2, 16, 64), inter=16, K=64, gate_up=e(4, 32))
    bad(B.grouped_gemm_swiglu_backward, B.BF16, off, x, e(2, 16, 64), inter=16, K=64, gate_up=e(4, 16))
    bad(B.grouped_gemm_swiglu_backward, B.BF16_NVFP4T, off, x, e(128, 8, dt=u8), inter=16, K=64, gate_up=e(4, 32))
    q, s, t = e(32, 32, dt=u8), e(32, 4, dt=u8), e(1, dt=f32)
    for fn in (B.gemv_block_scaled, B.gemv_swiglu):
        bad(fn, B.MXFP8, x, q, s, t)
        bad(fn, B.NVFP4, x, q, s)                                           # no FP32 scale
        bad(fn, B.NVFP4, x, q, s, t, t_scope="group")
        bad(fn, B.NVFP4, x, q, s, t, t_scope="row")                         # one scale for 32 rows
        bad(fn, B.NVFP4, x, q, e(32, 2, dt=u8), t)
        bad(fn, B.NVFP4, e(4, 96), q, s, t)
        bad(fn, B.NVFP4, x.float(), q, s, t)
        bad(fn, B.NVFP4, x, q, s, t)                                        # not on a GPU
    bad(B.gemv_swiglu, B.NVFP4, x, q[:31], s[:31], t)
    bad(B.gemv_block_scaled, B.NVFP4, x, q, s, t, out_dtype=torch.float16)
    bad(B.gemv_block_scaled, B.NVFP4, x, q, s, t, out=e(4, 32, dt=torch.float16))
    bad(B.gemv_block_scaled, B.NVFP4, x, q, s, t, out=e(4, 31))
    idx, wt, t2 = e(4, 2, dt=i32), e(4, 2, dt=f32), e(2, dt=f32)
    bad(B.moe_decode_gate_up, B.NVFP4, x, idx, q, s, t2)                    # how many experts
    bad(B.moe_decode_gate_up, B.NVFP4, x, idx, q, s, t2, experts=3)
    bad(B.moe_decode_gate_up, B.NVFP4, x, idx.long(), q, s, t2, experts=2)
    bad(B.moe_decode_gate_up, B.NVFP4, x, e(3, 2, dt=i32), q, s, t2, experts=2)
    bad(B.moe_decode_gate_up, B.NVFP4, x, idx, q, s, t, experts=2)          # one scale for two experts
    bad(B.moe_decode_gate_up, B.NVFP4, x, idx, q, s, t2, experts=2)         # not on a GPU
    h = e(4, 2, 64)
    bad(B.moe_decode_down, B.NVFP4, x, idx, wt, q, s, t2, experts=2)
    bad(B.moe_decode_down, B.NVFP4, h, idx, wt[:, :1], q, s, t2, experts=2)
    bad(B.moe_decode_down, B.NVFP4, h, idx, wt, q, s, t2, experts=2, out_dtype=torch.int32)
    bad(B.moe_decode_down, B.NVFP4, h, idx, wt, q, s, t2, experts=2, out=e(4, 15))
    bad(B.moe_decode_down, B.NVFP4, h, idx, wt, q, s, t2, experts=2)        # not on a GPU


def test_a_single_row_may_have_any_stride():
    """One row: nothing is addressed by its stride (the output's stride, looked at afterwards, is what is refused)."""
    def f(fn, rows, ld, ldy):
        tail = (F32, ldy, None) if fn == "gemv_block_scaled" else (ldy, None)
        return getattr(B.lib(), fn)(B.NVFP4, rows, 16, 64, P, ld, P, P, P, TENSOR, P, *tail)

    for fn in ("gemv_block_scaled", "gemv_swiglu"):
        assert f(fn, 2, 68, 8) == 3 and f(fn, 1, 68, 8) == 2 and f(fn, 1, (1 << 40) + 1, 8) == 2
        assert f(fn, 1, 63, 16) == 2                                        # a row stride below the row


def test_moe_decode_width_limit():
    """inter and hidden up to 65520: beyond it the size is what is refused, up to it the pointer."""
    def gate_up(n):
        return B.lib().moe_decode_gate_up(B.MXFP4, 4, 2, 8, n, 64, P, 64, P + 2, P, P, None, GROUP, P, None)

    def down(n):
        return B.lib().moe_decode_down(B.MXFP4, 4, 2, 8, n, 64, P, P + 2, P, P, P, None, GROUP, P, F32, P, 1 << 30, None)

    for f in (gate_up, down):
        assert f(65520) == 3 and f(65521) == 2 and f(65536) == 2
