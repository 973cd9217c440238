"""Edges of the gated feed-forward block and of the 4-bit matrix-vector products on the GPU: expert weights
past 32-bit offsets, a single row out of a buffer of any width, sums over no K, scale codes at the ends of
their range, gates around the zero of SwiGLU's derivative, the backward against BF16 weight transposes."""

import pytest
import torch

import microscaling_precision_quantization_amd as mxq
from microscaling_precision_quantization_amd import binding as B
from microscaling_precision_quantization_amd import pipeline
from tests import ffn_ref as R
from tests.test_gpu_ffn import BF, FMT, gen, randn, test_grouped_gemm_swiglu_backward as grouped_backward, weights4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [4, 8])
@pytest.mark.parametrize("I,K", [(65504, 65664), (65504, 131200)])
def test_decode_gate_up_of_an_expert_past_32_bits(tokens, I, K):
    """inter K past 2^32 (up rows more than 2^31 bytes behind their gates) and past 2^33 (more than 2^32), one
    expert, with few choices and with six and more."""
    assert I * K > (2 ** 32 if K < 2 ** 17 else 2 ** 33)
    # x of -1 and 1, scales of 2^-9 .. 2^-6: every product is a multiple of 2^-10 and at most 96 of them, and
    # 96 K < 2^24, so that sums are exact in binary32 in any order
    assert 96 * K < 2 ** 24
    g = gen(tokens)
    x = torch.where(randn(g, tokens, K) < 0, -1.0, 1.0).to(BF)
    q = torch.empty((2 * I, K // 2), dtype=torch.uint8, device="cuda")
    s = torch.empty((2 * I, K // 32), dtype=torch.uint8, device="cuda")
    for at in range(0, 2 * I, 8188):                        # 16 parts
        q[at:at + 8188].random_(0, 256, generator=g)
        s[at:at + 8188].random_(118, 122, generator=g)
    idx = torch.zeros((tokens, 1), dtype=torch.int32, device="cuda")
    h = mxq.moe_decode_gate_up(B.MXFP4, x, idx, q, s, experts=1)[:, 0]
    for lo in (0, I // 2 - 8, I - 40):
        rows = torch.cat([torch.arange(lo, lo + 40), torch.arange(I + lo, I + lo + 40)]).cuda()
        y = x.double() @ R.wide("mxfp4", q[rows], s[rows]).T
        want, tol, _ = R.gated(y, torch.zeros_like(y))
        R.check(h[:, lo:lo + 40], want, tol, f"h from column {lo}")


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_a_single_row_of_a_buffer_of_any_width(fmt):
    """One token's row: no second row is addressed, so the buffer's width does not matter."""
    K, I, E = 96, 40, 3
    g = gen(1)
    x = randn(g, 5, K + 3).to(BF)[:1, :K]
    assert x.stride(0) % 8
    w = randn(g, E * 2 * I, K, scale=0.2).to(BF)
    q, s, t = weights4(fmt, w, E)
    one = weights4(fmt, w[:2 * I])
    y, err = R.product(x.double(), R.wide(fmt, *one))
    R.check(mxq.gemv_block_scaled(FMT[fmt], x, *one), y, err + 2 * R.F32 * y.abs(), "y")
    want, tol, _ = R.gated(y, err + 2 * R.F32 * y.abs())
    R.check(mxq.gemv_swiglu(FMT[fmt], x, *one), want, tol, "h")
    for e in range(E):
        idx = torch.full((1, 1), e, dtype=torch.int32, device="cuda")
        got = mxq.moe_decode_gate_up(FMT[fmt], x, idx, q, s, t, experts=E)[:, 0]
        at = slice(e * 2 * I, (e + 1) * 2 * I)
        y, err = R.product(x.double(), R.wide(fmt, q[at], s[at], None if t is None else t[e:e + 1]))
        want, tol, _ = R.gated(y, err + 2 * R.F32 * y.abs())
        R.check(got, want, tol, f"h of expert {e}")


def k0_call(fn, dev, *args):
    B._call(fn, dev, *args)
    torch.cuda.synchronize()


@pytest.mark.parametrize("M,I", [(5, 24), (300, 272), (2601, 2416)])
def test_sums_over_no_k(M, I):
    """K = 0: h, (g | u) and dGU are zeros, h made again is silu(g) u. A call that hands buffers in, of which
    nothing is read."""
    buf = torch.full((4096,), float("nan"), dtype=BF, device="cuda")
    one = torch.ones(max(M, 2 * I), device="cuda")
    p, dev = buf.data_ptr(), buf.device
    off = torch.tensor([0, 0, M // 2, M], device="cuda")
    t = one.data_ptr()
    gu = randn(gen(M), M, 2 * I).to(BF)
    (_, _), (hw, htol) = R.through(torch.zeros(M, I, dtype=torch.float64, device="cuda"), 0.0, gu)
    new = lambda n: torch.full((M, n), float("nan"), dtype=BF, device="cuda")
    for fmt in (B.BF16, B.MXFP8, B.NVFP4):
        h, y = new(I), new(2 * I)
        k0_call("gemm_swiglu", dev, fmt, M, I, 0, p, p, t, 0, p, p, t, 1, h.data_ptr(), y.data_ptr(), None, 0)
        assert bool((h == 0).all()) and bool((y == 0).all()), fmt
    for fmt in (B.BF16, B.MXFP8):
        d, h = new(2 * I), new(I)
        k0_call("gemm_swiglu_backward", dev, fmt, M, I, 0, p, p, p, p, gu.data_ptr(), 0, d.data_ptr(), h.data_ptr(), None, 0)
        assert bool((d == 0).all()), fmt
        R.check(h, hw, htol, "h")
    for fmt in (B.BF16, B.NVFP4):
        h, y = new(I), new(2 * I)
        k0_call("grouped_gemm_swiglu", dev, fmt, 3, off.data_ptr(), M, I, 0, None, 0, p, p, t, 0, p, p, t, 2, h.data_ptr(),
                y.data_ptr(), None, 0)
        assert bool((h == 0).all()) and bool((y == 0).all()), fmt
    for fmt in (B.BF16, B.BF16_NVFP4T):
        if fmt == B.BF16_NVFP4T and I % 16:
            continue
        d, h = new(2 * I), new(I)
        k0_call("grouped_gemm_swiglu_backward", dev, fmt, 3, off.data_ptr(), M, I, 0, p, p, p, t, gu.data_ptr(), 0,
                d.data_ptr(), h.data_ptr(), None, 0)
        assert bool((d == 0).all()), fmt
        R.check(h, hw, htol, "h")


@pytest.mark.parametrize("code", [0, 1, 3, 252])
@pytest.mark.parametrize("rows", [1, 5, 20, 40])
def test_mxfp4_scale_codes_at_the_ends(code, rows):
    """Weights of q 2^(code - 127) from BF16's subnormal range to its largest, x such that the sums are ordinary
    numbers; plain, gated, over experts with few choices and with many, and down."""
    K, I = 160, 40
    g = gen(rows + code)
    x = (randn(g, rows, K) * 2.0 ** (120 if code < 100 else -112)).to(BF)
    assert bool(torch.isfinite(x).all())
    q = torch.randint(0, 256, (2 * I, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.full((2 * I, K // 32), code, dtype=torch.uint8, device="cuda")
    w = R.wide("mxfp4", q, s)
    y, err = R.product(x.double(), w)
    R.check(mxq.gemv_block_scaled(B.MXFP4, x, q, s), y, err + 2 * R.F32 * y.abs(), "y")
    want, tol, _ = R.gated(y, err)
    R.check(mxq.gemv_swiglu(B.MXFP4, x, q, s), want, tol, "h")
    idx = torch.zeros((rows, 1), dtype=torch.int32, device="cuda")
    got = mxq.moe_decode_gate_up(B.MXFP4, x, idx, q, s, experts=1)
    R.check(got[:, 0], want, tol, "h of the expert")
    wt = torch.full((rows, 1), 0.5, device="cuda")
    o = mxq.moe_decode_down(B.MXFP4, x[:, None].contiguous(), idx, wt, q, s, experts=1)
    R.check(o, 0.5 * y, err + 2 * R.F32 * y.abs(), "down")


def test_gates_around_the_zero_of_the_derivative():
    """silu'(g) vanishes at g = -1.27846...: the two terms of 1 + g (1 - sigma) cancel there, and d_gate is held
    to the size of what is added up, not to its own."""
    zero = torch.tensor([-1.2784645427610738], dtype=torch.float64, device="cuda")
    steps = torch.arange(-200, 200, device="cuda", dtype=torch.float64)
    g = (zero + torch.sign(steps) * torch.exp2(steps.abs() / 8 - 26)).float()
    M, I = g.numel(), 8
    gate_up = torch.ones(M, 2 * I, device="cuda")
    gate_up[:, :I] = g[:, None]
    d = torch.ones(M, 8, dtype=BF, device="cuda")
    w = torch.zeros(I, 8, dtype=BF, device="cuda")
    w[:, 0] = 1.0
    dgu, h = mxq.gemm_swiglu_backward(B.BF16, d, None, w, None, gate_up)
    (want, tol), (hw, htol) = R.through(torch.ones(M, I, dtype=torch.float64, device="cuda"), 0.0, gate_up)
    R.check(dgu, want, tol, "d_gate_up")
    R.check(h, hw, htol, "h")


class Experts:
    T, H, G, I, K, PAD = 96, 256, 16, 128, 3, 32

    def __init__(self, fused):
        d = torch.device("cuda")
        g = gen(3)
        plan = B.RoutePlan(self.T, self.G, self.K, self.PAD, dev=d)
        B.moe_route(randn(g, self.T, self.G), self.K, self.PAD, out=plan)
        self.m = pipeline.MoeNvfp4(self.T, self.H, self.G, self.I, plan, d, fused=fused)
        self.m.quantize_weights(randn(g, self.G * 2 * self.I, self.H, scale=0.1).to(BF),
                                randn(g, self.G * self.H, self.I, scale=0.1).to(BF))
        self.m.forward(randn(g, self.T, self.H).to(BF))
        live = (plan.row_index >= 0)[:, None]
        self.d_o = (randn(g, plan.slots, self.H, scale=1e-3) * live).to(BF)


@pytest.mark.parametrize("fused", [False, True])
def test_backward_through_swiglu_against_bf16_weight_transposes(fused):
    """fused_weights=False reads BF16 transposes of the weights that fused_weights=True makes on the way: the same
    operands, and so the same gradients but for the order of the sums."""
    c = Experts(fused)
    m, off = c.m, c.m.r.offsets.tolist()
    a = pipeline.MoeDequantBackward(m, through_swiglu=True)
    a.backward(c.d_o)
    b = pipeline.MoeDequantBackward(m, fused_weights=False, through_swiglu=True)
    b.dequantize_weights()
    b.backward(c.d_o)
    wd = B.dequantize(B.NVFP4, *m.wq["d"], t_scope="group", group_rows=c.H).double().view(c.G, c.H, c.I)
    wgu = B.dequantize(B.NVFP4, *m.wq["gu"], t_scope="group", group_rows=2 * c.I).double().view(c.G, 2 * c.I, c.H)
    for e in range(c.G):
        at = slice(off[e], off[e + 1])
        dh, err = R.product(c.d_o[at].double(), wd[e].T)
        (want, tol), _ = R.through(dh, err, m.gu[at])
        for r, name in ((a, "from the NVFP4 weights"), (b, "from BF16 transposes")):
            R.check(r.d_gu[at], want, tol, f"d_gate_up of expert {e} {name}")
            R.check(r.dx[at], *R.product(r.d_gu[at].double(), wgu[e].T), f"dx of expert {e} {name}")
            R.check(r.dw_gu[e], *R.product(r.d_gu[at].double().T, r.xT[0, :, at].double()), f"dw_gu of expert {e} {name}")
            R.check(r.dw_d[e], *R.product(c.d_o[at].double().T, r.hT[0, :, at].double()), f"dw_d of expert {e} {name}")


@pytest.mark.parametrize("through", [False, True])
def test_backward_without_its_weight_transposes_is_refused(through):
    c = Experts(True)
    b = pipeline.MoeDequantBackward(c.m, fused_weights=False, through_swiglu=through)
    d_gu = None if through else torch.zeros(c.m.S, 2 * c.I, dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        b.backward(c.d_o, d_gu)
    b.dequantize_weights()
    b.backward(c.d_o, d_gu)


@pytest.mark.parametrize("f32", [False, True])
def test_dense_backward_against_nvfp4_weights_as_one_group(f32):
    """A dense block's gradient against the forward's NVFP4 W_d: one expert of all rows."""
    grouped_backward("nvfp4", 272, 72, [300], [0], f32)
