"""The gated feed-forward block (gemm_swiglu and its backward, dense and per expert) and the 4-bit
matrix-vector products against FP64, with the bounds of tests/ffn_ref.py: formats, ragged sizes, empty
and padded experts, gates far out, rows behind the outputs, streams and graphs,
long K and tensors past 2^31 bytes."""

import pytest
import torch

import microscaling_precision_quantization_amd as mxq
from microscaling_precision_quantization_amd import binding as B
from tests import ffn_ref as R

pytestmark = pytest.mark.gpu
FMT = {"bf16": B.BF16, "mxfp8": B.MXFP8, "nvfp4": B.NVFP4, "mxfp4": B.MXFP4}
BF = torch.bfloat16


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, scale=1.0):
    return scale * torch.randn(shape, generator=g, device="cuda")


def guarded(*shape, dtype=BF):
    """A tensor in front of memory that must stay as it is: (tensor, check)."""
    n = 1
    for v in shape:
        n *= v
    flat = torch.full((n + 4096,), 7.0, dtype=dtype, device="cuda")
    flat[:n] = float("nan")

    def untouched():
        assert bool((flat[n:] == 7.0).all()), "memory behind the output was written"
    return flat[:n].view(shape), untouched


def operand(fmt, x, scope="row"):
    """(q, s, t) of BF16 x as the package quantizes it (per row, or one FP32 scale)."""
    if fmt == "bf16":
        return x, None, None
    if fmt == "mxfp8":
        return (*mxq.quantize_mxfp8(x, True, False)[:2], None)
    if fmt == "mxfp4":
        return (*mxq.quantize_mxfp4(x, True, False)[:2], None)
    return mxq.quantize_nvfp4_per_token(x) if scope == "row" else mxq.quantize_nvfp4(x, scope="tensor")


DENSE = [("bf16", 1, 8, 8), ("bf16", 5, 16, 40), ("bf16", 127, 72, 64), ("bf16", 300, 136, 200), ("bf16", 257, 392, 512),
         ("mxfp8", 1, 8, 32), ("mxfp8", 129, 72, 96), ("mxfp8", 200, 264, 128), ("mxfp8", 130, 136, 512),
         ("mxfp8", 64, 128, 1536),
         ("nvfp4", 1, 8, 32), ("nvfp4", 129, 72, 96), ("nvfp4", 200, 264, 64), ("nvfp4", 130, 136, 256),
         ("nvfp4", 64, 128, 1280)]
# few tiles and a long K: split, in even and uneven parts, the last one short
LONG = [("bf16", 3, 24, 1032), ("bf16", 130, 72, 7168), ("bf16", 1, 8, 5128), ("mxfp8", 5, 40, 1056), ("mxfp8", 140, 136, 2048),
        ("mxfp8", 64, 256, 7168), ("mxfp8", 9, 8, 1664), ("nvfp4", 5, 40, 1056), ("nvfp4", 140, 136, 2048),
        ("nvfp4", 64, 256, 7168), ("nvfp4", 9, 8, 1664)]
# more 128 x 128 tiles than CUs, fewer 256 x 256 than 192
MANY = [(f, 1300, 1672, k) for f, k in (("bf16", 72), ("bf16", 64), ("mxfp8", 96), ("mxfp8", 128), ("mxfp8", 512), ("nvfp4", 96),
                                        ("nvfp4", 128), ("nvfp4", 256))]
# enough 256 x 256 tiles for the large tile: 11 x 19 and more
LARGE = [("bf16", 2601, 2408, 72), ("bf16", 2601, 2408, 128), ("mxfp8", 2601, 2408, 96), ("mxfp8", 2601, 2408, 128),
         ("mxfp8", 2601, 2408, 512), ("nvfp4", 2601, 2408, 96), ("nvfp4", 2601, 2408, 128), ("nvfp4", 2601, 2408, 256)]


@pytest.mark.parametrize("fmt,M,I,K", DENSE + LONG + MANY + LARGE)
def test_gemm_swiglu(fmt, M, I, K):
    g = gen(M * 7 + I + K)
    x, w = randn(g, M, K).to(BF), randn(g, 2 * I, K, scale=2.0 / K ** 0.5).to(BF)
    a, b = operand(fmt, x), operand(fmt, w, "tensor")
    h, end = guarded(M, I)
    gu, gu_end = guarded(M, 2 * I)
    mxq.gemm_swiglu(FMT[fmt], a[0], a[1], b[0], b[1], tA=a[2], tB=b[2], out=(h, gu))
    y, err = R.product(R.wide(fmt, *a), R.wide(fmt, *b))
    want, tol, gu_tol = R.gated(y, err)
    R.check(gu, y, gu_tol, "gate_up")
    R.check(h, want, tol, "h")
    end(), gu_end()
    only, none = mxq.gemm_swiglu(FMT[fmt], a[0], a[1], b[0], b[1], tA=a[2], tB=b[2])
    assert none is None and torch.equal(only, h)            # the same bits without the projections kept


def test_gemm_swiglu_nvfp4_scales_per_row_and_per_tensor():
    g = gen(3)
    x, w = randn(g, 70, 96).to(BF), randn(g, 48, 96, scale=0.2).to(BF)
    for sa, sb in (("row", "row"), ("tensor", "tensor"), ("tensor", "row")):
        a, b = operand("nvfp4", x, sa), operand("nvfp4", w, sb)
        h, gu = mxq.gemm_swiglu(B.NVFP4, a[0], a[1], b[0], b[1], tA=a[2], tB=b[2], tA_scope=sa, tB_scope=sb,
                                keep_gate_up=True)
        y, err = R.product(R.wide("nvfp4", *a), R.wide("nvfp4", *b))
        want, tol, gu_tol = R.gated(y, err)
        R.check(gu, y, gu_tol, f"gate_up {sa} {sb}")
        R.check(h, want, tol, f"h {sa} {sb}")


def test_gates_far_out_give_zeros_and_no_nan():
    """Sums from the smallest to beyond where e^-g leaves binary32, in both directions."""
    far = torch.tensor([0.0, 1e-38, -1e-38, 1e-3, -1e-3, 20.0, -20.0, 87.0, -87.0, 89.0, -89.0, 103.0, -104.0, 1e4, -1e4,
                        3e30, -3e30], device="cuda")
    M, K = far.numel(), 8
    x = torch.zeros(M, K, device="cuda")
    x[:, 0], x[:, 1] = far, 1.0
    w = torch.zeros(16, K, device="cuda")
    w[:8, 0] = 1.0                                          # every gate is the row's value
    w[8:, 1] = torch.tensor([1.0, -1.0, 0.5, 3.0, -1e-20, 1e8, 0.0, -7.0], device="cuda")
    x, w = x.to(BF), w.to(BF)
    h, gu = mxq.gemm_swiglu(B.BF16, x, None, w, None, keep_gate_up=True)
    y, err = R.product(x.double(), w.double())
    want, tol, _ = R.gated(y, err)
    R.check(h, want, tol, "h")
    # backward on FP32 projections of that range
    gate_up = y.float().contiguous()
    d, wd = randn(gen(5), M, 16).to(BF), randn(gen(6), 8, 16).to(BF)
    dgu, h2 = mxq.gemm_swiglu_backward(B.BF16, d, None, wd, None, gate_up)
    dh, derr = R.product(d.double(), wd.double())
    (dd, dtol), (hh, htol) = R.through(dh, derr, gate_up)
    R.check(dgu, dd, dtol, "d_gate_up")
    R.check(h2, hh, htol, "h")


BACK = [c for c in DENSE + LONG + LARGE if c[0] != "nvfp4"] + [("bf16", 2600, 1672, 72), ("mxfp8", 2600, 1672, 96), ("mxfp8", 2600, 1672, 512),
                                                        ("bf16", 3200, 4104, 72), ("bf16", 3200, 4104, 64),
                                                        ("mxfp8", 3200, 4104, 512)]


@pytest.mark.parametrize("fmt,M,I,K", BACK)
@pytest.mark.parametrize("f32", [False, True])
def test_gemm_swiglu_backward(fmt, M, I, K, f32):
    g = gen(M * 5 + I + K)
    d, wdT = randn(g, M, K, scale=1e-3).to(BF), randn(g, I, K, scale=1.0 / K ** 0.5).to(BF)
    gate_up = randn(g, M, 2 * I, scale=2.0).to(torch.float32 if f32 else BF)
    a, b = operand(fmt, d), operand(fmt, wdT)
    dgu, end = guarded(M, 2 * I)
    h, h_end = guarded(M, I)
    mxq.gemm_swiglu_backward(FMT[fmt], a[0], a[1], b[0], b[1], gate_up, out=(dgu, h))
    dh, err = R.product(R.wide(fmt, *a), R.wide(fmt, *b))
    (want, tol), (hw, htol) = R.through(dh, err, gate_up)
    R.check(dgu, want, tol, "d_gate_up")
    R.check(h, hw, htol, "h")
    end(), h_end()
    only, none = mxq.gemm_swiglu_backward(FMT[fmt], a[0], a[1], b[0], b[1], gate_up, keep_h=False)
    assert none is None and torch.equal(only, dgu)


def test_backward_is_the_slope_of_the_forward():
    """d_gate_up against central differences in FP64 of <d, block output> along the projections."""
    g = gen(11)
    M, I, H = 6, 24, 40
    gate_up, wd, d = randn(g, M, 2 * I).to(BF), randn(g, H, I, scale=0.2).to(BF), randn(g, M, H).to(BF)
    dgu, _ = mxq.gemm_swiglu_backward(B.BF16, d, None, wd.T.contiguous(), None, gate_up)

    def value(y):
        gg, u = y.chunk(2, -1)
        return (((gg * torch.sigmoid(gg) * u) @ wd.double().T) * d.double()).sum()

    eps = 1e-4                                              # differences: an error of eps^2 f''' / 6, and rounding
    y0 = gate_up.double()
    for m, c in ((0, 0), (1, 5), (2, I - 1), (3, I), (4, I + 7), (5, 2 * I - 1)):
        step = torch.zeros_like(y0)
        step[m, c] = eps
        slope = (value(y0 + step) - value(y0 - step)) / (2 * eps)
        got = dgu[m, c].double()
        assert abs(got - slope) <= (R.BF16 + 1e-4) * abs(slope) + 1e-6, (m, c, got.item(), slope.item())


# ---------------------------------------------------------------------------- per expert

def slots(counts, pads, tokens, seed):
    """offsets and row_index of experts with `counts` rows and `pads` padding slots behind them."""
    off, rows = [0], []
    g = torch.Generator().manual_seed(seed)
    for n, p in zip(counts, pads):
        rows += torch.randint(0, tokens, (n,), generator=g).tolist() + [-1] * p
        off.append(off[-1] + n + p)
    return torch.tensor(off, device="cuda"), torch.tensor(rows, dtype=torch.int32, device="cuda")


EXPERTS = [([3, 0, 1, 130, 0, 40, 0], [0, 0, 2, 5, 3, 0, 0]), ([1], [0]), ([0, 700, 520, 385], [0, 4, 0, 7])]
# experts that fill 256-row tiles, and enough of those
TALL = [([0, 1800, 1100, 1500], [0, 8, 0, 5])]


@pytest.mark.parametrize("counts,pads", EXPERTS)
@pytest.mark.parametrize("fmt,I,K", [("bf16", 24, 40), ("bf16", 136, 128), ("nvfp4", 16, 32), ("nvfp4", 72, 64),
                                     ("nvfp4", 136, 256)])
def test_grouped_gemm_swiglu(fmt, I, K, counts, pads):
    G, T = len(counts), 150
    g = gen(sum(counts) + I + K)
    off, row = slots(counts, pads, T, 1)
    total = row.numel()
    x, w = randn(g, T, K).to(BF), randn(g, G * 2 * I, K, scale=2.0 / K ** 0.5).to(BF)
    a = operand(fmt, x)
    b = (w, None, None) if fmt == "bf16" else mxq.quantize_nvfp4(w, scope="group", group_rows=2 * I)
    h, end = guarded(total, I)
    gu, gu_end = guarded(total, 2 * I)
    mxq.grouped_gemm_swiglu(FMT[fmt], off, a[0], b[0], inter=I, K=K, sA=a[1], sB=b[1], tA=a[2], tB=b[2], a_row_index=row,
                            total=total, out=(h, gu))
    xs = torch.where((row >= 0)[:, None], R.wide(fmt, *a)[row.long().clamp(min=0)], 0.0)
    ws = R.wide(fmt, b[0], b[1], None if b[2] is None else b[2].repeat_interleave(2 * I)).view(G, 2 * I, K)
    for e in range(G):
        at = slice(int(off[e]), int(off[e + 1]))
        y, err = R.product(xs[at], ws[e])
        want, tol, gu_tol = R.gated(y, err)
        R.check(gu[at], y, gu_tol, f"gate_up of expert {e}")
        R.check(h[at], want, tol, f"h of expert {e}")
    end(), gu_end()
    assert not bool(h[row < 0].any()) and not bool(gu[row < 0].any())


@pytest.mark.parametrize("counts,pads", EXPERTS)
@pytest.mark.parametrize("fmt,I,K", [("bf16", 24, 40), ("bf16", 136, 128), ("nvfp4", 16, 32), ("nvfp4", 272, 72)])
@pytest.mark.parametrize("f32", [False, True])
def test_grouped_gemm_swiglu_backward(fmt, I, K, counts, pads, f32):
    G = len(counts)
    g = gen(sum(counts) * 3 + I + K)
    off, row = slots(counts, pads, 150, 2)
    total, live = row.numel(), (row >= 0)[:, None]
    d = (randn(g, total, K, scale=1e-3) * live).to(BF)
    gate_up = (randn(g, total, 2 * I, scale=2.0) * live).to(torch.float32 if f32 else BF)
    wd = randn(g, G * K, I, scale=0.1).to(BF)               # (K, inter) an expert, as the forward has it
    dgu, end = guarded(total, 2 * I)
    h, h_end = guarded(total, I)
    if fmt == "bf16":
        wT = wd.view(G, K, I).transpose(1, 2).contiguous().view(G * I, K)
        mxq.grouped_gemm_swiglu_backward(B.BF16, off, d, wT, inter=I, K=K, gate_up=gate_up, total=total, out=(dgu, h))
        ws = wd.double().view(G, K, I)
    else:
        q, s, t = mxq.quantize_nvfp4(wd, scope="group", group_rows=K)
        mxq.grouped_gemm_swiglu_backward(B.BF16_NVFP4T, off, d, q, inter=I, K=K, gate_up=gate_up, sB=s, tB=t, total=total,
                                         out=(dgu, h))
        ws = mxq.dequantize(B.NVFP4, q, s, t, t_scope="group", group_rows=K).double().view(G, K, I)
    for e in range(G):
        at = slice(int(off[e]), int(off[e + 1]))
        dh, err = R.product(d[at].double(), ws[e].T)
        (want, tol), (hw, htol) = R.through(dh, err, gate_up[at])
        R.check(dgu[at], want, tol, f"d_gate_up of expert {e}")
        R.check(h[at], hw, htol, f"h of expert {e}")
    end(), h_end()
    assert not bool(dgu[row < 0].any()) and not bool(h[row < 0].any())


@pytest.mark.parametrize("fmt", ["bf16", "nvfp4"])
@pytest.mark.parametrize("f32", [False, True])
def test_grouped_gemm_swiglu_backward_of_tall_experts(fmt, f32):
    test_grouped_gemm_swiglu_backward(fmt, 3088, 72, *TALL[0], f32)


@pytest.mark.parametrize("tA_scope", ["row", "tensor"])
def test_grouped_gemm_swiglu_with_a_scale_a_weight_row(tA_scope):
    G, T, I, K = 3, 60, 72, 96
    g = gen(12)
    off, row = slots([20, 0, 37], [0, 3, 0], T, 3)
    x, w = randn(g, T, K).to(BF), randn(g, G * 2 * I, K, scale=0.2).to(BF)
    a, b = operand("nvfp4", x, tA_scope), mxq.quantize_nvfp4_per_token(w)
    h, gu = mxq.grouped_gemm_swiglu(B.NVFP4, off, a[0], b[0], inter=I, K=K, sA=a[1], sB=b[1], tA=a[2], tB=b[2],
                                    tA_scope=tA_scope, tB_scope="row", a_row_index=row, total=60, keep_gate_up=True)
    xs = torch.where((row >= 0)[:, None], R.wide("nvfp4", *a)[row.long().clamp(min=0)], 0.0)
    ws = R.wide("nvfp4", *b).view(G, 2 * I, K)
    for e in range(G):
        at = slice(int(off[e]), int(off[e + 1]))
        y, err = R.product(xs[at], ws[e])
        want, tol, gu_tol = R.gated(y, err)
        R.check(gu[at], y, gu_tol, f"gate_up of expert {e}")
        R.check(h[at], want, tol, f"h of expert {e}")


@pytest.mark.parametrize("groups", [5, 64, 65, 255, 256, 257, 400])
def test_many_groups(groups):
    """Around the number of groups that a kernel looks through by itself; some empty, one of several tiles."""
    g = torch.Generator().manual_seed(groups)
    counts = torch.randint(0, 5, (groups,), generator=g).tolist()
    counts[groups // 3] = 150
    counts[-1] = groups % 2 * 3                             # the last one empty, or not
    test_grouped_gemm_swiglu("bf16", 136, 40, counts, [0] * groups)
    test_grouped_gemm_swiglu("nvfp4", 16, 32, counts, [0] * groups)
    test_grouped_gemm_swiglu_backward("nvfp4", 272, 40, counts, [0] * groups, True)


@pytest.mark.parametrize("groups", [2, 300])
def test_rejected_offsets_leave_the_outputs_unwritten(groups):
    g = gen(8)
    x, w = randn(g, 64, 64).to(BF), randn(g, groups * 32, 64).to(BF)
    for off in ([0, 40, 60], [0, 70, 64], [1, 30, 64], [0, -8, 64]):
        h = torch.full((64, 16), 5.0, dtype=BF, device="cuda")
        offsets = torch.tensor(off[:2] + off[2:] * (groups - 1), device="cuda")
        mxq.grouped_gemm_swiglu(B.BF16, offsets, x, w.view(groups, 32, 64), inter=16, K=64, total=64, out=(h, None))
        assert bool((h == 5.0).all()), off


# ---------------------------------------------------------------------------- matrix-vector products

GEMV = [(1, 1, 32), (1, 16, 128), (2, 40, 96), (3, 17, 160), (16, 100, 512), (17, 33, 1056), (32, 64, 2048), (33, 24, 64),
        (64, 200, 640), (1, 48, 7168)]


def weights4(fmt, w, groups=1):
    """(q, s, t) of stacked BF16 weights, one FP32 scale a group."""
    if fmt == "mxfp4":
        return operand("mxfp4", w)
    return mxq.quantize_nvfp4(w, scope="group", group_rows=w.shape[0] // groups)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("rows,N,K", GEMV)
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_gemv_block_scaled(fmt, rows, N, K, dtype):
    g = gen(rows + N + K)
    x, w = randn(g, rows, K).to(BF), randn(g, N, K, scale=0.1).to(BF)
    q, s, t = operand(fmt, w, "tensor")
    y, end = guarded(rows, N, dtype=dtype)
    mxq.gemv_block_scaled(FMT[fmt], x, q, s, t, out=y)
    want, err = R.product(x.double(), R.wide(fmt, q, s, t))
    tol = err + 2 * R.F32 * want.abs() + (R.half_step(want) if dtype == BF else 0.0)
    R.check(y, want, (1 + R.BF16) * tol, "y")
    end()
    assert torch.equal(mxq.gemv_block_scaled(FMT[fmt], x, q, s, t, out_dtype=dtype), y)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("rows,I,K", GEMV)
def test_gemv_swiglu(fmt, rows, I, K):
    g = gen(rows + 2 * I + K)
    x, w = randn(g, rows, K).to(BF), randn(g, 2 * I, K, scale=2.0 / K ** 0.5).to(BF)
    q, s, t = operand(fmt, w, "tensor")
    h, end = guarded(rows, I)
    mxq.gemv_swiglu(FMT[fmt], x, q, s, t, out=h)
    y, err = R.product(x.double(), R.wide(fmt, q, s, t))
    want, tol, _ = R.gated(y, err + 2 * R.F32 * y.abs())
    R.check(h, want, tol, "h")
    end()


def test_gemv_strided_rows_row_scales_and_strange_rows():
    """x and y inside wider buffers; one FP32 scale a weight row; Inf and NaN in a row of x stay in it."""
    g = gen(4)
    rows, N, K = 7, 50, 224
    big = randn(g, rows, K + 40).to(BF)
    big[:, K:] = float("nan")                               # beside the rows: never read
    x = big[:, :K]
    x[2, 5], x[4, 100] = float("inf"), float("nan")
    w = randn(g, N, K, scale=0.1).to(BF)
    q, s, t = mxq.quantize_nvfp4_per_token(w)
    out = torch.full((rows, N + 6), 7.0, device="cuda")
    mxq.gemv_block_scaled(B.NVFP4, x, q, s, t, t_scope="row", out=out[:, :N])
    assert bool((out[:, N:] == 7.0).all())
    fine = torch.tensor([0, 1, 3, 5, 6], device="cuda")
    want, err = R.product(x[fine].double(), R.wide("nvfp4", q, s, t))
    R.check(out[fine, :N], want, err + 3 * R.F32 * want.abs(), "y")
    assert not bool(torch.isfinite(out[4, :N]).any())
    hit = R.wide("nvfp4", q, s)[:, 5] != 0
    assert not bool(torch.isfinite(out[2, :N][hit]).any())


DECODE = [(1, 1, 4, 16, 32), (1, 8, 64, 40, 256), (3, 2, 5, 24, 96), (17, 8, 16, 72, 160), (33, 4, 40, 16, 128),
          (64, 6, 9, 33, 64), (64, 32, 32, 16, 32), (2, 3, 1024, 8, 32), (5, 2, 1, 20, 64),
          (64, 8, 96, 16, 160), (64, 16, 200, 24, 64), (21, 2, 4, 16424, 160)]   # 512 and 1024 choices, many tiles


def choices(T, k, E, seed, dead):
    g = torch.Generator().manual_seed(seed)
    idx = torch.stack([torch.randperm(max(E, k), generator=g)[:k] % E for _ in range(T)]).to(torch.int32)
    w = torch.rand((T, k), generator=g) + 0.1
    if dead:
        off = torch.rand((T, k), generator=g) < 0.3
        off[T // 2] = True                                  # a token without any
        idx[off] = torch.where(torch.rand(int(off.sum()), generator=g) < 0.5, -1, E + 3).to(torch.int32)
        w[off] = float("nan")                               # not read
    return idx.cuda(), w.cuda()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,k,E,I,K", DECODE)
@pytest.mark.parametrize("dead", [False, True])
def test_moe_decode_gate_up(fmt, T, k, E, I, K, dead):
    g = gen(T + k + E + I + K)
    x, w = randn(g, T, K).to(BF), randn(g, E * 2 * I, K, scale=2.0 / K ** 0.5).to(BF)
    q, s, t = weights4(fmt, w, E)
    idx, _ = choices(T, k, E, T + k, dead)
    h, end = guarded(T, k, I)
    mxq.moe_decode_gate_up(FMT[fmt], x, idx, q, s, t, experts=E, out=h)
    ws = R.wide(fmt, q, s, None if t is None else t.repeat_interleave(2 * I)).view(E, 2 * I, K)
    live = (idx >= 0) & (idx < E)
    e = torch.where(live, idx, 0).long()
    y, err = R.product(x.double(), ws.view(E * 2 * I, K))
    pick = lambda v: v.view(T, E, 2 * I).gather(1, e[:, :, None].expand(T, k, 2 * I))
    y = pick(y)
    want, tol, _ = R.gated(y, pick(err) + 2 * R.F32 * y.abs())
    R.check(h, want * live[:, :, None], tol, "h")
    assert not bool(h[~live].any())
    end()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,k,E,N,K", DECODE)
@pytest.mark.parametrize("dead", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_moe_decode_down(fmt, T, k, E, N, K, dead, dtype):
    g = gen(T + k + E + N + K + 1)
    h, w = randn(g, T, k, K).to(BF), randn(g, E * N, K, scale=0.1).to(BF)
    q, s, t = weights4(fmt, w, E)
    idx, weights = choices(T, k, E, T + k + 1, dead)
    live = (idx >= 0) & (idx < E)
    h[~live] = float("nan")                                 # not read
    y, end = guarded(T, N, dtype=dtype)
    mxq.moe_decode_down(FMT[fmt], h, idx, weights, q, s, t, experts=E, out=y)
    ws = R.wide(fmt, q, s, None if t is None else t.repeat_interleave(N)).view(E, N, K)
    want = torch.zeros((T, N), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(want)
    for c in live.nonzero().tolist():
        o, err = R.product(h[c[0], c[1]].double()[None], ws[int(idx[c[0], c[1]])])
        wt = weights[c[0], c[1]].double()
        want[c[0]] += wt * o[0]
        tol[c[0]] += wt * (err[0] + (k + 20) * R.F32 * (h[c[0], c[1]].double().abs()[None] @ ws[int(idx[c[0], c[1]])].abs().T)[0])
    R.check(y, want, (1 + R.BF16) * tol + (R.half_step(want) if dtype == BF else 0.0), "y")
    end()
    assert torch.equal(mxq.moe_decode_down(FMT[fmt], h, idx, weights, q, s, t, experts=E, out_dtype=dtype), y)


@pytest.mark.parametrize("T,k,E", [(3, 2, 5), (30, 3, 4)])
def test_decoding_with_a_scale_a_weight_row(T, k, E):
    """One FP32 scale a weight row, four choices at a time and 32; gemv_swiglu likewise. x inside a wider buffer."""
    I, H = 40, 96
    g = gen(T)
    x, idx = randn(g, T, H + 8).to(BF)[:, :H], choices(T, k, E, 5, False)[0]
    gu, d = (mxq.quantize_nvfp4_per_token(randn(g, E * n, c, scale=0.2).to(BF)) for n, c in ((2 * I, H), (H, I + 24)))
    e = idx.long()
    wide = R.wide("nvfp4", *gu).view(E, 2 * I, H)[e]
    y = (wide @ x.double()[:, None, :, None]).squeeze(-1)
    err = (R.SUM * H + 2 * R.F32) * (wide.abs() @ x.double().abs()[:, None, :, None]).squeeze(-1)
    want, tol, _ = R.gated(y, err)
    R.check(mxq.moe_decode_gate_up(B.NVFP4, x, idx, *gu, experts=E, t_scope="row"), want, tol, "h")
    h, weights = randn(g, T, k, I + 24).to(BF), torch.rand((T, k), generator=g, device="cuda")
    wide = R.wide("nvfp4", *d).view(E, H, I + 24)[e] * weights.double()[..., None, None]
    want = (wide @ h.double()[..., None]).squeeze(-1).sum(1)
    size = (wide.abs() @ h.double().abs()[..., None]).squeeze(-1).sum(1)
    got = mxq.moe_decode_down(B.NVFP4, h, idx, weights, *d, experts=E, t_scope="row")
    R.check(got, want, (R.SUM * (I + 24) + (k + 4) * R.F32) * size, "y")
    one = tuple(v[:2 * I] for v in gu)
    y, err = R.product(x.double(), R.wide("nvfp4", *one))
    want, tol, _ = R.gated(y, err + 2 * R.F32 * y.abs())
    R.check(mxq.gemv_swiglu(B.NVFP4, x, *one, t_scope="row"), want, tol, "gemv_swiglu")


def test_a_token_that_names_an_expert_twice():
    g = gen(9)
    T, k, E, I, H = 20, 4, 3, 24, 64
    x = randn(g, T, H).to(BF)
    idx = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    weights = torch.rand((T, k), generator=g, device="cuda")
    gu, d = weights4("nvfp4", randn(g, E * 2 * I, H, scale=0.2).to(BF), E), weights4("mxfp4", randn(g, E * H, 32).to(BF), E)
    h = mxq.moe_decode_gate_up(B.NVFP4, x, idx, *gu, experts=E)
    for t in range(T):
        for j in range(k):
            first = int((idx[t] == idx[t, j]).nonzero()[0])
            assert torch.equal(h[t, j], h[t, first])
    h = randn(g, T, k, 32).to(BF)
    y = mxq.moe_decode_down(B.MXFP4, h, idx, weights, *d, experts=E)
    ws = R.wide("mxfp4", d[0], d[1]).view(E, H, 32)
    o = (ws[idx.long()] @ h.double()[..., None]).squeeze(-1) * weights.double()[..., None]
    size = (ws[idx.long()].abs() @ h.double().abs()[..., None]).squeeze(-1) * weights.double()[..., None]
    R.check(y, o.sum(1), 200 * R.F32 * size.sum(1), "y")


def test_calls_on_another_stream_and_in_a_graph():
    """Every call captured once and replayed with new data, eager work in between; the eager calls run on
    another stream."""
    g = gen(21)
    T, I, H, E, k = 6, 64, 128, 8, 2
    gu, d = weights4("nvfp4", randn(g, E * 2 * I, H, scale=0.1).to(BF), E), weights4("nvfp4", randn(g, E * H, I, scale=0.1).to(BF), E)
    one = weights4("nvfp4", randn(g, 2 * I, H, scale=0.1).to(BF))
    wgu, wdT = randn(g, 2 * I, H, scale=0.1).to(BF), randn(g, I, H, scale=0.1).to(BF)
    x, dy = torch.empty(T, H, dtype=BF, device="cuda"), torch.empty(T, H, dtype=BF, device="cuda")
    idx = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    wt = torch.full((T, k), 0.5, device="cuda")
    off = torch.tensor([0, 1, 1, T], device="cuda")
    wgu3, wd3 = randn(g, 3 * 2 * I, H, scale=0.1).to(BF), weights4("nvfp4", randn(g, 3 * H, I, scale=0.1).to(BF), 3)

    def step():
        h, y = mxq.gemm_swiglu(B.BF16, x, None, wgu, None, keep_gate_up=True)
        dgu, h2 = mxq.gemm_swiglu_backward(B.BF16, dy, None, wdT, None, y)
        hg, yg = mxq.grouped_gemm_swiglu(B.BF16, off, x, wgu3, inter=I, K=H, total=T, keep_gate_up=True)
        dg, h3 = mxq.grouped_gemm_swiglu_backward(B.BF16_NVFP4T, off, dy, wd3[0], inter=I, K=H, gate_up=yg, sB=wd3[1],
                                                  tB=wd3[2], total=T)
        hd = mxq.moe_decode_gate_up(B.NVFP4, x, idx, *gu, experts=E)
        return [h, y, dgu, h2, hg, yg, dg, h3, hd, mxq.moe_decode_down(B.NVFP4, hd, idx, wt, *d, experts=E),
                mxq.gemv_swiglu(B.NVFP4, x, *one), mxq.gemv_block_scaled(B.NVFP4, x, *one)]

    def feed(seed):
        q = gen(seed)
        x.copy_(randn(q, T, H))
        dy.copy_(randn(q, T, H))
        idx.copy_(torch.randint(-1, E, (T, k), generator=q, device="cuda"))

    feed(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (1, 2, 3):
        feed(seed)
        graph.replay()
        torch.cuda.synchronize()
        replayed = [v.clone() for v in got]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            eager = step()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(replayed, eager)):
            assert torch.equal(a, b), (seed, i)


def two_calls(seed):
    """Two calls that need a workspace, and one that does not: a function of their inputs."""
    g = gen(seed)
    T, k, E, I, H = 9, 4, 6, 96, 512
    d = weights4("nvfp4", randn(g, E * H, I, scale=0.1).to(BF), E)
    idx, wt = choices(T, k, E, seed, False)
    h, x, wgu = randn(g, T, k, I).to(BF), randn(g, T, 7168).to(BF), randn(g, 48, 7168, scale=0.02).to(BF)
    one = weights4("mxfp4", randn(g, 304, k * I, scale=0.1).to(BF))

    def call():
        return (mxq.moe_decode_down(B.NVFP4, h, idx, wt, *d, experts=E), mxq.gemm_swiglu(B.BF16, x, None, wgu, None)[0],
                mxq.gemv_block_scaled(B.MXFP4, h.view(T, k * I), *one))
    return call, (h, x, wt)


def test_two_streams_at_once():
    calls = [two_calls(31)[0], two_calls(32)[0]]
    want = [c() for c in calls]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i].append(calls[i]())
    torch.cuda.synchronize()
    for i in (0, 1):
        for out in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(out, want[i]))


def test_two_graphs_and_eager_calls_between_them():
    calls, inputs = zip(two_calls(41), two_calls(42))
    for c in calls:
        c()
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for c, gr in zip(calls, graphs):
        with torch.cuda.graph(gr):
            outs.append(c())
    for turn in range(3):
        for t in inputs:
            for v in t:
                v.mul_(0.5 if turn % 2 else -2.0)
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        replayed = [[v.clone() for v in o] for o in outs]
        for c, o in zip(calls, replayed):
            assert all(torch.equal(a, b) for a, b in zip(c(), o)), turn


@pytest.mark.parametrize("rows", [1, 5, 40])
def test_gemv_with_a_long_k(rows):
    g = gen(rows)
    N, K = 24, 1 << 20
    x, t = randn(g, rows, K).to(BF), torch.full((1,), 2.0 ** -10, device="cuda")
    q = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.randint(0x28, 0x40, (N, K // 16), generator=g, device="cuda", dtype=torch.uint8)
    want, err = R.product(x.double(), R.wide("nvfp4", q, s, t))
    R.check(mxq.gemv_block_scaled(B.NVFP4, x, q, s, t), want, err + 2 * R.F32 * want.abs(), "y")


@pytest.mark.parametrize("rows", [2, 16, 40])
def test_gemv_with_weights_past_32_bits(rows):
    """2.2 GB of weights: the last rows lie past 2^31 bytes."""
    g = gen(rows)
    N, K = 66003, 65536
    x = randn(g, rows, K).to(BF)
    q = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.randint(110, 118, (N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    assert q.numel() > 2 ** 31
    y = mxq.gemv_block_scaled(B.MXFP4, x, q, s)
    for rows_of in (slice(0, 40), slice(N - 700, N)):
        want, err = R.product(x.double(), R.wide("mxfp4", q[rows_of], s[rows_of]))
        R.check(y[:, rows_of], want, err, "y")


def test_gated_outputs_past_32_bits():
    """(g | u) and its gradient of 2.2 GB."""
    g = gen(5)
    M, I, K = 270_000, 2048, 16
    x, w = randn(g, M, K).to(BF), randn(g, 2 * I, K, scale=0.5).to(BF)
    h, gu = mxq.gemm_swiglu(B.BF16, x, None, w, None, keep_gate_up=True)
    assert gu.numel() * 2 > 2 ** 31
    dy, wT = randn(g, M, K).to(BF), randn(g, I, K, scale=0.5).to(BF)
    dgu, h2 = mxq.gemm_swiglu_backward(B.BF16, dy, None, wT, None, gu)
    for at in (slice(0, 64), slice(M - 200, M)):
        y, err = R.product(x[at].double(), w.double())
        want, tol, gu_tol = R.gated(y, err)
        R.check(gu[at], y, gu_tol, "gate_up")
        R.check(h[at], want, tol, "h")
        (dg, dtol), (hb, htol) = R.through(*R.product(dy[at].double(), wT.double()), gu[at])
        R.check(dgu[at], dg, dtol, "d_gate_up")
        if h2 is not None:
            R.check(h2[at], hb, htol, "h made again")


def test_empty_calls():
    e = lambda *s, dt=BF: torch.empty(s, dtype=dt, device="cuda")
    h, gu = mxq.gemm_swiglu(B.BF16, e(0, 64), None, e(32, 64), None, keep_gate_up=True)
    assert h.shape == (0, 16) and gu.shape == (0, 32)
    dgu, _ = mxq.gemm_swiglu_backward(B.BF16, e(0, 64), None, e(16, 64), None, e(0, 32))
    assert dgu.shape == (0, 32)
    q, s, t = weights4("nvfp4", randn(gen(1), 32, 64).to(BF))
    assert mxq.gemv_block_scaled(B.NVFP4, e(0, 64), q, s, t).shape == (0, 32)
    assert mxq.gemv_swiglu(B.NVFP4, e(0, 64), q, s, t).shape == (0, 16)
    i0, w0 = e(0, 2, dt=torch.int32), e(0, 2, dt=torch.float32)
    assert mxq.moe_decode_gate_up(B.NVFP4, e(0, 64), i0, q, s, t, experts=1).shape == (0, 2, 16)
    assert mxq.moe_decode_down(B.NVFP4, e(0, 2, 64), i0, w0, q, s, t, experts=1).shape == (0, 32)
    off = torch.zeros(3, dtype=torch.int64, device="cuda")
    h, _ = mxq.grouped_gemm_swiglu(B.BF16, off, e(0, 64), e(2 * 32, 64), inter=16, K=64, total=0)
    assert h.shape == (0, 16)
    # K = 0: sums of nothing
    z, _ = mxq.grouped_gemm_swiglu(B.BF16, torch.tensor([0, 4], device="cuda"), randn(gen(2), 4, 8).to(BF),
                                   torch.zeros(32, 8, dtype=BF, device="cuda"), inter=16, K=8, total=4)
    assert not bool(z.any())
