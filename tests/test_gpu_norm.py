"""GPU parity of the norms around a block: the quantizing norm bit for bit against the oracle,
the others against FP64 within bounds that count roundings (u = 2^-24, one per binary32
operation; a BF16 result adds 2^-8 of itself)."""

import numpy as np
import pytest
import torch

from microscaling_precision_quantization_amd import binding as B
from microscaling_precision_quantization_amd import inputs
from oracle import mxfp4, mxfp8, norm, nvfp4
from tests.gpu_util import assert_bytes_equal, dev, dev_bf16, host

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF16 = 2.0 ** -8
EPS = 1e-6


def _values(seed, rows, cols, dtype, scale=1.0):
    """Hidden states of different magnitude per row; (device tensor, FP32 values)."""
    g = inputs.rng(300, seed)
    v = (g.standard_normal((rows, cols)) * g.lognormal(0, 1, (rows, 1)) * scale).astype(np.float32)
    if dtype == "f32":
        return dev(v), v
    bits = inputs.to_bf16_bits(v)
    return dev_bf16(bits), inputs.bf16_bits_to_float(bits)


def _weight(seed, cols):
    return (1 + 0.2 * inputs.rng(301, seed).standard_normal(cols)).astype(np.float32)


def _check_quantized(fmt, n_bits, q, s, t, what):
    if fmt == B.BF16:
        assert q is None and s is None and t is None
        return
    if fmt == B.NVFP4:
        eq, es, et = nvfp4.quantize_per_token(n_bits)
        assert_bytes_equal(host(t).view(np.uint32), et.view(np.uint32), f"{what}: t")
    else:
        assert t is None
        eq, es = (mxfp8 if fmt == B.MXFP8 else mxfp4).quantize_rowwise(n_bits)
    assert_bytes_equal(host(s), es, f"{what}: scales")
    assert_bytes_equal(host(q), eq, f"{what}: elements")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", [B.MXFP8, B.NVFP4, B.MXFP4, B.BF16])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (5, 512), (2, 2048), (7, 2080), (3, 4128), (2, 7168),
                                       (1, 8224), (2, 16384)])
def test_norm_quantize_is_bit_exact(rows, cols, fmt, dtype):
    x, xv = _values(cols, rows, cols, dtype)
    w = _weight(cols, cols)
    exp = norm.rmsnorm_bf16(xv, w, EPS)
    n, q, s, t, rstd = B.rmsnorm_quantize(x, dev(w), eps=EPS, fmt=fmt)
    assert_bytes_equal(host(n), exp, "n")
    _check_quantized(fmt, exp, q, s, t, f"{rows}x{cols}")
    assert_bytes_equal(host(rstd), norm.rstd(xv, EPS).astype(np.float32), "rstd")
    n2, q2, s2, t2, _ = B.rmsnorm_quantize(x, dev(w), eps=EPS, fmt=fmt, keep_n=False)
    assert (n2 is None) == (fmt != B.BF16)
    _check_quantized(fmt, exp, q2, s2, t2, f"{rows}x{cols} without n")


@pytest.mark.parametrize("cols,fmt", [(8, B.BF16), (40, B.BF16), (16, B.NVFP4), (48, B.NVFP4), (2064, B.NVFP4)])
def test_norm_quantize_narrow_and_odd_widths(cols, fmt):
    x, xv = _values(cols, 67, cols, "bf16")
    exp = norm.rmsnorm_bf16(xv, None, EPS)
    n, q, s, t, _ = B.rmsnorm_quantize(x, fmt=fmt, eps=EPS)
    assert_bytes_equal(host(n), exp, "n")
    _check_quantized(fmt, exp, q, s, t, str(cols))


@pytest.mark.parametrize("rows", [1, 255, 256, 1025, 4099])
def test_norm_quantize_many_rows(rows):
    """More rows than workgroups in flight; every row against the oracle."""
    x, xv = _values(rows, rows, 160, "bf16")
    w = _weight(0, 160)
    exp = norm.rmsnorm_bf16(xv, w, EPS)
    n, q, s, t, _ = B.rmsnorm_quantize(x, dev(w), eps=EPS, fmt=B.NVFP4)
    assert_bytes_equal(host(n), exp, "n")
    _check_quantized(B.NVFP4, exp, q, s, t, str(rows))


def test_norm_quantize_special_rows_strides_and_preallocated_outputs():
    """Zero rows, one large value, tiny and huge magnitudes, rows of a wider tensor; the bytes
    around the preallocated outputs stay as they were."""
    g = inputs.rng(302, 0)
    v = g.standard_normal((9, 64)).astype(np.float32)
    v[0] = 0.0
    v[1] = 0.0
    v[1, 5] = -3e38
    v[2] *= 1e-30
    v[3] *= 1e37
    v[4] = 2.0
    v[5, 1::2] = -0.0
    bits = inputs.to_bf16_bits(v)
    wide = torch.full((9, 200), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 64:128] = dev_bf16(bits)
    x = wide[:, 64:128]
    exp = norm.rmsnorm_bf16(inputs.bf16_bits_to_float(bits), None, EPS)
    for fmt in (B.MXFP8, B.MXFP4, B.NVFP4, B.BF16):
        per = 2 if fmt in (B.MXFP4, B.NVFP4) else 1
        blk = 16 if fmt == B.NVFP4 else 32
        guard = lambda r, c, dt: torch.full((r + 2, c), 85, dtype=dt, device="cuda")
        bn, bq, bs = guard(9, 64, torch.bfloat16), guard(9, 64 // per, torch.uint8), guard(9, 64 // blk, torch.uint8)
        bt, br = torch.full((11,), 85.0, device="cuda"), torch.full((11,), 85.0, device="cuda")
        has = fmt != B.BF16
        out = (bn[1:-1], bq[1:-1] if has else None, bs[1:-1] if has else None, bt[1:-1] if fmt == B.NVFP4 else None,
               br[1:-1])
        n, q, s, t, rstd = B.rmsnorm_quantize(x, eps=EPS, fmt=fmt, out=out)
        assert_bytes_equal(host(n), exp, "n")
        _check_quantized(fmt, exp, q, s, t, "special rows")
        assert_bytes_equal(host(rstd), norm.rstd(inputs.bf16_bits_to_float(bits), EPS).astype(np.float32), "rstd")
        for b in (bn, bq, bs, bt, br):
            assert bool((b[0] == 85).all()) and bool((b[-1] == 85).all())


def test_norm_quantize_outside_the_binary32_range():
    """Weights and rows at which binary32 products would leave the normal range, and weights that
    put many values next to BF16 rounding midpoints: still the correctly rounded values."""
    g = inputs.rng(304, 0)
    v = g.standard_normal((6, 512)).astype(np.float32)
    v[0] *= 2.0 ** -120
    v[1] *= 2.0 ** 115
    v[2, ::2] *= 2.0 ** -110
    v[3] = np.sign(v[3])                                     # r = 1 / sqrt(1 + eps)
    bits = inputs.to_bf16_bits(v)
    xv = inputs.bf16_bits_to_float(bits)
    for n, w in enumerate([np.ones(512), np.full(512, 2.0 ** 60), np.full(512, 2.0 ** -90),
                           1 + np.arange(512) / 256 + 2.0 ** -8,
                           np.where(np.arange(512) % 3, 1.0, 2.0 ** 30)]):
        w = w.astype(np.float32)
        for eps in (EPS, 1e-30):
            got = B.rmsnorm_quantize(dev_bf16(bits), dev(w), eps=eps, fmt=B.BF16)[0]
            with np.errstate(over="ignore"):
                assert_bytes_equal(host(got), norm.rmsnorm_bf16(xv, w, eps), f"weights {n}, eps {eps}")


def test_norm_quantize_equals_the_row_quantizers():
    x, _ = _values(9, 130, 512, "bf16")
    w = dev(_weight(9, 512))
    n, q, s, t, _ = B.rmsnorm_quantize(x, w, fmt=B.NVFP4)
    for a, b in zip((q, s, t), B.quantize_nvfp4_per_token(n)):
        assert torch.equal(a, b)
    _, q, s, _, _ = B.rmsnorm_quantize(x, w, fmt=B.MXFP8)
    assert torch.equal(q, B.quantize_mxfp8(n, colwise=False)[0]) and torch.equal(s, B.quantize_mxfp8(n, colwise=False)[1])
    _, q, s, _, _ = B.rmsnorm_quantize(x, w, fmt=B.MXFP4)
    assert torch.equal(q, B.quantize_mxfp4(n, colwise=False)[0]) and torch.equal(s, B.quantize_mxfp4(n, colwise=False)[1])


def _dx_bound(g, xh, r, extra, bf16, ref):
    """|dx - exact|: m = mean(g xh) is a sum of H products in at most 64 sequential steps, 8
    exchanges and 3 joins (76 u of the sum of magnitudes, with the roundings of g and xh); each
    of g, xh m, their difference and the product with r adds a few u."""
    m = np.mean(g * xh, axis=1, keepdims=True)
    mag = np.mean(np.abs(g * xh), axis=1, keepdims=True)
    b = np.abs(r) * (np.abs(xh) * 84 * U * mag + 8 * U * (np.abs(g) + np.abs(xh * m))) + extra
    return b + (BF16 * (np.abs(ref) + b) if bf16 else U * np.abs(ref)) + 1e-44


def _dw_bound(terms, rows):
    """Column sums: at most rows/512 + 1 sequential adds in a workgroup, then 512/4 + 3, plus four
    roundings of each term."""
    return (rows / 512 + 1 + 131 + 4) * U * np.sum(np.abs(terms), axis=0) + 1e-44


@pytest.mark.parametrize("xt,dt,two,res", [("bf16", "f32", True, True), ("bf16", "bf16", False, True),
                                           ("f32", "f32", False, False), ("f32", "bf16", True, True)])
@pytest.mark.parametrize("rows,cols", [(1, 8), (5, 96), (33, 2048), (3, 2056), (513, 264), (1100, 72), (6, 7168),
                                       (2, 16384)])
def test_norm_backward(rows, cols, xt, dt, two, res):
    x, xv = _values(rows, rows, cols, xt)
    dn, dnv = _values(rows + 1, rows, cols, dt, 1e-3)
    dn2, dn2v = _values(rows + 2, rows, cols, dt, 1e-3) if two else (None, 0.0)
    dr, drv = _values(rows + 3, rows, cols, xt, 1e-3) if res else (None, 0.0)
    w = _weight(rows, cols)
    rstd = norm.rstd(xv, EPS).astype(np.float32)
    dx, dw = B.rmsnorm_backward(dn, x, dev(rstd), dev(w), dn2=dn2, d_res=dr, res_scale=0.75)
    up = dnv.astype(np.float64) + dn2v
    ref, ref_w = norm.backward(up, xv, rstd, w)
    ref = ref + 0.75 * np.asarray(drv, np.float64)
    r = rstd.astype(np.float64)[:, None]
    xh = xv * r
    got = inputs.bf16_bits_to_float(host(dx)) if xt == "bf16" else host(dx)
    err = np.abs(got - ref)
    bound = _dx_bound(up * w, xh, r, 2 * U * np.abs(0.75 * np.asarray(drv)), xt == "bf16", ref)
    assert np.all(err <= bound), float(np.max(err / bound))
    terms = (np.abs(dnv.astype(np.float64)) + np.abs(dn2v)) * np.abs(xh)
    bound = _dw_bound(terms, rows)
    assert np.all(np.abs(host(dw) - ref_w) <= bound)
    again = B.rmsnorm_backward(dn, x, dev(rstd), dev(w), dn2=dn2, d_res=dr, res_scale=0.75)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    only = B.rmsnorm_backward(dn, x, dev(rstd), dev(w), dn2=dn2, d_res=dr, res_scale=0.75,
                              out=(torch.empty_like(x), None))
    assert torch.equal(only[0], dx) and only[1] is None


def test_norm_backward_without_weight_and_without_rows():
    x, xv = _values(1, 4, 64, "f32")
    dn, dnv = _values(2, 4, 64, "f32")
    rstd = norm.rstd(xv, EPS).astype(np.float32)
    dx, dw = B.rmsnorm_backward(dn, x, dev(rstd))
    assert dw is None
    ref, _ = norm.backward(dnv, xv, rstd, None)
    r = rstd.astype(np.float64)[:, None]
    assert np.all(np.abs(host(dx) - ref) <= _dx_bound(dnv.astype(np.float64), xv * r, r, 0.0, False, ref))
    w = torch.ones(64, device="cuda")
    dx, dw = B.rmsnorm_backward(dn[:0], x[:0], dev(rstd)[:0], w)
    assert dx.shape == (0, 64) and bool((dw == 0).all())


MODES = ["none", "token", "channel", "full"]


def _gate(seed, mode, rows, cols):
    g = inputs.rng(303, seed)
    shape = {"none": None, "token": (rows,), "channel": (cols,), "full": (rows, cols)}[mode]
    if shape is None:
        return None, None
    v = g.uniform(0.05, 1.0, shape).astype(np.float32)
    v.reshape(-1)[::5] *= -1
    return v, np.broadcast_to(v[:, None] if mode == "token" else v, (rows, cols))


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("xt,yt", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("rows,cols", [(1, 8), (5, 96), (33, 2048), (3, 2056), (1100, 72), (6, 7168), (2, 16384)])
def test_gate_residual_and_its_backward(rows, cols, xt, yt, mode):
    x, xv = _values(rows + 10, rows, cols, xt)
    y, yv = _values(rows + 11, rows, cols, yt)
    w = _weight(rows, cols)
    gate, gb = _gate(rows, mode, rows, cols)
    gt = None if gate is None else dev(gate)
    out, rstd = B.rmsnorm_gate_residual(x, y, dev(w), gt, gate_mode=mode, eps=EPS, branch_scale=0.625, res_scale=0.75)
    ref = norm.gate_residual(xv, yv, w, gb, EPS, 0.625, 0.75)
    got = inputs.bf16_bits_to_float(host(out)) if xt == "bf16" else host(out)
    r64 = norm.rstd(yv, EPS).astype(np.float64)
    # r, y r, w, gate, scale(, scale x token gate): at most 6 u of the branch; the sum: 2 u of each part
    arith = 8 * U * np.abs(ref - 0.75 * xv.astype(np.float64)) + 2 * U * np.abs(0.75 * xv) + U * np.abs(ref) + 1e-44
    bound = arith + (BF16 * (np.abs(ref) + arith) if xt == "bf16" else 0.0)
    assert np.all(np.abs(got - ref) <= bound), float(np.max(np.abs(got - ref) / bound))
    assert_bytes_equal(host(rstd), r64.astype(np.float32), "rstd")

    d, dv = _values(rows + 12, rows, cols, xt, 1e-3)
    dy, dw, dgate = B.rmsnorm_gate_residual_backward(d, y, rstd, dev(w), gt, gate_mode=mode, branch_scale=0.625)
    r = host(rstd).astype(np.float64)[:, None]
    yh, up = yv * r, 0.625 * dv.astype(np.float64)
    dn = up if gb is None else up * gb
    ref, ref_w = norm.backward(dn, yv, host(rstd), w)
    got = inputs.bf16_bits_to_float(host(dy)) if yt == "bf16" else host(dy)
    bound = _dx_bound(dn * w, yh, r, 0.0, yt == "bf16", ref)
    assert np.all(np.abs(got - ref) <= bound), float(np.max(np.abs(got - ref) / bound))
    assert np.all(np.abs(host(dw) - ref_w) <= _dw_bound(dn * yh, rows))
    terms = up * yh * w
    if mode == "none":
        assert dgate is None
    elif mode == "full":
        assert np.all(np.abs(host(dgate) - terms) <= 6 * U * np.abs(terms) + 1e-44)
    elif mode == "token":                                    # 64 sequential, 8 exchanges, 3 joins, 4 of a term
        assert np.all(np.abs(host(dgate) - terms.sum(1)) <= 84 * U * np.abs(terms).sum(1) + 1e-44)
    else:
        assert np.all(np.abs(host(dgate) - terms.sum(0)) <= _dw_bound(terms, rows))
    again = B.rmsnorm_gate_residual_backward(d, y, rstd, dev(w), gt, gate_mode=mode, branch_scale=0.625)
    assert torch.equal(again[0], dy) and torch.equal(again[1], dw) and (dgate is None or torch.equal(again[2], dgate))
    if dgate is not None:                                    # each output alone
        only = B.rmsnorm_gate_residual_backward(d, y, rstd, dev(w), gt, gate_mode=mode, branch_scale=0.625,
                                                out=(torch.empty_like(y), None, torch.empty_like(gt)))
        assert torch.equal(only[2], dgate) and torch.equal(only[0], dy)


def test_gate_residual_without_rows_or_weight():
    x, xv = _values(20, 3, 64, "f32")
    y, yv = _values(21, 3, 64, "f32")
    out, rstd = B.rmsnorm_gate_residual(x, y)
    ref = norm.gate_residual(xv, yv, None, None, EPS, 1.0, 1.0)
    assert np.all(np.abs(host(out) - ref) <= 8 * U * (np.abs(xv) + np.abs(ref - xv)))
    out, rstd = B.rmsnorm_gate_residual(x[:0], y[:0])
    assert out.shape == (0, 64) and rstd.shape == (0,)
    gate, w = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    dy, dw, dg = B.rmsnorm_gate_residual_backward(x[:0], y[:0], rstd, w, gate, gate_mode="channel")
    assert dy.shape == (0, 64) and bool((dw == 0).all()) and bool((dg == 0).all())


@pytest.mark.parametrize("mode", MODES)
def test_gate_residual_backward_without_weight(mode):
    rows, cols = 21, 136
    y, yv = _values(40, rows, cols, "f32")
    d, dv = _values(41, rows, cols, "f32", 1e-3)
    gate, gb = _gate(2, mode, rows, cols)
    gt = None if gate is None else dev(gate)
    rstd = norm.rstd(yv, EPS).astype(np.float32)
    dy, dw, dgate = B.rmsnorm_gate_residual_backward(d, y, dev(rstd), None, gt, gate_mode=mode)
    assert dw is None
    up, yh = dv.astype(np.float64), yv * rstd.astype(np.float64)[:, None]
    dn = up if gb is None else up * gb
    ref, _ = norm.backward(dn, yv, rstd, None)
    assert np.all(np.abs(host(dy) - ref) <= _dx_bound(dn, yh, rstd.astype(np.float64)[:, None], 0.0, False, ref))
    if mode != "none":
        axis = {"token": 1, "channel": 0, "full": ()}[mode]
        t = up * yh
        assert np.all(np.abs(host(dgate) - t.sum(axis)) <= 150 * U * np.abs(t).sum(axis) + 1e-44)


def test_norms_on_a_side_stream_and_with_one_workspace():
    """Calls on a stream of their own, one workspace for several calls in order."""
    x, _ = _values(30, 700, 256, "bf16")
    dn, _ = _values(31, 700, 256, "f32")
    w = dev(_weight(30, 256))
    n, q, s, t, rstd = B.rmsnorm_quantize(x, w)
    dx, dw = B.rmsnorm_backward(dn, x, rstd, w)
    ws = torch.empty(B.lib().mxq_workspace_bytes(B.OP_NORM_BACKWARD, 700, 256, 0), dtype=torch.uint8, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = B.rmsnorm_quantize(x, w)
        one = B.rmsnorm_backward(dn, x, got[4], w, workspace=ws)
        two = B.rmsnorm_backward(dn, x, got[4], w, workspace=ws)
    st.synchronize()
    assert torch.equal(got[1], q) and torch.equal(one[0], dx) and torch.equal(one[1], dw) and torch.equal(two[1], dw)
    with pytest.raises(ValueError, match="workspace"):
        B.rmsnorm_backward(dn, x, rstd, w, workspace=ws[:64])


def test_outputs_beyond_the_streaming_size_equal_smaller_calls():
    """More than 128 MB of BF16 output (non-temporal stores) against the same rows in small calls:
    every row's result is its own, whatever the call's size."""
    rows, cols = 16500, 4128
    assert rows * cols * 2 > 128 << 20
    g = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda s=1.0, dt=torch.bfloat16: (s * torch.randn((rows, cols), generator=g, device="cuda")).to(dt)
    x, dn, d_res, w = rand(), rand(1e-3, torch.float32), rand(1e-3), dev(_weight(0, cols))
    parts = [slice(0, 70), slice(8000, 8061), slice(rows - 33, rows)]
    for fmt in (B.MXFP8, B.NVFP4, B.MXFP4, B.BF16):
        whole = B.rmsnorm_quantize(x, w, fmt=fmt)
        for p in parts:
            for a, b in zip(whole, B.rmsnorm_quantize(x[p], w, fmt=fmt)):
                assert (a is None and b is None) or torch.equal(a[p], b)
    rstd = whole[4]
    dx, dw = B.rmsnorm_backward(dn, x, rstd, w, d_res=d_res, res_scale=0.5)
    for p in parts:
        assert torch.equal(dx[p], B.rmsnorm_backward(dn[p], x[p], rstd[p], w, d_res=d_res[p], res_scale=0.5)[0])
    ref = torch.zeros(cols, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(ref)
    for i in range(0, rows, 1100):
        t = dn[i:i + 1100].double() * x[i:i + 1100].double() * rstd[i:i + 1100, None].double()
        ref += t.sum(0)
        mag += t.abs().sum(0)
    assert bool(((dw.double() - ref).abs() <= (rows / 512 + 140) * U * mag).all())
    for mode, gate in (("none", None), ("token", torch.rand(rows, generator=g, device="cuda")),
                       ("full", torch.rand((rows, cols), generator=g, device="cuda"))):
        dy = B.rmsnorm_gate_residual_backward(d_res, x, rstd, w, gate, gate_mode=mode)[0]
        for p in parts:
            part = None if gate is None else gate[p]
            assert torch.equal(dy[p], B.rmsnorm_gate_residual_backward(d_res[p], x[p], rstd[p], w, part, gate_mode=mode)[0])


def test_more_rows_than_one_launch_takes():
    """2^21 rows to a launch: the rows on both sides of the seam equal calls of their own."""
    seam, rows, cols = 1 << 21, (1 << 21) + 9, 32
    g = torch.Generator(device="cuda").manual_seed(9)
    wide = torch.randn((rows, cols + 8), generator=g, device="cuda").bfloat16()
    x, y = wide[:, :cols], torch.randn((rows, cols), generator=g, device="cuda")
    w = dev(_weight(0, cols))
    gates = {"token": torch.randn(rows, generator=g, device="cuda"), "full": torch.randn_like(y)}
    parts = [slice(seam - 70, seam), slice(seam, rows)]
    for fmt in (B.MXFP8, B.MXFP4, B.NVFP4, B.BF16):
        whole = B.rmsnorm_quantize(x, w, fmt=fmt)
        for p in parts:
            for a, b in zip(whole, B.rmsnorm_quantize(x[p], w, fmt=fmt)):
                assert (a is None) == (b is None)
                assert a is None or torch.equal(a[p], b)
    for mode, gate in gates.items():
        res = x.contiguous()
        out, rstd = B.rmsnorm_gate_residual(res, y, w, gate, mode)
        for p in parts:
            o, r = B.rmsnorm_gate_residual(res[p], y[p], w, gate[p].clone(), mode)
            assert torch.equal(out[p], o) and torch.equal(rstd[p], r)


@pytest.mark.parametrize("xt,yt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
def test_gate_residual_beyond_the_streaming_size(xt, yt):
    """More than 128 MB of out and dy (non-temporal stores): every row equals a smaller call's."""
    rows, cols = 16500, 4104
    g = torch.Generator(device="cuda").manual_seed(12)
    make = lambda t: torch.randn((rows, cols), generator=g, device="cuda").to(torch.bfloat16 if t == "bf16" else torch.float32)
    x, y = make(xt), make(yt)
    w, gate = dev(_weight(3, cols)), torch.rand(cols, generator=g, device="cuda")
    assert x.numel() * x.element_size() > 128 << 20
    out, rstd = B.rmsnorm_gate_residual(x, y, w, gate, "channel", branch_scale=0.5, res_scale=0.75)
    dy, dw, dgate = B.rmsnorm_gate_residual_backward(x, y, rstd, w, gate, "channel", branch_scale=0.5)
    sums = torch.zeros(2, cols, dtype=torch.float64, device="cuda")
    for r0 in range(0, rows, 5000):
        r = slice(r0, min(r0 + 5000, rows))
        o, s = B.rmsnorm_gate_residual(x[r], y[r], w, gate, "channel", branch_scale=0.5, res_scale=0.75)
        assert torch.equal(out[r], o) and torch.equal(rstd[r], s)
        d, a, b = B.rmsnorm_gate_residual_backward(x[r], y[r], rstd[r].clone(), w, gate, "channel", branch_scale=0.5)
        assert torch.equal(dy[r], d)
        sums += torch.stack([a, b]).double()
    yh = y.double() * rstd.double()[:, None]
    mag = (0.5 * x.double() * yh).abs().sum(0)
    for got, ref, f in ((dw, sums[0], gate), (dgate, sums[1], w)):
        # both sides are ordered binary32 sums: at most 33 + 33 terms deep a workgroup and joined wave, and the factors
        assert bool(((got.double() - ref).abs() <= 2 * 80 * U * mag * f.abs().double()).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("log_w", [-3, 14, 15, 16, 18, 20, 40])
def test_norm_quantize_where_a_binary32_product_underflows(log_w, dtype):
    """A row statistic of one large element, others so small that x r leaves the binary32 range, and
    weights that bring the product back into BF16's: n is still the correctly rounded value, zeros
    and signs included."""
    cols = 512
    v = np.zeros((4, cols), np.float32)
    v[:, 0] = [2.0 ** 24, 2.0 ** 40, 2.0 ** 55, 2.0 ** 4]
    e = np.arange(1, cols)
    v[:, 1:] = np.where(e % 2, 1, -1) * np.ldexp(1 + (e % 5) / 8, -(90 + e % 60)).astype(np.float32)
    v[0, 1] = 2.0 ** -133
    x = dev(v)
    if dtype == "bf16":
        bits = inputs.to_bf16_bits(v)
        x, v = dev_bf16(bits), inputs.bf16_bits_to_float(bits)
    for w in (np.full(cols, 2.0 ** log_w), np.ldexp(1 + np.arange(cols) % 9 / 16, log_w)):
        w = w.astype(np.float32)
        exp = norm.rmsnorm_bf16(v, w, EPS)
        assert ((exp & 0x7FFF) - 1 < 0x7F).any()            # BF16 subnormals among them
        assert_bytes_equal(host(B.rmsnorm_quantize(x, dev(w), eps=EPS, fmt=B.BF16)[0]), exp, "n")
        n, q, s, t, _ = B.rmsnorm_quantize(x, dev(w), eps=EPS, fmt=B.NVFP4)
        assert_bytes_equal(host(n), exp, "n beside NVFP4")
        _check_quantized(B.NVFP4, exp, q, s, t, "underflow")


def test_rows_of_zeros_at_the_smallest_eps():
    """eps = 2^-252: r = 2^126 for a row of zeros, whose normed row is zero and whose gradients are
    those of the formula; a smaller eps only without a row statistic."""
    eps, cols = 2.0 ** -252, 64
    x, y = torch.full((3, cols), 3.0, device="cuda"), torch.zeros((3, cols), device="cuda")
    y[1, 0] = 1.0
    w = torch.full((cols,), 2.0, device="cuda")
    out, rstd = B.rmsnorm_gate_residual(x, y, w, eps=eps)
    want = x.clone()
    want[1, 0] += 16.0                                       # 1 / sqrt(1 / 64) times the weight
    assert torch.equal(out, want) and rstd.tolist() == [2.0 ** 126, 8.0, 2.0 ** 126]
    n, _, _, _, rstd = B.rmsnorm_quantize(y, w, eps=eps, fmt=B.BF16)
    assert torch.equal(n, (want - x).bfloat16()) and rstd.tolist() == [2.0 ** 126, 8.0, 2.0 ** 126]
    dx, dw = B.rmsnorm_backward(torch.full_like(y, 2.0 ** -100), y, rstd, w)
    assert bool((dx[0] == 2.0 ** 27).all()) and bool(torch.isfinite(dx).all()) and dw[1] == 0
    none = torch.empty((3, cols), dtype=torch.bfloat16, device="cuda")
    B.rmsnorm_quantize(y, w, eps=1e-200, fmt=B.BF16, out=(none, None, None, None, None))
    assert torch.equal(none, n)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("rows,cols,xt,yt", [(1100, 2048, "bf16", "f32"), (1537, 2056, "f32", "bf16"),
                                             (1030, 4104, "bf16", "bf16"), (1025, 8200, "f32", "f32")])
def test_norm_backwards_where_a_workgroup_takes_several_rows(rows, cols, xt, yt, mode):
    """512 workgroups of several waves, each with two to four rows in turn: the rows' sums meet in two
    buffers of LDS by turns. Every row, dgate and both column sums against FP64, and bit for bit
    against calls in which a workgroup has one row."""
    y, yv = _values(rows, rows, cols, yt)
    d, dv = _values(rows + 1, rows, cols, xt, 1e-3)
    w = _weight(rows, cols)
    gate, gb = _gate(rows, mode, rows, cols)
    gt, wt = None if gate is None else dev(gate), dev(w)
    rstd = norm.rstd(yv, EPS).astype(np.float32)
    rt = dev(rstd)
    dy, dw, dgate = B.rmsnorm_gate_residual_backward(d, y, rt, wt, gt, gate_mode=mode, branch_scale=0.625)
    for a in range(0, rows, 512):
        p = slice(a, min(a + 512, rows))
        gp = gt if mode in ("none", "channel") else gt[p].clone()           # a gate of its own allocation
        part = B.rmsnorm_gate_residual_backward(d[p], y[p], rt[p], wt, gp, gate_mode=mode, branch_scale=0.625)
        assert torch.equal(dy[p], part[0])
        if mode in ("token", "full"):
            assert torch.equal(dgate[p], part[2])
    r = rstd.astype(np.float64)[:, None]
    yh, up = yv * r, 0.625 * dv.astype(np.float64)
    dn = up if gb is None else up * gb
    ref, ref_w = norm.backward(dn, yv, rstd, w)
    got = inputs.bf16_bits_to_float(host(dy)) if yt == "bf16" else host(dy)
    # as _dx_bound and the dgate bounds count them; rows of 8200 join sixteen waves: 15 joins, not 3
    assert np.all(np.abs(got - ref) <= _dx_bound(dn * w, yh, r, np.abs(yh * r) * 12 * U * np.mean(np.abs(dn * w * yh), axis=1, keepdims=True),
                                                 yt == "bf16", ref))
    assert np.all(np.abs(host(dw) - ref_w) <= _dw_bound(dn * yh, rows))
    terms = up * yh * w
    if mode == "token":
        assert np.all(np.abs(host(dgate) - terms.sum(1)) <= 96 * U * np.abs(terms).sum(1) + 1e-44)
    elif mode == "channel":
        assert np.all(np.abs(host(dgate) - terms.sum(0)) <= _dw_bound(terms, rows))
    elif mode == "full":
        assert np.all(np.abs(host(dgate) - terms) <= 6 * U * np.abs(terms) + 1e-44)
    if mode == "none":                                       # the norm before a block: two gradients and a residual's
        dn2, dr = _values(rows + 2, rows, cols, xt, 1e-3)[0], _values(rows + 3, rows, cols, yt, 1e-3)[0]
        dx, dw = B.rmsnorm_backward(d, y, rt, wt, dn2=dn2, d_res=dr, res_scale=0.75)
        for a in range(0, rows, 512):
            p = slice(a, min(a + 512, rows))
            part = B.rmsnorm_backward(d[p], y[p], rt[p], wt, dn2=dn2[p], d_res=dr[p], res_scale=0.75)
            assert torch.equal(dx[p], part[0])
