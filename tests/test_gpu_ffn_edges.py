"""Edges of the gated feed-forward block and of the 4-bit matrix-vector products on the GPU: expert weights
past 32-bit offsets."""

import pytest
import torch

import microscaling_precision_quantization_amd as mxq
from microscaling_precision_quantization_amd import binding as B
from tests import ffn_ref as R
from tests.test_gpu_ffn import BF, gen, randn

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
