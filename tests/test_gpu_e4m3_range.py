"""Pages of an 8-bit pool whose V scales lie 2^20 and more apart, against the
bound that the few-rows kernel's number format gives."""
import numpy as np
import pytest

from e4m3_util import assert_within
from gpu_util import dev, host
from test_gpu_e4m3 import F16, F32, Case, wide_table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [16, 1])
@pytest.mark.parametrize("first", [0, 16, 48])
@pytest.mark.parametrize("low,lost", [(-10, 18), (-10, 30), (-14, 24), (0, 10)])
def test_outlier_page_of_little_weight(pkv, cuda_dev, page, first, low, lost):
    """16 tokens of V values near 2^10 and weights near 2^-lost of the others', whose V values are near
    2^low.  The product of weight and V scale is rounded to 11 (fp32 output: 22) bits, or, where that is
    more, to half of fp16's smallest in units of 2^-7 of the largest weight and V scale: by at most
    2^-32 |code| S for each token, S the largest scale, the sum of the weights being at least the
    largest of them."""
    import torch
    c = Case(pkv, cuda_dev, [64], 1, 1, 64, page)
    k = np.zeros((64, 1, 64), np.float16)
    v = c.rows(64, spread=False).astype(np.float64) * 2.0 ** low
    k[first:first + 16, :, 0] = -8.0 * np.log(2.0) * lost     # z = q . k / 8
    v[first:first + 16] *= 2.0 ** (10 - low)
    c.append([64], k=k, v=v.astype(np.float16))
    scales = c.vm.scale[c.table[0][:64 // page]]
    assert np.nanmax(scales) >= 2.0 ** (9 - low) * np.nanmin(scales)
    q = np.zeros((1, 1, 64), np.float16)
    q[:, :, 0] = 1.0
    blk = c.table[0][np.arange(64) // page]
    off = 2.0 ** -32 * np.abs(c.vm.code[blk, np.arange(64) % page]).sum(0) * np.nanmax(scales)   # [1, 64]
    table = dev(wide_table(c), cuda_dev)
    ws = pkv.make_workspace(c.pool, 1, 1, table.shape[1], 0)
    for f32 in (False, True):
        out = torch.empty((1, 1, 64), dtype=torch.float32 if f32 else torch.float16, device=cuda_dev)
        pkv.pf_paged_decode_attention(c.pool, 1, dev(q, cuda_dev), table, dev(c.lens, cuda_dev), c.scale(), out, 0, ws)
        want, tol = c.want(q, [0, 1], False, 2.0 ** -21 if f32 else F16, F32 if f32 else F16)
        # (want() allows for half of fp16's smallest subnormal, which fp32 output does not have)
        assert_within(host(out), want, tol - (2.0 ** -25 if f32 else 0.0) + off, f"f32={f32}")
