"""quantize_fp8 against exact arithmetic: every pair of mantissas of a value and
of its block's largest, in all of e4m3's range and one power of two below it."""
import pytest
import torch

import tensor_bf16_gemm_amd as gc
from gpu_util import log

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3 = torch.float8_e4m3fn


def nearest(x, top):
    """The e4m3 value nearest to 448 x / top, the even code of two as near.  448 x has at most 11
    bits and a midpoint of two codes times top at most 13, so that the doubles compared are exact."""
    codes = torch.arange(127, dtype=torch.uint8, device=DEV).view(E4M3).double()
    v = 448 * x.double().abs()
    index = torch.zeros(x.shape, dtype=torch.int64, device=DEV)
    for i in range(126):
        mid = (codes[i] + codes[i + 1]) / 2 * top.double()
        index += (v > mid) | ((v == mid) & (i % 2 == 1))
    return codes[index] * x.double().sign()


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("power", [0, 64, 99, 100, 127, -60, -99])
def test_every_code_is_the_nearest(rows, power):
    log(f"quantize_fp8 block_rows={rows} largest values from 2^{power}")
    mantissas = 1 + torch.arange(128, dtype=torch.float64, device=DEV) / 128
    top = mantissas * 2.0 ** power
    # down to 2^-19 of the largest: 448 * 2^-19 is below half of the least code, 2^-9
    x = (mantissas * torch.exp2(power - torch.arange(20, dtype=torch.float64, device=DEV))[:, None]).flatten()
    x = torch.cat([x, -x])
    blocks = -(-len(x) // 127)
    x = torch.nn.functional.pad(x, (0, 127 * blocks - len(x)))
    if rows == 1:
        # a row per largest value, which is in every block of it
        m = torch.cat([top[:, None, None].expand(-1, blocks, 1), x.view(1, blocks, 127).expand(128, -1, -1)], 2)
        m, top = m.reshape(128, -1), top[:, None]
    else:
        # a block per largest value
        m = torch.zeros((128, 128, 128), dtype=torch.float64, device=DEV)
        m.view(128, -1)[:, :len(x)] = x
        m[:, 127, 127] = top
        m, top = m.transpose(0, 1).reshape(128, -1), top.repeat_interleave(128)[None]
    m = torch.where(m.abs() > top, 0.0, m)                # (values above this row's or block's largest)
    given = m.bfloat16()
    assert torch.equal(given.double(), m)
    q, s = gc.quantize_fp8(given, block_rows=rows)
    assert torch.equal(q.double(), nearest(given, top))
    want = (m.abs().view(128, -1, 128).amax(2) if rows == 1 else top[:, ::128]) / 448
    assert torch.all((s.double() - want).abs() <= 2.0 ** -24 * 2 * want)
