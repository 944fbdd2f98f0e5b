"""Step-input calls at the edges of their ranges, against float64."""
import numpy as np
import pytest
import torch

from gpu_util import need_gpu, np_
from oracle import csa2_oracle as o
from serving_lightning_indexer_gb300 import csa2
from test_gpu_inputs import _sync_ok

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- quantiser
def _border_blocks(exponent, width):
    """Blocks of `width` bf16 values, one for every bf16 mantissa of the block's maximum: the
    maximum, then every value of the 16 binades below it, as many blocks as that takes, and
    zeros of both signs."""
    blocks = []
    for k in range(128):
        top = (1 + k / 128) * 2.0 ** exponent
        vals = np.array([(1 + j / 128) * 2.0 ** (exponent - e) for e in range(17) for j in range(128)])
        vals = vals[vals < top]
        vals[::2] *= -1
        n = -(-len(vals) // (width - 1))
        b = np.zeros((n, width))
        b[:, 0] = top
        flat = np.where(np.arange(n * (width - 1)) % 3 == 0, -0.0, 0.0)
        flat[:len(vals)] = vals
        b[:, 1:] = flat.reshape(n, width - 1)
        blocks.append(b)
    return np.concatenate(blocks)


@pytest.mark.parametrize("exponent", [0, 1, 6, -100, 120, 127])
@pytest.mark.parametrize("rows", [1, 128])
def test_quant_fp8_borders_go_to_the_even_code(rows, exponent):
    """x * 448 / a of bf16 x and a lies on a border between two codes or at least 2^-14 of
    itself away from one (448 x has 11 bits, border * a at most 13): the float64 quotient,
    rounded to fp32 on its way to e4m3, is on the same side, so the codes are equal."""
    dev = need_gpu()
    if rows == 1:
        v = _border_blocks(exponent, 128)                 # a block a row
    else:
        v = _border_blocks(exponent, 128 * 128).reshape(-1, 128)   # a tile of 128 rows
    x = torch.tensor(v, dtype=torch.float64).to(torch.bfloat16)
    assert np.array_equal(x.double().numpy(), v)
    codes = torch.empty(v.shape, dtype=torch.uint8, device=dev)
    scale = torch.empty(len(v) // rows, 1, device=dev)
    csa2.quant_fp8(x.to(dev), codes, scale, block_rows=rows)
    _sync_ok()
    a = np.abs(v).reshape(-1, rows * 128).max(axis=1).repeat(rows)[:, None]
    want = torch.tensor(v * 448.0 / a).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(np_(scale)[:, 0], (a[::rows, 0].astype(np.float32) / np.float32(448)))
    bad = np_(codes) != want
    assert not bad.any(), f"{bad.sum()} of {bad.size} codes"


# ---------------------------------------------------------------- the batch's arrays
def test_batch_plan_writes_a_window_right_before_and_around_the_lengths():
    """One allocation: the lengths between the rows of the window and right behind its last row."""
    dev = need_gpu()
    i32 = dict(dtype=torch.int32, device=dev)
    ctx, new = [0, 100, 17, 3, 500, 0, 64, 9], [1, 1, 2, 0, 1, 1, 1, 1]
    buf = torch.full((8 * 256 + 8,), -7, **i32)
    buf[:8] = torch.tensor(ctx, **i32)
    buf[2048:] = torch.tensor(new, **i32)
    wide = buf[:2048].view(8, 256)
    csa2.batch_plan(buf[:8], buf[2048:], 1, swa_ring=130, swa_slot=wide[:, 128:])
    _sync_ok()
    want = np.full(2056, -7)
    want[:8], want[2048:] = ctx, new
    want[:2048].reshape(8, 256)[:, 128:] = o.batch_plan(ctx, new, 1, ring=130, n_swa=128)[0]["swa_slot"]
    assert np.array_equal(np_(buf), want)
