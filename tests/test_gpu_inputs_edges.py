"""Step-input calls at the edges of their ranges, against float64."""
import numpy as np
import pytest
import torch

from gpu_util import need_gpu, np_
from oracle import csa2_oracle as o
from serving_lightning_indexer_gb300 import csa2
from test_gpu_inputs import _codes, _gen, _sync_ok

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


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


# ---------------------------------------------------------------- projection
def _linear64(x, xs, w, ws):
    """The product of the decoded codes with their scales in float64, and that of the magnitudes."""
    T, K = x.shape
    xd = x.view(torch.float8_e4m3fn).double() * xs.double().repeat_interleave(128, 1)[:, :K]
    wd = w.view(torch.float8_e4m3fn).double() * ws.double().repeat_interleave(128, 0)[:len(w)].repeat_interleave(128, 1)[:, :K]
    return xd @ wd.t(), xd.abs() @ wd.abs().t()


def test_fp8_linear_one_row_through_both_kernels():
    """Whole numbers whose sums are exact in any order, so that a row's fp32 output has the
    same bits whether 8 rows or 1,300 are projected, rotated columns included."""
    dev = need_gpu()
    g = _gen(dev, 41)
    table = torch.tensor([0x00, 0x38, 0xB8, 0x40, 0xC0], dtype=torch.uint8, device=dev)   # 0, 1, -1, 2, -2
    T, N, K = 1300, 1024, 400
    x = table[torch.randint(0, 5, (T, K), generator=g, device=dev)]
    w = table[torch.randint(0, 5, (N, K), generator=g, device=dev)]
    xs, ws = torch.ones(T, 4, device=dev), torch.ones(8, 4, device=dev)
    pos = torch.randint(0, 2 ** 31 - 1, (T,), generator=g, device=dev, dtype=torch.int64).to(torch.int32)
    many = torch.empty(T, N, device=dev)
    csa2.fp8_linear(x, xs, w, ws, many, row_pos=pos, rope_head=256)
    for n in (8, 20, 60):
        few = torch.empty(n, N, device=dev)
        csa2.fp8_linear(x[:n], xs[:n], w, ws, few, row_pos=pos[:n], rope_head=256)
        _sync_ok()
        assert torch.equal(few, many[:n]), f"{n}: {(few != many[:n]).sum().item()} of {few.numel()} values differ"
    # the unrotated columns are the sums themselves
    y, _ = _linear64(x, xs, w, ws)
    keep = (torch.arange(N, device=dev) % 256) < 192
    assert torch.equal(many[:, keep].double(), y[:, keep])


def _rope64(y, pos, head, theta=10000.0):
    rate = theta ** (-torch.arange(32, dtype=torch.float64, device=y.device) / 32)
    ang = pos.double()[:, None] * rate
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    z = y.reshape(len(y), -1, head).clone()
    a, b = z[..., head - 64::2].clone(), z[..., head - 63::2].clone()
    z[..., head - 64::2], z[..., head - 63::2] = a * c - b * s, a * s + b * c
    return z.reshape(y.shape)


@pytest.mark.parametrize("T", [8, 60, 1300])
def test_fp8_linear_turns_fp32_output_to_fp32(T):
    """Exact sums, so that the turn's own error shows.  Of a pair's length: the angle 2^-23.3
    (its top bits as fp32: half a step of 2^7 in 2^32 turns) and 2^-26 (the rate); sine and
    cosine of 2 steps of 2^-24 each, 2^-22.5 together; a product's and a sum's rounding 2^-23:
    2^-21.2 in all.  float64's own angle is off by 2^-33 here."""
    dev = need_gpu()
    g = _gen(dev, 42)
    table = torch.tensor([0x00, 0x38, 0xB8, 0x40, 0xC0], dtype=torch.uint8, device=dev)
    x = table[torch.randint(0, 5, (T, 272), generator=g, device=dev)]
    w = table[torch.randint(0, 5, (1024, 272), generator=g, device=dev)]
    xs, ws = torch.ones(T, 3, device=dev), torch.ones(8, 3, device=dev)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device=dev, dtype=torch.int32)
    out = torch.empty(T, 1024, device=dev)
    csa2.fp8_linear(x, xs, w, ws, out, row_pos=pos, rope_head=128)
    _sync_ok()
    y = _linear64(x, xs, w, ws)[0]
    err = (out.double() - _rope64(y, pos, 128)).abs().view(T, -1, 2)
    length = torch.linalg.vector_norm(y.view(T, -1, 2), dim=-1, keepdim=True)
    assert bool((err <= 2.0 ** -21.2 * length).all()), f"worst {(err / length.clamp(min=1e-30)).max().log2().item()}"


# (T, N, K).  On 152 SMs a CTA of the few-rows kernel has 34 blocks (153 column tiles leave
# no CTAs to split the input dims over), 33 (60 tiles split by 2), 32 (K = 65,536 split by
# 16), 16 (the attention query's 256 tiles); the last is the many-rows kernel's, 256 a CTA.
DEEP = [(8, 19500, 4240), (24, 19500, 4240), (64, 7680, 8208), (5, 130, 65536), (20, 130, 65536), (40, 130, 65536),
        (8, 32768, 2048), (4096, 130, 65536)]


@pytest.mark.parametrize("w_ready", [False, True])
@pytest.mark.parametrize("T,N,K", DEEP)
def test_fp8_linear_over_many_blocks(T, N, K, w_ready):
    """The rings of stages, accumulators and scale segments go round several times.  Error:
    (130 + 2 blocks) roundings of the sum of magnitudes, then the output's."""
    dev = need_gpu()
    g = _gen(dev, T + N + K)
    x, xs = _codes((T, K), g, dev, 1)
    w, ws = _codes((N, K), g, dev, 128)
    y, mag = _linear64(x, xs, w, ws)
    torch.cuda.synchronize()
    tol = (130 + 2 * xs.shape[1]) * U * mag
    out = torch.full((T, N), 7.0, device=dev)
    csa2.fp8_linear(x, xs, w, ws, out, w_ready=w_ready)
    _sync_ok()
    assert bool(((out.double() - y).abs() <= U * y.abs() + tol).all())
    if N % 512 == 0:
        pos = torch.randint(0, 1 << 20, (T,), generator=g, device=dev, dtype=torch.int32)
        out = torch.zeros(T, N, dtype=torch.bfloat16, device=dev)
        csa2.fp8_linear(x, xs, w, ws, out, row_pos=pos, rope_head=512, w_ready=w_ready)
        _sync_ok()
        y = _rope64(y, pos, 512)
        # a pair's values share their errors; RoPE's own are 2^-20 of the pair
        z, t = y.abs().view(T, -1, 2), tol.view(T, -1, 2)
        both = (t.sum(-1) + 2.0 ** -20 * z.sum(-1))[..., None].expand_as(z).reshape(T, N)
        assert bool(((out.double() - y).abs() <= 2.0 ** -8 * (y.abs() + both) + both).all())


@pytest.mark.parametrize("T", [4, 40, 1300])
@pytest.mark.parametrize("ex,ew", [(-63, -63), (-120, -6), (60, 60), (100, -100)])
def test_fp8_linear_scales_at_the_ends_of_the_range(T, ex, ew):
    """Products of two scales down to 2^-126, fp32's smallest normal number, are exact."""
    dev = need_gpu()
    g = _gen(dev, 43)
    table = torch.tensor([0x00, 0x38, 0xB8], dtype=torch.uint8, device=dev)
    K, N = 272, 256
    x = table[torch.randint(0, 3, (T, K), generator=g, device=dev)]
    w = table[torch.randint(0, 3, (N, K), generator=g, device=dev)]
    xs, ws = torch.full((T, 3), 2.0 ** ex, device=dev), torch.full((2, 3), 2.0 ** ew, device=dev)
    out = torch.empty(T, N, device=dev)
    csa2.fp8_linear(x, xs, w, ws, out)
    _sync_ok()
    assert torch.equal(out.double(), _linear64(x, xs, w, ws)[0])


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


def test_batch_plan_records_counts_past_31_bits_without_row_arrays():
    """The counts of places stop at 2^31 - 1, also where only they are asked for."""
    dev = need_gpu()
    i32 = dict(dtype=torch.int32, device=dev)
    big = 2 ** 31 - 1
    zero = torch.zeros(2, **i32)
    for new, bad in (([big, big], True), ([big, 1], True), ([big - 3, 2], False)):
        start = torch.full((3,), -9, **i32)
        csa2.batch_plan(zero, torch.tensor(new, **i32), 2, row_start=start)
        torch.cuda.synchronize()
        assert csa2.check_device_error() == (6 if bad else 0), new
        if not bad:
            assert np_(start).tolist() == [0, new[0], sum(new)]
