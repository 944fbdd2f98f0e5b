"""GPU parity of the step-input calls: csa2_quant_fp8, csa2_fp8_linear and
csa2_batch_plan against the float64 oracle.

Tolerances, from the arithmetic (u = 2^-24, half a step of fp32):
  * a code: the kernel's value to round is y * f with f = 448 / a, two fp32
    roundings; with a norm, y carries the rounded root of a sum of K squares
    (each of at most K / 256 + 13 additions in a chain) and two products, and a
    carries the same.  So the value is within e = (2 + [norm] 2 (K / 256 + 24)) u
    relative of the exact one, and its code within half a step of that: 2^-4
    relative above 2^-6, 2^-10 below.
  * a scale: the same e, and 2 u for its own roundings.
  * a projection: products of codes are exact in fp32; a block's 128 products and
    the sum over blocks are at most 128 + 2 * blocks roundings in a chain, and the
    two scales two more: e = (130 + 2 blocks) u sum_k |x w| (all scaled).  RoPE adds
    2^-20 of the pair's magnitudes (the angle: 1e-8 rad from the rate, 2^-23 * pi
    from its fp32 value; sin and cos; two products and a sum).  Then half a step of
    the output's type.
"""
import numpy as np
import pytest
import torch

from gpu_util import need_gpu, np_
from oracle import csa2_oracle as o
from serving_lightning_indexer_gb300 import csa2
from serving_lightning_indexer_gb300 import workloads as W

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _sync_ok():
    torch.cuda.synchronize()
    assert csa2.check_device_error() == 0


def _gen(dev, seed):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g


def _assert_codes(codes, v, e, what):
    """e4m3 codes (uint8 array) round the exact values v, known to a relative e."""
    d = o.fp8_e4m3_table()[codes]
    a = np.minimum(np.abs(v), 448.0)
    half = np.maximum(2.0 ** -4 * a, 2.0 ** -10)
    err = np.abs(d - np.clip(v, -448.0, 448.0))
    bad = err > half * (1 + 2 * e) + 2 * e * a
    assert not bad.any(), f"{what}: {bad.sum()} codes off, worst {err.max()}"


def _quant_case(T, K, rows, norm, seed, ld_extra=0):
    dev = need_gpu()
    g = _gen(dev, seed)
    buf = torch.randn(T, K + ld_extra, generator=g, device=dev).to(torch.bfloat16)
    x = buf[:, :K]
    x[:, ::37] *= 30.0
    gamma = 1.0 + 0.1 * torch.randn(K, generator=g, device=dev) if norm else None
    nb, rb = -(-K // 128), -(-T // rows)
    codes = torch.full((T + 1, K + 32), 0x55, dtype=torch.uint8, device=dev)
    scale = torch.full((rb + 1, nb + 3), -1.0, device=dev)
    return x, gamma, codes, scale, nb, rb


@pytest.mark.parametrize("T,K,rows,norm", [
    (1, 16, 1, False), (1, 7168, 1, False), (5, 528, 1, False), (33, 2000, 1, False), (130, 128, 1, False),
    (1, 16, 1, True), (3, 144, 1, True), (8, 7168, 1, True), (17, 4096, 1, True), (2, 4112, 1, True), (2, 8208, 1, True),
    (2, 16384, 1, True), (1, 16, 128, False), (127, 144, 128, False), (128, 128, 128, False), (300, 2000, 128, False),
])
def test_quant_fp8_matches_oracle(T, K, rows, norm):
    x, gamma, codes, scale, nb, rb = _quant_case(T, K, rows, norm, seed=T * 7 + K, ld_extra=48)
    csa2.quant_fp8(x, codes[:T, :K], scale[:rb, :nb], gamma=gamma, eps=1e-5, block_rows=rows)
    _sync_ok()
    y = np_(x.float()).astype(np.float64)
    if norm:
        y = o.rms_norm_rows(y, np_(gamma).astype(np.float64), 1e-5)
    s, m = o.e4m3_block_scales(y, rows)
    e = (2 + (2 * (K / 256 + 24) if norm else 0)) * U
    assert np.all(np.abs(np_(scale)[:rb, :nb] - s) <= (e + 2 * U) * s)
    _assert_codes(np_(codes)[:T, :K], y * o.expand_blocks(m, rows, T, K), e, "quant")
    # nothing outside is touched
    assert (np_(codes)[T:] == 0x55).all() and (np_(codes)[:T, K:] == 0x55).all()
    assert (np_(scale)[rb:] == -1).all() and (np_(scale)[:rb, nb:] == -1).all()


@pytest.mark.parametrize("rows", [1, 128])
def test_quant_fp8_special_values(rows):
    dev = need_gpu()
    x = torch.zeros(4, 640, dtype=torch.bfloat16, device=dev)
    x[0, 3], x[0, 4], x[0, 5] = float("inf"), float("-inf"), float("nan")
    x[0, 6], x[0, 7] = -7.0, 3.5                         # the block's finite values keep their codes
    x[1, 130] = 2.0 ** -133                              # a subnormal bf16: below the floor
    x[1, 256] = 3.3895313892515355e38                    # the largest bf16
    x[2, 384:512] = float("nan")                         # nothing finite
    x[3, 512] = -0.0
    codes, scale = torch.empty(4, 640, dtype=torch.uint8, device=dev), torch.empty(4 if rows == 1 else 1, 5, device=dev)
    csa2.quant_fp8(x, codes, scale, block_rows=rows)
    _sync_ok()
    c, s = np_(codes), np_(scale)
    v = o.fp8_e4m3_table()[c]
    assert np.isnan(v[0, 3:6]).all() and v[0, 6] == -448.0 and v[0, 7] == 224.0
    assert s[0, 0] == np.float32(7.0 / 448.0) and np.isnan(v).sum() == 3 + 128
    r1 = 1 if rows == 1 else 0
    assert s[r1, 1] == np.float32(2.0 ** -120) and v[1, 130] == 0.0
    assert v[1, 256] == 448.0 and s[r1, 2] == np.float32(3.3895313892515355e38) / np.float32(448)
    assert s[2 if rows == 1 else 0, 3] == 1.0 and np.isnan(v[2, 384:512]).all()
    assert s[3 if rows == 1 else 0, 4] == 1.0 and not v[3].any()


def test_quant_fp8_norm_of_a_zero_row_and_of_a_nan_row():
    dev = need_gpu()
    x = torch.zeros(3, 256, dtype=torch.bfloat16, device=dev)
    x[1] = 1.0
    x[2, 200] = float("nan")
    x[2, 0] = 1.0
    gamma = torch.ones(256, device=dev)
    codes, scale = torch.empty(3, 256, dtype=torch.uint8, device=dev), torch.empty(3, 2, device=dev)
    csa2.quant_fp8(x, codes, scale, gamma=gamma, eps=1e-6)
    _sync_ok()
    v, s = o.fp8_e4m3_table()[np_(codes)], np_(scale)
    assert not v[0].any() and (s[0] == 1).all() and (v[1] == 448.0).all()
    assert np.isnan(v[2]).all() and (s[2] == 1).all()   # the norm of a row with a NaN is NaN throughout


# ---------------------------------------------------------------- projections
def _codes(shape, g, dev, rows):
    """Random codes with scales, as csa2_quant_fp8 lays them out (NaN codes left out)."""
    T, K = shape
    c = torch.randint(0, 256, (T, K), generator=g, device=dev, dtype=torch.uint8)
    c = torch.where((c & 0x7F) == 0x7F, c & 0x80, c)
    s = 0.01 + torch.rand(-(-T // rows), -(-K // 128), generator=g, device=dev)
    return c, s


def _decode(c):
    return o.fp8_e4m3_table()[np_(c)]


def _linear_ref(x, xs, w, ws, pos, head, theta):
    xd, wd, xs, ws = _decode(x), _decode(w), np_(xs).astype(np.float64), np_(ws).astype(np.float64)
    y = o.fp8_linear(xd, xs, wd, ws)
    mag = o.fp8_linear(np.abs(xd), xs, np.abs(wd), ws)
    tol = (130 + 2 * xs.shape[1]) * U * mag
    if head:
        T, N = y.shape
        z, t = np.abs(y).reshape(T, -1, head), tol.reshape(T, -1, head)
        pair = z[..., head - 64::2] + z[..., head - 63::2]
        both = t[..., head - 64::2] + t[..., head - 63::2] + 2.0 ** -20 * pair
        t[..., head - 64::2] = t[..., head - 63::2] = both
        y = o.rope_heads(y, np_(pos), head, theta)
    return y, tol


def _check_linear(T, N, K, out, head=0, seed=0, theta=10000.0, x=None, xs=None, w=None, ws=None, extra=0, w_ready=False):
    dev = need_gpu()
    g = _gen(dev, seed)
    if x is None:
        x, xs = _codes((T, K), g, dev, 1)
    if w is None:
        w, ws = _codes((N, K), g, dev, 128)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device=dev, dtype=torch.int32) if head else None
    kind = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.uint8}[out]
    big = torch.full((T + 1, N + extra), 77, dtype=kind, device=dev)
    osc = torch.full((T + 1, N // 128 + 2), -5.0, device=dev) if out == "fp8" else None
    csa2.fp8_linear(x, xs, w, ws, big[:T, :N], out_scale=osc[:T, :N // 128] if out == "fp8" else None, row_pos=pos,
                    rope_head=head, rope_theta=theta, w_ready=w_ready)
    _sync_ok()
    y, tol = _linear_ref(x, xs, w, ws, pos, head, theta)
    got = np_(big.float() if out == "bf16" else big)
    assert (got[T:] == 77).all() and (got[:T, N:] == 77).all(), "written outside the output"
    got = got[:T, :N]
    if out == "fp8":
        s, _ = o.e4m3_block_scales(y, 1)
        gs = np_(osc).astype(np.float64)
        assert (gs[T:] == -5).all() and (gs[:T, N // 128:] == -5).all()
        gs = gs[:T, :N // 128]
        top = tol.reshape(T, -1, 128).max(axis=2)
        assert np.all(np.abs(gs - s) <= (top / 448.0 + 4 * U * s)), "scales"
        gsx = o.expand_blocks(gs, 1, T, N)
        d = o.fp8_e4m3_table()[got] * gsx
        half = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * gsx)
        slack = tol + o.expand_blocks(top, 1, T, N) + 4 * U * np.abs(y)   # value and scale errors
        assert np.all(np.abs(d - y) <= half + 1.2 * slack), f"codes: worst {np.abs(d - y).max()}"
    else:
        step = {"fp32": U, "bf16": 2.0 ** -8}[out]
        bad = np.abs(got - y) > step * (np.abs(y) + tol) + tol
        assert not bad.any(), f"T={T} N={N} K={K} {out}: {bad.sum()} outside, worst {np.abs(got - y).max()}"


SHAPES = [(1, 1, 16), (1, 512, 7168), (2, 130, 144), (7, 1001, 1360), (8, 4096, 2048), (16, 256, 128), (17, 384, 4112),
          (33, 640, 640), (64, 512, 7168), (65, 96, 2000), (128, 128, 256), (129, 257, 400), (200, 1024, 1024),
          (333, 1001, 1360), (512, 512, 7168), (1000, 300, 272), (1300, 1001, 2064), (1300, 1000, 2192), (2500, 300, 1040), (2700, 2001, 400), (2700, 2000, 144)]


@pytest.mark.parametrize("T,N,K", SHAPES)
@pytest.mark.parametrize("out", ["fp32", "bf16"])
def test_fp8_linear_matches_oracle(T, N, K, out):
    _check_linear(T, N, K, out, seed=T + N + K, extra=0 if (T + N) % 2 else 24)


@pytest.mark.parametrize("T,N,K,out,head", [
    (1, 128, 128, "fp8", 0), (8, 4096, 2048, "fp8", 128), (3, 1024, 144, "bf16", 512), (130, 512, 272, "fp8", 0),
    (130, 768, 1040, "fp8", 128), (16, 1024, 2048, "fp8", 512), (33, 512, 640, "fp8", 256), (40, 1536, 528, "fp32", 256),
    (257, 2048, 512, "bf16", 512), (300, 640, 2048, "fp8", 128), (700, 4096, 384, "fp8", 128), (90, 384, 784, "bf16", 128),
    (1300, 1024, 2064, "fp8", 128), (1300, 1152, 2192, "bf16", 384), (1300, 4096, 272, "fp8", 128), (1411, 4352, 1040, "bf16", 256),
])
def test_fp8_linear_rope_and_e4m3_output(T, N, K, out, head):
    _check_linear(T, N, K, out, head, seed=T * N + K, extra=32)


@pytest.mark.parametrize("T", [6, 1300])
def test_fp8_linear_rope_far_positions_and_other_thetas(T):
    """Positions up to 2^31 - 1 (the float64 angle is off by under 2^-21 there); the thetas in
    turn, as a thread keeps the last one's rates."""
    dev = need_gpu()
    g = _gen(dev, 17)
    x, xs = _codes((T, 272), g, dev, 1)
    w, ws = _codes((1024, 272), g, dev, 128)
    pos = torch.randint(2 ** 31 - 5000, 2 ** 31 - 1, (T,), generator=g, device=dev, dtype=torch.int64).to(torch.int32)
    outs = {}
    for theta in (500000.0, 0.0, 10000.0, 500000.0):
        out = torch.empty(T, 1024, device=dev)
        csa2.fp8_linear(x, xs, w, ws, out, row_pos=pos, rope_head=512, rope_theta=theta)
        if theta in outs:
            assert torch.equal(out, outs[theta])
        outs[theta] = out
    _sync_ok()
    assert torch.equal(outs[0.0], outs[10000.0]) and not torch.equal(outs[0.0], outs[500000.0])
    for theta in (10000.0, 500000.0):
        y, tol = _linear_ref(x, xs, w, ws, pos, 512, theta)
        z = np.abs(y).reshape(T, -1, 512)
        extra = np.zeros_like(z)
        extra[..., 448::2] = extra[..., 449::2] = 2.0 ** -21 * 1.5 * (z[..., 448::2] + z[..., 449::2])
        assert np.all(np.abs(np_(outs[theta]) - y) <= tol + extra.reshape(T, -1) + U * np.abs(y))


@pytest.mark.parametrize("T", [16, 300])
def test_fp8_linear_padded_rows_stay_in_their_rows(T):
    """Rows that batch_plan pads (position -1) change no other row."""
    dev = need_gpu()
    g = _gen(dev, 18)
    x, xs = _codes((T, 512), g, dev, 1)
    w, ws = _codes((512, 512), g, dev, 128)
    pos = torch.arange(T, dtype=torch.int32, device=dev)
    a, b = torch.empty(T, 512, device=dev), torch.empty(T, 512, device=dev)
    csa2.fp8_linear(x, xs, w, ws, a, row_pos=pos, rope_head=128)
    pos[T // 2:] = -1
    csa2.fp8_linear(x, xs, w, ws, b, row_pos=pos, rope_head=128)
    _sync_ok()
    assert torch.equal(a[:T // 2], b[:T // 2]) and torch.isfinite(b).all()


def test_fp8_linear_prefill_width_rows():
    """A prefill chunk's attention query projection, on sampled rows (the oracle takes whole rows)."""
    dev = need_gpu()
    g = _gen(dev, 5)
    T, N, K = 4096, 32768, 2048
    x, xs = _codes((T, K), g, dev, 1)
    w, ws = _codes((N, K), g, dev, 128)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device=dev, dtype=torch.int32)
    out = torch.empty(T, N, dtype=torch.bfloat16, device=dev)
    csa2.fp8_linear(x, xs, w, ws, out, row_pos=pos, rope_head=512)
    _sync_ok()
    pick = torch.tensor([0, 1, 127, 128, 2049, 4095], device=dev)
    y, tol = _linear_ref(x[pick], xs[pick], w, ws, pos[pick], 512, 10000.0)
    got = np_(out[pick].float())
    assert np.all(np.abs(got - y) <= 2.0 ** -8 * (np.abs(y) + tol) + tol)


def test_fp8_linear_takes_strided_rows():
    dev = need_gpu()
    g = _gen(dev, 11)
    x, xs = _codes((50, 512), g, dev, 1)
    w, ws = _codes((300, 640), g, dev, 128)
    xs3 = torch.full((50, 7), 9.0, device=dev)
    xs3[:, :3] = xs[:, :3]
    ws4 = torch.full((3, 8), 9.0, device=dev)
    ws4[:, :3] = ws[:, :3]
    _check_linear(50, 300, 272, "bf16", x=x[:, :272], xs=xs3[:, :3], w=w[:, 16:288], ws=ws4[:, :3])
    # every second row of a wider matrix
    _check_linear(25, 300, 272, "fp32", x=x[::2, :272], xs=xs3[::2, :3], w=w[:, :272], ws=ws4[:, :3])


@pytest.mark.parametrize("T", [3, 40, 300])
def test_fp8_linear_nan_and_infinity_stay_in_their_rows(T):
    dev = need_gpu()
    g = _gen(dev, 12)
    x, xs = _codes((T, 400), g, dev, 1)
    w, ws = _codes((256, 400), g, dev, 128)
    clean = torch.empty(T, 256, device=dev)
    csa2.fp8_linear(x, xs, w, ws, clean)
    x2, xs2 = x.clone(), xs.clone()
    x2[0, 399] = 0x7F                       # NaN code
    xs2[1, 2] = float("inf")
    xs2[2, 0] = 0.0
    got = torch.empty(T, 256, device=dev)
    csa2.fp8_linear(x2, xs2, w, ws, got)
    codes, sc = torch.empty(T, 256, dtype=torch.uint8, device=dev), torch.empty(T, 2, device=dev)
    csa2.fp8_linear(x2, xs2, w, ws, codes, out_scale=sc)
    _sync_ok()
    assert torch.isnan(got[0]).all() and not torch.isfinite(got[1]).any() and torch.isfinite(got[2]).all()
    assert torch.equal(got[3:], clean[3:])
    assert (codes[:2] == 0x7F).all() and (sc[:2] == 1).all() and not ((codes[2:] & 0x7F) == 0x7F).any()


def test_fp8_linear_zero_weights_give_zero_codes():
    dev = need_gpu()
    x, xs = _codes((9, 256), _gen(dev, 1), dev, 1)
    w, ws = torch.zeros(128, 256, dtype=torch.uint8, device=dev), torch.ones(1, 2, device=dev)
    codes, sc = torch.full((9, 128), 3, dtype=torch.uint8, device=dev), torch.zeros(9, 1, device=dev)
    csa2.fp8_linear(x, xs, w, ws, codes, out_scale=sc)
    _sync_ok()
    assert not (codes & 0x7F).any() and (sc == 1).all()


@pytest.mark.parametrize("T", [8, 256])
def test_fp8_linear_is_repeatable(T):
    dev = need_gpu()
    g = _gen(dev, 13)
    x, xs = _codes((T, 7168), g, dev, 1)
    w, ws = _codes((512, 7168), g, dev, 128)
    outs = [torch.empty(T, 512, device=dev) for _ in range(3)]
    for y in outs:
        csa2.fp8_linear(x, xs, w, ws, y)
    _sync_ok()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("T", [12, 50, 700])
def test_fp8_linear_on_two_streams_and_in_a_graph(T):
    dev = need_gpu()
    g = _gen(dev, 14)
    x, xs = _codes((T, 1024), g, dev, 1)
    w, ws = _codes((4096, 1024), g, dev, 128)
    want = torch.empty(T, 4096, device=dev)
    csa2.fp8_linear(x, xs, w, ws, want)
    torch.cuda.synchronize()
    a, b = torch.empty_like(want), torch.empty_like(want)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        with torch.cuda.stream(s1):
            csa2.fp8_linear(x, xs, w, ws, a)
        csa2.fp8_linear(x, xs, w, ws, b, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)
    # captured: quantise, project; the weights' codes are not the previous launch's
    h = torch.randn(T, 1024, generator=g, device=dev).to(torch.bfloat16)
    codes, sc, y = torch.empty_like(x), torch.empty_like(xs), torch.empty_like(want)
    with torch.cuda.stream(s1):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s1):
            csa2.quant_fp8(h, codes, sc)
            csa2.fp8_linear(codes, sc, w, ws, y, w_ready=True)
    for k in range(3):
        h.copy_(torch.randn(T, 1024, generator=g, device=dev))
        gr.replay()
        torch.cuda.synchronize()
        y2 = torch.empty_like(want)
        c2, s2_ = torch.empty_like(x), torch.empty_like(xs)
        csa2.quant_fp8(h, c2, s2_)
        csa2.fp8_linear(c2, s2_, w, ws, y2)
        torch.cuda.synchronize()
        assert torch.equal(codes, c2) and torch.equal(y, y2)


def test_quantise_weights_then_project_at_once():
    """Weights quantised by the launch before the projection, without w_ready."""
    dev = need_gpu()
    g = _gen(dev, 15)
    h = torch.randn(16, 2048, generator=g, device=dev).to(torch.bfloat16)
    hc, hs = torch.empty(16, 2048, dtype=torch.uint8, device=dev), torch.empty(16, 16, device=dev)
    csa2.quant_fp8(h, hc, hs)
    for k in range(4):
        wt = (torch.randn(8192, 2048, generator=g, device=dev) * (k + 1)).to(torch.bfloat16)
        wc, ws = torch.empty(8192, 2048, dtype=torch.uint8, device=dev), torch.empty(64, 16, device=dev)
        y = torch.empty(16, 8192, device=dev)
        csa2.quant_fp8(wt, wc, ws, block_rows=128)
        csa2.fp8_linear(hc, hs, wc, ws, y)
        _sync_ok()
        ref, tol = _linear_ref(hc, hs, wc, ws, None, 0, 0.0)
        assert np.all(np.abs(np_(y) - ref) <= U * np.abs(ref) + tol)


# ---------------------------------------------------------------- the batch's arrays
def _plan_run(ctx, new, m, table=None, free=None, head=None, ring=0, ring_id=None, n_swa=128, cap=None, ecap=None, pad=False):
    dev = need_gpu()
    B = len(ctx)

    def t(v):
        return None if v is None else torch.tensor(np.asarray(v), dtype=torch.int32, device=dev)

    cap = sum(max(n, 0) for n in new) if cap is None else cap
    ecap = cap if ecap is None else ecap
    o_ = {"row_start": (B + 1,), "row_seq": (cap,), "row_pos": (cap,), "n_visible": (B,), "entry_start": (B + 1,),
          "entry_pos": (ecap,), "entry_row": (ecap,)}
    if table is not None:
        o_["entry_slot"] = (ecap,)
    if free is not None:
        o_["free_head_out"] = (1,)
    if ring:
        o_["swa_new"], o_["swa_slot"] = (cap,), (cap, n_swa)
    bufs = {k: torch.full(s, -77, dtype=torch.int32, device=dev) for k, s in o_.items()}
    pt = t(table)
    csa2.batch_plan(t(ctx), t(new), m, page_table=pt, free_pages=t(free), free_head=t(None if head is None else [head]),
                    swa_ring=ring, ring_id=t(ring_id), pad=pad, **bufs)
    torch.cuda.synchronize()
    rc = csa2.check_device_error()
    return {k: np_(v) for k, v in bufs.items()}, None if pt is None else np_(pt), rc


def _plan_check(ctx, new, m, table=None, free=None, head=None, ring=0, ring_id=None, n_swa=128, cap=None, ecap=None,
                pad=False):
    got, pt, rc = _plan_run(ctx, new, m, table, free, head, ring, ring_id, n_swa, cap, ecap, pad)
    want, wpt, bad = o.batch_plan(ctx, new, m, table, free, head or 0, ring, ring_id, n_swa)
    for k, v in got.items():
        w = np.array(want[k], dtype=np.int64).reshape((-1,) + v.shape[1:])
        n = min(len(w), len(v))
        bad = bad or len(w) > len(v)
        assert np.array_equal(v[:n], w[:n]), k
        assert (v[n:] == ((0 if k == "entry_pos" else -1) if pad else -77)).all(), f"{k} behind the last"
    if pt is not None:
        assert np.array_equal(pt, wpt)
    assert rc == (6 if bad else 0)


def _batch(B, max_ctx, max_new, m, seed, zero=0.2):
    r = np.random.default_rng(seed)
    ctx, new = r.integers(0, max_ctx + 1, B), r.integers(0, max_new + 1, B)
    new[r.random(B) < zero] = 0
    stride = (max_ctx + max_new) // m // 64 + 1
    pages = r.permutation(B * stride * 2)
    table = np.full((B, stride), -1)
    for b in range(B):
        held = -(-(ctx[b] // m) // 64)
        table[b, :held] = pages[b * stride:b * stride + held]
    return ctx.tolist(), new.tolist(), table, pages[B * stride:], r.permutation(B).tolist()


@pytest.mark.parametrize("B,max_ctx,max_new,m", [(1, 0, 1, 1), (1, 70, 300, 2), (8, 5000, 1, 1), (8, 5000, 1, 2), (33, 700, 40, 2),
                                                 (257, 300, 9, 1), (1000, 90, 3, 2), (8192, 20, 1, 1), (3, 10, 700, 1)])
def test_batch_plan_matches_oracle(B, max_ctx, max_new, m):
    ctx, new, table, free, rid = _batch(B, max_ctx, max_new, m, seed=B + max_new)
    _plan_check(ctx, new, m, table, free, 5, 127 + max_new, rid)
    _plan_check(ctx, new, m, table, free, None, 127 + max_new, None, cap=sum(new) + 70, ecap=sum(new) + 3, pad=False)
    _plan_check(ctx, new, m, table, free, 0, 63 + max_new, rid, n_swa=64, cap=sum(new) + 70, pad=True)
    _plan_check(ctx, new, m, table, free, 0, 12 + max_new, rid, n_swa=13)


def test_batch_plan_without_a_free_list_reads_the_table():
    r = np.random.default_rng(3)
    table = r.permutation(40).reshape(4, 10)
    _plan_check([0, 64, 100, 319], [64, 1, 200, 0], 1, table)
    _plan_check([1, 127, 128, 639], [1, 1, 1, 1], 2, table, ring=128)
    _plan_check([7, 8], [3, 4], 2)                                    # rows and entries only


def test_batch_plan_resting_batch_and_nothing_visible():
    _plan_check([0, 0, 0], [0, 0, 0], 2, np.full((3, 1), -1), [], None, 128, cap=4, pad=True)
    _plan_check([0, 1], [1, 0], 2, np.full((2, 1), -1), [3], 0, 128)  # one token of two: no entry yet


@pytest.mark.parametrize("case", [
    dict(ctx=[5, -3], new=[2, 2], m=1), dict(ctx=[5, 3], new=[2, -2], m=1), dict(ctx=[2 ** 31 - 2, 3], new=[2, 1], m=1),
    dict(ctx=[0], new=[129], m=1, table=np.full((1, 2), -1), free=[4, 5, 6]),       # past the table
    dict(ctx=[0, 60], new=[65, 9], m=1, table=np.array([[-1, -1], [9, -1]]), free=[4, 5], head=0),  # list ends
    dict(ctx=[0], new=[5], m=1, table=np.full((1, 1), -1), free=[4], head=1),
    dict(ctx=[70], new=[1], m=1, table=np.full((1, 2), -1)),                        # a held page is missing
    dict(ctx=[200, 3], new=[9, 1], m=1, ring=135), dict(ctx=[200, 3], new=[9, 1], m=1, ring=5),
    dict(ctx=[200, 3], new=[1, 1], m=1, ring=128, ring_id=[0, -1]),
    dict(ctx=[200, 3], new=[1, 1], m=1, ring=1 << 20, ring_id=[2048, 0]),           # slots past INT32_MAX
    dict(ctx=[200, 3], new=[9, 4], m=2, cap=7, ecap=2, ring=200),                   # more rows and entries than room
])
def test_batch_plan_records_what_does_not_fit(case):
    _plan_check(**{"n_swa": 128, **case})
    assert csa2.check_device_error() == 0


def test_batch_plan_in_a_graph_follows_the_lengths():
    dev = need_gpu()
    B, cap, m = 6, 24, 1
    ctx = torch.tensor([0, 63, 64, 100, 5, 7], dtype=torch.int32, device=dev)
    new = torch.ones(B, dtype=torch.int32, device=dev)
    table = torch.full((B, 8), -1, dtype=torch.int32, device=dev)
    table[:, :2] = torch.arange(12, dtype=torch.int32, device=dev).view(6, 2)
    table0 = table.clone()
    free = torch.arange(100, 130, dtype=torch.int32, device=dev)
    head, head2 = torch.zeros(1, dtype=torch.int32, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    seq, pos, slot = (torch.full((cap,), -9, dtype=torch.int32, device=dev) for _ in range(3))
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            csa2.batch_plan(ctx, new, m, page_table=table, free_pages=free, free_head=head, free_head_out=head2,
                            row_seq=seq, row_pos=pos, entry_slot=slot, pad=True)
            head.copy_(head2)
            ctx.add_(new)
    c, t, h = [0, 63, 64, 100, 5, 7], np_(table0), 0
    for n in ([1] * 6, [0, 4, 2, 0, 9, 1], [0] * 6, [3] * 6):
        new.copy_(torch.tensor(n, dtype=torch.int32))
        gr.replay()
        torch.cuda.synchronize()
        want, t, bad = o.batch_plan(c, n, m, t, np_(free), h)
        assert not bad and csa2.check_device_error() == 0
        k = sum(n)
        assert np_(seq)[:k].tolist() == want["row_seq"] and np_(pos)[:k].tolist() == want["row_pos"]
        assert np_(slot)[:k].tolist() == want["entry_slot"] and (np_(seq)[k:] == -1).all() and (np_(slot)[k:] == -1).all()
        assert np.array_equal(np_(table), t)
        c, h = [a + b for a, b in zip(c, n)], want["free_head_out"][0]


@pytest.mark.parametrize("first,W", [(0, 64), (4, 64), (3, 64), (1, 30)])
def test_batch_plan_writes_a_strided_window(first, W):
    dev = need_gpu()
    i32 = dict(dtype=torch.int32, device=dev)
    wide = torch.full((50, 80), -7, **i32)
    ctx, new = [0, 100, 17, 3], [9, 20, 0, 11]
    csa2.batch_plan(torch.tensor(ctx, **i32), torch.tensor(new, **i32), 1, swa_ring=90, swa_slot=wide[:, first:first + W])
    _sync_ok()
    want = np.array(o.batch_plan(ctx, new, 1, ring=90, n_swa=W)[0]["swa_slot"])
    got = np_(wide)
    assert np.array_equal(got[:40, first:first + W], want)
    assert (got[40:] == -7).all() and (got[:, :first] == -7).all() and (got[:, first + W:] == -7).all()


def test_batch_plan_more_rows_than_31_bits_count():
    dev = need_gpu()
    i32 = dict(dtype=torch.int32, device=dev)
    big = 2 ** 31 - 1
    start, seq, pos = torch.zeros(4, **i32), torch.full((40,), -9, **i32), torch.full((40,), -9, **i32)
    csa2.batch_plan(torch.tensor([0, 0, 5], **i32), torch.tensor([big, big, 1], **i32), 2, row_start=start, row_seq=seq, row_pos=pos)
    torch.cuda.synchronize()
    assert csa2.check_device_error() == 6
    assert np_(start).tolist() == [0, big, big, big] and (np_(seq) == 0).all() and np_(pos).tolist() == list(range(40))


def test_decode_step_finds_its_newest_entries():
    dev = need_gpu()
    from serving_lightning_indexer_gb300.decode_step import DecodeStep
    lengths = [4096, 130, 64, 2]
    step = DecodeStep(lengths, seed=3, device=dev, layers=(2, 20))
    torch.cuda.synchronize()
    assert csa2.check_device_error() == 0
    for ci, m in ((0, 2), (3, 1)):
        c = step.caches[ci]
        pt = np_(c.pc.page_table)
        e = [n // m - 1 for n in lengths]
        assert np_(c.entry_slot_new).tolist() == [int(pt[b, x // 64]) * 64 + x % 64 for b, x in enumerate(e)]
        assert np_(c.entry_pos_new).tolist() == [x * m for x in e]


@pytest.mark.parametrize("T", [24, 2200])
def test_offsets_past_32_bits(T):
    """Rows 2^20 elements apart (T = 2200: the last ones past 2^31 elements), and T = 24 rows 2^27 apart."""
    dev = need_gpu()
    g = _gen(dev, 31)
    ld = 1 << (20 if T == 2200 else 27)
    K, N = 272, 96
    hidden = torch.empty(T * ld, dtype=torch.bfloat16, device=dev).view(T, ld)[:, :K]
    hidden.copy_(torch.randn(T, K, generator=g, device=dev))
    codes = torch.empty(T * ld, dtype=torch.uint8, device=dev).view(T, ld)[:, 64:64 + K]
    scale = torch.empty(T, 3, device=dev)
    csa2.quant_fp8(hidden, codes, scale)
    w, ws = _codes((N, K), g, dev, 128)
    out = torch.empty(T * ld, dtype=torch.bfloat16, device=dev).view(T, ld)[:, 128:128 + N]
    csa2.fp8_linear(codes, scale, w, ws, out)
    _sync_ok()
    c2, s2, o2 = torch.empty(T, K, dtype=torch.uint8, device=dev), torch.empty(T, 3, device=dev), torch.empty(T, N, dtype=torch.bfloat16, device=dev)
    csa2.quant_fp8(hidden.contiguous(), c2, s2)
    csa2.fp8_linear(c2, s2, w, ws, o2)
    _sync_ok()
    assert torch.equal(codes.contiguous(), c2) and torch.equal(scale, s2) and torch.equal(out.contiguous(), o2)
    y, tol = _linear_ref(c2, s2, w, ws, None, 0, 0.0)
    assert np.all(np.abs(np_(o2.float()) - y) <= 2.0 ** -8 * (np.abs(y) + tol) + tol)


# ---------------------------------------------------------------- together, as a step uses them
def test_a_step_from_lengths_and_hidden_states():
    """Two decode steps of three sequences: batch_plan, quant_fp8 and fp8_linear make every
    input of the entry build, the indexer, the selection and the attention."""
    dev = need_gpu()
    g = _gen(dev, 21)
    B, H, m = 3, 1024, 1
    lengths = [700, 64, 1500]
    pc = W.make_paged_cache(lengths, seed=5, device=dev)
    pages = pc.index_k.shape[0]
    ik = torch.cat([pc.index_k, torch.zeros(8, 8448, dtype=torch.uint8, device=dev)])
    mk = torch.cat([pc.main_kv, torch.zeros(8 * 64, 288, dtype=torch.uint8, device=dev)])
    table = torch.full((B, 32), -1, dtype=torch.int32, device=dev)
    table[:, :pc.page_table.shape[1]] = pc.page_table
    free = torch.arange(pages, pages + 8, dtype=torch.int32, device=dev)
    al = W.make_attn_layer(B, seed=6, device=dev)

    def weights(n):
        wc, ws = torch.empty(n, H, dtype=torch.uint8, device=dev), torch.empty(-(-n // 128), H // 128, device=dev)
        csa2.quant_fp8((torch.randn(n, H, generator=g, device=dev) / 32).to(torch.bfloat16), wc, ws, block_rows=128)
        return wc, ws

    w_kv, w_iq, w_q = weights(512), weights(32 * 128), weights(64 * 512)
    w_ik, k_gamma = W.make_index_projection(seed=8, device=dev)
    gamma, norm = torch.ones(512, device=dev), torch.ones(H, device=dev)
    iw = torch.randn(B, 32, generator=g, device=dev)
    i32 = dict(dtype=torch.int32, device=dev)
    ctx, new = torch.tensor(lengths, **i32), torch.ones(B, **i32)
    head, head2 = torch.zeros(1, **i32), torch.zeros(1, **i32)
    seq, pos, vis, slot, epos, erow = (torch.empty(B, **i32) for _ in range(6))
    swa_new, swa_slot = torch.empty(B, **i32), torch.empty(B, 128, **i32)
    for step in range(2):
        h = torch.randn(B, H, generator=g, device=dev).to(torch.bfloat16)
        csa2.batch_plan(ctx, new, m, page_table=table, free_pages=free, free_head=head, free_head_out=head2, row_seq=seq,
                        row_pos=pos, n_visible=vis, entry_slot=slot, entry_pos=epos, entry_row=erow, swa_ring=128,
                        swa_new=swa_new, swa_slot=swa_slot)
        hc, hs = torch.empty(B, H, dtype=torch.uint8, device=dev), torch.empty(B, H // 128, device=dev)
        csa2.quant_fp8(h, hc, hs, gamma=norm)
        Cm = torch.empty(B, 512, dtype=torch.bfloat16, device=dev)
        csa2.fp8_linear(hc, hs, *w_kv, Cm)
        q8, qs = torch.empty(B, 32 * 128, dtype=torch.uint8, device=dev), torch.empty(B, 32, device=dev)
        csa2.fp8_linear(hc, hs, *w_iq, q8, out_scale=qs, row_pos=pos, rope_head=128)
        q = torch.empty(B, 64 * 512, dtype=torch.bfloat16, device=dev)
        csa2.fp8_linear(hc, hs, *w_q, q, row_pos=pos, rope_head=512, w_ready=True)
        csa2.compress_m2(Cm, None, m, gamma, mk, entry_slot=slot, entry_pos=epos, w_ik=w_ik, k_gamma=k_gamma, index_k=ik)
        r = csa2.rows(B, B, row_seq=seq, n_visible=vis)
        scores = torch.empty(B, 1536, device=dev)
        csa2.index_score(q8.view(B, 32, 128), qs, iw, ik, table, r, scores)
        tp, ts = torch.empty(B, 512, **i32), torch.empty(B, 512, **i32)
        csa2.topk_with_candidates(scores, r, 512, tp, ts, table)
        out = torch.empty(B, 64, 512, device=dev)
        csa2.sparse_attn(q.view(B, 64, 512), mk, ts, al.swa_kv, swa_slot, al.sink, out, q_pos=pos, out_inv_rope=True)
        _sync_ok()
        lengths = [n + 1 for n in lengths]
        assert np_(vis).tolist() == lengths and np_(pos).tolist() == [n - 1 for n in lengths]
        pt = np_(table)
        assert np_(slot).tolist() == [int(pt[b, (n - 1) // 64]) * 64 + (n - 1) % 64 for b, n in enumerate(lengths)]
        kv = o.kv_project(o.fp8_e4m3_table()[np_(hc)] * o.expand_blocks(np_(hs).astype(np.float64), 1, B, H),
                          (o.fp8_e4m3_table()[np_(w_kv[0])] * o.expand_blocks(np_(w_kv[1]).astype(np.float64), 128, 512, H)).T)
        assert np.abs(np_(Cm.float()) - kv).max() <= 2.0 ** -8 * np.abs(kv).max() * 1.01
        for b, n in enumerate(lengths):
            ref = o.index_scores_row(np_(q8).reshape(B, 32, 128)[b], np_(qs)[b], np_(iw)[b], np_(ik), pt[b], n)
            got = np_(scores)[b, :n].astype(np.float64)
            assert np.all(np.abs(got - ref) <= 1e-3 * np.maximum(np.abs(ref), 1e-2 * np.sqrt((ref ** 2).mean())))
            assert n - 1 in np_(tp)[b].tolist() or n > 512
            oo, _ = o.attention_row(np_(q.view(B, 64, 512)[b].float()).astype(np.float64), np_(mk), np_(ts)[b], np_(al.swa_kv),
                                    np_(swa_slot)[b], np_(al.sink).astype(np.float64), 512 ** -0.5, q_pos=n - 1,
                                    inv_rope_theta=10000.0)
            assert np.abs(np_(out)[b] - oo).max() <= 2e-2
        ctx.add_(new)
        head.copy_(head2)
    assert np_(head)[0] == 1   # the second sequence's 65th entry took one page
