"""GPU parity of the calls around the layers: csa2_add_norm_fp8, csa2_lora_linear and
csa2_logprobs against the float64 oracle.

Tolerances, from the arithmetic (u = 2^-24, half a step of fp32):
  * the residual: the sum of a bf16 and a bf16 or fp32 value is rounded once to fp32,
    and where it is rounded again to bf16 the first rounding cannot reach a border
    (the terms' 8 bits leave the sum exact in 24 wherever it comes near one): equal.
  * the norm: a thread's 16 V squares (V = 1, 2, 4), 5 shuffle steps, 8 warps, the
    division and eps are 16 V + 16 roundings of a sum of positive terms, half of that
    after the root; root, reciprocal and two products 4 more: e = (8 V + 12) u.  A
    code's value adds its block's maximum (e) and factor and product (2 u).
  * an inner product v: 128 products of a block, exact in fp32, and blocks in at most
    150 + blocks / 16 roundings; then its bf16 value, 2^-8 of it, or two, 2^-16, or
    three, 2^-24.
  * an adapter's addition: exact products, at most 2 rank + 8 roundings; the whole sum
    those of csa2_fp8_linear and one for each of the parts that are added (at most 40
    here).  RoPE and the output's step as for csa2_fp8_linear.
  * R = sum e^d and W = sum d e^d over all but the largest logit, d = x - M <= 0, with
    Q = sum d^2 e^d: a term's exponent has two roundings (2 u |d|), its rescalings as
    many (they add up to |d| at most), and ex2 2^-22; a term and a rescaling factor, a
    thread's additions and the merges are c = elements of a thread + 8 batches + 100
    more.  So dR <= u (4 |W| + c R), dW <= u (4 Q + c |W|).
"""
import numpy as np
import pytest
import torch

from gpu_util import need_gpu, np_
from oracle import csa2_oracle as o
from serving_lightning_indexer_gb300 import csa2
from test_gpu_inputs import U, _assert_codes, _codes, _decode, _gen, _sync_ok

pytestmark = pytest.mark.gpu
INF = float("inf")
FP32_END = 2.0 ** 128 - 2.0 ** 103   # rounds to infinity, and everything above it


def f64(t):
    return np_(t.float()).astype(np.float64)


# ---------------------------------------------------------------- residual, norm, codes
def _norm_case(T, K, kind, seed, extra=0):
    dev = need_gpu()
    g = _gen(dev, seed)
    x = (0.5 * torch.randn(T, K + extra, generator=g, device=dev)).to(torch.bfloat16)[:, :K]
    res = torch.randn(T, K + extra, generator=g, device=dev)
    res[:, ::37] *= 20.0
    gamma = 1.0 + 0.1 * torch.randn(K, generator=g, device=dev)
    return dev, x, res.to(kind)[:, :K], gamma


def _check_norm(x, res, gamma, eps, r_out, codes, scale, y):
    T, K = x.shape
    V = 1 if K <= 4096 else (2 if K <= 8192 else 4)
    e = (8 * V + 12) * U
    r, want = o.add_norm_rows(f64(x), np_(res.double()), f64(gamma), eps, fp32=res.dtype == torch.float32)
    assert np.array_equal(np_(r_out.double()), r)
    if y is not None:
        assert np.all(np.abs(f64(y) - want) <= (2.0 ** -8 * (1 + e) + e) * np.abs(want))
    if codes is not None:
        s, m = o.e4m3_block_scales(want, 1)
        assert np.all(np.abs(np_(scale) - s) <= (e + 2 * U) * s)
        _assert_codes(np_(codes), want * o.expand_blocks(m, 1, T, K), 2 * e + 2 * U, "add_norm")


@pytest.mark.parametrize("T,K", [(1, 16), (3, 144), (8, 7168), (17, 512), (5, 528), (4, 1024), (2, 4096), (2, 4112), (3, 8192),
                                 (3, 8208), (2, 16384), (1003, 2064), (300, 7168)])
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_add_norm_matches_oracle(T, K, kind):
    dev, x, res, gamma = _norm_case(T, K, kind, T + K, extra=48)
    nb = -(-K // 128)
    r_out = torch.full((T + 1, K + 16), 3.0, dtype=kind, device=dev)
    codes = torch.full((T + 1, K + 32), 0x55, dtype=torch.uint8, device=dev)
    scale = torch.full((T + 1, nb + 3), -1.0, device=dev)
    y = torch.full((T + 1, K + 8), 5.0, dtype=torch.bfloat16, device=dev)
    csa2.add_norm_fp8(x, res, r_out[:T, :K], gamma, codes=codes[:T, :K], scale=scale[:T, :nb], y=y[:T, :K], eps=1e-5)
    _sync_ok()
    _check_norm(x, res, gamma, 1e-5, r_out[:T, :K], codes[:T, :K], scale[:T, :nb], y[:T, :K])
    for t, fill in ((r_out, 3.0), (y, 5.0)):     # nothing outside is touched
        assert (t[T:] == fill).all() and (t[:T, K:] == fill).all()
    assert (codes[T:] == 0x55).all() and (codes[:T, K:] == 0x55).all() and (scale[T:] == -1).all() and (scale[:T, nb:] == -1).all()


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,K", [(6, 640), (9, 7168)])
def test_add_norm_in_place_and_each_output_alone(T, K, kind):
    dev, x, res, gamma = _norm_case(T, K, kind, 3)
    full = [torch.empty(T, K, dtype=kind, device=dev), torch.empty(T, K, dtype=torch.uint8, device=dev),
            torch.empty(T, -(-K // 128), device=dev), torch.empty(T, K, dtype=torch.bfloat16, device=dev)]
    csa2.add_norm_fp8(x, res, full[0], gamma, codes=full[1], scale=full[2], y=full[3])
    here, codes, scale, y = res.clone(), torch.empty_like(full[1]), torch.empty_like(full[2]), torch.empty_like(full[3])
    csa2.add_norm_fp8(x, here, here, gamma, codes=codes, scale=scale)
    assert torch.equal(here, full[0]) and torch.equal(codes, full[1]) and torch.equal(scale, full[2])
    here = res.clone()
    csa2.add_norm_fp8(x, here, here, gamma, y=y)
    _sync_ok()
    assert torch.equal(here, full[0]) and torch.equal(y, full[3])
    # the codes are those of csa2_quant_fp8 on the stored residual
    if kind is torch.bfloat16:
        csa2.quant_fp8(here, codes, scale, gamma=gamma)
        _sync_ok()
        v, s = o.add_norm_rows(f64(x), f64(res), f64(gamma), 1e-6)[1], np_(scale).astype(np.float64)
        assert np.all(np.abs(s - np_(full[2])) <= 100 * U * s) and v.shape == (T, K)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,K,unit", [(2000, 1040, False), (600, 7168, False), (300, 16384, False), (700, 528, True), (100, 7168, True)])
def test_add_norm_codes_are_the_exact_quotients(T, K, unit, kind):
    """Codes of r * gamma * 448 / a, a the block's largest |r * gamma|, rounded to fp32 and no
    more before the code: every code is that of the quotient in 64 bits (2^-52 off), or of
    what is 2^-40 less or more of it, where the kernel's two-part products are 2^-45 off.
    With gamma of ones and bf16 r many lie on a border."""
    dev, x, res, gamma = _norm_case(T, K, kind, T)
    if unit:
        gamma.fill_(1.0)
    nb = -(-K // 128)
    r, codes, scale = torch.empty_like(res), torch.empty(T, K, dtype=torch.uint8, device=dev), torch.empty(T, nb, device=dev)
    csa2.add_norm_fp8(x, res, r, gamma, codes=codes, scale=scale)
    _sync_ok()
    v = torch.nn.functional.pad(r.double() * gamma.double(), (0, nb * 128 - K)).view(T, nb, 128)
    q = (v * 448.0 / v.abs().amax(-1, keepdim=True)).view(T, -1)[:, :K]
    less, want, more = ((q * (1.0 + d)).clamp(-448.0, 448.0).float().to(torch.float8_e4m3fn).float()
                        for d in (-2.0 ** -40, 0.0, 2.0 ** -40))
    got = codes.view(torch.float8_e4m3fn).float()
    assert bool(((got == less) | (got == want) | (got == more)).all())
    assert int((got != want).sum()) <= 2 and int((less != more).sum()) <= 2 + q.numel() * (2.0 ** -7 if unit else 2.0 ** -18)


def test_add_norm_special_rows():
    dev = need_gpu()
    x = torch.zeros(6, 256, dtype=torch.bfloat16, device=dev)
    res = torch.zeros(6, 256, dtype=torch.bfloat16, device=dev)
    x[1], res[1] = 1.0, -1.0                            # the sum is zero throughout
    x[2, 3], res[2, 3], res[2, 4] = INF, -INF, 1.0      # NaN
    res[3, 200], res[3, 1] = INF, 2.0                   # the norm of a row with an infinity
    x[4], res[4] = 3e38, 3e38                           # the sum leaves bf16
    x[5] = 2.0 ** 70                                    # the squares leave fp32
    gamma = torch.ones(256, device=dev)
    r, codes = torch.empty_like(res), torch.empty(6, 256, dtype=torch.uint8, device=dev)
    scale, y = torch.empty(6, 2, device=dev), torch.empty_like(res)
    csa2.add_norm_fp8(x, res, r, gamma, codes=codes, scale=scale, y=y)
    _sync_ok()
    v, s = o.fp8_e4m3_table()[np_(codes)], np_(scale)
    assert not v[:2].any() and (s[:2] == 1).all() and not y[:2].any()
    assert np.isnan(v[2]).all() and (s[2] == 1).all() and torch.isnan(y[2]).all() and torch.isnan(r[2, 3])
    assert np.isnan(v[3, 200]) and not v[3, :200].any() and (s[3] == 1).all() and r[3, 200] == INF
    assert torch.isinf(r[4]).all() and np.isnan(v[4]).all()
    assert (r[5] == 2.0 ** 70).all() and not v[5].any() and (s[5] == 1).all()


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", [256, 5120, 8208])
def test_add_norm_products_below_fp32(K, kind):
    """r * gamma next to fp32's smallest values, where the norm is not."""
    dev, x, res, gamma = _norm_case(3, K, kind, 8)
    x, res = x * 2.0 ** -50, res * 2.0 ** -50
    gamma.mul_(2.0 ** -40)
    x[1], res[1] = x[1] * 2.0 ** -10, res[1] * 2.0 ** -10
    gamma[:128] *= 2.0 ** -10
    r, codes = torch.empty_like(res), torch.empty(3, K, dtype=torch.uint8, device=dev)
    scale, y = torch.empty(3, -(-K // 128), device=dev), torch.empty(3, K, dtype=torch.bfloat16, device=dev)
    csa2.add_norm_fp8(x, res, r, gamma, codes=codes, scale=scale, y=y, eps=1e-37)
    _sync_ok()
    _check_norm(x, res, gamma, float(np.float32(1e-37)), r, codes, scale, y)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", [256, 5120, 8208])
def test_add_norm_products_past_fp32(K, kind):
    """r * gamma leaves fp32 where the norm does not, and where the squares do (zeros)."""
    dev, x, res, gamma = _norm_case(4, K, kind, 7)
    x[0], x[1], x[2], x[3] = x[0] * 2.0 ** 30, x[1] * 2.0 ** -90, x[2] * 2.0 ** 100, x[3]
    res[0], res[1], res[2] = res[0] * 2.0 ** 30, res[1] * 2.0 ** -90, res[2] * 2.0 ** 100
    gamma.mul_(2.0 ** 100)
    gamma[K // 2:] *= 2.0 ** -230
    nb = -(-K // 128)
    r, y = torch.empty_like(res), torch.empty(4, K, dtype=torch.bfloat16, device=dev)
    codes, scale = torch.empty(4, K, dtype=torch.uint8, device=dev), torch.empty(4, nb, device=dev)
    csa2.add_norm_fp8(x, res, r, gamma, codes=codes, scale=scale, y=y)
    _sync_ok()
    assert not codes[2].bitwise_and(0x7F).any() and not y[2].any() and (scale[2] == 1).all()
    half = K // 2
    for t in (0, 1, 3):     # gamma is 2^-130 in the second half: what is not told from zero there
        _, want = o.add_norm_rows(f64(x[t:t + 1]), np_(res[t:t + 1].double()), f64(gamma), 1e-6, fp32=kind == torch.float32)
        e = 44 * U
        got = f64(y[t:t + 1])
        assert np.all(np.abs(got - want)[:, :half] <= (2.0 ** -8 * (1 + e) + e) * np.abs(want)[:, :half])
        assert np.all(np.abs(got - want)[:, half:] <= 2.0 ** -8 * np.abs(want)[:, half:] + 2.0 ** -133)
        first = half // 128
        s, m = o.e4m3_block_scales(want, 1)
        assert np.all(np.abs(np_(scale[t:t + 1]) - s)[:, :first] <= (e + 2 * U) * s[:, :first])
        _assert_codes(np_(codes[t:t + 1])[:, :first * 128], (want * o.expand_blocks(m, 1, 1, K))[:, :first * 128], 2 * e + 2 * U, "past")


# ---------------------------------------------------------------- adapters
def _adapters(n, N, K, R, g, dev):
    a = (torch.randn(n, R, K, generator=g, device=dev) / K ** 0.5).to(torch.bfloat16)
    b = torch.randn(n, N, R, generator=g, device=dev).to(torch.bfloat16)
    return a, b, 0.5 + torch.rand(n, generator=g, device=dev)


def _ids(T, n, run, g, dev):
    ids = torch.randint(-1, n, (-(-T // run),), generator=g, device=dev, dtype=torch.int32)
    return ids.repeat_interleave(run)[:T].contiguous()


def _lora_ref(x, xs, w, ws, a, b, ids, s, pos, head, theta, planes):
    nb, R = xs.shape[1], a.shape[1]
    T, K = x.shape
    xd, wd, xs_, ws_ = _decode(x), _decode(w), np_(xs).astype(np.float64), np_(ws).astype(np.float64)
    y = o.fp8_linear(xd, xs_, wd, ws_)
    mag = o.fp8_linear(np.abs(xd), xs_, np.abs(wd), ws_)
    xr = xd * o.expand_blocks(xs_, 1, T, K)
    af, bf, sf, idn = f64(a), f64(b), f64(s), np_(ids)
    add = o.lora_rows(xr, af, bf, idn, sf)
    add_mag = o.lora_rows(np.abs(xr), np.abs(af), np.abs(bf), idn, sf)
    out_mag = np.zeros_like(add)       # sum_r |v| |b|
    for t, i in enumerate(idn):
        if i >= 0:
            out_mag[t] = np.abs(bf[i]) @ np.abs(sf[i] * (af[i] @ xr[t]))
    tol = (170 + 2 * nb) * U * (mag + out_mag) + (150 + nb / 16) * U * add_mag
    tol += (2.0 ** (-8 * planes) + (2 * R + 8) * U) * out_mag
    y = y + add
    if head:
        N = y.shape[1]
        z, t = np.abs(y).reshape(T, -1, head), tol.reshape(T, -1, head)
        pair = z[..., head - 64::2] + z[..., head - 63::2]
        both = t[..., head - 64::2] + t[..., head - 63::2] + 2.0 ** -20 * pair
        t[..., head - 64::2] = t[..., head - 63::2] = both
        y = o.rope_heads(y, np_(pos), head, theta)
        assert y.shape == (T, N)
    return y, tol


def _check_out(got, osc, y, tol, out, T, N):
    if out == "fp8":
        s, _ = o.e4m3_block_scales(y, 1)
        gs = np_(osc).astype(np.float64)
        top = tol.reshape(T, -1, 128).max(axis=2)
        assert np.all(np.abs(gs - s) <= (top / 448.0 + 4 * U * s)), "scales"
        gsx = o.expand_blocks(gs, 1, T, N)
        d = o.fp8_e4m3_table()[np_(got)] * gsx
        half = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * gsx)
        slack = tol + o.expand_blocks(top, 1, T, N) + 4 * U * np.abs(y)
        assert np.all(np.abs(d - y) <= half + 1.2 * slack), f"codes: worst {np.abs(d - y).max()}"
    else:
        step = {"fp32": U, "bf16": 2.0 ** -8}[out]
        g = f64(got) if out == "bf16" else np_(got).astype(np.float64)
        bad = np.abs(g - y) > step * (np.abs(y) + tol) + tol
        assert not bad.any(), f"{bad.sum()} of {bad.size} outside, worst {np.abs(g - y).max()} where {tol[bad].min()}"


KIND = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.uint8}


def _check_lora(T, N, K, out, R, n, run=1, head=0, seed=0, w_ready=False, extra=0, factor=True):
    dev = need_gpu()
    g = _gen(dev, seed)
    x, xs = _codes((T, K), g, dev, 1)
    w, ws = _codes((N, K), g, dev, 128)
    a, b, s = _adapters(n, N, K, R, g, dev)
    ids = _ids(T, n, run, g, dev)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device=dev, dtype=torch.int32) if head else None
    big = torch.full((T + 1, N + extra), 77, dtype=KIND[out], device=dev)
    osc = torch.full((T + 1, N // 128 + 2), -5.0, device=dev) if out == "fp8" else None
    csa2.lora_linear(x, xs, w, ws, a, b, ids, big[:T, :N], adapter_scale=s if factor else None,
                     out_scale=osc[:T, :N // 128] if out == "fp8" else None, row_pos=pos, rope_head=head, w_ready=w_ready)
    _sync_ok()
    assert (big[T:] == 77).all() and (big[:T, N:] == 77).all(), "written outside the output"
    if out == "fp8":
        assert (osc[T:] == -5).all() and (osc[:T, N // 128:] == -5).all()
    # every row without an adapter is the shared projection's
    base = torch.empty(T, N, dtype=KIND[out], device=dev)
    base_s = torch.empty(T, N // 128, device=dev) if out == "fp8" else None
    csa2.fp8_linear(x, xs, w, ws, base, out_scale=base_s, row_pos=pos, rope_head=head)
    _sync_ok()
    none = ids < 0
    assert torch.equal(big[:T, :N][none], base[none])
    pick = torch.arange(T, device=dev) if T * N * K < 1 << 31 else torch.unique(torch.cat([
        torch.tensor([0, 1, T // 2, T - 1], device=dev), torch.randint(0, T, (12,), generator=g, device=dev)]))
    y, tol = _lora_ref(x[pick], xs[pick], w, ws, a, b, ids[pick], s if factor else torch.ones_like(s),
                       pos[pick] if head else None, head, 10000.0, {"bf16": 1, "fp32": 2, "fp8": 3}[out])
    _check_out(big[:T, :N][pick], osc[:T, :N // 128][pick] if out == "fp8" else None, y, tol, out, len(pick), N)


@pytest.mark.parametrize("T,N,K,R,n,run", [
    (1, 1, 16, 8, 1, 1), (1, 512, 7168, 16, 3, 1), (8, 512, 7168, 16, 8, 1), (7, 1001, 1360, 24, 2, 1), (16, 256, 128, 64, 20, 1),
    (17, 384, 4112, 72, 4, 3), (32, 640, 640, 128, 5, 1), (33, 640, 640, 40, 40, 1), (64, 4096, 2048, 32, 16, 1),
    (65, 96, 2000, 8, 70, 1), (129, 257, 400, 128, 3, 1), (333, 1001, 1360, 24, 5, 40), (500, 300, 272, 56, 200, 1),
    (1300, 1001, 2064, 64, 6, 100), (1300, 1001, 2064, 16, 300, 1), (2500, 300, 1040, 48, 9, 128), (2700, 2001, 400, 64, 4, 700),
    (4100, 2304, 272, 16, 33, 7)])
@pytest.mark.parametrize("out", ["fp32", "bf16"])
def test_lora_linear_matches_oracle(T, N, K, R, n, run, out):
    _check_lora(T, N, K, out, R, n, run, seed=T + N + R, extra=0 if (T + N) % 2 else 24, w_ready=T % 2 == 1)


@pytest.mark.parametrize("T,N,K,R,n,run,out,head", [
    (8, 4096, 2048, 64, 4, 1, "fp8", 128), (3, 1024, 144, 8, 2, 1, "bf16", 512), (16, 1024, 2048, 128, 16, 1, "fp8", 512),
    (40, 1536, 528, 16, 7, 1, "fp32", 256), (130, 768, 1040, 32, 3, 20, "fp8", 128), (257, 2048, 512, 80, 5, 64, "bf16", 512),
    (1300, 1024, 2064, 64, 4, 200, "fp8", 128), (1300, 4096, 272, 16, 3, 1, "fp8", 0), (2048, 4352, 1040, 64, 2, 512, "bf16", 256)])
def test_lora_linear_rope_and_e4m3_output(T, N, K, R, n, run, out, head):
    _check_lora(T, N, K, out, R, n, run, head, seed=T * N + K, extra=32, factor=T % 2 == 0)


@pytest.mark.parametrize("T", [9, 40, 300, 1400])
def test_lora_linear_special_adapters(T):
    """NaN and infinities of an adapter stay in its rows; ids outside the range count as none
    and are reported; a batch without adapters is the projection."""
    dev = need_gpu()
    g = _gen(dev, 5)
    K, N, R, n = 2064, 512, 32, 4
    x, xs = _codes((T, K), g, dev, 1)
    w, ws = _codes((N, K), g, dev, 128)
    a, b, s = _adapters(n, N, K, R, g, dev)
    ids = (torch.arange(T, device=dev, dtype=torch.int32) % (n + 1)) - 1
    clean, got, base = (torch.empty(T, N, device=dev) for _ in range(3))
    csa2.lora_linear(x, xs, w, ws, a, b, ids, clean, adapter_scale=s)
    a2, b2 = a.clone(), b.clone()
    a2[1, 3, 7], b2[2, :, 5], a2[2, 5, 0] = float("nan"), INF, INF
    csa2.lora_linear(x, xs, w, ws, a2, b2, ids, got, adapter_scale=s)
    csa2.fp8_linear(x, xs, w, ws, base)
    _sync_ok()
    for i in (-1, 0, 3):
        assert torch.equal(got[ids == i], clean[ids == i])
    assert torch.isnan(got[ids == 1]).all() and not torch.isfinite(got[ids == 2]).any()
    # a row's own NaN stays in it
    x2 = x.clone()
    x2[4, 0] = 0x7F
    csa2.lora_linear(x2, xs, w, ws, a, b, ids, got, adapter_scale=s)
    _sync_ok()
    rest = torch.arange(T, device=dev) != 4
    assert torch.isnan(got[4]).all() and torch.equal(got[rest], clean[rest])
    bad = ids.clone()
    bad[2], bad[5] = n, -2
    csa2.lora_linear(x, xs, w, ws, a, b, bad, got, adapter_scale=s)
    torch.cuda.synchronize()
    assert csa2.check_device_error() == 6 and csa2.check_device_error() == 0
    assert torch.equal(got[2], base[2]) and torch.equal(got[5], base[5])
    # the other rows by the oracle, not bit by bit: the tile's list of adapters has changed,
    # and with it which CTA of a cluster adds which adapter's products, so the same fp32
    # terms are added in another order (at most the roundings that _lora_ref counts)
    bad[2] = bad[5] = -1
    pick = torch.arange(min(T, 40), device=dev)
    y, tol = _lora_ref(x[pick], xs[pick], w, ws, a, b, bad[pick], s, None, 0, 10000.0, 2)
    _check_out(got[pick], None, y, tol, "fp32", len(pick), N)
    csa2.lora_linear(x, xs, w, ws, a, b, torch.full_like(ids, -1), got, adapter_scale=s)
    _sync_ok()
    assert torch.equal(got, base)


@pytest.mark.parametrize("T,K,N", [(8, 7168, 512), (300, 2048, 1024), (1300, 2064, 1000)])
def test_lora_linear_repeats_and_takes_strides_streams_and_graphs(T, K, N):
    dev = need_gpu()
    g = _gen(dev, 6)
    sets = []
    for k in range(3):     # other inputs each time: a late read or an early write shows
        x, xs = _codes((T, K + 32), g, dev, 1)
        xs3 = torch.rand(T, xs.shape[1] + 2, generator=g, device=dev)
        xs3 = xs3[:, :-(-K // 128)]
        w, ws = _codes((N, K), g, dev, 128)
        a, b, s = _adapters(5, N, K, 48, g, dev)
        sets.append((x[:, :K], xs3, w, ws, a, b, _ids(T, 5, 3, g, dev), s))
    want = []
    for q in sets:
        y = torch.empty(T, N, device=dev)
        csa2.lora_linear(*q[:7], y, adapter_scale=q[7])
        _sync_ok()
        want.append(y)
    outs = [[torch.empty(T, N, device=dev) for _ in sets] for _ in range(4)]
    for row in outs[:2]:   # one behind the other
        for q, y in zip(sets, row):
            csa2.lora_linear(*q[:7], y, adapter_scale=q[7])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(4):     # side by side
        for q, y, st in zip(sets, outs[2], streams):
            csa2.lora_linear(*q[:7], y, adapter_scale=q[7], stream=st)
    torch.cuda.synchronize()
    ws = torch.empty(csa2.lora_workspace_size(T, 48), dtype=torch.uint8, device=dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for q, y in zip(sets, outs[3]):
            csa2.lora_linear(*q[:7], y, adapter_scale=q[7], ws=ws)
        csa2.lora_linear(*sets[0][:7], outs[3][0], adapter_scale=sets[0][7])
    for row in outs[3]:
        row.zero_()
    graph.replay()
    graph.replay()
    _sync_ok()
    for row in outs:
        for y, ref in zip(row, want):
            assert torch.equal(y, ref)


@pytest.mark.parametrize("T,N,K,R,n,run,out", [
    (5, 128, 65536, 16, 2, 1, "fp8"), (200, 128, 32768, 64, 3, 50, "fp8"), (16, 128, 16, 96, 16, 1, "fp8"),
    (64, 8192, 128, 104, 9, 1, "bf16"), (48, 20000, 144, 8, 48, 1, "fp32"), (1500, 1024, 528, 8, 4, 90, "fp8"),
    (1500, 1024, 528, 40, 4, 90, "bf16"), (1500, 4097, 528, 120, 3, 500, "fp32"), (1400, 640, 272, 128, 1400, 1, "fp8"),
    (1400, 640, 272, 96, 1, 1400, "fp32"), (20000, 257, 144, 32, 11, 333, "bf16"), (2305, 512, 7168, 64, 8, 100, "fp8")])
def test_lora_linear_at_the_edges_of_its_kernels(T, N, K, R, n, run, out):
    """The longest and shortest rows, each way that a block of b is copied beside each kind of
    tile, a tile in which every row has an adapter of its own, one adapter for all."""
    _check_lora(T, N, K, out, R, n, run, seed=T + N + R, extra=16, w_ready=T % 3 == 0)


@pytest.mark.parametrize("T,N,K,R", [(8, 512, 2048, 24), (70, 2048, 528, 64), (300, 512, 1040, 16), (1400, 700, 272, 72)])
def test_lora_linear_leaves_an_old_workspace_unread(T, N, K, R):
    """What an earlier call left, NaN in every place, has no part in the result."""
    dev = need_gpu()
    g = _gen(dev, 31)
    x, xs = _codes((T, K), g, dev, 1)
    w, ws = _codes((N, K), g, dev, 128)
    a, b, s = _adapters(4, N, K, R, g, dev)
    ids = _ids(T, 4, 3, g, dev)
    want, got = torch.empty(T, N, device=dev), torch.empty(T, N, device=dev)
    need = csa2.lora_workspace_size(T, R)
    space = torch.zeros(need + 64, dtype=torch.uint8, device=dev)
    csa2.lora_linear(x, xs, w, ws, a, b, ids, want, adapter_scale=s, ws=space[:need])
    space.fill_(0xFF)
    csa2.lora_linear(x, xs, w, ws, a, b, ids, got, adapter_scale=s, ws=space[:need])
    _sync_ok()
    assert torch.equal(got, want) and (space[need:] == 0xFF).all()


@pytest.mark.parametrize("T", [8, 300, 1400])
def test_lora_linear_graphs_may_share_a_workspace(T):
    """Two captured calls with one workspace, replayed in turn, and an eager one between."""
    dev = need_gpu()
    g = _gen(dev, 33)
    K, N, R = 1040, 512, 64
    sets, want, graphs, outs = [], [], [], []
    space = torch.empty(csa2.lora_workspace_size(T, R), dtype=torch.uint8, device=dev)
    for k in range(2):
        x, xs = _codes((T, K), g, dev, 1)
        w, ws = _codes((N, K), g, dev, 128)
        a, b, s = _adapters(5, N, K, R, g, dev)
        sets.append((x, xs, w, ws, a, b, _ids(T, 5, 2, g, dev)))
        want.append(torch.empty(T, N, device=dev))
        csa2.lora_linear(*sets[k], want[k])
        torch.cuda.synchronize()
        outs.append(torch.empty(T, N, device=dev))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[k]):
            for _ in range(3):
                csa2.lora_linear(*sets[k], outs[k], ws=space)
    eager = torch.empty(T, N, device=dev)
    for _ in range(5):
        for k in (0, 1):
            graphs[k].replay()
            csa2.lora_linear(*sets[1 - k], eager, ws=space)
            assert torch.equal(outs[k], want[k]) and torch.equal(eager, want[1 - k])
    _sync_ok()


@pytest.mark.parametrize("T,N,K,R,n", [(8, 512, 2048, 16, 8), (64, 4096, 512, 32, 20), (400, 512, 1040, 64, 7), (1400, 700, 272, 24, 9)])
def test_lora_linear_graph_follows_its_inputs(T, N, K, R, n):
    """A replay takes the adapters, their factors, the rows' ids and the codes as they are then,
    from batches without an adapter to ones where each row has another."""
    dev = need_gpu()
    g = _gen(dev, 41)
    x, xs = _codes((T, K), g, dev, 1)
    w, ws = _codes((N, K), g, dev, 128)
    a, b, s = _adapters(n, N, K, R, g, dev)
    ids = torch.full((T,), -1, dtype=torch.int32, device=dev)
    y, want = torch.empty(T, N, device=dev), torch.empty(T, N, device=dev)
    csa2.lora_linear(x, xs, w, ws, a, b, ids, y, adapter_scale=s, w_ready=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        csa2.lora_linear(x, xs, w, ws, a, b, ids, y, adapter_scale=s, w_ready=True)
    for step in range(6):
        ids.copy_([torch.full_like(ids, -1), torch.arange(T, device=dev, dtype=torch.int32) % n, _ids(T, n, 1, g, dev),
                   torch.full_like(ids, n - 1), _ids(T, n, 5, g, dev), ids.flip(0)][step])
        a.mul_(-1.5)
        s.add_(0.25)
        x2, _ = _codes((T, K), g, dev, 1)
        x.copy_(x2)
        graph.replay()
        csa2.lora_linear(x, xs, w, ws, a, b, ids, want, adapter_scale=s)
        _sync_ok()
        assert torch.equal(y, want)


@pytest.mark.parametrize("T", [5, 70, 1300])
def test_lora_linear_many_adapters(T):
    """A hundred thousand adapters, of which the rows use the first and the last ones."""
    dev = need_gpu()
    g = _gen(dev, 43)
    K, N, R, n = 272, 128, 8, 100003
    x, xs = _codes((T, K), g, dev, 1)
    w, ws = _codes((N, K), g, dev, 128)
    a, b, s = _adapters(n, N, K, R, g, dev)
    ids = torch.randint(0, 9, (T,), generator=g, device=dev, dtype=torch.int32)
    ids[::2] = n - 1 - ids[::2]
    y = torch.empty(T, N, device=dev)
    csa2.lora_linear(x, xs, w, ws, a, b, ids, y, adapter_scale=s)
    _sync_ok()
    used, at = torch.unique(ids, return_inverse=True)
    u = used.long()
    ref, tol = _lora_ref(x, xs, w, ws, a[u], b[u], at.int(), s[u], None, 0, 10000.0, 2)
    _check_out(y, None, ref, tol, "fp32", T, N)


def test_rows_further_apart_than_32_bits():
    """Row strides that put the last row past 2^32 bytes and 2^31 elements."""
    dev = need_gpu()
    g = _gen(dev, 35)
    T, K, far = 6, 2048, (1 << 29) - 64
    room = torch.empty(2 * ((T - 1) * far + K), dtype=torch.uint8, device=dev)
    wide = torch.as_strided(room.view(torch.bfloat16), (T, K), (far, 1))
    x = (0.5 * torch.randn(T, K, generator=g, device=dev)).to(torch.bfloat16)
    # residual and log probabilities
    wide.copy_(x)
    res, gamma = torch.randn(T, K, generator=g, device=dev), torch.ones(K, device=dev)
    r_out, y = torch.empty_like(res), torch.empty_like(x)
    csa2.add_norm_fp8(wide, res, r_out, gamma, y=y)
    _sync_ok()
    _check_norm(x, res, gamma, 1e-6, r_out, None, None, y)
    wide.zero_()
    csa2.add_norm_fp8(x, x, wide, gamma, y=y)      # x and the residual may be one tensor
    _sync_ok()
    assert torch.equal(wide, 2 * x)
    csa2.add_norm_fp8(x, res, r_out, gamma, y=wide)
    _sync_ok()
    _check_norm(x, res, gamma, 1e-6, r_out, None, None, wide)
    _check_logprobs(wide, torch.tensor([1, 2047, 5, -1, 7, 9], dtype=torch.int32, device=dev), 4)
    # the adapters' projection
    codes, xs = _codes((T, K), g, dev, 1)
    w, ws = _codes((256, K), g, dev, 128)
    a, b, s = _adapters(2, 256, K, 16, g, dev)
    ids = torch.tensor([1, 0, 1, -1, 0, 1], dtype=torch.int32, device=dev)
    apart = torch.as_strided(room, (T, K), (2 * far, 1))
    apart.copy_(codes)
    want, got = torch.empty(T, 256, device=dev), torch.empty(T, 256, device=dev)
    csa2.lora_linear(codes, xs, w, ws, a, b, ids, want, adapter_scale=s)
    csa2.lora_linear(apart, xs, w, ws, a, b, ids, got, adapter_scale=s)
    _sync_ok()
    assert torch.equal(got, want)
    out = torch.as_strided(room.view(torch.float32), (T, 256), (far // 2, 1))
    csa2.lora_linear(codes, xs, w, ws, a, b, ids, out, adapter_scale=s)
    _sync_ok()
    assert torch.equal(out, want)


def test_lora_linear_binding_refuses():
    dev = need_gpu()
    g = _gen(dev, 1)
    x, xs = _codes((4, 256), g, dev, 1)
    w, ws = _codes((128, 256), g, dev, 128)
    a, b, s = _adapters(2, 128, 256, 16, g, dev)
    ids, y = torch.zeros(4, dtype=torch.int32, device=dev), torch.empty(4, 128, device=dev)
    with pytest.raises(ValueError, match="a, b"):
        csa2.lora_linear(x, xs, w, ws, a[:, :8].contiguous(), b, ids, y)
    with pytest.raises(ValueError, match="contiguous"):
        csa2.lora_linear(x, xs, w, ws, a[:, ::2], b, ids, y)
    with pytest.raises(TypeError, match="b: "):
        csa2.lora_linear(x, xs, w, ws, a, b.float(), ids, y)
    with pytest.raises(ValueError, match="row_adapter"):
        csa2.lora_linear(x, xs, w, ws, a, b, ids[:3], y)
    with pytest.raises(TypeError, match="row_adapter"):
        csa2.lora_linear(x, xs, w, ws, a, b, None, y)
    with pytest.raises(TypeError, match="ws: "):
        csa2.lora_linear(x, xs, w, ws, a, b, ids, y, ws=torch.empty(8, device=dev))
    with pytest.raises(csa2.Csa2Error, match="needed"):
        csa2.lora_linear(x, xs, w, ws, a, b, ids, y, ws=torch.empty(16, dtype=torch.uint8, device=dev))


# ---------------------------------------------------------------- log probabilities
def _logits(T, V, kind, g, dev, mask=0.0, spread=2.0):
    x = spread * torch.randn(T, V, generator=g, device=dev)
    x.scatter_add_(1, torch.randint(0, V, (T, 3), generator=g, device=dev), 12.0 * torch.rand(T, 3, generator=g, device=dev))
    if mask:
        x = torch.where(torch.rand(T, V, generator=g, device=dev) < mask, -INF, x)
    return x.to(kind)


def _check_logprobs(x, token, n, splits_elements=None, ids_stride=0):
    dev = x.device
    T, V = x.shape
    lp, en, ls = (torch.full((T + 1,), 9.0, device=dev) for _ in range(3))
    ti = torch.full((T + 1, n + ids_stride), -9, dtype=torch.int32, device=dev)
    tl = torch.full((T + 1, n + ids_stride), 9.0, device=dev)
    csa2.logprobs(x, token=token, logprob=lp[:T], entropy=en[:T], lse=ls[:T], top_id=ti[:T, :n] if n else None,
                  top_logprob=tl[:T, :n] if n else None)
    _sync_ok()
    assert lp[T] == 9 and en[T] == 9 and ls[T] == 9 and (ti[T] == -9).all() and (ti[:, n:] == -9).all() and (tl[:, n:] == 9).all()
    xd, tk = np_(x.double()), np_(token)
    c = V / 256 + 8 * (V / 1024 + 1) + 100
    for t in range(T):
        wl, we, ws, wi, wt = o.logprobs_row(xd[t], int(tk[t]), n)
        # the output is fp32: from half a step past its largest value on it is -inf (the
        # lowest logit next to the largest one is 6.8e38 below it)
        wl, wt = (np.where(np.asarray(v) <= -FP32_END, -INF, v) for v in (wl, wt))
        fin = np.isfinite(xd[t])
        if not fin.any():
            assert float(ls[t]) == -INF and float(en[t]) == 0.0 and float(lp[t]) == wl
        else:
            top = xd[t][fin].max()
            d = np.where(fin, xd[t], top) - top
            e = np.where(fin, np.exp(d), 0.0)
            e[int(np.argmax(np.where(fin, xd[t], -INF)))] = 0.0
            with np.errstate(over="ignore", invalid="ignore"):
                d = np.where(e > 0, d, 0.0)
                R, W, Q = e.sum(), -(e * d).sum(), (e * d * d).sum()
            lt = np.log1p(R)
            d_lt = U * (4 * W + c * R) / (1 + R) + 2 * U * lt
            d_h = d_lt + U * (4 * Q + c * W) / (1 + R) + W / (1 + R) ** 2 * U * (4 * W + c * R) + 4 * U * (lt + W / (1 + R))
            assert abs(float(ls[t]) - ws) <= d_lt + U * abs(ws)
            assert abs(float(en[t]) - we) <= d_h, (t, float(en[t]), we, d_h)
            if np.isfinite(wl):
                assert abs(float(lp[t]) - wl) <= d_lt + 2 * U * abs(wl) + U * abs(wl), (t, float(lp[t]), wl)
            else:
                assert float(lp[t]) == wl
            ok = np.isfinite(wt)
            gt = f64(tl[t, :n])
            assert np.array_equal(np.isfinite(gt), ok) and (gt[~ok] == -INF).all()
            assert np.all(np.abs(gt[ok] - wt[ok]) <= d_lt + 3 * U * np.abs(wt[ok]))
        assert np_(ti)[t, :n].tolist() == wi.tolist(), t


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,V,n", [(1, 1, 3), (3, 2, 2), (2, 31, 32), (5, 257, 20), (4, 1023, 1), (3, 4097, 5), (700, 130, 7), (8, 8192, 20),
                                   (1, 32000, 0), (2, 50001, 32), (3, 131072, 20), (40, 20011, 1), (333, 5003, 5), (2, 300007, 17)])
def test_logprobs_match_oracle(T, V, n, kind):
    dev = need_gpu()
    g = _gen(dev, T + V)
    x = _logits(T, V, kind, g, dev)
    token = torch.randint(-1, V, (T,), generator=g, device=dev, dtype=torch.int32)
    token[0] = int(x[0].float().argmax())
    _check_logprobs(x, token, n, ids_stride=3)


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,V,n", [(3, 512, 9), (3, 513, 9), (759, 1500, 3), (760, 1500, 3), (760, 10000, 0), (760, 10001, 2),
                                   (76, 8192, 4), (77, 8192, 4), (304, 4000, 5), (305, 4000, 5), (153, 4000, 0), (5, 4095, 6),
                                   (19, 65536, 6), (38, 65536, 32), (9, 32768, 7), (9, 32767, 7), (10, 32768, 7), (4, 2047, 3),
                                   (4, 4097, 3), (1, 1 << 21, 32)])
def test_logprobs_at_the_edges_of_their_kernels(T, V, n, kind):
    dev = need_gpu()
    g = _gen(dev, T + V)
    x = _logits(T, V, kind, g, dev, mask=0.3)
    _check_logprobs(x, torch.randint(-1, V, (T,), generator=g, device=dev, dtype=torch.int32), n)


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift", [0, 1, 3, 5])
def test_logprobs_rows_anywhere(kind, shift):
    """Rows that start off a 16-byte border, in a wider matrix whose other columns would win."""
    dev = need_gpu()
    g = _gen(dev, 8)
    for T, V in ((6, 1003), (2, 40003), (3, 5)):
        wide = torch.full((T, V + 11), 1000.0, dtype=kind, device=dev)
        x = wide[:, shift:shift + V]
        x.copy_(_logits(T, V, kind, g, dev))
        _check_logprobs(x, torch.randint(0, V, (T,), generator=g, device=dev, dtype=torch.int32), 6)


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [5, 700, 9001, 70001])
def test_logprobs_masks_ties_and_special_values(V, kind):
    dev = need_gpu()
    g = _gen(dev, 9)
    low = torch.finfo(kind).min
    rows = [_logits(1, V, kind, g, dev, mask=0.95)[0], torch.full((V,), -INF, dtype=kind, device=dev),
            torch.full((V,), low, dtype=kind, device=dev), torch.zeros(V, dtype=kind, device=dev)]
    r = torch.full((V,), -INF, dtype=kind, device=dev)
    r[V - 1] = -3.0                                   # one token left
    rows.append(r)
    r = _logits(1, V, kind, g, dev)[0]
    r[V // 2], r[0], r[V - 1] = float("nan"), INF, -INF
    rows.append(r)
    r = torch.full((V,), low, dtype=kind, device=dev)
    r[V // 3], r[V // 2] = torch.finfo(kind).max, 1.0
    rows.append(r)
    rows.append(torch.full((V,), float("nan"), dtype=kind, device=dev))
    r = torch.zeros(V, dtype=kind, device=dev)
    r[::2] = -0.0                                     # equal values
    rows.append(r)
    rows.append((torch.arange(V, device=dev) % 3).to(kind))   # many ties at the top
    x = torch.stack(rows)
    token = torch.tensor([0, 0, V - 1, 1, V - 1, 0, V // 2, 0, 2, -1], dtype=torch.int32, device=dev)
    for n in (1, 4, 32):
        _check_logprobs(x, token, n)


@pytest.mark.parametrize("V", [40000, 131072, 1 << 20])
def test_logprobs_alternatives_side_by_side(V):
    """The best tokens in one run of a thread, ascending, descending, and in more candidates than the list holds."""
    dev = need_gpu()
    x = torch.zeros(5, V, device=dev)
    x[0] = torch.arange(V, device=dev) / V
    x[1] = -x[0]
    x[2, 7::1024] = 5.0 + torch.arange(len(x[2, 7::1024]), device=dev) / V      # of one thread
    x[3, 4096:4096 + 8192] = 3.0
    x[3, 4096:4096 + 8192:5] = 4.0
    x[4].view(-1)[: V // 1024 * 1024].view(-1, 1024)[:, :128] = 1.0 + torch.rand(V // 1024, 128, generator=_gen(dev, 2), device=dev)
    _check_logprobs(x, torch.tensor([0, 1, 2, 3, -1], dtype=torch.int32, device=dev), 32)


def test_logprobs_bad_tokens_are_reported():
    dev = need_gpu()
    x = _logits(4, 100, torch.float32, _gen(dev, 1), dev)
    token = torch.tensor([0, 100, -2, -1], dtype=torch.int32, device=dev)
    lp = torch.full((4,), 5.0, device=dev)
    csa2.logprobs(x, token=token, logprob=lp)
    torch.cuda.synchronize()
    assert csa2.check_device_error() == 6 and lp[1:].tolist() == [0.0, 0.0, 0.0] and lp[0] < 0


def test_logprobs_streams_graphs_and_single_outputs():
    dev = need_gpu()
    g = _gen(dev, 3)
    x = _logits(8, 50000, torch.float32, g, dev)
    token = torch.randint(0, 50000, (8,), generator=g, device=dev, dtype=torch.int32)
    full = {"logprob": torch.empty(8, device=dev), "entropy": torch.empty(8, device=dev), "lse": torch.empty(8, device=dev),
            "top_id": torch.empty(8, 9, dtype=torch.int32, device=dev), "top_logprob": torch.empty(8, 9, device=dev)}
    csa2.logprobs(x, token=token, **full)
    for k, v in full.items():
        alone = torch.zeros_like(v)
        csa2.logprobs(x, token=token if k == "logprob" else None, **{k: alone})
        assert torch.equal(alone, v), k
    again = {k: torch.zeros_like(v) for k, v in full.items()}
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    csa2.logprobs(x, token=token, stream=st, **again)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    third = {k: torch.zeros_like(v) for k, v in full.items()}
    with torch.cuda.graph(graph):
        csa2.logprobs(x, token=token, **third)
    graph.replay()
    graph.replay()
    _sync_ok()
    for k, v in full.items():
        assert torch.equal(again[k], v) and torch.equal(third[k], v), k


def test_binding_checks_of_the_alternatives():
    dev = need_gpu()
    x = torch.zeros(2, 64, device=dev)
    with pytest.raises(ValueError, match="top_logprob"):
        csa2.logprobs(x, top_id=torch.zeros(2, 3, dtype=torch.int32, device=dev), top_logprob=torch.zeros(2, 4, device=dev))
    with pytest.raises(ValueError, match="row stride"):
        csa2.logprobs(x, top_id=torch.zeros(2, 3, dtype=torch.int32, device=dev), top_logprob=torch.zeros(2, 4, device=dev)[:, :3])
    with pytest.raises(TypeError, match="logits"):
        csa2.logprobs(x.half(), entropy=torch.zeros(2, device=dev))
    with pytest.raises(csa2.Csa2Error, match="no output"):
        csa2.logprobs(x)


# ---------------------------------------------------------------- as they are used
@pytest.mark.parametrize("T", [8, 200])
def test_from_a_layers_output_to_the_answers_probabilities(T):
    """The last layer's output joins the residual, its norm's codes go through the head with
    the requests' adapters, and the logits become probabilities: every step against the
    oracle on what the step before it wrote, then the whole run as one graph."""
    dev = need_gpu()
    g = _gen(dev, 21)
    H, V, R, n = 1024, 5000, 16, 3
    _, x, res, gamma = _norm_case(T, H, torch.bfloat16, 22)
    w, ws = _codes((V, H), g, dev, 128)
    ws.mul_(1e-3)
    a, b, s = _adapters(n, V, H, R, g, dev)
    ids = _ids(T, n, 2, g, dev)
    token = torch.randint(0, V, (T,), generator=g, device=dev, dtype=torch.int32)
    r, codes = torch.empty_like(res), torch.empty(T, H, dtype=torch.uint8, device=dev)
    scale, logits = torch.empty(T, H // 128, device=dev), torch.empty(T, V, device=dev)
    o_ = {"logprob": torch.empty(T, device=dev), "entropy": torch.empty(T, device=dev),
          "top_id": torch.empty(T, 4, dtype=torch.int32, device=dev)}

    def step():
        csa2.add_norm_fp8(x, res, r, gamma, codes=codes, scale=scale)
        csa2.lora_linear(codes, scale, w, ws, a, b, ids, logits, adapter_scale=s, w_ready=True)
        csa2.logprobs(logits, token=token, **o_)

    torch.cuda.synchronize()
    step()
    _sync_ok()
    _check_norm(x, res, gamma, 1e-6, r, codes, scale, None)
    y, tol = _lora_ref(codes, scale, w, ws, a, b, ids, s, None, 0, 10000.0, 2)
    _check_out(logits, None, y, tol, "fp32", T, V)
    _check_logprobs(logits, token, 4)
    first = [t.clone() for t in (r, codes, scale, logits, *o_.values())]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            step()
    for t in (r, codes, scale, logits, *o_.values()):
        t.zero_()
    graph.replay()
    _sync_ok()
    for t, f in zip((r, codes, scale, logits, *o_.values()), first):
        assert torch.equal(t, f)
