"""How many bits of the adapters' inner products reach csa2_lora_linear's output.

Inputs whose sums round next to nothing, so that a part of v that is left out shows.  The
projection's own weights are zero and a row of x has one code, 1, in each block of 128, so
v[t][r] is a sum of one term a block.  Tolerance, from the arithmetic (u = 2^-24, v's terms in
absolute value where a magnitude is meant):
  * v: the scale times a code's product, an addition a block, the warps' or CTAs' additions (8 at
    most with a term that is not zero beside each), adapter_scale: (blocks + 10) u;
  * its bf16 parts: each rounding leaves half a step, so two leave 2^-17 of v (2^-8, of whose
    binade's lower end at most 2^-9 is left, half a step of which is 2^-17), three nothing;
  * an output: rank products, each in as many parts, and the sums of the blocks of ranks:
    (2 rank + 8) u; then half a step of its type, at the binade of the value itself.
"""
import numpy as np
import pytest
import torch

from gpu_util import need_gpu, np_
from serving_lightning_indexer_gb300 import csa2
from test_gpu_inputs import U, _gen, _sync_ok

pytestmark = pytest.mark.gpu


def _inputs(T, N, K, R, n, seed, run=1):
    dev = need_gpu()
    g = _gen(dev, seed)
    nb = -(-K // 128)
    x = torch.zeros(T, K, dtype=torch.uint8, device=dev)
    for b in range(nb):
        at = b * 128 + torch.randint(0, min(128, K - b * 128), (T,), generator=g, device=dev)
        x[torch.arange(T, device=dev), at] = 0x38                                  # 1.0
    xs = 0.5 + torch.rand(T, nb, generator=g, device=dev)
    w, ws = torch.zeros(N, K, dtype=torch.uint8, device=dev), torch.ones(-(-N // 128), nb, device=dev)
    a = torch.randn(n, R, K, generator=g, device=dev).to(torch.bfloat16)
    b = torch.randn(n, N, R, generator=g, device=dev).to(torch.bfloat16)
    one = torch.arange(N, device=dev) % 2 == 0                                     # a single rank's product
    hot = torch.arange(N, device=dev)[:, None] // 2 % R == torch.arange(R, device=dev)
    b = torch.where(one[:, None] & ~hot, torch.zeros_like(b), b)
    ids = torch.randint(-1, n, (-(-T // run),), generator=g, device=dev, dtype=torch.int32).repeat_interleave(run)[:T].contiguous()
    return x, xs, w, ws, a, b, ids, 0.5 + torch.rand(n, generator=g, device=dev)


def _reference(x, xs, a, b, ids, s):
    T, K = x.shape
    xr = x.view(torch.float8_e4m3fn).double() * xs.double().repeat_interleave(128, dim=1)[:, :K]
    y, mag, out_mag = (torch.zeros(T, b.shape[1], dtype=torch.float64, device=x.device) for _ in range(3))
    for i in range(a.shape[0]):
        at = (ids == i).nonzero()[:, 0]
        if len(at):
            v, va = xr[at] @ a[i].double().t() * s[i].double(), xr[at] @ a[i].double().abs().t() * s[i].double()
            bi = b[i].double().t()
            y[at], out_mag[at], mag[at] = v @ bi, v.abs() @ bi.abs(), va @ bi.abs()
    return np_(y), np_(mag), np_(out_mag)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,N,K,R,n", [
    (1, 130, 16, 8, 1), (8, 512, 384, 16, 8), (8, 512, 384, 64, 8), (16, 1001, 272, 128, 5), (24, 640, 384, 64, 4), (32, 384, 144, 104, 9),
    (48, 256, 384, 40, 5), (64, 512, 2048, 72, 6),                                  # tiles of up to 64 rows
    (40, 20000, 256, 64, 16), (64, 20001, 272, 24, 7), (33, 19584, 144, 128, 3), (64, 19712, 384, 8, 12),   # up to 64 rows of 128
    (40, 12700, 4096, 64, 3), (64, 12700, 4096, 40, 5),                             # the same, two CTAs a tile
    (65, 20000, 144, 64, 4), (500, 300, 272, 56, 60), (1300, 1000, 2064, 64, 6), (1300, 1001, 2064, 16, 30), (2700, 2001, 400, 72, 4)])
def test_lora_output_has_the_inner_products_bits(T, N, K, R, n, out):
    x, xs, w, ws, a, b, ids, s = _inputs(T, N, K, R, n, T + N + R)
    y = torch.empty(T, N, dtype=out, device=x.device)
    space = torch.full((csa2.lora_workspace_size(T, R),), 0xFF, dtype=torch.uint8, device=x.device)   # NaN wherever it is not written
    csa2.lora_linear(x, xs, w, ws, a, b, ids, y, adapter_scale=s, ws=space)
    _sync_ok()
    want, mag, out_mag = _reference(x, xs, a, b, ids, s)
    tol = (-(-K // 128) + 10) * U * mag + ((2.0 ** -17 if out is torch.bfloat16 else 0.0) + (2 * R + 8) * U) * out_mag
    top = np.abs(want) + tol
    half = np.where(top > 0, np.exp2(np.floor(np.log2(np.where(top > 0, top, 1.0)))), 0.0) * torch.finfo(out).eps / 2
    err = np.abs(np_(y.double()) - want)
    assert np.all(err <= half + tol), (int((err > half + tol).sum()), float((err / (half + tol + 1e-300)).max()))


@pytest.mark.parametrize("T,N,K,R,n,run", [
    (4096, 512, 7168, 64, 4, 128), (4096, 512, 7168, 64, 9, 64), (4096, 512, 7168, 64, 30, 43), (4096, 256, 7168, 128, 4, 128),
    (4096, 256, 7168, 128, 9, 60), (4096, 512, 7168, 16, 60, 16), (19000, 256, 2064, 64, 5, 128), (19000, 128, 2064, 32, 40, 50),
    (200, 128, 32768, 64, 3, 50), (2432, 256, 16384, 48, 3, 300)])
def test_lora_scales_of_long_shares(T, N, K, R, n, run):
    """Nine blocks of input dims and more to a CTA of the many-rows kernel, with one adapter a tile,
    two, three and more: a row's sums take the scales of their own blocks, again and again."""
    x, xs, w, ws, a, b, ids, s = _inputs(T, N, K, R, n, T + N + R + run, run)
    xs *= 2.0 ** (torch.arange(xs.shape[1], device=xs.device) % 7 - 3)
    y, again = torch.empty(T, N, device=x.device), torch.empty(T, N, device=x.device)
    csa2.lora_linear(x, xs, w, ws, a, b, ids, y, adapter_scale=s)
    for _ in range(20):
        csa2.lora_linear(x, xs, w, ws, a, b, ids, again, adapter_scale=s)
        assert torch.equal(y, again)
    _sync_ok()
    want, mag, out_mag = _reference(x, xs, a, b, ids, s)
    assert np.all(np.abs(np_(y.double()) - want) <= U * np.abs(want) + (-(-K // 128) + 10) * U * mag + (2 * R + 8) * U * out_mag)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,N,K,R,n", [(8, 512, 384, 16, 4), (64, 20000, 256, 8, 5), (1300, 1000, 2064, 64, 6)])
def test_lora_inner_products_next_to_the_largest_number(T, N, K, R, n, out):
    """Between bf16's largest number and fp32's an inner product is finite, and so is the output
    of a small b; an inner product that leaves fp32 is an infinity in its own rows."""
    x, xs, w, ws, a, b, ids, s = _inputs(T, N, K, R, n, T + N + R)
    x[:, 128:], xs[:, 0] = 0, 1.0                # one term: v = a's power of two times the factor
    sign = torch.where(a > 0, 1.0, -1.0)
    a = (sign * 2.0 ** 127).to(torch.bfloat16)
    s = (2.0 - 2.0 ** -10 + 2.0 ** -16 * torch.arange(n, device=x.device)).float()      # 3.401e38 and above
    b = b * 2.0 ** -20
    ids[0], ids[1] = 0, n - 1
    y = torch.empty(T, N, dtype=out, device=x.device)
    csa2.lora_linear(x, xs, w, ws, a, b, ids, y, adapter_scale=s)
    _sync_ok()
    want, _, out_mag = _reference(x, xs, a, b, ids, s)
    got = np_(y.double())
    assert np.isfinite(got).all() and np.abs(want).max() > 2.0 ** 107
    assert np.all(np.abs(got - want) <= torch.finfo(out).eps / 2 * np.abs(want) + (2.0 ** -17 + (2 * R + 8) * U) * out_mag)
    s[0] = 4.0
    again = torch.empty_like(y)
    csa2.lora_linear(x, xs, w, ws, a, b, ids, again, adapter_scale=s)
    _sync_ok()
    assert not torch.isfinite(again[ids == 0][:, ::2]).any() and torch.equal(again[ids != 0], y[ids != 0])
