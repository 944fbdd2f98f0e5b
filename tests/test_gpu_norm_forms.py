"""csa2_add_norm_fp8 in each form that its launch takes, with the bound of that form, and its codes
beside those of csa2_quant_fp8 on the residual that it stored.

u = 2^-24.  A thread adds the squares of 16 V columns (V runs: one up to K = 4,096, and up to 8,192
for at most two rows an SM, else two), five shuffle steps, at most 16 warps; the division and eps are
two more.  Of a sum of positive terms half of that is left by the root: 8 V + 11; root, reciprocal and two
products: e = (8 V + 15) u of a value.  Its block's maximum has the same, a scale two roundings more.

csa2_quant_fp8 takes its codes from values of such an error (K / 256 + 13 additions in a chain, two
products, and the same in the maximum), this call from exact quotients: a code may differ where the
quotient is that near to a border.
"""
import numpy as np
import pytest
import torch

from gpu_util import np_
from oracle import csa2_oracle as o
from serving_lightning_indexer_gb300 import csa2
from test_gpu_inputs import U, _sync_ok
from test_gpu_layers import _norm_case, f64

pytestmark = pytest.mark.gpu


def _run(T, K, kind, seed):
    dev, x, res, gamma = _norm_case(T, K, kind, seed)
    r, codes = torch.empty_like(res), torch.empty(T, K, dtype=torch.uint8, device=dev)
    scale, y = torch.empty(T, -(-K // 128), device=dev), torch.empty(T, K, dtype=torch.bfloat16, device=dev)
    csa2.add_norm_fp8(x, res, r, gamma, codes=codes, scale=scale, y=y)
    _sync_ok()
    return x, res, gamma, r, codes, scale, y


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", [16, 512, 2064, 4096, 4112, 7168, 8192, 8208, 12288, 16384])
@pytest.mark.parametrize("many", [False, True])
def test_add_norm_within_the_bound_of_its_form(K, kind, many):
    sms = torch.cuda.get_device_properties(0).multi_processor_count if torch.cuda.is_available() else 0
    T = 2 * sms + many                       # the last of the few rows, the first of the many
    x, res, gamma, r, codes, scale, y = _run(T, K, kind, K + many)
    e = (8 * (1 if K <= 4096 or (K <= 8192 and not many) else 2) + 15) * U
    eps = float(np.float32(1e-6))
    pick = torch.cat([torch.arange(8, device=x.device), torch.arange(T - 8, T, device=x.device)])
    want_r, want = o.add_norm_rows(f64(x[pick]), np_(res[pick].double()), f64(gamma), eps, fp32=kind is torch.float32)
    assert np.array_equal(np_(r[pick].double()), want_r)
    assert np.all(np.abs(f64(y[pick]) - want) <= (2.0 ** -8 * (1 + e) + e) * np.abs(want))
    s, _ = o.e4m3_block_scales(want, 1)
    assert np.all(np.abs(np_(scale[pick]) - s) <= (e + 2 * U) * s)


@pytest.mark.parametrize("T,K", [(4, 144), (700, 528), (300, 7168), (900, 4096), (40, 16384)])
def test_add_norm_codes_beside_the_quantisers(T, K):
    x, res, gamma, r, codes, scale, y = _run(T, K, torch.bfloat16, T + K)
    other, other_s = torch.empty_like(codes), torch.empty_like(scale)
    csa2.quant_fp8(r, other, other_s, gamma=gamma, eps=1e-6)
    _sync_ok()
    assert bool(((scale - other_s).abs() <= (2 * (K / 256 + 24) + 60) * U * scale).all())
    nb = -(-K // 128)
    v = torch.nn.functional.pad(r.double() * gamma.double(), (0, nb * 128 - K)).view(T, nb, 128)
    q = (v * 448.0 / v.abs().amax(-1, keepdim=True)).view(T, -1)[:, :K]
    e = (2 + 2 * (K / 256 + 24)) * U
    low, high = ((q * (1.0 + d)).clamp(-448.0, 448.0).float().to(torch.float8_e4m3fn).float() for d in (-e, e))
    a, b = codes.view(torch.float8_e4m3fn).float(), other.view(torch.float8_e4m3fn).float()
    same = (codes & 0x7F) + (codes & 0x80) * (a != 0) == (other & 0x7F) + (other & 0x80) * (b != 0)
    assert bool((same | ((low != high) & ((b == low) | (b == high)))).all())
    assert int((~same).sum()) <= 2 + q.numel() * 2.0 ** -14      # borders are 2^-4 apart, 2 e wide: 2^-15 at K = 16,384
