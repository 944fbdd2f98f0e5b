"""CPU pins of the oracle's functions around the layers: the residual's addition and
norm, low-rank adapters, log probabilities."""
import math

import numpy as np
import pytest
import torch

from oracle import csa2_oracle as o


def test_bf16_round_is_torchs():
    r = np.random.default_rng(0)
    v = np.concatenate([r.normal(size=2000) * np.exp2(r.integers(-140, 120, 2000)), [0.0, 1.00390625, 1.01171875, 3.4e38, -3.4e38]])
    v = v.astype(np.float32)
    want = torch.from_numpy(v).to(torch.bfloat16).double().numpy()
    assert np.array_equal(o.bf16_round(v.astype(np.float64)), want)


@pytest.mark.parametrize("fp32", [False, True])
def test_add_norm_rows_matches_torch(fp32):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(5, 96, generator=g).to(torch.bfloat16)
    res = torch.randn(5, 96, generator=g).to(torch.float32 if fp32 else torch.bfloat16)
    gamma = torch.rand(96, generator=g, dtype=torch.float64)
    r, y = o.add_norm_rows(x.double().numpy(), res.double().numpy(), gamma.numpy(), 1e-5, fp32)
    kept = (x.double() + res.double()).to(res.dtype)
    assert np.array_equal(r, kept.double().numpy())
    want = torch.nn.functional.rms_norm(kept.double(), (96,), gamma, 1e-5)
    assert np.allclose(y, want.numpy(), rtol=1e-12)


def test_lora_rows_is_the_double_loop():
    r = np.random.default_rng(2)
    x, a, b = r.normal(size=(4, 6)), r.normal(size=(3, 2, 6)), r.normal(size=(3, 5, 2))
    s, ids = r.random(3), [2, -1, 0, 2]
    got = o.lora_rows(x, a, b, ids, s)
    for t, i in enumerate(ids):
        for n in range(5):
            want = 0.0
            if i >= 0:
                for q in range(2):
                    want += s[i] * b[i, n, q] * sum(a[i, q, k] * x[t, k] for k in range(6))
            assert math.isclose(got[t, n], want, rel_tol=1e-12, abs_tol=1e-12)


def test_a_low_rank_update_is_a_change_of_the_weights():
    r = np.random.default_rng(3)
    x, w = r.normal(size=(3, 16)), r.normal(size=(7, 16))
    a, b = r.normal(size=(1, 4, 16)), r.normal(size=(1, 7, 4))
    assert np.allclose(x @ w.T + o.lora_rows(x, a, b, [0, 0, 0], [0.5]), x @ (w + 0.5 * b[0] @ a[0]).T)


def test_logprobs_row_matches_torch():
    g = torch.Generator().manual_seed(4)
    x = 5 * torch.randn(300, generator=g, dtype=torch.float64)
    x[7] = -math.inf
    lp, entropy, lse, ids, best = o.logprobs_row(x.numpy(), 11, 9)
    p = torch.softmax(x, 0)
    assert math.isclose(lse, torch.logsumexp(x, 0).item(), rel_tol=1e-13)
    assert math.isclose(lp, math.log(p[11].item()), rel_tol=1e-12)
    assert math.isclose(entropy, torch.distributions.Categorical(probs=p).entropy().item(), rel_tol=1e-7)
    want = torch.sort(x, descending=True, stable=True)
    assert ids.tolist() == want.indices[:9].tolist()
    assert np.allclose(best, torch.log(p[want.indices[:9]]).numpy(), rtol=1e-12)


def test_logprobs_row_by_hand():
    lp, entropy, lse, ids, best = o.logprobs_row([0.0, -math.inf, 0.0, math.nan, math.inf], 1, 4)
    assert lp == -math.inf and math.isclose(entropy, math.log(2)) and math.isclose(lse, math.log(2))
    assert ids.tolist() == [0, 2, -1, -1] and best[2] == -math.inf and math.isclose(best[0], -math.log(2))
    assert o.logprobs_row([-math.inf, math.nan], 0, 1)[:3] == (-math.inf, 0.0, -math.inf)
    assert o.logprobs_row([-math.inf], -1, 0)[0] == 0.0
    low = -3.4028234663852886e38
    lp, entropy, lse, ids, _ = o.logprobs_row([low, low, low, low], 2, 2)
    assert math.isclose(lp, -math.log(4)) and math.isclose(entropy, math.log(4)) and ids.tolist() == [0, 1]
    # next to a likely token the others' sum is the log probability
    assert math.isclose(o.logprobs_row([0.0, -40.0], 0)[0], -math.exp(-40.0), rel_tol=1e-12)
