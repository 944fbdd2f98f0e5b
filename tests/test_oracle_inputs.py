"""CPU pins of the oracle's step-input functions: block scales, the projection on
codes, the heads' RoPE, and the batch's rows, pages and slots."""
import numpy as np
import pytest
import torch

from oracle import csa2_oracle as o


def test_block_scales_by_hand():
    y = np.zeros((3, 200))
    y[0, 5], y[0, 130], y[1, 199], y[2, 0] = -896.0, 7.0, 1e-44, np.inf
    y[2, 1] = 2.0
    s, m = o.e4m3_block_scales(y, 1)
    assert s.tolist() == [[2.0, 7.0 / 448.0], [1.0, 2.0 ** -120], [2.0 / 448.0, 1.0]]
    assert m[0, 0] == 0.5 and m[1, 1] == 2.0 ** 120
    tile, _ = o.e4m3_block_scales(y, 128)
    assert tile.tolist() == [[2.0, 7.0 / 448.0]]
    assert o.expand_blocks(s, 1, 3, 200)[0].tolist() == [2.0] * 128 + [7.0 / 448.0] * 72


def test_block_scale_makes_the_largest_value_448():
    y = np.random.default_rng(0).normal(size=(5, 384))
    s, m = o.e4m3_block_scales(y, 1)
    v = np.abs(y * o.expand_blocks(m, 1, 5, 384)).reshape(5, 3, 128).max(axis=2)
    assert np.allclose(v, 448.0, rtol=1e-15) and np.allclose(s * m, 1.0, rtol=1e-15)


def test_rms_norm_rows_matches_torch():
    x = torch.randn(4, 96, dtype=torch.float64)
    g = torch.rand(96, dtype=torch.float64)
    want = torch.nn.functional.rms_norm(x, (96,), g, 1e-5)
    assert np.allclose(o.rms_norm_rows(x.numpy(), g.numpy(), 1e-5), want.numpy(), rtol=1e-12)


def test_fp8_linear_is_the_double_loop():
    r = np.random.default_rng(1)
    x, w = r.normal(size=(3, 144)), r.normal(size=(130, 144))
    xs, ws = r.random((3, 2)), r.random((2, 2))
    want = np.zeros((3, 130))
    for t in range(3):
        for n in range(130):
            for k in range(144):
                want[t, n] += x[t, k] * xs[t, k // 128] * w[n, k] * ws[n // 128, k // 128]
    assert np.allclose(o.fp8_linear(x, xs, w, ws), want, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("head", [128, 512])
def test_rope_heads_is_the_keys_rotation(head):
    r = np.random.default_rng(2)
    y = r.normal(size=(2, 2 * head))
    pos = np.array([0, 70001])
    got = o.rope_heads(y, pos, head, 10000.0)
    assert np.array_equal(got[0], y[0])
    z = y[1].reshape(2, head)[:, -64:].reshape(2, 32, 2)
    z = (z[..., 0] + 1j * z[..., 1]) * np.exp(1j * 70001 * 10000.0 ** (-np.arange(32) / 32.0))
    assert np.allclose(got[1].reshape(2, head)[:, -64::2], z.real) and np.allclose(got[1].reshape(2, head)[:, -63::2], z.imag)
    assert np.array_equal(got[1].reshape(2, head)[:, :-64], y[1].reshape(2, head)[:, :-64])
    # one head of the latent's width: the rotation of the entries
    one = r.normal(size=(3, 512))
    assert np.allclose(o.rope_heads(one, np.array([3, 9, 1000]), 512, 10000.0),
                       o.rope_interleaved(one, np.array([3, 9, 1000]), 10000.0))


def test_batch_plan_worked_example():
    # m = 2; sequence 0 holds 127 tokens (63 entries, 1 page) and gets 4 (entries 63, 64: page 1 is new);
    # sequence 1 rests with 5 tokens; sequence 2 is new with 3 tokens (entry 0, page 0 is new)
    table = np.array([[7, -1], [3, -1], [-1, -1]])
    out, pt, bad = o.batch_plan([127, 5, 0], [4, 0, 3], 2, table, [40, 41, 42], 1, ring=8, ring_id=[2, 0, 1], n_swa=4)
    assert not bad and pt.tolist() == [[7, 41], [3, -1], [42, -1]]
    assert out["row_start"] == [0, 4, 4, 7] and out["row_seq"] == [0, 0, 0, 0, 2, 2, 2]
    assert out["row_pos"] == [127, 128, 129, 130, 0, 1, 2] and out["n_visible"] == [65, 2, 1]
    assert out["entry_start"] == [0, 2, 2, 3] and out["entry_pos"] == [126, 128, 0]
    assert out["entry_slot"] == [7 * 64 + 63, 41 * 64, 42 * 64] and out["entry_row"] == [0, 2, 5]
    assert out["free_head_out"] == [3]
    assert out["swa_new"] == [16 + 7, 16, 17, 18, 8, 9, 10]
    assert out["swa_slot"][0] == [16 + 4, 16 + 5, 16 + 6, 16 + 7] and out["swa_slot"][4] == [-1, -1, -1, 8]


def test_batch_plan_reports_what_does_not_fit():
    assert o.batch_plan([0], [65], 1, np.full((1, 1), -1), [5, 6])[2]               # second page past the table
    out, pt, bad = o.batch_plan([0, 0], [64, 1], 1, np.full((2, 1), -1), [5])       # free list ends
    assert bad and pt.tolist() == [[5], [-1]] and out["entry_slot"][-1] == -1
    assert o.batch_plan([3], [1], 1, np.full((1, 1), -1))[2]                        # the table lacks a held page
    assert not o.batch_plan([100], [5], 1, ring=8, n_swa=4)[2]                      # 4 - 1 + 5 = 8 slots
    out, _, bad = o.batch_plan([100], [6], 1, ring=8, n_swa=4)                      # one too few: the oldest key is gone
    assert bad and out["swa_slot"][0] == [-1, 98 % 8, 99 % 8, 100 % 8]
