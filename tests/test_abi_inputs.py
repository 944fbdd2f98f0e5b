"""Host-side checks of the step-input calls that need no GPU: struct layout, and
refusals by status code without a launch."""
import ctypes as C
import os
import subprocess
import tempfile

import pytest
import torch

from conftest import ROOT

FAKE = 0x10000  # a non-null, 16-B aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    from serving_lightning_indexer_gb300 import _build, csa2
    _build.build()
    return csa2.load()


def test_ctypes_structs_match_c_layout():
    from serving_lightning_indexer_gb300 import csa2
    pairs = [("csa2_quant_fp8_args", csa2.QuantFp8Args), ("csa2_fp8_linear_args", csa2.Fp8LinearArgs),
             ("csa2_batch_plan_args", csa2.BatchPlanArgs)]
    body = "".join(f'printf("%zu\\n", sizeof({c}));\n' + "".join(
        f'printf("%zu\\n", offsetof({c}, {f[0]}));\n' for f in py._fields_) for c, py in pairs)
    with tempfile.TemporaryDirectory() as d:
        with open(os.path.join(d, "s.c"), "w") as f:
            f.write(f'#include <stdio.h>\n#include <stddef.h>\n#include "csa2.h"\nint main(void) {{\n{body}return 0;\n}}\n')
        exe = os.path.join(d, "s")
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), os.path.join(d, "s.c"), "-o", exe], check=True)
        got = list(map(int, subprocess.run([exe], capture_output=True, text=True).stdout.split()))
    want = []
    for _, py in pairs:
        want += [C.sizeof(py)] + [getattr(py, f[0]).offset for f in py._fields_]
    assert got == want


def _quant(**kw):
    from serving_lightning_indexer_gb300 import csa2
    base = dict(x=FAKE, ld_x=256, T=4, K=256, block_rows=1, gamma=None, eps=1e-6, codes=FAKE, ld_codes=256, scale=FAKE,
                ld_scale=2)
    return csa2.QuantFp8Args(**{**base, **kw})


@pytest.mark.parametrize("kw,code,word", [
    ({"x": None}, 1, b"x/codes/scale"), ({"codes": None}, 1, b"x/codes/scale"), ({"scale": None}, 1, b"x/codes/scale"),
    ({"T": 0}, 2, b"T must"), ({"K": 0}, 2, b"K=0"), ({"K": 24}, 2, b"K=24"), ({"K": 16400, "ld_x": 16400}, 2, b"K=16400"),
    ({"block_rows": 64}, 4, b"block_rows"), ({"block_rows": 128, "gamma": FAKE}, 4, b"gamma"),
    ({"eps": -1.0}, 2, b"eps"), ({"eps": float("nan")}, 2, b"eps"), ({"eps": float("inf")}, 2, b"eps"),
    ({"ld_x": 240}, 2, b"stride"), ({"ld_codes": 240}, 2, b"stride"), ({"ld_scale": 1}, 2, b"stride"),
    ({"x": FAKE + 8}, 3, b"16-B"), ({"codes": FAKE + 4}, 3, b"16-B"), ({"gamma": FAKE + 4}, 3, b"16-B"),
    ({"ld_x": 260}, 3, b"ld_x"), ({"ld_codes": 264}, 3, b"ld_codes"), ({"scale": FAKE + 2}, 3, b"4-B"),
    ({"T": 2 ** 31 - 1, "K": 16384, "ld_x": 16384, "ld_codes": 16384, "ld_scale": 128}, 2, b"too many"),
])
def test_quant_fp8_refusals(lib, kw, code, word):
    a = _quant(**kw)
    assert lib.csa2_quant_fp8(C.byref(a), None) == code
    assert word in lib.csa2_last_error_detail()
    assert lib.csa2_quant_fp8(None, None) == 1


def _linear(**kw):
    from serving_lightning_indexer_gb300 import csa2
    base = dict(x=FAKE, ld_x=256, x_scale=FAKE, ld_x_scale=2, w=FAKE, ld_w=256, w_scale=FAKE, ld_w_scale=2, T=4, N=512,
                K=256, out_format=1, out=FAKE, ld_out=512, out_scale=None, ld_out_scale=0, row_pos=None, rope_head=0,
                rope_theta=0.0, w_ready=0)
    return csa2.Fp8LinearArgs(**{**base, **kw})


@pytest.mark.parametrize("kw,code,word", [
    ({"x": None}, 1, b"NULL"), ({"x_scale": None}, 1, b"NULL"), ({"w": None}, 1, b"NULL"), ({"w_scale": None}, 1, b"NULL"),
    ({"out": None}, 1, b"NULL"), ({"T": 0}, 2, b"T=0"), ({"N": 0}, 2, b"N=0"), ({"N": -5}, 2, b"N=-5"),
    ({"N": (1 << 28) + 1, "ld_out": 1 << 29}, 2, b"2^28"),
    ({"K": 8}, 2, b"K=8"), ({"K": 264}, 2, b"K=264"), ({"K": 65552, "ld_x": 65552, "ld_w": 65552}, 2, b"K=65552"),
    ({"ld_x": 240}, 2, b"stride"), ({"ld_w": 240}, 2, b"stride"), ({"ld_out": 511}, 2, b"stride"),
    ({"ld_x_scale": 1}, 2, b"stride"), ({"ld_w_scale": 1}, 2, b"stride"), ({"ld_x": 1 << 39}, 2, b"2^39"),
    ({"out_format": 3}, 4, b"out_format"), ({"out_format": -1}, 4, b"out_format"),
    ({"x": FAKE + 8}, 3, b"16-B"), ({"w": FAKE + 1}, 3, b"16-B"), ({"out": FAKE + 8}, 3, b"16-B"),
    ({"ld_x": 264}, 3, b"ld_x"), ({"ld_w": 264}, 3, b"ld_w"), ({"x_scale": FAKE + 2}, 3, b"4-B"),
    ({"out_format": 2}, 1, b"out_scale"), ({"out_format": 2, "out_scale": FAKE, "ld_out_scale": 3}, 2, b"ld_out_scale"),
    ({"out_format": 2, "out_scale": FAKE, "ld_out_scale": 4, "N": 500}, 2, b"multiple of 128"),
    ({"out_format": 2, "out_scale": FAKE, "ld_out_scale": 4, "ld_out": 520}, 3, b"ld_out"),
    ({"rope_head": 128}, 1, b"row_pos"), ({"rope_head": 64, "row_pos": FAKE}, 2, b"rope_head=64"),
    ({"rope_head": 192, "row_pos": FAKE}, 2, b"rope_head=192"), ({"rope_head": 384, "row_pos": FAKE}, 2, b"rope_head=384"),
    ({"rope_head": -128, "row_pos": FAKE}, 2, b"rope_head=-128"),
    ({"rope_head": 128, "row_pos": FAKE, "rope_theta": -1.0}, 2, b"rope_theta"),
    ({"rope_head": 128, "row_pos": FAKE, "rope_theta": float("nan")}, 2, b"rope_theta"),
    ({"w_ready": 2}, 2, b"w_ready"),
])
def test_fp8_linear_refusals(lib, kw, code, word):
    a = _linear(**kw)
    assert lib.csa2_fp8_linear(C.byref(a), None) == code
    assert word in lib.csa2_last_error_detail()
    assert lib.csa2_fp8_linear(None, None) == 1


@pytest.mark.parametrize("kw,code,word", [
    ({"ctx_len": None}, 1, b"ctx_len"), ({"new_len": None}, 1, b"ctx_len"), ({"B": 0}, 2, b"B=0"), ({"B": 8193}, 2, b"B=8193"),
    ({"ratio_m": 3}, 4, b"ratio_m"), ({"page_table": FAKE}, 2, b"pt_stride"), ({"entry_slot": FAKE}, 1, b"page_table"),
    ({"free_pages": FAKE}, 1, b"page_table"), ({"page_table": FAKE, "pt_stride": 1, "free_pages": FAKE, "n_free": -1}, 2, b"n_free"),
    ({"free_head": FAKE}, 1, b"free_pages"), ({"free_head_out": FAKE}, 1, b"free_pages"),
    ({"page_table": FAKE, "pt_stride": 1, "free_pages": FAKE, "free_head": FAKE, "free_head_out": FAKE}, 4, b"free_head_out"),
    ({"max_rows": -1}, 2, b"max_rows"), ({"max_entries": -1}, 2, b"max_entries"), ({"swa_new": FAKE}, 2, b"swa_ring"),
    ({"swa_slot": FAKE, "swa_ring": 128}, 2, b"n_swa=0"), ({"swa_slot": FAKE, "swa_ring": 128, "n_swa": 129, "ld_swa": 129}, 2, b"n_swa"),
    ({"swa_slot": FAKE, "swa_ring": 128, "n_swa": 8, "ld_swa": 7}, 2, b"ld_swa"), ({"pad": 2}, 2, b"pad"),
    ({"row_pos": FAKE + 2}, 3, b"4-B"),
])
def test_batch_plan_refusals(lib, kw, code, word):
    from serving_lightning_indexer_gb300 import csa2
    a = csa2.BatchPlanArgs(**{**dict(B=2, ctx_len=FAKE, new_len=FAKE, ratio_m=1), **kw})
    assert lib.csa2_batch_plan(C.byref(a), None) == code
    assert word in lib.csa2_last_error_detail()
    assert lib.csa2_batch_plan(None, None) == 1


def test_binding_refuses_what_it_cannot_pass():
    from serving_lightning_indexer_gb300 import csa2
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        csa2.quant_fp8(x, x, x)
    with pytest.raises(TypeError):
        csa2.quant_fp8([1.0], x, x)
    with pytest.raises(ValueError, match="CUDA"):
        csa2.fp8_linear(x.view(torch.uint8), x, x, x, x)
    n = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        csa2.batch_plan(n, n)


@pytest.mark.parametrize("T", [(1 << 30) + 1, (1 << 31) - 1])
def test_fp8_linear_refuses_rows_past_its_counters(lib, T):
    assert lib.csa2_fp8_linear(C.byref(_linear(T=T)), None) == 2
    assert b"2^30" in lib.csa2_last_error_detail()


_IN, _OUT = 0x100000, 0x200000   # 4-B aligned, never dereferenced, a megabyte apart


@pytest.mark.parametrize("kw", [
    {"n_visible": _IN}, {"n_visible": _IN + 7 * 4}, {"n_visible": _IN - 7 * 4}, {"row_start": _IN - 8 * 4},
    {"entry_start": _IN + 0x1000}, {"row_pos": _IN + 0x1000 - 15 * 4, "max_rows": 16},
    {"entry_pos": _IN + 7 * 4, "max_entries": 1}, {"swa_new": _IN, "swa_ring": 8, "max_rows": 1},
    {"swa_slot": _IN - 0x1000, "swa_ring": 8, "n_swa": 4, "ld_swa": 1024, "max_rows": 2},
    {"ring_id": _OUT, "row_seq": _OUT + 4, "max_rows": 3},
    {"page_table": _OUT, "pt_stride": 4, "free_pages": _OUT + 31 * 4, "n_free": 9},
    {"page_table": _OUT, "pt_stride": 4, "free_pages": _IN + 0x2000, "n_free": 9, "free_head": _OUT},
    {"page_table": _OUT, "pt_stride": 4, "free_pages": _IN + 0x2000, "n_free": 9, "free_head_out": _IN + 0x2000 + 32},
])
def test_batch_plan_refuses_outputs_over_inputs(lib, kw):
    """ctx_len and new_len of 8 sequences at _IN and _IN + 0x1000: a write over a word that
    other CTAs still read."""
    from serving_lightning_indexer_gb300 import csa2
    a = csa2.BatchPlanArgs(**{**dict(B=8, ctx_len=_IN, new_len=_IN + 0x1000, ratio_m=1), **kw})
    assert lib.csa2_batch_plan(C.byref(a), None) == 4
    assert b"overlaps" in lib.csa2_last_error_detail()
