"""Host-side checks of the calls around the layers that need no GPU: struct layout, and
refusals by status code without a launch."""
import ctypes as C
import os
import subprocess
import tempfile

import pytest
import torch

from conftest import ROOT

FAKE = 0x10000000  # non-null, 16-B aligned addresses that are never dereferenced, 16 MB apart
STEP = 1 << 24


@pytest.fixture(scope="module")
def lib():
    from serving_lightning_indexer_gb300 import _build, csa2
    _build.build()
    return csa2.load()


def test_ctypes_structs_match_c_layout():
    from serving_lightning_indexer_gb300 import csa2
    pairs = [("csa2_add_norm_fp8_args", csa2.AddNormFp8Args), ("csa2_lora_linear_args", csa2.LoraLinearArgs),
             ("csa2_logprobs_args", csa2.LogprobsArgs)]
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


def _norm(**kw):
    from serving_lightning_indexer_gb300 import csa2
    base = dict(x=FAKE, ld_x=256, residual=FAKE + STEP, ld_residual=256, residual_out=FAKE + 2 * STEP, ld_residual_out=256,
                residual_f32=0, T=4, K=256, gamma=FAKE + 3 * STEP, eps=1e-6, codes=FAKE + 4 * STEP, ld_codes=256,
                scale=FAKE + 5 * STEP, ld_scale=2, y=FAKE + 6 * STEP, ld_y=256)
    return csa2.AddNormFp8Args(**{**base, **kw})


@pytest.mark.parametrize("kw,code,word", [
    ({"x": None}, 1, b"NULL"), ({"residual": None}, 1, b"NULL"), ({"residual_out": None}, 1, b"NULL"), ({"gamma": None}, 1, b"NULL"),
    ({"codes": None, "scale": None, "y": None}, 1, b"one of codes, y"), ({"scale": None}, 1, b"together"),
    ({"codes": None}, 1, b"together"), ({"T": 0}, 2, b"T must"), ({"K": 0}, 2, b"K=0"), ({"K": 24}, 2, b"K=24"),
    ({"K": 16400}, 2, b"K=16400"), ({"residual_f32": 2}, 4, b"residual_f32"), ({"eps": -1.0}, 2, b"eps"),
    ({"eps": float("nan")}, 2, b"eps"), ({"ld_x": 240}, 2, b"stride"), ({"ld_residual": 240}, 2, b"stride"),
    ({"ld_residual_out": 240}, 2, b"stride"), ({"ld_codes": 240}, 2, b"stride"), ({"ld_scale": 1}, 2, b"stride"),
    ({"ld_y": 240}, 2, b"stride"), ({"ld_y": 1 << 29}, 2, b"2^29"), ({"x": FAKE + 8}, 3, b"16-B"), ({"residual": FAKE + STEP + 4}, 3, b"16-B"),
    ({"residual_out": FAKE + 2 * STEP + 2}, 3, b"16-B"), ({"codes": FAKE + 4 * STEP + 8}, 3, b"16-B"), ({"y": FAKE + 6 * STEP + 8}, 3, b"16-B"),
    ({"gamma": FAKE + 3 * STEP + 4}, 3, b"16-B"), ({"ld_x": 260}, 3, b"16-B"), ({"ld_residual": 260}, 3, b"16-B"),
    ({"ld_residual_out": 258, "residual_f32": 1}, 3, b"16-B"), ({"ld_codes": 264}, 3, b"16-B"), ({"ld_y": 260}, 3, b"16-B"),
    ({"scale": FAKE + 2}, 3, b"4-B"),
    # outputs over inputs and over each other
    ({"residual_out": FAKE + STEP, "ld_residual_out": 512}, 4, b"input"), ({"residual_out": FAKE}, 4, b"input"),
    ({"residual_out": FAKE + STEP + 1024}, 4, b"input"), ({"codes": FAKE + 16}, 4, b"input"), ({"y": FAKE}, 4, b"input"),
    ({"y": FAKE + 3 * STEP + 1008}, 4, b"input"), ({"scale": FAKE + 3 * STEP}, 4, b"input"),
    ({"codes": FAKE + 6 * STEP + 512}, 4, b"outputs"), ({"y": FAKE + 2 * STEP}, 4, b"outputs"),
    ({"scale": FAKE + 4 * STEP + 1020, "ld_scale": 64}, 4, b"outputs"),
    # windows of one buffer whose rows meet
    ({"ld_residual": 512, "ld_residual_out": 512, "residual_out": FAKE + STEP + 504 * 2}, 4, b"input"),
    ({"ld_residual": 512, "ld_residual_out": 512, "residual_out": FAKE + STEP + 248 * 2}, 4, b"input"),
])
def test_add_norm_refusals(lib, kw, code, word):
    assert lib.csa2_add_norm_fp8(C.byref(_norm(**kw)), None) == code
    assert word in lib.csa2_last_error_detail()
    assert lib.csa2_add_norm_fp8(None, None) == 1


def _lora(base=None, **kw):
    from serving_lightning_indexer_gb300 import csa2
    lin = dict(x=FAKE, ld_x=256, x_scale=FAKE, ld_x_scale=2, w=FAKE, ld_w=256, w_scale=FAKE, ld_w_scale=2, T=4, N=512,
               K=256, out_format=1, out=FAKE, ld_out=512, out_scale=None, ld_out_scale=0, row_pos=None, rope_head=0,
               rope_theta=0.0, w_ready=0)
    args = dict(base=csa2.Fp8LinearArgs(**{**lin, **(base or {})}), row_adapter=FAKE, n_adapters=3, rank=16, a=FAKE, b=FAKE,
                adapter_scale=FAKE)
    return csa2.LoraLinearArgs(**{**args, **kw})


@pytest.mark.parametrize("base,kw,code,word", [
    ({"x": None}, {}, 1, b"csa2_lora_linear: x/"), ({"T": 0}, {}, 2, b"T=0"), ({"K": 264}, {}, 2, b"K=264"),
    ({"out_format": 2}, {}, 1, b"out_scale"), ({"rope_head": 128}, {}, 1, b"row_pos"), ({"w_ready": 2}, {}, 2, b"w_ready"),
    ({"T": (1 << 20) + 1}, {}, 2, b"2^20"), ({}, {"row_adapter": None}, 1, b"row_adapter"), ({}, {"a": None}, 1, b"row_adapter/a/b"),
    ({}, {"b": None}, 1, b"row_adapter/a/b"), ({}, {"rank": 0}, 2, b"rank=0"), ({}, {"rank": 12}, 2, b"rank=12"),
    ({}, {"rank": 136}, 2, b"rank=136"), ({}, {"rank": -8}, 2, b"rank=-8"), ({}, {"n_adapters": 0}, 2, b"n_adapters=0"),
    ({}, {"n_adapters": (1 << 21) + 1}, 2, b"n_adapters"), ({"N": 1}, {"n_adapters": (1 << 23) + 1, "rank": 128}, 2, b"rank at most"), ({}, {"a": FAKE + 8}, 3, b"16-B"), ({}, {"b": FAKE + 8}, 3, b"16-B"),
    ({}, {"row_adapter": FAKE + 2}, 3, b"4-B"), ({}, {"adapter_scale": FAKE + 2}, 3, b"4-B"),
])
def test_lora_linear_refusals(lib, base, kw, code, word):
    from serving_lightning_indexer_gb300 import csa2
    a = _lora(base, **kw)
    assert lib.csa2_lora_linear(C.byref(a), FAKE, 1 << 30, None) == code
    assert word in lib.csa2_last_error_detail()
    size = C.c_size_t(7)
    assert lib.csa2_workspace_size(csa2.CALL_LORA_LINEAR, C.cast(C.byref(a), C.c_void_p), C.byref(size)) == code
    assert lib.csa2_lora_linear(None, FAKE, 1 << 30, None) == 1


def test_lora_linear_workspace(lib):
    from serving_lightning_indexer_gb300 import csa2
    a = _lora()
    size = C.c_size_t(0)
    assert lib.csa2_workspace_size(csa2.CALL_LORA_LINEAR, C.cast(C.byref(a), C.c_void_p), C.byref(size)) == 0
    assert size.value >= 2 * 2 * 4 * 16 and size.value == csa2.lora_workspace_size(4, 16)
    assert lib.csa2_lora_linear(C.byref(a), None, size.value, None) == 7
    assert lib.csa2_lora_linear(C.byref(a), FAKE, size.value - 1, None) == 7 and b"needed" in lib.csa2_last_error_detail()
    assert lib.csa2_lora_linear(C.byref(a), FAKE + 8, size.value, None) == 3


@pytest.mark.parametrize("T", [1, 15, 16, 17, 64, 127, 128, 129, 1000, 1 << 20])
@pytest.mark.parametrize("rank", [8, 24, 128])
def test_lora_workspace_holds_every_tile_height(lib, T, rank):
    """Inner products [3][T][rank, to a multiple of 64] in bf16, then (rows + 4) words for each tile of 16, 32, 64 or 128 rows."""
    from serving_lightning_indexer_gb300 import csa2
    v = -(-6 * T * (-(-rank // 64) * 64) // 256) * 256
    assert csa2.lora_workspace_size(T, rank) >= v + max(-(-T // rows) * (rows + 4) * 4 for rows in (16, 32, 64, 128))


def _logprobs(**kw):
    from serving_lightning_indexer_gb300 import csa2
    base = dict(logits=FAKE, ld_logits=1000, logits_f32=1, T=4, V=1000, token=FAKE, logprob=FAKE, entropy=FAKE, lse=FAKE, n_top=5,
                top_id=FAKE, top_logprob=FAKE, ld_top=5)
    return csa2.LogprobsArgs(**{**base, **kw})


@pytest.mark.parametrize("kw,code,word", [
    ({"logits": None}, 1, b"logits"), ({"token": None}, 1, b"together"), ({"logprob": None}, 1, b"together"),
    ({"token": None, "logprob": None, "entropy": None, "lse": None, "top_id": None, "top_logprob": None, "n_top": 0}, 1, b"no output"),
    ({"T": 0}, 2, b"T=0"), ({"T": (1 << 27) + 1}, 2, b"T="), ({"V": 0}, 2, b"V=0"), ({"V": (1 << 30) + 1, "ld_logits": 1 << 31}, 2, b"V="),
    ({"logits_f32": 2}, 4, b"logits_f32"), ({"n_top": 33, "ld_top": 33}, 2, b"n_top"), ({"n_top": -1}, 2, b"n_top"),
    ({"n_top": 0}, 1, b"n_top"), ({"top_id": None, "top_logprob": None}, 1, b"n_top"), ({"ld_logits": 999}, 2, b"stride"),
    ({"ld_top": 4}, 2, b"stride"), ({"ld_logits": 1 << 32}, 2, b"2^32"), ({"logits": FAKE + 2}, 3, b"logits"),
    ({"logits": FAKE + 1, "logits_f32": 0}, 3, b"logits"), ({"token": FAKE + 2}, 3, b"4-B"), ({"top_id": FAKE + 1}, 3, b"4-B"),
])
def test_logprobs_refusals(lib, kw, code, word):
    assert lib.csa2_logprobs(C.byref(_logprobs(**kw)), None) == code
    assert word in lib.csa2_last_error_detail()
    assert lib.csa2_logprobs(None, None) == 1


def test_binding_refuses_what_it_cannot_pass():
    from serving_lightning_indexer_gb300 import csa2
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    u, f, i = x.view(torch.uint8), x.float(), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        csa2.add_norm_fp8(x, x, x, f[0])
    with pytest.raises(TypeError):
        csa2.add_norm_fp8(None, x, x, f[0])
    with pytest.raises(ValueError, match="CUDA"):
        csa2.lora_linear(u, f, u, f, x[None], x[None], i, f)
    with pytest.raises(ValueError, match="CUDA"):
        csa2.logprobs(f)
    with pytest.raises(TypeError):
        csa2.logprobs([1.0])
