"""Outputs over inputs or over each other: refused by csa2_lora_linear and csa2_logprobs on the
host, and nothing else is.  Layouts that share a buffer without a byte in common are run on a
GPU; here the rule itself is tried against all bytes of small layouts."""
import ctypes as C
import os
import re
import subprocess

import pytest
import torch

from conftest import ROOT
from gpu_util import need_gpu

FAKE, STEP = 0x10000000, 1 << 24   # addresses that are never dereferenced: every call here is refused


@pytest.fixture(scope="module")
def lib():
    from serving_lightning_indexer_gb300 import _build, csa2
    _build.build()
    return csa2.load()


def _lora(base, kw):
    from serving_lightning_indexer_gb300 import csa2
    lin = dict(x=FAKE, ld_x=256, x_scale=FAKE + STEP, ld_x_scale=2, w=FAKE + 2 * STEP, ld_w=256, w_scale=FAKE + 3 * STEP, ld_w_scale=2,
               T=4, N=512, K=256, out_format=1, out=FAKE + 4 * STEP, ld_out=512, out_scale=None, ld_out_scale=0, row_pos=None,
               rope_head=0, rope_theta=0.0, w_ready=0)
    return csa2.LoraLinearArgs(**{**dict(base=csa2.Fp8LinearArgs(**{**lin, **base}), row_adapter=FAKE + 5 * STEP, n_adapters=3, rank=16,
                                         a=FAKE + 6 * STEP, b=FAKE + 7 * STEP, adapter_scale=FAKE + 8 * STEP), **kw})


WS = FAKE + 16 * STEP
FP8 = {"out_format": 2, "ld_out_scale": 4, "out_scale": FAKE + 10 * STEP}


@pytest.mark.parametrize("base,kw,ws,word", [
    ({"out": FAKE + 512}, {}, WS, b"input"), ({"out": FAKE + STEP + 16}, {}, WS, b"input"), ({"out": FAKE + 2 * STEP + 512 * 255}, {}, WS, b"input"),
    ({"out": FAKE + 3 * STEP}, {}, WS, b"input"), ({"out": FAKE + 5 * STEP}, {}, WS, b"input"), ({"out": FAKE + 6 * STEP + 3 * 16 * 256 * 2 - 16}, {}, WS, b"input"),
    ({"out": FAKE + 7 * STEP}, {}, WS, b"input"), ({"out": FAKE + 8 * STEP}, {}, WS, b"input"),
    ({"rope_head": 128, "row_pos": FAKE + 9 * STEP, "out": FAKE + 9 * STEP}, {}, WS, b"input"),
    ({**FP8, "out_scale": FAKE + STEP + 28}, {}, WS, b"input"), ({**FP8, "out_scale": FAKE + 4 * STEP + 4 * 512 - 4}, {}, WS, b"outputs"),
    ({}, {}, FAKE, b"input"), ({}, {}, FAKE + 4 * STEP, b"outputs"), (FP8, {}, FAKE + 10 * STEP, b"outputs"), ({}, {}, FAKE + 5 * STEP, b"input"),
    ({"ld_out": 1 << 62, "T": 2, "out": FAKE}, {}, WS, b"input"),
])
def test_lora_linear_refuses_overlaps(lib, base, kw, ws, word):
    a = _lora(base, kw)
    assert lib.csa2_lora_linear(C.byref(a), ws, 1 << 24, None) == 4
    assert word in lib.csa2_last_error_detail()


@pytest.mark.parametrize("kw,word", [
    ({"lse": FAKE + 3996}, b"input"), ({"logprob": FAKE + 4 * 4000 - 4}, b"input"), ({"entropy": FAKE}, b"input"), ({"top_id": FAKE + 16}, b"input"),
    ({"top_logprob": FAKE + 4000}, b"input"), ({"top_logprob": FAKE + 4 * STEP + 16}, b"outputs"), ({"lse": FAKE + 2 * STEP + 12}, b"outputs"),
    ({"ld_logits": 1100, "ld_top": 1100, "top_id": FAKE + 4 * 996}, b"input"), ({"ld_logits": 1100, "lse": FAKE + 4 * 1098}, b"input"),
])
def test_logprobs_refuses_overlaps(lib, kw, word):
    from serving_lightning_indexer_gb300 import csa2
    base = dict(logits=FAKE, ld_logits=1000, logits_f32=1, T=4, V=1000, token=FAKE + STEP, logprob=FAKE + 2 * STEP, entropy=FAKE + 3 * STEP,
                lse=FAKE + 6 * STEP, n_top=5, top_id=FAKE + 4 * STEP, top_logprob=FAKE + 5 * STEP, ld_top=5)
    assert lib.csa2_logprobs(C.byref(csa2.LogprobsArgs(**{**base, **kw})), None) == 4
    assert word in lib.csa2_last_error_detail()


def test_the_rule_is_exact(tmp_path):
    """ByteRows::meets as it stands in the library's source, against sets of bytes."""
    with open(os.path.join(ROOT, "serving_lightning_indexer_gb300", "csrc", "csa2_api.cu")) as f:
        text = f.read()
    rule = re.search(r"struct ByteRows \{.*?\n\};", text, re.S).group(0)
    src = tmp_path / "meets.cpp"
    src.write_text("#include <stdint.h>\n#include <stdio.h>\n#include <stdlib.h>\n#include <set>\n" + rule + r"""
int main() {
  srand(7);
  for (int k = 0; k < 200000; ++k) {
    ByteRows r[2];
    std::set<long long> bytes[2];
    for (int i = 0; i < 2; ++i) {
      const long long n = 1 + rand() % 9, rows = 1 + rand() % 6, ld = n + rand() % 12, at = 1000 + rand() % 90;
      r[i] = ByteRows{reinterpret_cast<const void*>(at), n, rows, i && rand() % 3 == 0 && r[0].ld >= n ? r[0].ld : ld};
      for (long long q = 0; q < rows; ++q)
        for (long long b = 0; b < n; ++b) bytes[i].insert(at + q * r[i].ld + b);
    }
    bool meet = false;
    for (long long b : bytes[0]) meet = meet || bytes[1].count(b);
    if (r[0].meets(r[1]) != meet || r[1].meets(r[0]) != meet) return printf("case %d\n", k), 1;
  }
  return 0;
}
""")
    exe = str(tmp_path / "meets")
    subprocess.run(["g++", "-O1", "-std=c++17", str(src), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


@pytest.mark.gpu
def test_outputs_between_the_rows_of_an_input():
    """Results in the columns behind the logits, and an output whose rows lie between an input's."""
    from serving_lightning_indexer_gb300 import csa2
    dev = need_gpu()
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    T, V, n = 9, 5000, 6
    wide = torch.zeros(T, V + 32, device=dev)
    x = wide[:, :V]
    x.copy_(torch.randn(T, V, generator=g, device=dev))
    want = [torch.empty(T, n, dtype=torch.int32, device=dev), torch.empty(T, n, device=dev), torch.empty(T, device=dev)]
    csa2.logprobs(x, top_id=want[0], top_logprob=want[1], lse=want[2])
    ids, top, lse = wide.view(torch.int32)[:, V:V + n], wide[:, V + n:V + 2 * n], wide[3, V + 2 * n:V + 2 * n + T]
    csa2.logprobs(x, top_id=ids, top_logprob=top, lse=lse)
    torch.cuda.synchronize()
    assert torch.equal(ids, want[0]) and torch.equal(top, want[1]) and torch.equal(lse, want[2])
    with pytest.raises(csa2.Csa2Error, match="overlaps an input"):
        csa2.logprobs(x, lse=wide[3, V - 1:V - 1 + T])
    # codes in the first half of each row, the projection in the second
    T, K, N = 5, 256, 128
    room = torch.zeros(T, 1024, dtype=torch.uint8, device=dev)
    codes = room[:, :K]
    codes.copy_(torch.randint(0, 120, (T, K), generator=g, device=dev, dtype=torch.uint8))
    w = torch.randint(0, 120, (N, K), generator=g, device=dev, dtype=torch.uint8)
    xs, ws = torch.ones(T, 2, device=dev), torch.ones(1, 2, device=dev)
    a, b = (torch.randn(2, *s, generator=g, device=dev).to(torch.bfloat16) for s in ((16, K), (N, 16)))
    ids = torch.tensor([0, 1, -1, 1, 0], dtype=torch.int32, device=dev)
    first, second = torch.empty(T, N, device=dev), room[:, 512:].view(torch.float32)
    csa2.lora_linear(codes, xs, w, ws, a, b, ids, first)
    csa2.lora_linear(codes, xs, w, ws, a, b, ids, second)
    torch.cuda.synchronize()
    assert csa2.check_device_error() == 0 and torch.equal(first, second)
    with pytest.raises(csa2.Csa2Error, match="overlaps an input"):
        csa2.lora_linear(codes, xs, w, ws, a, b, ids, room[:, :512].view(torch.float32))
