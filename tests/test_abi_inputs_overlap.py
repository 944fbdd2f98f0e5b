"""csa2_batch_plan's check of outputs against inputs: which windows and tables it refuses
(no GPU: a call that passes the checks ends at the missing device)."""
import ctypes as C

import pytest
import torch

from test_abi_inputs import lib  # noqa: F401  (fixture)

_IN, _OUT = 0x100000, 0x200000   # 4-B aligned, never dereferenced, a megabyte apart


def _call(lib, **kw):  # noqa: F811
    from serving_lightning_indexer_gb300 import csa2
    a = csa2.BatchPlanArgs(**{**dict(B=8, ctx_len=_IN, new_len=_IN + 0x1000, ratio_m=1), **kw})
    rc = lib.csa2_batch_plan(C.byref(a), None)
    return rc, lib.csa2_last_error_detail()


WINDOW = dict(swa_ring=200, n_swa=128, ld_swa=256, max_rows=8)   # columns of a matrix of 256: 8 rows, 1,920 words


@pytest.mark.parametrize("kw", [
    {**WINDOW, "swa_slot": _IN - 1920 * 4 + 4}, {**WINDOW, "swa_slot": _IN + 7 * 4},
    {**WINDOW, "swa_slot": _IN - 256 * 4 + 4 * 7}, {**WINDOW, "swa_slot": _IN - (256 + 127) * 4},
    {**WINDOW, "swa_slot": _IN - 128 * 4, "ld_swa": 135},     # the second row starts on the last length
    {**WINDOW, "swa_slot": _IN - 127 * 4, "max_rows": 1, "ld_swa": 1 << 62},
    # the table is read for entry_slot, free pages or not
    {"page_table": _OUT, "pt_stride": 4, "entry_slot": _OUT, "max_entries": 1},
    {"page_table": _OUT, "pt_stride": 4, "entry_slot": _OUT + 31 * 4, "max_entries": 1},
    {"page_table": _OUT, "pt_stride": 4, "entry_slot": _OUT + 0x1000, "entry_row": _OUT - 4, "max_entries": 2},
    {"page_table": _OUT, "pt_stride": 4, "entry_slot": _OUT + 0x1000, "max_entries": 2, "row_seq": _OUT + 8, "max_rows": 1},
    {"page_table": _OUT, "pt_stride": 4, "entry_slot": _OUT + 0x1000, "max_entries": 2, "n_visible": _OUT - 7 * 4},
    {"page_table": _OUT, "pt_stride": 4, "free_pages": _IN + 0x2000, "n_free": 9, "entry_slot": _OUT, "max_entries": 2},
    {"page_table": _OUT, "pt_stride": 4, "free_pages": _IN + 0x2000, "n_free": 9, "entry_slot": _OUT + 0x1000,
     "row_pos": _OUT + 4, "max_entries": 2, "max_rows": 1},
])
def test_batch_plan_refuses_an_output_over_what_it_reads(lib, kw):  # noqa: F811
    rc, detail = _call(lib, **kw)
    assert rc == 4 and b"overlaps" in detail


@pytest.mark.skipif(torch.cuda.is_available(), reason="a call that passes the checks would be launched")
@pytest.mark.parametrize("kw", [
    {**WINDOW, "swa_slot": _IN - 1920 * 4},                   # the last row ends where the lengths begin
    {**WINDOW, "swa_slot": _IN + 8 * 4},                      # the first row begins where they end
    {**WINDOW, "swa_slot": _IN - 128 * 4},                    # they lie between two rows
    {**WINDOW, "swa_slot": _IN - 128 * 4, "ld_swa": 136},
    {**WINDOW, "swa_slot": _IN - 128 * 4, "max_rows": 1, "ld_swa": 1 << 62},
    {**WINDOW, "swa_slot": _IN - 128 * 4, "ld_swa": 1 << 62},
    {**WINDOW, "swa_slot": _IN, "max_rows": 0},
    {"page_table": _OUT, "pt_stride": 4, "entry_slot": _OUT + 32 * 4, "entry_pos": _OUT - 8, "max_entries": 2},
    {"page_table": _OUT, "pt_stride": 4, "free_pages": _OUT + 32 * 4, "n_free": 9, "entry_slot": _OUT - 8, "max_entries": 2},
])
def test_batch_plan_takes_an_output_beside_what_it_reads(lib, kw):  # noqa: F811
    rc, detail = _call(lib, **kw)
    assert rc == 5 and b"overlaps" not in detail
