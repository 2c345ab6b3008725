"""Refusals of the copy that lays codes and scales out, without a GPU: every
argument error is reported before any HIP call."""

import pytest

nsd = pytest.importorskip("newton_schulz_dmuon_amd")
from newton_schulz_dmuon_amd import _lib  # noqa: E402

A, B = 0x7F0000000000, 0x7F0100000000
BAD, MIS, ALIAS = _lib.ERR_INVALID_ARG, _lib.ERR_MISALIGNED, _lib.ERR_ALIAS


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), BAD), (dict(rows=(1 << 29) + 1), BAD), (dict(cols=-16), BAD), (dict(cols=24), BAD),
    (dict(cols=(1 << 29) + 16), BAD), (dict(rows=1 << 22, cols=(1 << 14) + 16), BAD), (dict(row_step=-1), BAD),
    (dict(col_step=-1), BAD), (dict(row_step=1 << 62), BAD), (dict(col_step=1 << 62), BAD), (dict(row_step=1 << 46), BAD),
    (dict(src=None), BAD), (dict(out=None), BAD), (dict(out=B + 8), MIS), (dict(src=B), ALIAS), (dict(out=A + 256), ALIAS),
    (dict(src=B - 63 * 256 - 127), ALIAS), (dict(src=B + 64 * 128 - 1), ALIAS), (dict(rows=0, src=None), _lib.OK),
    (dict(cols=0, out=None), _lib.OK)])
def test_copy_refusals(kw, want):
    d = dict(src=A, rows=64, cols=128, row_step=256, col_step=1, out=B)
    d.update(kw)
    assert _lib.load().dmuon_q4_copy(*(d[n] for n in ("src", "rows", "cols", "row_step", "col_step", "out")), None) == want
