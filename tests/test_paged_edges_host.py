"""The paged 8-bit cache without a GPU: refusals of calls whose output overlaps what they read."""
import pytest

import attention_decode_b200 as nsnq
from test_paged_host import FAKE, OTHER, _append, _attn, lib  # noqa: F401

FAR = 0x30000


@pytest.mark.parametrize("change", [
    dict(q=FAR, qo=FAKE), dict(q=FAR, qo=FAKE + 256 * 3 * 2), dict(q=FAR, qo=OTHER + 16), dict(q=FAR, qo=FAR + 1024),
    dict(q=FAR, qo=FAR - 16), dict(q=FAR, qt=1024, qo=FAR + 4096), dict(q=FAR, qo=OTHER - 16, dt=nsnq.NSNQ_F32, qt=512),
])
def test_append_refuses_overlapping_queries(lib, change):  # noqa: F811
    assert _append(lib, **change) == nsnq.NSNQ_ERR_INVALID_ARG and b"overlaps" in lib.nsnq_last_error()


@pytest.mark.parametrize("change", [
    dict(out=FAKE), dict(out=FAKE + 4080), dict(out=FAKE - 16), dict(out=FAKE - 8000, od=nsnq.NSNQ_F32),
    dict(n=1, cu=None, B=1, mr=1, qt=7, out=FAKE + 512),
])
def test_attention_refuses_an_output_over_its_queries(lib, change):  # noqa: F811
    got = _attn(lib, **dict(dict(wsb=1 << 40), **change))
    assert got == nsnq.NSNQ_ERR_INVALID_ARG and b"overlaps" in lib.nsnq_last_error(), lib.nsnq_last_error()
