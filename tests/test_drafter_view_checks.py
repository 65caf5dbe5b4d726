"""Which views of q and o, and which scales, stv_paged_attn takes: checked on the host, so no
GPU is needed, nor used where there is one: the workspace is too small."""
import pytest

import speculative_tree_verify_bit_gb300 as stv
from test_drafter_checks import BAD, D, SMALL, call_attn, lib, rows, shape  # noqa: F401  (lib: a fixture)

HD, HQ = 128, 24
ROW = 2 * HQ * HD


@pytest.mark.parametrize("q,o,n_rows,fits", [
    # beside q in its rows, on either side
    (rows(D, ROW, HD, HQ), rows(D + 2 * HQ * HD, ROW, HD, HQ), 2, True),
    (rows(D + 2 * HQ * HD, ROW, HD, HQ), rows(D, ROW, HD, HQ), 2, True),
    # the other half of each head
    (rows(D, ROW, 2 * HD, HQ), rows(D + 2 * HD, ROW, 2 * HD, HQ), 2, True),
    (rows(D, ROW, 2 * HD, HQ), rows(D + 2 * HD, ROW, 2 * HD, HQ), 1, True),
    (rows(D + 2 * HD, ROW, 2 * HD, HQ), rows(D, ROW, 2 * HD, HQ), 7, True),
    # over q by one element, by a head, in another row
    (rows(D, ROW, 2 * HD, HQ), rows(D + 2 * HD - 2, ROW, 2 * HD, HQ), 2, False),
    (rows(D, ROW, 2 * HD, HQ), rows(D + 4 * HD, ROW, 2 * HD, HQ), 2, False),
    (rows(D, ROW, HD, HQ), rows(D + 2 * ROW, ROW, HD, HQ), 2, False),
    (rows(D, ROW, HD, HQ), rows(D + 2 * ROW, ROW, HD, HQ), 1, True),
    (rows(D, ROW, HD, HQ), rows(D + 2 * HQ * HD - 2, ROW, HD, HQ), 3, False),
    (rows(D, ROW, HD, HQ), rows(D + 2 * HQ * HD, ROW + HD, HD, HQ), 2, False),
])
def test_o_beside_q(lib, q, o, n_rows, fits):  # noqa: F811
    rc = call_attn(lib, q=q, o=o, n_rows=n_rows, n=1, s=shape(hd=HD), ws_bytes=0)
    assert rc == BAD if not fits else rc in (SMALL, stv.STV_ERR_CUDA), rc


@pytest.mark.parametrize("scale,fits", [(1e-45, True), (1.0, True), (2.3e38, True), (2.4e38, False), (3.4e38, False)])
def test_scales(lib, scale, fits):  # noqa: F811
    """The kernels multiply by scale log2(e), which has to be finite."""
    rc = call_attn(lib, spec=stv.make_attn(scale=scale), ws_bytes=0)
    assert rc == BAD if not fits else rc in (SMALL, stv.STV_ERR_CUDA), rc
