"""Windows and numbers of first tokens past 32 bits mean what they say: no window, all tokens."""
import pytest
import torch

from tests._gpu import ra_lib, check_status
from tests.test_gpu_serving import batch, dev, paged
from tests.test_gpu_window import i32, packed, parts

pytestmark = pytest.mark.gpu
FAR = 2 ** 31 - 1


@pytest.fixture(scope="module")
def ra():
    return ra_lib()


@pytest.mark.parametrize("window,sink,like", [(2 ** 32 + 5, 0, (FAR, 0)), (2 ** 64 + 1, 0, (FAR, 0)), (9, 2 ** 32 + 3, (9, FAR)),
                                              (2 ** 31, 2 ** 33, (FAR, FAR))])
def test_reach_past_32_bits(ra, window, sink, like):
    x, do, qsl = packed(1, [90, 40], 4, 2, 64)
    xd, dd, sd = dev(x, do, qsl)
    q, k, v = parts(xd, 4, 2)
    o, lse = ra.window_attn_fwd(q, k, v, sd, window, n_sink=sink)
    want = ra.window_attn_fwd(q, k, v, sd, like[0], n_sink=like[1])
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    for a, b in zip(ra.window_attn_bwd(dd, q, k, v, o, lse, sd, window, n_sink=sink),
                    ra.window_attn_bwd(dd, q, k, v, o, lse, sd, like[0], n_sink=like[1])):
        assert torch.equal(a, b)
    ctx = [70, 33]
    kc, vc, table, _ = paged(2, ctx, 2, 64, 16, 16, 1, 1)
    qp, qslp = batch(2, [20, 1], 4, 64)
    args = dev(qp, kc, vc, table, qslp, i32(*ctx))
    for a, b in zip(ra.cp_window_attn(*args, window, 16, 1, 1, n_sink=sink), ra.cp_window_attn(*args, like[0], 16, 1, 1, n_sink=like[1])):
        assert torch.equal(a, b)
    check_status(ra)


def test_windows_below_one_are_still_refused(ra):
    x, _, qsl = packed(1, [9], 2, 1, 64)
    xd, sd = dev(x, qsl)
    for window, sink in ((0, 0), (-1, 0), (-2 ** 31, 0), (5 - 2 ** 32, 0), (4, -1), (4, 3 - 2 ** 32)):
        with pytest.raises(ra.RingAttnError):
            ra.window_attn_fwd(*parts(xd, 2, 1), sd, window, n_sink=sink)
