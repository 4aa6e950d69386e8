"""Window attention's gradient where o and lse are those of more keys than the call's, and these others hold little weight:
the sum of P is next to 1 and yet delta must not be taken from these keys alone.  Tolerances: those of
tests/test_gpu_window.py; their term 2^-8 sum |dO||O| of each delta, there for the rounding of o, is not used up by it here
(the oracle has the rounded o too) and is what a row may be off by whose other keys cannot be told from rounding."""
import numpy as np
import pytest
import torch

from oracle import window as O
from tests._gpu import ra_lib, check_status
from tests.test_gpu_serving import BF, dev
from tests.test_gpu_window import assert_grads, packed, parts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ra():
    return ra_lib()


def more_keys(q, k, v, do, qsl, window, sink, weight, size):
    """o and lse with other keys that hold `weight` of each row, whose values point where dO does, `size` long each way."""
    ref = O.window_attn(q, k, v, qsl, window, sink)
    w = weight[..., None]
    o = torch.from_numpy(ref[0]) * (1 - w) + size * torch.sign(do.double()) * w
    return o.to(BF), (torch.from_numpy(ref[1]) - torch.log1p(-weight)).float()


@pytest.mark.parametrize("n,window,sink", [([300, 41], 60, 3), ([700], 600, 0), ([3] * 40, 2, 0)], ids=["short", "long", "pairs"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lo,hi,size", [(1e-4, 9e-4, 100.0), (1e-5, 1e-4, 100.0), (1e-4, 9e-4, 1.0), (1e-7, 1e-5, 1000.0)])
def test_other_keys_of_little_weight(ra, n, window, sink, d, lo, hi, size):
    Hq, Hkv, T = 6, 2, sum(n)
    x, do, qsl = packed(d, n, Hq, Hkv, d)
    x[:, :Hq] = x[:, :Hq].abs()                   # what delta is off by adds up in dK
    q, k, v = parts(x, Hq, Hkv)
    g = torch.Generator().manual_seed(5)
    weight = lo * (hi / lo) ** torch.rand((T, Hq), generator=g, dtype=torch.float64)
    o, lse = more_keys(q, k, v, do, qsl, window, sink, weight, size)
    want, bound = O.window_attn_grad(do, q, k, v, qsl, window, sink, o=o, lse=lse)
    xd, dd, sd, od, ld = dev(x, do, qsl, o, lse)
    got = ra.window_attn_bwd(dd, *parts(xd, Hq, Hkv), od, ld, sd, window, n_sink=sink)
    check_status(ra)
    assert_grads(got, (want, bound))


@pytest.mark.parametrize("d", [64, 128])
def test_all_keys_are_still_told(ra, d):
    """With o and lse of these keys the rounding of o stays out of dK, as before: with it dK is off by 0.003 of its norm and more
    where values share a direction; without it by dS's own rounding, at most 2^-8 of each term and sqrt(1/3) of that on
    average, and 2^-11 for the weights."""
    n, Hq, Hkv, window = [500], 8, 2, 400
    x, do, qsl = packed(d + 1, n, Hq, Hkv, d)
    x[:, :Hq] = x[:, :Hq].abs()
    x[:, Hq + Hkv:] += 2.0
    q, k, v = parts(x, Hq, Hkv)
    ref = O.window_attn(q, k, v, qsl, window, 0)
    want = O.window_attn_grad(do, q, k, v, qsl, window, 0)[0][1]
    o, lse = torch.from_numpy(ref[0]).to(BF), torch.from_numpy(ref[1]).float()
    xd, dd, sd, od, ld = dev(x, do, qsl, o, lse)
    dk = ra.window_attn_bwd(dd, *parts(xd, Hq, Hkv), od, ld, sd, window, out_dtype=torch.float32)[1].double().cpu().numpy()
    check_status(ra)
    assert np.linalg.norm(dk - want) <= (3 ** -0.5 * 2.0 ** -8 + 2.0 ** -11) * np.linalg.norm(want)
