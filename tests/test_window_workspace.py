"""A workspace that lies over an input or an output of the window attention and the chunk attention is refused on the host,
before any CUDA call (no GPU needed)."""
import ctypes
import os

import pytest

from tests.test_window_refusals import caller, c_f

MB = 1 << 20


@pytest.fixture(scope="module")
def ra():
    from context_long_sequence_ring_gb300 import build, ringattn
    if not os.path.exists(build.LIB):
        build.build()
    return ringattn


def at(mb, more=0):
    return ctypes.c_void_p((1 << 32) + mb * MB + more)      # never dereferenced


def refused(ra, st):
    return st == ra.RA_ERR_INVALID_ARG and "workspace must not overlap" in ra.last_error()


def sweep(ra, run, need, sizes):
    """Each tensor over the workspace's last 16 bytes, at its start, and with its own last bytes at its start."""
    ws = 512
    for x, size in sizes.items():
        for byte in (need - 16, 0, -((size - 1) // 16) * 16):
            assert refused(ra, run(ws=at(ws), n=need, **{x: at(ws, byte)})), (x, byte)


def test_packed(ra):
    T, R, Hq, Hkv, d = 100, 2, 8, 2, 128
    base = dict(q=at(1), qrs=1536, k=at(2), krs=1536, v=at(3), vrs=1536, o=at(7), lse=at(8), do=at(10), qsl=at(5), T=T, R=R,
                Hq=Hq, Hkv=Hkv, d=d, window=100, sink=4, scale=c_f(0.0), dt=0, ws=at(512), n=0, dq=at(11), dqrs=1536, dk=at(12),
                dkrs=1536, dv=at(13), dvrs=1536)
    fwd = caller(ra, "ra_window_attn_fwd", "q qrs k krs v vrs qsl T R Hq Hkv d window sink scale o dt lse ws n", base)
    bwd = caller(ra, "ra_window_attn_bwd", "q qrs k krs v vrs o lse do qsl T R Hq Hkv d window sink scale dq dqrs dk dkrs dv dvrs "
                                           "dt ws n", base)
    n = ctypes.c_size_t(0)
    assert ra.lib().ra_window_attn_workspace_size(T, R, Hq, Hkv, d, ctypes.byref(n)) == 0
    rows, kv = 2 * ((T - 1) * 1536 + Hq * d), 2 * ((T - 1) * 1536 + Hkv * d)
    common = dict(q=rows, k=kv, v=kv, qsl=12, lse=T * Hq * 4)
    es = 4                                       # of outputs in RA_F32
    sweep(ra, fwd, n.value, dict(common, o=T * Hq * d * es))
    sweep(ra, bwd, n.value, dict(common, o=T * Hq * d * 2, do=T * Hq * d * 2, dq=es * ((T - 1) * 1536 + Hq * d),
                                       dk=es * ((T - 1) * 1536 + Hkv * d), dv=es * ((T - 1) * 1536 + Hkv * d)))


@pytest.mark.parametrize("name", ["ra_cp_window_attn", "ra_cp_chunk_attn"])
def test_paged(ra, name):
    window = "window" in name
    T, R, Hq, Hkv, d, bs, W, nb = 50, 3, 8, 2, 64, 32, 2, 9
    base = dict(q=at(1), k=at(2), v=at(3), table=at(4), qsl=at(5), ctx=at(6), T=T, R=R, Hq=Hq, Hkv=Hkv, d=d, bs=bs, I=16,
                pcp=1, dcp=W, max_vb=4, nb=nb, window=100, sink=4, causal=1, scale=c_f(0.0), o=at(7), dt=1, lse=at(8), ws=at(512),
                n=0)
    run = caller(ra, name, "q k v table qsl ctx T R Hq Hkv d bs I pcp dcp max_vb nb " + ("window sink" if window else "causal") +
                 " scale o dt lse ws n", base)
    n = ctypes.c_size_t(0)
    assert getattr(ra.lib(), name + "_workspace_size")(Hq, Hkv, d, ctypes.byref(n)) == 0
    cache = W * nb * Hkv * bs * d * 2
    sweep(ra, run, n.value, dict(q=T * Hq * d * 2, k=cache, v=cache, table=R * 4 * 4, qsl=16, ctx=12, o=T * Hq * d * 2,
                                       lse=T * Hq * 4))
