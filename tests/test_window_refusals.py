"""Host-side refusals of the window attention, the rotating store and the rotary positions with several axes, and sizes
with nothing to do: validation happens before any CUDA call (no GPU needed)."""
import ctypes
import os

import pytest
import torch

c_f, c_d = ctypes.c_float, ctypes.c_double


@pytest.fixture(scope="module")
def ra():
    from context_long_sequence_ring_gb300 import build, ringattn
    if not os.path.exists(build.LIB):
        build.build()
    return ringattn


def at(x):
    return ctypes.c_void_p(x << 24)      # never dereferenced


def caller(ra, name, order, base):
    def run(**kw):
        assert set(kw) <= set(base), kw
        a = dict(base, **kw)
        return getattr(ra.lib(), name)(*[a[k] for k in order.split()], None)
    return run


def test_cp_window_attn(ra):
    run = caller(ra, "ra_cp_window_attn", "q k v table qsl ctx T R Hq Hkv d bs I pcp dcp max_vb nb window sink scale o dt lse ws n",
                 dict(q=at(1), k=at(2), v=at(3), table=at(4), qsl=at(5), ctx=at(6), T=4, R=2, Hq=8, Hkv=2, d=128, bs=32, I=16,
                      pcp=1, dcp=1, max_vb=4, nb=9, window=100, sink=4, scale=c_f(0.0), o=at(7), dt=1, lse=at(8), ws=at(9),
                      n=1 << 30))
    bad, no = ra.RA_ERR_INVALID_ARG, ra.RA_ERR_UNSUPPORTED
    assert run(window=0) == bad and "window" in ra.last_error()
    assert run(window=-2 ** 31) == bad and run(sink=-1) == bad and "n_sink" in ra.last_error()
    assert run(Hq=7) == bad and "multiple of Hkv" in ra.last_error()
    assert run(R=0) == bad and run(T=-1) == bad and run(T=2 ** 29) == bad and run(nb=2 ** 31) == bad
    assert run(I=24) == bad and "interleave" in ra.last_error()
    assert run(d=96) == no and run(Hq=130) == no and run(bs=24, I=8) == no
    assert run(dt=2) == bad and run(n=1000) == bad and "workspace" in ra.last_error()
    for x in ("q", "k", "v", "o", "ws"):
        assert run(**{x: None}) == bad and "NULL" in ra.last_error()
        assert run(**{x: ctypes.c_void_p((1 << 28) + 8)}) == bad and "aligned" in ra.last_error()
    for x in ("table", "qsl", "ctx"):
        assert run(**{x: None}) == bad
    assert run(T=0) == ra.RA_OK and run(T=0, q=None) == ra.RA_OK
    n = ctypes.c_size_t(0)
    assert ra.lib().ra_cp_window_attn_workspace_size(8, 2, 128, ctypes.byref(n)) == 0 and n.value > 0
    assert ra.lib().ra_cp_window_attn_workspace_size(0, 2, 128, ctypes.byref(n)) == bad
    assert ra.lib().ra_cp_window_attn_workspace_size(8, 2, 128, None) == bad


def test_window_attn(ra):
    base = dict(q=at(1), qrs=1536, k=at(2), krs=1536, v=at(3), vrs=1536, o=at(7), lse=at(8), do=at(10), qsl=at(5), T=4, R=2,
                Hq=8, Hkv=2, d=128, window=100, sink=4, scale=c_f(0.0), dt=1, ws=at(9), n=1 << 32, dq=at(11), dqrs=1536,
                dk=at(12), dkrs=1536, dv=at(13), dvrs=1536)
    fwd = caller(ra, "ra_window_attn_fwd", "q qrs k krs v vrs qsl T R Hq Hkv d window sink scale o dt lse ws n", base)
    bwd = caller(ra, "ra_window_attn_bwd", "q qrs k krs v vrs o lse do qsl T R Hq Hkv d window sink scale dq dqrs dk dkrs dv dvrs "
                                           "dt ws n", base)
    bad, no = ra.RA_ERR_INVALID_ARG, ra.RA_ERR_UNSUPPORTED
    for run in (fwd, bwd):
        assert run(window=0) == bad and "window" in ra.last_error()
        assert run(sink=-1) == bad and run(R=0) == bad and run(T=-1) == bad and run(T=2 ** 29) == bad
        assert run(Hq=7) == bad and "multiple of Hkv" in ra.last_error()
        assert run(d=96) == no and run(Hq=130) == no and run(dt=2) == bad
        assert run(qrs=1020) == bad and run(krs=255) == bad and run(vrs=248) == bad and "strides" in ra.last_error()
        assert run(qrs=1537) == bad and run(krs=257) == bad and "multiples" in ra.last_error()
        assert run(n=64) == bad and "workspace" in ra.last_error()
        for x in ("q", "k", "v", "o", "ws"):
            assert run(**{x: None}) == bad
            assert run(**{x: ctypes.c_void_p((1 << 28) + 8)}) == bad and "aligned" in ra.last_error()
        assert run(qsl=None) == bad
        assert run(T=0) == ra.RA_OK
    for x in ("lse", "do", "dq", "dk", "dv"):
        assert bwd(**{x: None}) == bad
    for x in ("do", "dq", "dk", "dv"):
        assert bwd(**{x: ctypes.c_void_p((1 << 28) + 8)}) == bad and "aligned" in ra.last_error()
    assert bwd(dqrs=1000) == bad and bwd(dkrs=1537) == bad and bwd(dvrs=1540) == bad and "16 bytes" in ra.last_error()
    n = ctypes.c_size_t(0)
    size = ra.lib().ra_window_attn_workspace_size
    assert size(1000, 2, 8, 2, 128, ctypes.byref(n)) == 0 and n.value > 0
    assert size(1000, 2, 8, 2, 128, None) == bad and size(-1, 2, 8, 2, 128, ctypes.byref(n)) == bad
    assert size(2 ** 29, 2, 8, 2, 128, ctypes.byref(n)) == bad and size(1000, 0, 8, 2, 128, ctypes.byref(n)) == bad


def test_rope_apply_axes(ra):
    f = (c_d * 32)(*[0.5] * 32)
    ax = (ctypes.c_int32 * 32)(*[i % 3 for i in range(32)])
    run = caller(ra, "ra_rope_apply_axes", "src srs shs dst drs dhs rows H d rot dt style pos n f axis m back",
                 dict(src=at(1), srs=512, shs=64, dst=at(2), drs=512, dhs=64, rows=5, H=8, d=64, rot=64, dt=1, style=0, pos=at(3),
                      n=3, f=f, axis=ax, m=c_d(1.0), back=0))
    bad = ra.RA_ERR_INVALID_ARG
    assert run(n=2) == bad and "axis" in ra.last_error()
    assert run(n=0) == bad and run(n=17) == bad and run(axis=None) == bad
    assert run(axis=(ctypes.c_int32 * 32)(*[-1] * 32)) == bad
    assert run(rot=66) == bad and run(rot=7) == bad and run(rot=0) == bad
    assert run(f=None) == bad and run(f=(c_d * 32)(*[7.0] * 32)) == bad and run(f=(c_d * 32)(*[float("nan")] * 32)) == bad
    assert run(m=c_d(float("inf"))) == bad and run(dt=3) == bad and run(style=2) == bad
    assert run(src=None) == bad and run(pos=None) == bad and run(dst=None) == bad
    assert run(dst=at(1), drs=1024) == bad and "overlap" in ra.last_error()
    assert run(dhs=32) == bad and "alias" in ra.last_error()
    assert run(srs=-1) == bad and run(rows=-1) == bad
    assert run(src=ctypes.c_void_p((1 << 24) + 1)) == bad
    assert run(rows=0) == ra.RA_OK


def test_cp_rope_append(ra):
    f = (c_d * 32)(*[0.5] * 32)
    ax = (ctypes.c_int32 * 32)(*[i % 3 for i in range(32)])
    run = caller(ra, "ra_cp_rope_append", "k krs khs v vrs vhs q qrs qhs qo qors qohs kc vc table qsl ctx T R Hq Hkv d dt bs I pcp "
                                          "dcp max_vb nb pos n rot style f axis m",
                 dict(k=at(1), krs=768, khs=64, v=at(2), vrs=768, vhs=64, q=at(3), qrs=768, qhs=64, qo=at(4), qors=512, qohs=64,
                      kc=at(5), vc=at(6), table=at(7), qsl=at(8), ctx=at(9), T=4, R=2, Hq=8, Hkv=2, d=64, dt=1, bs=20, I=4,
                      pcp=1, dcp=2, max_vb=4, nb=9, pos=at(10), n=3, rot=64, style=0, f=f, axis=ax, m=c_d(1.0)))
    bad, no = ra.RA_ERR_INVALID_ARG, ra.RA_ERR_UNSUPPORTED
    assert run(I=3) == bad and run(R=0) == bad and run(nb=0) == bad and run(T=-1) == bad and run(T=2 ** 31) == bad
    assert run(dt=2) == bad and run(d=68, rot=0, f=None) == no and run(d=2048) == bad
    assert run(n=2) == bad and run(axis=None) == bad and run(pos=None) == bad and "positions" in ra.last_error()
    assert run(rot=66) == bad and run(rot=0) == bad and run(f=None) == bad and "rot" in ra.last_error()
    assert run(style=2) == bad and run(m=c_d(float("nan"))) == bad
    for x in ("k", "v", "qo", "kc", "vc", "table", "qsl", "ctx"):
        assert run(**{x: None}) == bad and "NULL" in ra.last_error()
    assert run(kc=ctypes.c_void_p((5 << 24) + 8)) == bad and "aligned" in ra.last_error()
    assert run(k=ctypes.c_void_p((1 << 24) + 1)) == bad and "aligned" in ra.last_error()
    assert run(krs=-1) == bad and run(vhs=2 ** 41) == bad and run(qors=-1) == bad
    assert run(kc=at(6)) == bad and run(k=at(5)) == bad and run(v=at(6)) == bad and run(q=at(5)) == bad and run(qo=at(6)) == bad
    assert "overlap" in ra.last_error()
    assert run(qo=at(3)) == bad and run(qo=at(1)) == bad and run(qohs=32) == bad and "alias" in ra.last_error()
    assert run(T=0) == ra.RA_OK
    assert run(T=0, q=None, Hq=0) == ra.RA_OK


def test_the_binding_checks_shapes_before_the_library(ra):
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    s = torch.zeros(2, dtype=torch.int32)
    f = torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError):
        ra.window_attn_fwd(x, x, x, s, 4)                       # not on a GPU
    with pytest.raises(ValueError):
        ra.window_attn_bwd(x, x, x, x, x, torch.zeros((3, 2)), s, 4)
    with pytest.raises(ValueError):
        ra.cp_window_attn(x, x, x, s, s, s, 4, 16, 1, 1)
    with pytest.raises(ValueError):
        ra.rope_apply_axes(x, torch.zeros((2, 3), dtype=torch.int32), f, torch.zeros(32, dtype=torch.int32))
    with pytest.raises(ValueError):
        ra.cp_rope_append(x, x, x, x, s, s, s, 16, 1, 1)
