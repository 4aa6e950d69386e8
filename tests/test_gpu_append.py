"""GPU parity of the store that rotates new keys on their way into the sharded paged cache, and of rotary positions with
several axes, against the float64 oracle and against the calls that they are made of.  Tolerances of a rotation as in
tests/test_gpu_serving.py: 2^-19 (|a| + |b|) plus the output's rounding."""
import numpy as np
import pytest
import torch

from oracle import window as O
from tests._gpu import ra_lib, check_status
from tests.test_gpu_serving import BF, DEV, assert_chunk, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ra():
    return ra_lib()


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


def assert_turned(y, ref, x, rot, style, mscale, dt):
    """|error| <= 2^-19 mscale (|a| + |b|) + half a step; what is not turned is equal."""
    y, x = y.double().cpu().numpy(), x.double().cpu().numpy()
    half = rot // 2
    mag = np.zeros_like(x)
    u, v = (slice(0, half), slice(half, rot)) if style == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    mag[..., u] = mag[..., v] = np.abs(x[..., u]) + np.abs(x[..., v])
    step = 2.0 ** -8 if dt == BF else 2.0 ** -24
    assert (np.abs(y - ref) <= 2.0 ** -19 * mscale * mag + step * np.abs(ref)).all()
    assert np.array_equal(y[..., rot:], x[..., rot:])


# ---------------------------------------------------------------------- rotary positions with several axes

# rows, H, extra heads, d, rot, axis (by pair), style
AXES = [
    (1, 1, 0, 32, 32, "sections", "half"),
    (7, 3, 2, 128, 128, "sections", "half"),
    (33, 5, 0, 80, 40, "turns", "interleaved"),
    (64, 40, 8, 128, 64, "turns", "half"),
    (50, 4, 1, 72, 24, "sections", "interleaved"),
    (19, 2, 0, 22, 10, "turns", "half"),          # no whole words
    (19, 2, 0, 21, 6, "sections", "interleaved"),
    (300, 9, 0, 256, 256, "sections", "half"),
]


def axis_of(kind, half, n):
    return i32(*[(i * n // half if kind == "sections" else i % n) for i in range(half)])


@pytest.mark.parametrize("case", AXES, ids=lambda c: "r%d-h%d.%d-d%d.%d-%s-%s" % c)
@pytest.mark.parametrize("dt", [BF, torch.float32])
@pytest.mark.parametrize("n_axes", [2, 3, 16])
def test_axes(ra, case, dt, n_axes):
    rows, H, extra, d, rot, kind, style = case
    g = torch.Generator().manual_seed(rows)
    x = torch.randn((rows, H + extra, d), generator=g).to(dt)
    pos = torch.randint(0, 2 ** 24, (n_axes, rows), generator=g).to(torch.int32)
    f, m = ra.rope_frequencies(rot, scaling="yarn", factor=4.0)
    axis = axis_of(kind, rot // 2, n_axes)
    xd, pd = dev(x, pos)
    for backward in (False, True):
        y = ra.rope_apply_axes(xd[:, :H], pd, f, axis, m, style, backward)
        check_status(ra)
        ref = O.rope_apply_axes(x[:, :H], pos.numpy(), f.numpy(), axis.numpy(), m, style, backward)
        assert_turned(y, ref, x[:, :H], rot, style, m, dt)
        # strided out, and in place
        z = torch.full((rows, H + 2, d), 7.0, dtype=dt, device=DEV)
        ra.rope_apply_axes(xd[:, :H], pd, f, axis, m, style, backward, out=z[:, 1:1 + H])
        assert torch.equal(z[:, 1:1 + H], y) and (z[:, 0] == 7).all() and (z[:, -1] == 7).all()
        w = xd.clone()
        ra.rope_apply_axes(w[:, :H], pd, f, axis, m, style, backward, out=w[:, :H])
        assert torch.equal(w[:, :H], y) and torch.equal(w[:, H:], xd[:, H:])
        # equal positions on all axes: one axis, to the bit
        same = pd[:1].expand(n_axes, rows).contiguous()
        a = ra.rope_apply_axes(xd[:, :H], same, f, axis, m, style, backward)
        assert torch.equal(a, ra.rope_apply(xd[:, :H], pd[0].contiguous(), f, m, style, backward=backward))
    check_status(ra)


def test_axes_strides_and_the_gradient(ra):
    """Rows and heads in other orders, unaligned starts; the gradient is the transpose, against differences."""
    g = torch.Generator().manual_seed(5)
    rows, H, d, rot = 40, 6, 64, 48
    f, _ = ra.rope_frequencies(rot)
    axis = axis_of("sections", rot // 2, 3)
    pos = torch.randint(0, 5000, (3, rows), generator=g).to(torch.int32).to(DEV)
    x = torch.randn((rows, H, d), generator=g).to(DEV)
    want = ra.rope_apply_axes(x, pos, f, axis)
    for view in (x.transpose(0, 1).contiguous().transpose(0, 1), torch.empty((rows, H, d + 1), device=DEV)[:, :, 1:].copy_(x),
                 torch.empty((rows, 2 * H, d), device=DEV)[:, ::2].copy_(x)):
        assert torch.equal(ra.rope_apply_axes(view, pos, f, axis), want)
    # one row for all: stride 0
    one = ra.rope_apply_axes(x[:1].expand(rows, H, d), pos, f, axis)
    assert torch.equal(one, ra.rope_apply_axes(x[:1].expand(rows, H, d).contiguous(), pos, f, axis))
    dy = torch.randn((rows, H, d), generator=g).to(DEV)
    dx = ra.rope_apply_axes(dy, pos, f, axis, backward=True).double().cpu().numpy()
    check_status(ra)
    loss = lambda t: (O.rope_apply_axes(t, pos.cpu().numpy(), f.numpy(), axis.numpy()) * dy.double().cpu().numpy()).sum()  # noqa: E731
    xs = x.double().cpu().numpy()
    for seed in range(3):
        u = np.random.default_rng(seed).standard_normal(xs.shape)
        diff = (loss(xs + 1e-3 * u) - loss(xs - 1e-3 * u)) / 2e-3
        assert abs(diff - (dx * u).sum()) <= 2.0 ** -18 * np.abs(u).sum() * float(dy.abs().max()) + 1e-6


def test_axes_bad_positions(ra):
    x = torch.randn((3, 2, 16), device=DEV)
    f, _ = ra.rope_frequencies(16)
    axis = i32(0, 0, 0, 0, 1, 1, 1, 1)
    for bad in (-1, 2 ** 24, -2 ** 31):
        pos = torch.zeros((3, 3), dtype=torch.int32, device=DEV)
        pos[1, 1] = bad
        y = ra.rope_apply_axes(x, pos, f, axis)
        assert ra.device_status() == ra.RA_ERR_DEVICE_BOUNDS and torch.equal(y, x)
        pos[1, 1], pos[2, 1] = 0, bad                   # of an axis that no pair has: not looked at
        ra.rope_apply_axes(x, pos, f, axis)
        check_status(ra)
    assert ra.rope_apply_axes(x[:0], torch.zeros((2, 0), dtype=torch.int32, device=DEV), f, axis).shape == (0, 2, 16)
    check_status(ra)


# ---------------------------------------------------------------------- the store

# ctx, n, Hq, Hkv, d, rot, bs, I, pcp, dcp, axes, style
STORES = [
    ([1], [1], 4, 2, 128, 128, 128, 16, 1, 1, 0, "half"),
    ([1, 2, 129, 127], [1, 1, 1, 1], 8, 1, 64, 32, 16, 16, 1, 1, 0, "interleaved"),
    ([300, 5, 77], [3, 5, 1], 6, 2, 128, 128, 32, 4, 2, 2, 0, "half"),
    ([257, 0, 300, 128], [33, 0, 300, 128], 6, 2, 64, 64, 64, 16, 1, 2, 3, "half"),
    ([700], [260], 5, 5, 80, 40, 128, 128, 2, 4, 3, "interleaved"),
    ([130, 500, 20], [130, 66, 20], 16, 1, 64, 48, 16, 1, 1, 3, 0, "half"),
    ([40, 33], [7, 5], 3, 3, 72, 22, 8, 2, 1, 1, 0, "half"),        # pairs that are no whole words
    ([40, 33], [7, 5], 3, 3, 72, 22, 24, 8, 1, 2, 2, "interleaved"),
    ([90], [90], 2, 2, 64, 0, 5, 5, 1, 1, 0, "half"),               # nothing turned, odd blocks
    ([2000], [600], 40, 8, 128, 128, 128, 16, 2, 4, 0, "half"),
]


def store_inputs(case, dt, seed=0, before=0, after=0):
    ctx, n, Hq, Hkv, d, rot, bs, I, pcp, dcp, axes, style = case
    g = torch.Generator().manual_seed(seed + sum(ctx))
    W, V = pcp * dcp, bs * pcp * dcp
    nvb = [-(-x // V) for x in ctx]
    nb = sum(nvb) + 2
    ids = torch.randperm(nb, generator=g).to(torch.int32)
    table = torch.full((len(ctx), max(nvb) + 1), -1, dtype=torch.int32)
    at = 0
    for r, m in enumerate(nvb):
        table[r, :m] = ids[at:at + m]
        at += m
    qsl = torch.tensor(np.concatenate([[before], before + np.cumsum(n)]), dtype=torch.int32)
    T = int(qsl[-1]) + after
    x = torch.randn((T, Hq + 2 * Hkv, d), generator=g).to(dt)
    kc, vc = (torch.randn((W, nb, Hkv, bs, d), generator=g).to(dt) for _ in range(2))
    pos = torch.randint(0, 2 ** 20, (axes or 1, T), generator=g).to(torch.int32)
    return x, kc, vc, table, qsl, pos


def turned(ra, x, pos, f, axis, m, style):
    if f is None:
        return x.clone()
    return ra.rope_apply(x, pos[0].contiguous(), f, m, style) if axis is None else ra.rope_apply_axes(x, pos, f, axis, m, style)


@pytest.mark.parametrize("case", STORES, ids=lambda c: "%s-%s-h%d.%d-d%d.%d-b%d.%d-w%d-a%d-%s" % (
    c[0], c[1], c[2], c[3], c[4], c[5], c[6], c[7], c[8] * c[9], c[10], c[11]))
@pytest.mark.parametrize("dt", [BF, torch.float32])
def test_store(ra, case, dt):
    ctx, n, Hq, Hkv, d, rot, bs, I, pcp, dcp, axes, style = case
    x, kc, vc, table, qsl, pos = store_inputs(case, dt, before=2, after=3)
    f, m, axis = None, 1.0, None
    if rot:
        f, m = ra.rope_frequencies(rot, scaling="yarn", factor=2.0)
        axis = axis_of("sections", rot // 2, axes) if axes else None
    xd, kd, vd, td, sd, pd, cd = dev(x, kc, vc, table, qsl, pos, i32(*ctx))
    q, k, v = xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:]
    kt, qt = turned(ra, k, pd, f, axis, m, style), turned(ra, q, pd, f, axis, m, style)
    check_status(ra)
    want_k, want_v = O.cp_rope_append(kt.double().cpu(), v.double().cpu(), kc, vc, table.numpy(), qsl, ctx, bs, I, pcp, dcp)
    if rot:
        p = pos.numpy()
        full = O.rope_apply_axes(k.double().cpu(), p if axes else p[:1], f.numpy(), axis.numpy() if axes else [0] * (rot // 2),
                                 m, style)
        assert_turned(kt, full, k, rot, style, m, dt)
    given = None if f is None else (pd if axes else pd[0].contiguous())
    qo = torch.full((x.shape[0], Hq, d), 7.0, dtype=dt, device=DEV)
    a, b = kd.clone(), vd.clone()
    got = ra.cp_rope_append(k, v, a, b, td, sd, cd, I, pcp, dcp, positions=given, inv_freq=f, axis=axis, mscale=m, style=style,
                            q=q, q_out=qo)
    check_status(ra)
    assert got is qo
    assert np.array_equal(a.double().cpu().numpy(), want_k) and np.array_equal(b.double().cpu().numpy(), want_v)
    mine = slice(2, x.shape[0] - 3)
    assert torch.equal(qo[mine], qt[mine]) and (qo[:2] == 7).all() and (qo[-3:] == 7).all()
    # without q, and with q in place
    a, b = kd.clone(), vd.clone()
    assert ra.cp_rope_append(k, v, a, b, td, sd, cd, I, pcp, dcp, positions=given, inv_freq=f, axis=axis, mscale=m,
                             style=style) is None
    y = xd.clone()
    a2, b2 = kd.clone(), vd.clone()
    yq, yk, yv = y[:, :Hq], y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:]
    ra.cp_rope_append(yk, yv, a2, b2, td, sd, cd, I, pcp, dcp, positions=given, inv_freq=f, axis=axis, mscale=m, style=style,
                      q=yq, q_out=yq)
    check_status(ra)
    for c in (a, a2):
        assert np.array_equal(c.double().cpu().numpy(), want_k)
    for c in (b, b2):
        assert np.array_equal(c.double().cpu().numpy(), want_v)
    assert torch.equal(yq[mine], qt[mine]) and torch.equal(y[:, Hq:], xd[:, Hq:])
    assert torch.equal(yq[:2], q[:2]) and torch.equal(yq[-3:], q[-3:])


# the same with so many tokens that a warp takes one instead of a block
MANY_TOKENS = [
    ([1500], [1111], 6, 2, 128, 128, 32, 4, 1, 2, 0, "half"),
    ([5, 0, 997, 3, 800], [5, 0, 700, 1, 300], 5, 3, 64, 32, 16, 16, 1, 1, 3, "interleaved"),
    ([i % 9 + 3 for i in range(700)], [i % 4 for i in range(700)], 4, 1, 80, 40, 16, 2, 1, 2, 0, "half"),
    ([1300, 40], [1233, 7], 3, 3, 72, 22, 8, 2, 1, 1, 2, "interleaved"),       # pairs that are no whole words
    ([2000], [913], 9, 1, 64, 0, 5, 5, 1, 1, 0, "half"),                       # nothing turned
    ([1000], [908], 1, 1, 8, 8, 16, 16, 1, 1, 0, "half"),                      # less work than a warp has threads
]


@pytest.mark.parametrize("case", MANY_TOKENS, ids=lambda c: "n%d-h%d.%d-d%d.%d-a%d-%s" % (
    sum(c[1]), c[2], c[3], c[4], c[5], c[10], c[11]))
@pytest.mark.parametrize("dt", [BF, torch.float32])
def test_store_many_tokens(ra, case, dt):
    test_store(ra, case, dt)


def test_store_positions_default_to_the_place(ra):
    case = ([300, 41], [30, 41], 4, 2, 64, 64, 16, 4, 1, 2, 0, "half")
    ctx, n, Hq, Hkv, d, rot, bs, I, pcp, dcp, _, style = case
    x, kc, vc, table, qsl, _ = store_inputs(case, BF)
    f, _ = ra.rope_frequencies(rot)
    xd, kd, vd, td, sd, cd = dev(x, kc, vc, table, qsl, i32(*ctx))
    q, k, v = xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:]
    place = torch.cat([torch.arange(c - m, c, dtype=torch.int32) for c, m in zip(ctx, n)]).to(DEV)
    a, b, a2, b2 = kd.clone(), vd.clone(), kd.clone(), vd.clone()
    qo = ra.cp_rope_append(k, v, a, b, td, sd, cd, I, pcp, dcp, inv_freq=f, q=q)
    q2 = ra.cp_rope_append(k, v, a2, b2, td, sd, cd, I, pcp, dcp, positions=place, inv_freq=f, q=q)
    check_status(ra)
    assert torch.equal(a, a2) and torch.equal(b, b2) and torch.equal(qo, q2)
    # the four calls that it replaces
    slot = ra.cp_slot_mapping(sd, place, td, bs, I, pcp, dcp)
    a3, b3 = kd.clone(), vd.clone()
    ra.cp_kv_scatter(ra.rope_apply(k, place, f), v.contiguous(), slot, a3, b3)
    check_status(ra)
    assert torch.equal(a, a3) and torch.equal(b, b3) and torch.equal(qo, ra.rope_apply(q, place, f))


def test_store_strides(ra):
    """k and v in another order of rows and heads, off their words, and one row for all tokens."""
    case = ([50], [33], 4, 2, 64, 32, 16, 16, 1, 1, 0, "interleaved")
    ctx, n, Hq, Hkv, d, rot, bs, I, pcp, dcp, _, style = case
    x, kc, vc, table, qsl, pos = store_inputs(case, BF)
    f, _ = ra.rope_frequencies(rot)
    xd, kd, vd, td, sd, pd, cd = dev(x, kc, vc, table, qsl, pos[0].contiguous(), i32(*ctx))
    k, v = xd[:, Hq:Hq + Hkv].contiguous(), xd[:, Hq + Hkv:].contiguous()

    def run(k, v):
        a, b = kd.clone(), vd.clone()
        ra.cp_rope_append(k, v, a, b, td, sd, cd, I, pcp, dcp, positions=pd, inv_freq=f, style=style)
        check_status(ra)
        return a, b

    want = run(k, v)
    off = torch.empty((33, Hkv, d + 1), dtype=BF, device=DEV)[:, :, 1:]
    off2 = torch.empty((33, Hkv, d + 4), dtype=BF, device=DEV)[:, :, 4:]
    for kk, vv in ((k.transpose(0, 1).contiguous().transpose(0, 1), v), (off.copy_(k), v), (k, off2.copy_(v))):
        assert all(torch.equal(a, b) for a, b in zip(run(kk, vv), want))
    same = k[:1].expand(33, Hkv, d)
    assert all(torch.equal(a, b) for a, b in zip(run(same, same), run(same.contiguous(), same.contiguous())))


@pytest.mark.parametrize("T", [1, 33])
def test_store_in_place_in_a_projection_by_heads(ra, T):
    """q, k and v of each head side by side, [T, H, 3, d], q turned in place between them."""
    case = ([50], [T], 2, 2, 64, 64, 16, 16, 1, 1, 0, "half")
    ctx, n, H, _, d, rot, bs, I, pcp, dcp, _, style = case
    _, kc, vc, table, qsl, pos = store_inputs(case, BF)
    x = torch.randn((T, H, 3, d), generator=torch.Generator().manual_seed(3)).to(BF).to(DEV)
    f, _ = ra.rope_frequencies(rot)
    kd, vd, td, sd, pd, cd = dev(kc, vc, table, qsl, pos[0].contiguous(), i32(*ctx))
    a, b, y = kd.clone(), vd.clone(), x.clone()
    want = ra.cp_rope_append(x[:, :, 1], x[:, :, 2], kd, vd, td, sd, cd, I, pcp, dcp, positions=pd, inv_freq=f, q=x[:, :, 0])
    ra.cp_rope_append(y[:, :, 1], y[:, :, 2], a, b, td, sd, cd, I, pcp, dcp, positions=pd, inv_freq=f, q=y[:, :, 0],
                      q_out=y[:, :, 0])
    check_status(ra)
    assert torch.equal(a, kd) and torch.equal(b, vd) and torch.equal(y[:, :, 0], want) and torch.equal(y[:, :, 1:], x[:, :, 1:])
    with pytest.raises(ra.RingAttnError):      # k itself
        ra.cp_rope_append(y[:, :, 0], y[:, :, 2], a, b, td, sd, cd, I, pcp, dcp, positions=pd, inv_freq=f, q=y[:, :, 0],
                          q_out=y[:, :, 0])


def test_store_many_requests_and_empty_ones(ra):
    rng = np.random.default_rng(3)
    n = rng.choice([0, 0, 0, 1, 1, 2, 5], size=700)
    ctx = (n + rng.integers(0, 40, size=700)).tolist()
    case = (ctx, n.tolist(), 2, 1, 64, 64, 16, 4, 1, 1, 0, "half")
    x, kc, vc, table, qsl, pos = store_inputs(case, BF)
    f, _ = ra.rope_frequencies(64)
    xd, kd, vd, td, sd, pd, cd = dev(x, kc, vc, table, qsl, pos, i32(*ctx))
    k, v = xd[:, 2:3], xd[:, 3:]
    kt = ra.rope_apply(k, pd[0].contiguous(), f)
    want = O.cp_rope_append(kt.double().cpu(), v.double().cpu(), kc, vc, table.numpy(), qsl, ctx, 16, 4, 1, 1)
    ra.cp_rope_append(k, v, kd, vd, td, sd, cd, 4, 1, 1, positions=pd[0].contiguous(), inv_freq=f)
    check_status(ra)
    assert np.array_equal(kd.double().cpu().numpy(), want[0]) and np.array_equal(vd.double().cpu().numpy(), want[1])


def test_store_bad_blocks_places_and_ranges(ra):
    case = ([40, 33], [7, 5], 4, 2, 64, 64, 16, 16, 1, 1, 0, "half")
    ctx, n, Hq, Hkv, d, rot, bs, I, pcp, dcp, _, style = case
    x, kc, vc, table, qsl, pos = store_inputs(case, BF)
    f, _ = ra.rope_frequencies(rot)
    xd, kd, vd, td, sd, pd, cd = dev(x, kc, vc, table, qsl, pos[0].contiguous(), i32(*ctx))
    k, v = xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:]

    def run(table=td, qsl=sd, ctx=cd, positions=pd):
        a, b = kd.clone(), vd.clone()
        ra.cp_rope_append(k, v, a, b, table, qsl, ctx, I, pcp, dcp, positions=positions, inv_freq=f)
        return ra.device_status(), a, b

    st, good_k, good_v = run()
    assert st == 0
    for bad in (-1, kc.shape[1], 2 ** 31 - 1, -2 ** 31):
        t = td.clone()
        t[1, 2] = bad                                    # token 32 of request 1
        st, a, b = run(table=t)
        assert st == ra.RA_ERR_DEVICE_BOUNDS
        blk = int(table[1, 2])
        assert torch.equal(a[0, blk], kd[0, blk]) and torch.equal(b[0, blk], vd[0, blk])
        rest = [i for i in range(kc.shape[1]) if i != blk]
        assert torch.equal(a[0, rest], good_k[0, rest]) and torch.equal(b[0, rest], good_v[0, rest])
    for c in (i32(3, 33), i32(40, 2 ** 31 - 1), i32(-2 ** 31, 33), i32(40, 65)):
        st, a, b = run(ctx=c.to(DEV))                    # places below 0 or past the table
        assert st == ra.RA_ERR_DEVICE_BOUNDS
    for s in (i32(0, 9, 4), i32(-3, 7, 12), i32(0, 7, 13), i32(0, 2 ** 31 - 1, 12)):
        st, a, b = run(qsl=s.to(DEV))
        assert st == ra.RA_ERR_DEVICE_BOUNDS
    for bad in (-1, 2 ** 24):
        p = pd.clone()
        p[3] = bad
        st, a, b = run(positions=p)
        assert st == ra.RA_ERR_DEVICE_BOUNDS and torch.equal(b, good_v)
    check_status(ra)


def test_store_no_tokens(ra):
    case = ([40], [7], 4, 2, 64, 64, 16, 16, 1, 1, 0, "half")
    x, kc, vc, table, _, _ = store_inputs(case, BF)
    f, _ = ra.rope_frequencies(64)
    kd, vd, td = dev(kc, vc, table)
    e = torch.zeros((0, 2, 64), dtype=BF, device=DEV)
    s = torch.zeros(2, dtype=torch.int32, device=DEV)
    q = ra.cp_rope_append(e, e, kd, vd, td, s, i32(40).to(DEV), 16, 1, 1, inv_freq=f, q=torch.zeros((0, 4, 64), dtype=BF, device=DEV))
    check_status(ra)
    assert q.shape == (0, 4, 64) and torch.equal(kd.cpu(), kc)


def test_store_replayed_with_other_lengths_on_two_streams(ra):
    Hq, Hkv, d, bs, I, pcp, dcp, T = 4, 2, 64, 16, 4, 1, 2, 60
    f, _ = ra.rope_frequencies(64)
    sets = []
    for _ in range(2):
        st = dict(x=torch.zeros((T, Hq + 2 * Hkv, d), dtype=BF, device=DEV), kc=torch.zeros((2, 40, Hkv, bs, d), dtype=BF, device=DEV),
                  vc=torch.zeros((2, 40, Hkv, bs, d), dtype=BF, device=DEV), t=torch.zeros((3, 12), dtype=torch.int32, device=DEV),
                  s=torch.zeros(4, dtype=torch.int32, device=DEV), c=torch.zeros(3, dtype=torch.int32, device=DEV),
                  p=torch.zeros(T, dtype=torch.int32, device=DEV), qo=torch.zeros((T, Hq, d), dtype=BF, device=DEV))

        def call(st=st):
            x = st["x"]
            ra.cp_rope_append(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], st["kc"], st["vc"], st["t"], st["s"], st["c"], I, pcp, dcp,
                              positions=st["p"], inv_freq=f, q=x[:, :Hq], q_out=st["qo"])

        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        sets.append((st, g, torch.cuda.Stream()))
    for ctx, n in [([100, 3, 64], [1, 1, 1]), ([70, 40, 1], [30, 9, 1]), ([5, 120, 0], [5, 20, 0]), ([9, 9, 9], [0, 0, 0])]:
        want = []
        for i, (st, g, stream) in enumerate(sets):
            case = (ctx, n, Hq, Hkv, d, 64, bs, I, pcp, dcp, 0, "half")
            x, kc, vc, table, qsl, pos = store_inputs(case, BF, seed=i, after=T - sum(n))
            nb = kc.shape[1]
            st["x"].copy_(x)
            st["kc"][:, :nb], st["vc"][:, :nb] = kc.to(DEV), vc.to(DEV)
            st["t"].fill_(-1)
            st["t"][:, :table.shape[1]] = table.to(DEV)
            st["s"].copy_(qsl)
            st["c"].copy_(i32(*ctx))
            st["p"].copy_(pos[0])
            st["qo"].fill_(7.0)
            kt = ra.rope_apply(st["x"][:, Hq:Hq + Hkv], st["p"], f)
            want.append((O.cp_rope_append(kt.double().cpu(), x[:, Hq + Hkv:], kc, vc, table.numpy(), qsl, ctx, bs, I, pcp, dcp),
                         ra.rope_apply(st["x"][:, :Hq], st["p"], f), nb))
        torch.cuda.synchronize()
        for st, g, stream in sets:
            with torch.cuda.stream(stream):
                g.replay()
        torch.cuda.synchronize()
        check_status(ra)
        for (st, _, _), ((wk, wv), qt, nb) in zip(sets, want):
            assert np.array_equal(st["kc"][:, :nb].double().cpu().numpy(), wk)
            assert np.array_equal(st["vc"][:, :nb].double().cpu().numpy(), wv)
            m = sum(n)
            assert torch.equal(st["qo"][:m], qt[:m]) and (st["qo"][m:] == 7).all()


def test_store_past_32_bit_offsets(ra):
    """Blocks at the far end of caches of more than 2^31 elements."""
    NB, Hkv, bs, d = 17000, 8, 128, 128
    kc, vc = (torch.zeros((1, NB, Hkv, bs, d), dtype=BF, device=DEV) for _ in range(2))
    x = torch.randn((300, 2 * Hkv, d), generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    table = i32(NB - 1, 0, NB - 2).view(1, 3).to(DEV)
    f, _ = ra.rope_frequencies(d)
    ra.cp_rope_append(x[:, :Hkv], x[:, Hkv:], kc, vc, table, i32(0, 300).to(DEV), i32(300).to(DEV), 16, 1, 1, inv_freq=f)
    pos = torch.arange(300, dtype=torch.int32, device=DEV)
    k, v = ra.cp_kv_gather(kc, vc, table, i32(0, 300).to(DEV), pos, 16, 1, 1)
    check_status(ra)
    assert torch.equal(v, x[:, Hkv:]) and torch.equal(k, ra.rope_apply(x[:, :Hkv], pos, f))
    assert int((vc != 0).any(dim=4).sum()) == 300 * Hkv


# ---------------------------------------------------------------------- together

def test_serving_steps_with_a_window(ra):
    """A prompt in pieces and then tokens one by one, as a server with a window runs them: each step stores and
    attends, and a block that has left the window is given to another request at once."""
    Hq, Hkv, d, bs, I, pcp, dcp, window, sink = 8, 2, 64, 16, 4, 1, 2, 70, 3
    V, L = bs * pcp * dcp, 420
    g = torch.Generator().manual_seed(4)
    x = torch.randn((L, Hq + 2 * Hkv, d), generator=g).to(BF).to(DEV)
    f, m = ra.rope_frequencies(d, 10000.0, "linear", 4.0)
    pos = torch.arange(L, dtype=torch.int32, device=DEV)
    q, k = ra.rope_apply(x[:, :Hq], pos, f, m), ra.rope_apply(x[:, Hq:Hq + Hkv], pos, f, m)
    ref = O.window_attn(q.double().cpu(), k.double().cpu(), x[:, Hq + Hkv:].double().cpu(), [0, L], window, sink)
    kc = torch.full((2, 8, Hkv, bs, d), float("nan"), dtype=BF, device=DEV)
    vc = torch.full_like(kc, float("nan"))
    table, free = torch.full((1, L // V + 1), -1, dtype=torch.int32), list(range(8))
    at = 0
    for n in (100, 90, 60) + (1,) * 40 + (4, 7, 60, 59):
        for vb in range(-(-(at + n) // V)):
            if table[0, vb] < 0 and (vb * V >= at or (vb + 1) * V > at):
                table[0, vb] = free.pop(0)
        sd, cd, td = dev(i32(0, n), i32(at + n), table)
        part = x[at:at + n]
        qo = ra.cp_rope_append(part[:, Hq:Hq + Hkv], part[:, Hq + Hkv:], kc, vc, td, sd, cd, I, pcp, dcp, inv_freq=f, mscale=m,
                               q=part[:, :Hq])
        o, lse = ra.cp_window_attn(qo, kc, vc, td, sd, cd, window, I, pcp, dcp, n_sink=sink)
        check_status(ra)
        assert_chunk(o, lse, ref, slice(at, at + n))
        at += n
        for vb in range(1, table.shape[1]):             # blocks that the next query does not see
            if table[0, vb] >= 0 and (vb + 1) * V <= at - window + 1:
                b = int(table[0, vb])
                kc[:, b] = vc[:, b] = float("nan")
                free.append(b)
                table[0, vb] = -1
    assert at == L


def test_training_step_with_a_window(ra):
    """Rotation, attention and the way back to the projection's rows, against differences of the oracle."""
    n, Hq, Hkv, d, window, sink = [130, 61], 4, 2, 64, 40, 2
    T = sum(n)
    g = torch.Generator().manual_seed(6)
    x = torch.randn((T, Hq + 2 * Hkv, d), generator=g).to(BF)
    do = torch.randn((T, Hq, d), generator=g).to(BF)
    f, _ = ra.rope_frequencies(48)
    axis = axis_of("sections", 24, 3)
    pos = torch.randint(0, 300, (3, T), generator=g).to(torch.int32)
    qsl = [0, 130, 191]
    xd, dd, pd, sd = dev(x, do, pos, i32(*qsl))
    qk = ra.rope_apply_axes(xd[:, :Hq + Hkv], pd, f, axis, style="interleaved")
    v = xd[:, Hq + Hkv:]
    o, lse = ra.window_attn_fwd(qk[:, :Hq], qk[:, Hq:], v, sd, window, n_sink=sink)
    dx = torch.empty((T, Hq + 2 * Hkv, d), device=DEV)
    ra.window_attn_bwd(dd, qk[:, :Hq], qk[:, Hq:], v, o, lse, sd, window, n_sink=sink, dq=dx[:, :Hq], dk=dx[:, Hq:Hq + Hkv],
                       dv=dx[:, Hq + Hkv:])
    ra.rope_apply_axes(dx[:, :Hq + Hkv], pd, f, axis, style="interleaved", backward=True, out=dx[:, :Hq + Hkv])
    check_status(ra)
    dof = do.double().numpy()

    def loss(t):
        r = O.rope_apply_axes(t[:, :Hq + Hkv], pos.numpy(), f.numpy(), axis.numpy(), 1.0, "interleaved")
        return (O.window_attn(r[:, :Hq], r[:, Hq:], t[:, Hq + Hkv:], qsl, window, sink)[0] * dof).sum()

    xs, got = x.double().numpy(), dx.double().cpu().numpy()
    for seed in range(4):
        u = np.random.default_rng(seed).standard_normal(xs.shape)
        diff = (loss(xs + 1e-5 * u) - loss(xs - 1e-5 * u)) / 2e-5
        # q, k and P, dS, O rounded to bf16 (2^-8 of values of a few units), independent over T*H*d directions of size 1:
        # sqrt(191 * 8 * 64) * 2^-8 * 4 = 4.9
        assert abs(diff - (got * u).sum()) <= 4.9
