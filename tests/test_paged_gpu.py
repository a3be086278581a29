"""The paged serving calls against their float64 oracle: page bookkeeping, rotary positions and their gradient, the
cache write, attention over the pages, and a run of them together.

Tolerances.  The page step is whole numbers: equal.  A rotation is two products and a sum in float32 of a table
rounded to float32 (relative 2^-24 each, so at most 4 * 2^-24 of |a| + |b|), then one rounding to the output type
(half a step: 2^-8 relative in bf16, 2^-24 in float32).  The attention's weights are rounded to bf16 (2^-8 relative)
with sums in float32 (2^-12 covers the score's, the exponential's and the sum's float32 errors for the scores used here:
40 log2 units * 2^-24 * 128 terms < 2^-11.6 in the worst case is carried by the factor 1 + 2^-3), then the result is
rounded to bf16; the oracle turns that into a bound per element."""
import numpy as np
import pytest
import torch

import oracle.paged_ref as pr
from differential_attention_04_b200 import api

pytestmark = pytest.mark.gpu

P_ERR, OUT_ERR, FLOOR = 2.0 ** -8 * (1 + 2.0 ** -3), 2.0 ** -8, 1e-6
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from differential_attention_04_b200.build import build
    build()
    torch.cuda.set_device(0)
    api.set_wait_limit_ns(0)
    api.device_status()
    yield
    assert api.device_status() == api.OK


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def f64(t):
    return t.detach().cpu().double().numpy()


# ------------------------------------------------------------------ the page step --
def _step_case(seed, S, page, hi, new_hi, extra, width_extra=2):
    r = np.random.default_rng(seed)
    ctx = r.integers(0, hi + 1, S)
    new = r.integers(0, new_hi + 1, S)
    new[r.random(S) < 0.1] = -1
    held = -(-ctx // page)
    want = -(-(ctx + np.maximum(new, 0)) // page)
    need = int(np.where(new < 0, 0, want - held).sum())
    total = int(held.sum()) + need + extra
    ids = r.permutation(total)
    table = np.full((S, int(want.max(initial=1)) + width_extra), -1)
    at = 0
    for s in range(S):
        table[s, :held[s]] = ids[at:at + held[s]]
        at += held[s]
    head = int(r.integers(0, max(total, 1)))
    ring = np.full(max(total, 1), -1)
    ring[(head + np.arange(total - at)) % len(ring)] = ids[at:]
    return ctx, new, table, ring, [head, total - at], page, int(np.maximum(new, 0).sum())


def _check_step(case, T, in_place):
    ctx, new, table, ring, pool, page, _ = case
    want = pr.paged_step(ctx, new, table, ring, pool, page, T)
    dt, dr, dp = i32(table), i32(ring), i32(pool)
    po = dp if in_place else torch.full((2,), 99, dtype=torch.int32, device=DEV)
    cu, kv, pos, slots, info = api.paged_step(i32(ctx), i32(new), dt, dr, dp, page, T, pool_out=None if in_place else po)
    for name, a, b in zip(("table", "ring", "pool", "cu_q", "kv_lens", "positions", "slots", "info"),
                          (dt, dr, po, cu, kv, pos, slots, info), want):
        assert np.array_equal(a.cpu().numpy(), np.asarray(b)), name
    if not in_place:
        assert dp.tolist() == list(pool)
    return info.tolist()


@pytest.mark.parametrize("seed,S,page,hi,new_hi,extra,pad", [
    (1, 1, 16, 0, 0, 1, 0), (2, 1, 16, 5, 1, 3, 4), (3, 64, 64, 3000, 1, 9, 0), (4, 33, 1, 40, 7, 5, 1),
    (5, 700, 16, 900, 300, 0, 77), (6, 513, 256, 5000, 600, 1, 3), (7, 8192, 32, 64, 3, 11, 100)])
@pytest.mark.parametrize("in_place", [False, True])
def test_step(seed, S, page, hi, new_hi, extra, pad, in_place):
    case = _step_case(seed, S, page, hi, new_hi, extra)
    assert _check_step(case, case[6] + pad, in_place)[3] == 0


@pytest.mark.parametrize("in_place", [False, True])
def test_step_that_fails_takes_nothing(in_place):
    ctx, new, table, ring, pool, page, T = _step_case(11, 90, 16, 400, 40, 6)
    bad = lambda **k: _check_step((k.get("ctx", ctx), k.get("new", new), k.get("table", table), ring,
                                   k.get("pool", pool), page, T), k.get("T", T), in_place)
    assert bad(pool=[pool[0], 2])[3] == 1
    assert bad(T=T - 1)[3] == 4
    assert bad(table=table[:, :4])[3] & 2
    over = ctx.copy()
    over[89] = -1
    assert bad(ctx=over)[3] == 8
    huge = new.copy()
    huge[3], huge[4] = 2 ** 31 - 1 - ctx[3], 2 ** 31 - 1 - ctx[4]
    assert bad(new=huge)[3] & 7 == 7
    assert bad(pool=[len(ring), 5])[3] & 16 and bad(pool=[-1, 5])[3] & 16
    full = bad(pool=[pool[0], len(ring)])
    assert full[2] > 0 and full[3] == 16


def test_step_pool_beside_its_output():
    # pool_out shares one word with pool: the new head and count are still those of the old pair
    case = _step_case(12, 200, 16, 300, 20, 4)
    ctx, new, table, ring, pool, page, T = case
    buf = i32([7, pool[0], pool[1], 8])
    api.paged_step(i32(ctx), i32(new), i32(table), i32(ring), buf[1:3], page, T, pool_out=buf[0:2])
    assert buf.tolist() == pr.paged_step(ctx, new, table, ring, pool, page, T)[2] + [pool[1], 8]


# -------------------------------------------------------------------- rotations --
KINDS = {"plain": api.ROPE_PLAIN, "linear": api.ROPE_LINEAR, "ntk": api.ROPE_NTK, "yarn": api.ROPE_YARN}


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("n,rot", [(1, 4), (70000, 64), (257, 126)])
def test_tables(kind, n, rot):
    s = 1.0 if kind == "plain" else 4.0
    t = f64(api.rope_table_scaled(n, rot, 10000.0, KINDS[kind], s, orig_len=2048))
    theta, m = pr.rope_frequencies(rot, 10000.0, kind, s, 2048)
    a = np.arange(n)[:, None] * theta
    # float32 rounding of cos and sin, and of the angle: 2^-53 relative in theta, a few steps of pow and sincos
    tol = m * (2.0 ** -24 + 8 * 2.0 ** -53 * (np.abs(a) + 1))
    assert (np.abs(t[..., 0] - m * np.cos(a)) <= tol).all() and (np.abs(t[..., 1] - m * np.sin(a)) <= tol).all()
    if kind == "plain":
        assert torch.equal(api.rope_table_scaled(n, rot), api.rope_table(n, rot))


def _rope_tol(x, want, m, dtype):
    """|a| + |b| of each pair is at most sqrt(2) |(a, b)| = sqrt(2) |(a', b')| / m; taken as the row's largest."""
    pair = np.abs(x).max(-1, keepdims=True) * 2
    return np.abs(want) * torch.finfo(dtype).eps / 2 * 1.01 + 6 * 2.0 ** -24 * pair * max(m, 1)


def _table_angles(n, rot, kind):
    s = 1.0 if kind == "plain" else 4.0
    t = api.rope_table_scaled(n, rot, 10000.0, KINDS[kind], s)
    theta, m = pr.rope_frequencies(rot, 10000.0, kind, s)
    return t, theta, m


@pytest.mark.parametrize("T,H,Hkv,d,rot,kind", [(1, 1, 1, 8, 2, "plain"), (37, 3, 0, 64, 64, "linear"),
                                                (130, 5, 2, 128, 128, "yarn"), (65, 2, 2, 128, 32, "ntk"),
                                                (19, 2, 1, 24, 22, "plain"), (33, 1, 3, 256, 112, "yarn"),
                                                (5, 40, 8, 256, 2, "plain"), (1029, 12, 12, 64, 48, "plain")])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(T, H, Hkv, d, rot, kind, half, dtype, inverse):
    r = np.random.default_rng(T + d + rot)
    n_pos = 777
    table, theta, m = _table_angles(n_pos, rot, kind)
    pos = r.integers(0, n_pos, T)
    pos[r.random(T) < 0.1] = -1
    g = torch.Generator(device=DEV).manual_seed(T)
    q = torch.randn(T, H, 2, d, generator=g, device=DEV).to(dtype)
    k = torch.randn(T, Hkv, 2, d, generator=g, device=DEV).to(dtype) if Hkv else None
    lay = api.ROPE_HALF if half else api.ROPE_INTERLEAVED
    out = tuple(None if x is None else torch.full_like(x, 7.0) for x in (q, k))
    api.rope(q, k, i32(pos), table, lay, inverse, out=out)
    for x, y in zip((q, k), out):
        if x is None:
            continue
        want = pr.rope(f64(x), pos, theta, m, half, inverse)
        live = pos >= 0
        assert (np.abs(f64(y) - want)[live] <= _rope_tol(f64(x), want, m, dtype)[live]).all()
        assert (f64(y)[~live] == 7).all()
    mine = tuple(None if x is None else x.clone() for x in (q, k))
    api.rope(*mine, i32(pos), table, lay, inverse, out=mine)  # in place
    for x, y, z in zip((q, k), out, mine):
        if x is not None:
            assert torch.equal(z[pos >= 0], y[pos >= 0]) and torch.equal(z[pos < 0], x[pos < 0])


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("kind,rot", [("plain", 64), ("yarn", 40)])
def test_rope_gradient(half, kind, rot):
    """The inverse call is the transpose: <R x, g> = <x, R^T g>, and it agrees with differences of the oracle."""
    table, theta, m = _table_angles(4000, rot, kind)
    g = torch.Generator(device=DEV).manual_seed(5)
    T, d = 29, 64
    x, dy = (torch.randn(T, 3, 2, d, generator=g, device=DEV) for _ in range(2))
    pos = np.random.default_rng(1).integers(0, 4000, T)
    lay = api.ROPE_HALF if half else api.ROPE_INTERLEAVED
    dx, _ = api.rope(dy, None, i32(pos), table, lay, inverse=True)
    loss = lambda z: float((pr.rope(z, pos, theta, m, half) * f64(dy)).sum())
    x64, h = f64(x), 1e-3
    for at in [(0, 0, 0, 0), (3, 1, 1, 5), (28, 2, 0, rot // 2), (11, 0, 1, rot - 1), (9, 2, 1, d - 1)]:
        e = np.zeros_like(x64)
        e[at] = h
        diff = (loss(x64 + e) - loss(x64 - e)) / (2 * h)  # linear: no truncation, rounding below 1e-9
        assert abs(float(dx[at]) - diff) <= 1e-5
    y, _ = api.rope(x, None, i32(pos), table, lay)
    a, b = float((y.double() * dy.double()).sum()), float((x.double() * dx.double()).sum())
    assert abs(a - b) <= 1e-5 * float((y.abs() * dy.abs()).sum())


def test_rope_position_behind_the_table():
    table = api.rope_table(16, 64)
    q = torch.randn(4, 2, 2, 64, device=DEV)
    out = torch.zeros_like(q)
    api.rope(q, None, i32([0, 16, 2 ** 31 - 1, 15]), table, out=(out, None))
    assert api.device_status() == api.ERR_BOUNDS
    assert (out[1:3] == 0).all() and torch.equal(out[0], q[0]) and (out[3] != 0).all()


# ------------------------------------------------------------------- the cache write --
@pytest.mark.parametrize("T,H,Hkv,d,rot,page,half", [(1, 2, 2, 64, 64, 16, False), (77, 6, 2, 128, 64, 16, True),
                                                     (300, 12, 12, 128, 128, 64, False), (50, 3, 1, 40, 6, 8, True),
                                                     (9, 4, 4, 128, 0, 32, False)])
def test_append(T, H, Hkv, d, rot, page, half):
    r = np.random.default_rng(T)
    pages = -(-T // page) + 2
    g = torch.Generator(device=DEV).manual_seed(T)
    bf = lambda *s: torch.randn(*s, generator=g, device=DEV).bfloat16()
    q, k, v = bf(T, H, 2, d), bf(T, Hkv, 2, d), bf(T, Hkv, 2 * d)
    kc, vc = bf(pages, page, Hkv, 2, d), bf(pages, page, Hkv, 2 * d)
    slots = r.permutation(pages * page)[:T]
    slots[r.random(T) < 0.15] = -1
    pos = r.integers(0, 500, T)
    table, theta, m = _table_angles(500, rot, "yarn") if rot else (None, np.zeros(0), 1.0)
    want_k, want_v = f64(kc).reshape(-1, Hkv, 2, d), f64(vc).reshape(-1, Hkv, 2 * d)
    rot_of = lambda x: pr.rope(f64(x), pos, theta, m, half) if rot else f64(x)
    live = slots >= 0
    want_k[slots[live]], want_v[slots[live]] = rot_of(k)[live], f64(v)[live]
    qo = api.kv_append(q, k, v, i32(pos) if rot else None, i32(slots), table, kc, vc,
                       api.ROPE_HALF if half else api.ROPE_INTERLEAVED)
    got_k = f64(kc).reshape(want_k.shape)
    tol = _rope_tol(want_k, want_k, m, torch.bfloat16) if rot else 0
    assert (np.abs(got_k - want_k) <= tol).all() and np.array_equal(f64(vc).reshape(want_v.shape), want_v)
    rest = np.ones(len(want_k), bool)
    rest[slots[live]] = False
    assert np.array_equal(got_k[rest], want_k[rest])
    assert (np.abs(f64(qo) - rot_of(q)) <= (_rope_tol(f64(q), rot_of(q), m, torch.bfloat16) if rot else 0)).all()


def test_append_slot_behind_the_cache():
    q, k, v = torch.randn(3, 1, 2, 64, device=DEV).bfloat16(), torch.ones(3, 1, 2, 64, device=DEV).bfloat16(), \
        torch.ones(3, 1, 128, device=DEV).bfloat16()
    kc, vc = torch.zeros(2, 16, 1, 2, 64, device=DEV).bfloat16(), torch.zeros(2, 16, 1, 128, device=DEV).bfloat16()
    out = api.kv_append(q, k, v, None, i32([31, 32, 2 ** 31 - 1]), None, kc, vc)
    assert api.device_status() == api.ERR_BOUNDS
    assert torch.equal(out, q) and float(kc.float().sum()) == 128 and float(vc[1, 15].float().sum()) == 128


# -------------------------------------------------------------------- the attention --
def _cache(seed, kv, H, Hkv, d, page, T, spare=2, garbage=None, scale=1.0):
    """Inputs on the device: q, caches, table.  Pages are permuted; rows behind kv_lens hold `garbage`."""
    r = np.random.default_rng(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    kv = np.asarray(kv)
    held = -(-kv // page)
    total = int(held.sum()) + spare
    ids = r.permutation(total)
    table = np.full((len(kv), max(1, int(held.max()))), -1)
    bf = lambda *s: (torch.randn(*s, generator=g, device=DEV) * scale).bfloat16()
    q, kc, vc = bf(T, H, 2, d), bf(total, page, Hkv, 2, d), bf(total, page, Hkv, 2 * d)
    at = 0
    for s, n in enumerate(held):
        table[s, :n] = ids[at:at + n]
        at += n
        if garbage is not None and kv[s] % page:
            kc[ids[at - 1], kv[s] % page:] = garbage
            vc[ids[at - 1], kv[s] % page:] = garbage
    if garbage is not None:
        for p in ids[at:]:
            kc[p], vc[p] = garbage, garbage
    return q, kc, vc, table


def _check(got, q, kc, vc, table, cu, kv, lam, w, causal=True, c2=None, li=0.4, p_err=P_ERR):
    want, tol = pr.extend(f64(q), np.nan_to_num(f64(kc)), np.nan_to_num(f64(vc)), table, cu, kv, lam, li, f64(w), 1e-5,
                          causal, c2, p_err=p_err, out_err=OUT_ERR)
    live = ~np.isnan(want[:, 0, 0])
    err = np.abs(f64(got)[live] - want[live])
    over = err - tol[live] - FLOOR
    assert np.isfinite(err).all() and (over <= 0).all(), f"worst {over.max():.3e} at {np.unravel_index(over.argmax(), over.shape)}"
    return live


def _extend(seed, new, kv, H, Hkv, d, page, causal=True, pad=0, garbage=float("nan"), mode=api.MODE_DIFF, max_new=None,
            scale=1.0):
    cu = np.concatenate([[0], np.cumsum(new)])
    T = int(cu[-1]) + pad
    q, kc, vc, table = _cache(seed, kv, H, Hkv, d, page, T, garbage=garbage, scale=scale)
    lam = torch.tensor([0.3], device=DEV)
    w = torch.linspace(0.5, 1.5, 2 * d, device=DEV)
    plan = api.extend_plan(i32(cu), i32(kv), T, H, Hkv, d, max(new) if max_new is None else max_new, causal)
    out = torch.full((T, H, 2 * d), 5.0, device=DEV).bfloat16()
    api.diffattn_extend(q, kc, vc, i32(table), plan, lam, 0.4, w, mode=mode, out=out)
    l32 = float(lam)
    c2 = {api.MODE_DIFF: -l32, api.MODE_SUM: l32, api.MODE_LAMBDA_ZERO: 0.0}[mode]
    live = _check(out, q, kc, vc, table, cu, kv, l32, w, causal, c2)
    assert (out[torch.as_tensor(~live)] == 5.0).all()
    return out


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,kv,H,Hkv,page", [
    ([1], [1], 1, 1, 16), ([1], [77], 2, 2, 16), ([1], [128], 1, 1, 64), ([1], [129], 3, 1, 16),
    ([1, 1, 1], [1, 600, 1100], 2, 2, 128), ([1] * 5, [16, 15, 17, 64, 300], 7, 1, 32), ([8], [8], 2, 2, 256),
    ([5, 5], [400, 5], 2, 2, 16), ([2, 1, 3], [130, 255, 257], 4, 2, 16), ([9], [300], 1, 1, 16),
    ([16, 1], [200, 40], 2, 1, 64), ([40], [40], 2, 2, 16), ([130, 1, 17], [385, 700, 17], 2, 2, 16),
    ([128], [128], 1, 1, 128), ([129], [129], 1, 1, 256), ([257, 3], [300, 130], 3, 1, 32),
    ([100, 0, 1], [333, 50, 9], 10, 2, 64), ([33], [513], 7, 1, 256)])
def test_extend(d, new, kv, H, Hkv, page):
    _extend(sum(new) + sum(kv), new, kv, H, Hkv, d, page, pad=3)


@pytest.mark.parametrize("new,kv", [([1, 4], [100, 33]), ([64, 1], [300, 200]), ([150], [150])])
@pytest.mark.parametrize("mode", [api.MODE_DIFF, api.MODE_SUM, api.MODE_LAMBDA_ZERO])
def test_extend_modes_without_mask(new, kv, mode):
    _extend(3, new, kv, 2, 1, 64, 32, causal=False, mode=mode)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,kv", [([4], [0]), ([1, 1], [0, 20]), ([6, 1], [2, 0]), ([150, 20], [60, 0]),
                                    ([300], [170]), ([260], [0])])
@pytest.mark.parametrize("causal", [True, False])
def test_extend_rows_that_see_nothing(d, new, kv, causal):
    out = _extend(9, new, kv, 2, 2, d, 16, causal=causal, pad=1)
    at = 0
    for n, L in zip(new, kv):
        blind = n if L == 0 else max(0, n - L) if causal else 0
        assert (out[at:at + blind] == 0).all()
        at += n


@pytest.mark.parametrize("new,kv", [([1, 7], [200, 90]), ([200], [450])])
def test_extend_large_scores(new, kv):
    # scores of hundreds: the running maximum moves by far more than a rescaling threshold
    _extend(4, new, kv, 2, 2, 128, 16, scale=5.0)


def test_extend_shared_keys_of_128_heads():
    _extend(6, [1, 2], [70, 150], 128, 1, 64, 16)
    _extend(6, [3], [140], 100, 1, 128, 64)


def test_extend_bound_above_the_need():
    # the host's bound of new tokens only has to be a bound
    a = _extend(8, [1, 3], [300, 200], 4, 2, 128, 16, max_new=900)
    b = _extend(8, [1, 3], [300, 200], 4, 2, 128, 16, max_new=3)
    assert torch.equal(a, b)


def test_extend_many_requests():
    r = np.random.default_rng(0)
    new = np.where(r.random(300) < 0.8, 1, r.integers(0, 30, 300)).tolist()
    kv = [int(n + r.integers(0, 60)) for n in new]
    _extend(10, new, kv, 2, 1, 64, 16, pad=5)


def test_extend_split_over_a_long_context():
    # few rows and many keys: the work of a row is split and joined
    _extend(12, [1, 2], [9000, 5000], 1, 1, 128, 256)
    _extend(13, [20, 130], [6000, 3001], 1, 1, 64, 128)


def _plain(new, kv, H, Hkv, d, page, seed=2, pad=0):
    cu = np.concatenate([[0], np.cumsum(new)])
    T = int(cu[-1]) + pad
    q, kc, vc, table = _cache(seed, kv, H, Hkv, d, page, T)
    lam, w = torch.tensor([0.3], device=DEV), torch.ones(2 * d, device=DEV)
    plan = api.extend_plan(i32(cu), i32(kv), T, H, Hkv, d, max(new))
    return q, kc, vc, table, cu, plan, lam, w


@pytest.mark.parametrize("new,kv", [([1, 2], [50, 300]), ([140], [300])])
@pytest.mark.parametrize("bad", [-1, 10 ** 6, 2 ** 31 - 1, -2 ** 31])
def test_extend_bad_page_reads_as_zeros(new, kv, bad):
    q, kc, vc, table, cu, plan, lam, w = _plain(new, kv, 2, 2, 64, 16)
    table[-1, 3] = bad
    out = api.diffattn_extend(q, kc, vc, i32(table), plan, lam, 0.4, w)
    assert api.device_status() == api.ERR_BOUNDS
    _check(out, q, kc, vc, table, cu, kv, float(lam), w)


@pytest.mark.parametrize("new,kv", [([1, 2], [50, 300]), ([140], [300])])
def test_extend_table_too_narrow(new, kv):
    q, kc, vc, table, cu, plan, lam, w = _plain(new, kv, 2, 2, 128, 16)
    table = np.ascontiguousarray(table[:, :7])
    out = api.diffattn_extend(q, kc, vc, i32(table), plan, lam, 0.4, w)
    assert api.device_status() == api.ERR_BOUNDS
    _check(out, q, kc, vc, table, cu, kv, float(lam), w)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("S,n,L", [(64, 1, 2 ** 30), (1, 1, 2 ** 31 - 257), (1, 140, 2 ** 31 - 257), (9, 40, 2 ** 27)])
def test_extend_lengths_far_beyond_the_table(S, n, L, d):
    """Lengths that no table of the call could hold are reported, at once and with nothing computed."""
    q, kc, vc, table, cu, _, lam, w = _plain([n] * S, [200] * S, 4, 2, d, 16)
    plan = api.extend_plan(i32(cu), i32([L] * S), S * n, 4, 2, d, n)
    out = torch.full((S * n, 4, 2 * d), 3.0, device=DEV).bfloat16()
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e0.record()
    api.diffattn_extend(q, kc, vc, i32(table), plan, lam, 0.4, w, out=out)
    e1.record()
    assert api.device_status() == api.ERR_BOUNDS
    assert (out == 3.0).all() and e0.elapsed_time(e1) < 50


def test_extend_plan_of_bad_offsets():
    """Requests whose entries do not fit are left out, and say so; the others are computed."""
    kv = [40, 60, 30]
    q, kc, vc, table, _, _, lam, w = _plain([1, 2, 1], kv, 2, 2, 64, 16, pad=4)
    T = q.shape[0]
    good = api.diffattn_extend(q, kc, vc, i32(table), api.extend_plan(i32([0, 1, 3, 4]), i32(kv), T, 2, 2, 64, 2),
                               lam, 0.4, w)
    for cu, lens, keep in [([0, 1, 9, 10], kv, [0]), ([0, 1, 3, 4], [40, -5, 30], [0, 3]),
                           ([0, 1, -2, 4], [40, 60, 30], [0]), ([0, 1, 4, 5], kv, [0])]:
        plan = api.extend_plan(i32(cu), i32(lens), T, 2, 2, 64, 2)
        out = torch.full_like(good, 3.0)
        api.diffattn_extend(q, kc, vc, i32(table), plan, lam, 0.4, w, out=out)
        assert api.device_status() == api.ERR_BOUNDS
        for t in keep:
            assert torch.equal(out[t], good[t])
        assert (out[1] == 3.0).all()


def test_extend_is_repeatable_and_shares_its_plan():
    q, kc, vc, table, cu, plan, lam, w = _plain([1, 1, 3, 200, 40], [900, 4000, 700, 1500, 40], 6, 3, 128, 16)
    bt = i32(table)
    want = api.diffattn_extend(q, kc, vc, bt, plan, lam, 0.4, w)
    ws = torch.full((max(16, api.extend_workspace_size(plan)),), 255, dtype=torch.uint8, device=DEV)
    assert torch.equal(want, api.diffattn_extend(q, kc, vc, bt, plan, lam, 0.4, w, workspace=ws))
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for i in range(9):
        with torch.cuda.stream(streams[i % 3]):
            streams[i % 3].wait_stream(torch.cuda.default_stream())
            outs.append(api.diffattn_extend(q, kc, vc, bt, plan, lam, 0.4, w))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)


@pytest.mark.parametrize("d", [64, 128])
def test_extend_forced_timeout_is_reported_and_context_survives(d):
    """Every wait of the many-row kernels is bounded: with a limit of 1 ns they give up, say so and return."""
    new, kv = [200, 64, 300], [700, 300, 300]
    q, kc, vc, table, cu, plan, lam, w = _plain(new, kv, 3, 3, d, 16)
    assert api.device_status() == api.OK
    api.set_wait_limit_ns(1)
    try:
        api.diffattn_extend(q, kc, vc, i32(table), plan, lam, 0.4, w)
        torch.cuda.synchronize()
    finally:
        api.set_wait_limit_ns(0)
    assert api.device_status() == api.ERR_TIMEOUT
    out = api.diffattn_extend(q, kc, vc, i32(table), plan, lam, 0.4, w)
    assert api.device_status() == api.OK
    _check(out, q, kc, vc, table, cu, kv, float(lam), w)


def test_extend_offsets_behind_32_bits():
    """Pages behind 2^31 elements and 2^32 bytes of the cache."""
    Hkv, d, page = 4, 128, 64
    pages = (2 ** 31 // (page * Hkv * 2 * d)) + 40
    kc = torch.empty(pages, page, Hkv, 2, d, dtype=torch.bfloat16, device=DEV)
    vc = torch.empty(pages, page, Hkv, 2 * d, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    for new, kv in (([1, 1], [200, 130]), ([130], [330])):
        held = [-(-x // page) for x in kv]
        table = np.full((len(kv), max(held)), -1)
        at = pages
        for s, n in enumerate(held):
            for j in range(n):
                at -= 1
                table[s, j] = at
        first = at
        T = sum(new)
        small = tuple(torch.randn(pages - first, *c.shape[1:], generator=g, device=DEV).bfloat16() for c in (kc, vc))
        cu = np.concatenate([[0], np.cumsum(new)])
        # written through the cache write: one row per slot
        rows = (pages - first) * page
        slots = i32(np.arange(first * page, pages * page))
        q0 = torch.zeros(rows, Hkv, 2, d, dtype=torch.bfloat16, device=DEV)
        api.kv_append(q0, small[0].view(rows, Hkv, 2, d), small[1].view(rows, Hkv, 2 * d), None, slots, None, kc, vc)
        q = torch.randn(T, Hkv, 2, d, generator=g, device=DEV).bfloat16()
        lam, w = torch.tensor([0.3], device=DEV), torch.ones(2 * d, device=DEV)
        plan = api.extend_plan(i32(cu), i32(kv), T, Hkv, Hkv, d, max(new))
        out = api.diffattn_extend(q, kc, vc, i32(table), plan, lam, 0.4, w)
        _check(out, q, *small, np.where(table >= 0, table - first, -1), cu, kv, float(lam), w)


def _check_on_device(got, q, kc, vc, table, cu, kv, lam, w, causal, li=0.4):
    """The oracle's formulas and its bound in float64 torch on the device, for sizes where numpy takes too long."""
    H, d, page, Hkv = q.shape[1], q.shape[3], kc.shape[1], kc.shape[2]
    G = H // Hkv
    for s, L in enumerate(kv):
        a, b = int(cu[s]), int(cu[s + 1])
        n = b - a
        if n == 0:
            continue
        ids = torch.as_tensor(table[s, :-(-L // page)], device=DEV).long()
        k, v = kc[ids].view(-1, Hkv, 2, d)[:L].double(), vc[ids].view(-1, Hkv, 2 * d)[:L].double()
        see = torch.arange(L, device=DEV)[None] <= (torch.arange(n, device=DEV)[:, None] + (L - n) if causal else L)
        for h in range(H):
            o = e = 0.0
            for m, c in ((0, 1.0), (1, -lam)):
                x = (q[a:b, h, m].double() @ k[:, h // G, m].T / d ** 0.5).masked_fill(~see, -torch.inf)
                p = torch.softmax(x, -1)
                o, e = o + c * p @ v[:, h // G], e + P_ERR * abs(c) * p @ v[:, h // G].abs()
            rms = ((o * o).mean(-1, keepdim=True) + 1e-5).sqrt()
            ne = (e * e).mean(-1, keepdim=True).sqrt()
            y = (1 - li) * w.double() * o / rms
            tol = ((1 - li) * w.double()).abs() * (e + o.abs() * ne / rms) / rms / (1 - ne / rms)
            tol = tol + OUT_ERR * (y.abs() + tol) + FLOOR
            err = (got[a:b, h].double() - y).abs()
            assert bool((err <= tol).all()), (s, h, float((err - tol).max()))


@pytest.mark.parametrize("d,new,kv,H,Hkv,page,causal", [
    (64, [1500], [1700], 32, 32, 16, True),        # whole items in rounds, then split ones
    (128, [1000, 400, 1], [1000, 5000, 700], 16, 16, 64, True),
    (128, [600, 0, 300, 7], [2500, 40, 300, 900], 24, 4, 256, True),
    (64, [129] * 40, [129] * 40, 8, 8, 128, True),  # two tiles of one unit and two
    (128, [260, 512], [3000, 512], 10, 10, 32, False),
    (64, [40] * 9 + [1] * 9, [777] * 18, 14, 2, 16, True),
    (128, [8, 1, 4, 5], [20000, 9000, 131, 64], 4, 4, 64, True)])
def test_extend_larger(d, new, kv, H, Hkv, page, causal):
    cu = np.concatenate([[0], np.cumsum(new)])
    q, kc, vc, table = _cache(17, kv, H, Hkv, d, page, int(cu[-1]), garbage=float("nan"))
    lam, w = torch.tensor([0.3], device=DEV), torch.linspace(0.5, 1.5, 2 * d, device=DEV)
    plan = api.extend_plan(i32(cu), i32(kv), int(cu[-1]), H, Hkv, d, max(new), causal)
    out = api.diffattn_extend(q, kc, vc, i32(table), plan, lam, 0.4, w)
    _check_on_device(out, q, kc, vc, table, cu, kv, float(lam), w, causal)


_rng = np.random.default_rng(2025)
RANDOM_STEPS = []
for _ in range(16):
    _G, _d, _page = int(_rng.choice([1, 1, 2, 3, 5, 7])), int(_rng.choice([64, 128])), int(_rng.choice([16, 32, 64, 256]))
    _top = int(_rng.choice([2, 9, 17, 300]))
    _new = [int(x) for x in _rng.integers(0, _top, int(_rng.integers(1, 14)))]
    _kv = [int(n + (0 if _rng.random() < 0.3 else _rng.integers(0, 1500))) for n in _new]
    RANDOM_STEPS.append((_d, _new, _kv, _G * int(_rng.integers(1, 5)), _G, _page, bool(_rng.random() < 0.8)))


@pytest.mark.parametrize("d,new,kv,H,G,page,causal", RANDOM_STEPS)
def test_extend_random_steps(d, new, kv, H, G, page, causal):
    cu = np.concatenate([[0], np.cumsum(new)])
    T = int(cu[-1]) + 2
    q, kc, vc, table = _cache(sum(kv) + d, kv, H, H // G, d, page, T, garbage=float("inf"))
    lam, w = torch.tensor([0.3], device=DEV), torch.linspace(0.5, 1.5, 2 * d, device=DEV)
    plan = api.extend_plan(i32(cu), i32(kv), T, H, H // G, d, max(new), causal)
    out = torch.full((T, H, 2 * d), 5.0, device=DEV).bfloat16()
    api.diffattn_extend(q, kc, vc, i32(table), plan, lam, 0.4, w, out=out)
    _check_on_device(out, q, kc, vc, table, cu, kv, float(lam), w, causal)
    assert (out[T - 2:] == 5.0).all()


@pytest.mark.parametrize("seed", range(10))
def test_step_random(seed):
    r = np.random.default_rng(seed + 100)
    case = _step_case(seed + 50, int(r.integers(1, 900)), int(r.choice([1, 3, 16, 24, 256])), int(r.integers(0, 4000)),
                      int(r.integers(0, 400)), int(r.integers(0, 20)))
    assert _check_step(case, case[6] + int(r.integers(0, 50)), bool(seed & 1))[3] == 0


def test_binding_and_marshalling_module_make_the_same_calls(monkeypatch):
    from differential_attention_04_b200 import _lib
    assert _lib.marshal()
    q, kc, vc, bt, cu, plan, lam, w = _plain([1, 5, 30], [40, 70, 30], 4, 2, 64, 16)
    T = q.shape[0]
    g = torch.Generator(device=DEV).manual_seed(8)
    k, v = (torch.randn(T, 2, n, generator=g, device=DEV).bfloat16().view(T, 2, *s) for n, s in ((128, (2, 64)), (128, (128,))))
    tab = api.rope_table(200, 32)
    case = _step_case(77, 40, 16, 300, 20, 5)

    def run():
        ctx, new, table, ring, pool, page, n = case
        dt, dr, dp, po = i32(table), i32(ring), i32(pool), i32([0, 0])
        res = [*api.paged_step(i32(ctx), i32(new), dt, dr, dp, page, n + 3, pool_out=po), dt, dr, po]
        out = tuple(torch.zeros_like(t) for t in res[:5])
        dt2, dr2 = i32(table), i32(ring)
        res += list(api.paged_step(i32(ctx), i32(new), dt2, dr2, dp, page, n + 3, out=out)) + [dp, dt2]
        pos, slots = i32(np.arange(T)), i32(np.arange(T)[::-1].copy())
        res += list(api.rope(q, k, pos, tab, api.ROPE_HALF, True)) + [api.rope(q.float(), None, pos, tab)[0]]
        a, b = kc.clone(), vc.clone()
        res += [api.kv_append(q, k, v, pos, slots, tab, a, b, api.ROPE_HALF), a, b]
        a, b = kc.clone(), vc.clone()
        res += [api.kv_append(q, k, v, None, slots, None, a, b), a, b]
        ws = torch.empty(max(16, api.extend_workspace_size(plan)), dtype=torch.uint8, device=DEV)
        out = torch.zeros(T, 4, 128, device=DEV).bfloat16()
        return res + [api.diffattn_extend(q, kc, vc, i32(bt), plan, lam, 0.4, w, workspace=ws, out=out)]

    fast = run()
    # refusals by the library come through with their status, and the checks' with their messages
    refuse = lambda: [pytest.raises(api.DiffAttnError, api.rope, q, None, i32(np.arange(T)), tab, 7).value.status,
                      str(pytest.raises(ValueError, api.rope, q, None, i32(np.arange(T))[:-1], tab).value),
                      str(pytest.raises(ValueError, api.kv_append, q, k, v.transpose(1, 2), i32(np.arange(T)),
                                        i32(np.arange(T)), tab, kc, vc).value)]
    said = refuse()
    monkeypatch.setattr(_lib, "_marshal", False)
    assert not _lib.marshal()
    for x, y in zip(fast, run()):
        assert torch.equal(x, y)
    assert refuse() == said


def test_binding_refuses_tensors_without_storage():
    """A batched tensor of torch.vmap looks like any other until its address is asked for."""
    pos, tab = i32([0, 1, 2, 3]), api.rope_table(8, 64, device=DEV)
    kc, vc = torch.zeros(2, 16, 2, 2, 64, device=DEV).bfloat16(), torch.zeros(2, 16, 2, 128, device=DEV).bfloat16()
    plan = api.extend_plan(i32([0, 4]), i32([4]), 4, 2, 2, 64, 4)
    ws = torch.empty(api.extend_workspace_size(plan), dtype=torch.uint8, device=DEV)
    lam, w, bt = torch.tensor([0.3], device=DEV), torch.ones(128, device=DEV), i32([[0]])
    x, v = torch.randn(3, 4, 2, 2, 64, device=DEV).bfloat16(), torch.randn(3, 4, 2, 128, device=DEV).bfloat16()
    lens = torch.ones(3, 1, dtype=torch.int32, device=DEV)
    for f in (lambda a, b, n: api.rope(a, None, pos, tab)[0], lambda a, b, n: api.kv_append(a, a, b, pos, pos, tab, kc, vc),
              lambda a, b, n: api.diffattn_extend(a, kc, vc, bt, plan, lam, 0.4, w, workspace=ws, out=b),
              lambda a, b, n: api.paged_step(n, n, bt, i32([1]), i32([0, 1]), 16, 4)[0]):
        with pytest.raises((RuntimeError, ValueError)):
            torch.vmap(f)(x, v, lens)
    assert not kc.any() and not vc.any()


def test_debug_build_gives_the_same_bits():
    from differential_attention_04_b200 import _lib
    from differential_attention_04_b200.build import build
    q, kc, vc, table, cu, plan, lam, w = _plain([1, 1, 3, 200, 40], [900, 4000, 700, 1500, 40], 6, 3, 128, 16)
    pos, rot = i32(np.arange(q.shape[0])), api.rope_table(300, 128)
    run = lambda: (api.diffattn_extend(q, kc, vc, i32(table), plan, lam, 0.4, w), api.rope(q, None, pos, rot)[0])
    want = run()
    build(debug=True)
    _lib.use_debug_library(True)
    try:
        got = run()
        assert api.device_status() == api.OK
    finally:
        _lib.use_debug_library(False)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_extend_without_a_plan_of_its_sizes():
    q, kc, vc, table, cu, plan, lam, w = _plain([1, 140], [50, 300], 2, 2, 64, 16)
    out = torch.full((q.shape[0], 2, 128), 3.0, device=DEV).bfloat16()
    for bad in (plan._replace(buf=torch.zeros_like(plan.buf)), plan._replace(buf=torch.full_like(plan.buf, 255)),
                plan._replace(max_new=139)):
        api.diffattn_extend(q, kc, vc, i32(table), bad, lam, 0.4, w, out=out)
        assert api.device_status() == api.ERR_BOUNDS
        assert (out == 3.0).all()


def test_extend_of_no_rows_and_of_empty_requests():
    lam, w = torch.tensor([0.3], device=DEV), torch.ones(128, device=DEV)
    kc, vc = torch.zeros(2, 16, 2, 2, 64, device=DEV).bfloat16(), torch.zeros(2, 16, 2, 128, device=DEV).bfloat16()
    bt = i32([[0], [1]])
    for T, most in ((0, 0), (0, 5), (5, 5), (300, 300)):
        plan = api.extend_plan(i32([0, 0, 0]), i32([3, 0]), T, 4, 2, 64, most)
        out = torch.full((T, 4, 128), 3.0, device=DEV).bfloat16()
        api.diffattn_extend(torch.zeros(T, 4, 2, 64, device=DEV).bfloat16(), kc, vc, bt, plan, lam, 0.4, w, out=out)
        assert (out == 3.0).all()
    assert api.device_status() == api.OK


def test_extend_requests_on_the_same_pages():
    """A shared prompt: two requests' tables name the same pages (each with its own last one)."""
    q, kc, vc, table, cu, _, lam, w = _plain([1, 140], [50, 300], 2, 2, 64, 16)
    shared = np.full((3, 19), -1)
    shared[0], shared[1] = table[1], table[1]
    shared[2, :3] = table[1, :3]
    cu, kv = [0, 1, 140, 141], [300, 290, 48]
    plan = api.extend_plan(i32(cu), i32(kv), q.shape[0], 2, 2, 64, 139)
    out = api.diffattn_extend(q, kc, vc, i32(shared), plan, lam, 0.4, w)
    _check(out, q, kc, vc, shared, cu, kv, float(lam), w)


# ------------------------------------------------------------------ a run of them together --
def _serve(schedule, x, H, Hkv, d, page, table, pages, T, check):
    """Two layers' caches served through the steps of `schedule` (new tokens per request); x: per layer (q, k, v) of
    every request's tokens.  One graph of the step is captured at the second step and replayed from then on."""
    S = len(schedule[0])
    dev = dict(device=DEV)
    ring = torch.arange(pages, dtype=torch.int32, **dev)
    pool = i32([0, pages])
    bt = torch.full((S, pages), -1, dtype=torch.int32, **dev)
    ctx, new = torch.zeros(S, dtype=torch.int32, **dev), torch.zeros(S, dtype=torch.int32, **dev)
    step_out = tuple(torch.empty(n, dtype=torch.int32, **dev) for n in (S + 1, S, T, T, 4))
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, **dev)
    qkv = [(bf(T, H, 2, d), bf(T, Hkv, 2, d), bf(T, Hkv, 2 * d)) for _ in x]
    caches = [(torch.full((pages, page, Hkv, 2, d), float("nan"), **dev).bfloat16(),
               torch.full((pages, page, Hkv, 2 * d), float("nan"), **dev).bfloat16()) for _ in x]
    qr, outs = [bf(T, H, 2, d) for _ in x], [bf(T, H, 2 * d) for _ in x]
    most = max(max(s) for s in schedule)
    cu, kv, pos, slots, info = step_out
    need = int(api.lib().diffattn_extend_plan_size(S, T, H, Hkv, d, most))
    pbuf = torch.empty(max(16, need), dtype=torch.uint8, **dev)
    ws = torch.empty(max(16, api.extend_workspace_size(api.ExtendPlan(pbuf, S, T, H, Hkv, d, most))),
                     dtype=torch.uint8, **dev)
    lam, w = torch.tensor([0.3], **dev), torch.ones(2 * d, **dev)

    def step():
        api.paged_step(ctx, new, bt, ring, pool, page, T, out=step_out)
        plan = api.extend_plan(cu, kv, T, H, Hkv, d, most, buf=pbuf)
        for (q, k, v), (kc, vc), r, o in zip(qkv, caches, qr, outs):
            api.kv_append(q, k, v, pos, slots, table, kc, vc, out=r)
            api.diffattn_extend(r, kc, vc, bt, plan, lam, 0.4, w, workspace=ws, out=o)
        ctx.copy_(kv)

    graph = None
    seen = [0] * S
    for at, lens in enumerate(schedule):
        new.copy_(i32(lens))
        for (q, k, v), rows in zip(qkv, x):
            for dst, src in zip((q, k, v), rows):
                dst[:sum(lens)] = torch.cat([src[s][seen[s]:seen[s] + n] for s, n in enumerate(lens)])
        if at == 1:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        step() if graph is None else graph.replay()
        torch.cuda.synchronize()
        assert info.tolist()[3] == 0 and info.tolist()[0] == sum(lens)
        for layer, o in enumerate(outs):
            row = 0
            for s, n in enumerate(lens):
                check(layer, s, seen[s], o[row:row + n])
                row += n
        seen = [a + b for a, b in zip(seen, lens)]
    del graph
    return bt, ring, pool, ctx


@pytest.mark.parametrize("H,Hkv,d,page", [(2, 2, 128, 16), (6, 2, 64, 32)])
def test_serving_matches_the_dense_prefill(H, Hkv, d, page):
    """Prompts in chunks, drafted tokens and single tokens through the pages give what one dense causal prefill of
    each whole sequence gives."""
    total = [310, 47, 166]
    schedule = [[200, 40, 0], [100, 1, 160], [1, 1, 1], [5, 1, 1], [1, 1, 1], [1, 1, 1], [1, 1, 1], [1, 1, 1]]
    assert [sum(c) for c in zip(*schedule)] == total
    g = torch.Generator(device=DEV).manual_seed(3)
    bf = lambda *s: torch.randn(*s, generator=g, device=DEV).bfloat16()
    x, dense = [], []
    table = api.rope_table(400, d)
    lam, w = torch.tensor([0.3], device=DEV), torch.ones(2 * d, device=DEV)
    for _ in range(2):
        q, k, v = ([bf(n, h, 2, d) for n in total] for h in (H, Hkv, Hkv))
        v = [t.reshape(t.shape[0], Hkv, 2 * d) for t in v]
        x.append((q, k, v))
        rows = []
        for a, b, c, n in zip(q, k, v, total):
            pos = torch.arange(n, dtype=torch.int32, device=DEV)
            ar, br = api.rope(a, b, pos, table)
            rep = lambda t: t.repeat_interleave(H // Hkv, 1)[None].contiguous()
            rows.append(api.diffattn_fwd(ar[None], rep(br), rep(c), lam, 0.4, w, 1e-5, True)[0])
        dense.append(rows)

    def check(layer, s, first, got):
        want = dense[layer][s][first:first + got.shape[0]].double()
        # both round their weights and their result to bf16, from the same bf16 queries, keys and values
        err = (got.double() - want).norm() / want.norm() if got.shape[0] else torch.zeros(())
        assert float(err) <= 2 * 5e-3 and float((got.double() - want).abs().max() if got.shape[0] else 0) <= 2 * 2e-2

    pages = sum(-(-n // page) for n in total) + 1
    bt, ring, pool, ctx = _serve(schedule, x, H, Hkv, d, page, table, pages, 270, check)
    held = [-(-n // page) for n in total]
    assert pool.tolist()[1] == pages - sum(held) and ctx.tolist() == total
    used = [int(p) for s, n in enumerate(held) for p in bt[s, :n]]
    assert len(set(used)) == len(used)


@pytest.mark.parametrize("args", [("--S", "9", "--H", "4", "--Hkv", "2", "--lmin", "1", "--lmax", "300", "--new", "50"),
                                  ("--S", "3", "--H", "2", "--Hkv", "2", "--d", "64", "--lmin", "10", "--lmax", "900")])
def test_serve_command(args, capsys):
    from differential_attention_04_b200 import run_case
    run_case.main(["serve", "--iters", "2", "--page", "16", *args])
    assert capsys.readouterr().out.count("serve iter") == 2
