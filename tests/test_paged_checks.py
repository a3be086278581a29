"""Refusals of the paged serving calls, by the library and by the binding,
before any CUDA call (no GPU needed)."""
import ctypes

import pytest
import torch

from differential_attention_04_b200 import _lib, api
from differential_attention_04_b200.build import build

INV, UNS, WS = api.ERR_INVALID_ARG, api.ERR_UNSUPPORTED, api.ERR_WORKSPACE
nul, fake, odd = None, ctypes.c_void_p(4096), ctypes.c_void_p(4104)


@pytest.fixture(scope="module")
def L():
    build()
    return _lib.lib()


def test_step_refusals(L):
    f = lambda S=2, width=3, F=9, P=16, T=4, a=fake, pos=fake: L.diffattn_paged_step(
        a, a, S, a, width, a, F, a, a, P, T, a, a, pos, pos, a, nul)
    assert f(S=0) == INV and f(width=0) == INV and f(F=0) == INV and f(P=0) == INV and f(T=-1) == INV
    assert f(a=nul) == INV and f(pos=nul) == INV and f(a=ctypes.c_void_p(4098)) == INV
    assert f(S=8193) == UNS


def test_rope_refusals(L):
    t = lambda n=8, rot=64, base=1e4, kind=0, s=1.0, orig=4096, bf=32.0, bs=1.0, p=fake: \
        L.diffattn_rope_table_scaled(n, rot, base, kind, s, orig, bf, bs, p, nul)
    assert t(n=0) == INV and t(rot=7) == INV and t(rot=0) == INV and t(base=0.0) == INV and t(p=nul) == INV
    assert t(kind=4) == INV and t(kind=-1) == INV and t(kind=1, s=0.5) == INV and t(kind=2, s=float("nan")) == INV
    assert t(kind=2, rot=2, s=2.0) == INV and t(kind=3, s=2.0, orig=0) == INV and t(kind=3, s=2.0, bf=1.0) == INV
    assert t(n=1 << 26) == INV
    r = lambda q=fake, k=fake, pos=fake, tab=fake, n_pos=8, T=4, H=2, Hk=2, d=64, rot=64, dt=1, lay=0, qo=fake, \
        ko=fake: L.diffattn_rope(q, k, pos, tab, n_pos, T, H, Hk, d, rot, dt, lay, 0, qo, ko, nul)
    assert r(T=0) == api.OK and r(T=-1) == INV and r(H=0) == INV and r(Hk=-1) == INV
    assert r(q=nul) == INV and r(k=nul) == INV and r(pos=nul) == INV and r(tab=nul) == INV and r(qo=nul) == INV
    assert r(ko=nul) == INV and r(n_pos=0) == INV and r(rot=66) == INV and r(rot=7) == INV and r(rot=0) == INV
    assert r(dt=2) == INV and r(lay=2) == INV and r(q=odd) == INV and r(ko=odd) == INV and r(d=60, rot=60) == UNS
    assert r(d=264) == UNS and r(T=1 << 24) == INV
    a = lambda q=fake, k=fake, pos=fake, sl=fake, tab=fake, T=4, H=2, Hk=2, d=64, rot=64, P=3, ps=16, kc=fake: \
        L.diffattn_kv_append(q, k, k, pos, sl, tab, 8, T, H, Hk, d, rot, 0, P, ps, q, kc, kc, nul)
    assert a(T=0) == api.OK and a(T=-1) == INV and a(Hk=0) == INV and a(q=nul) == INV and a(sl=nul) == INV
    assert a(k=nul) == INV and a(kc=nul) == INV and a(kc=odd) == INV and a(P=0) == INV and a(ps=0) == INV
    assert a(pos=nul) == INV and a(P=1 << 20, ps=1 << 12) == INV and a(d=60, rot=60) == UNS
    assert a(tab=nul, pos=nul, d=60) == UNS and a(tab=nul, sl=nul) == INV


def test_extend_refusals(L):
    size = lambda S=2, T=8, H=4, Hk=2, d=64, mx=4: (L.diffattn_extend_plan_size(S, T, H, Hk, d, mx),
                                                    L.diffattn_extend_workspace_size(S, T, H, Hk, d, mx))
    assert size()[0] > 0
    for bad in (dict(S=0), dict(T=-1), dict(H=0), dict(Hk=0), dict(Hk=3), dict(d=0), dict(d=96), dict(mx=-1),
                dict(H=129, Hk=1), dict(S=1 << 16), dict(T=1 << 24)):
        assert size(**bad) == (0, 0), bad
    pl = lambda cu=fake, plan=fake, n=1 << 30, Hk=2, d=64: L.diffattn_extend_plan(cu, cu, 2, 8, 4, Hk, d, 4, 1, plan,
                                                                                  n, nul)
    assert pl(cu=nul) == INV and pl(plan=nul) == WS and pl(n=size()[0] - 1) == WS and pl(plan=odd) == WS
    assert pl(Hk=3) == INV and pl(d=32) == UNS
    ex = lambda q=fake, bt=fake, width=3, P=5, ps=16, plan=fake, pn=1 << 30, T=8, H=4, Hk=2, d=64, mx=4, eps=1e-5, \
        mode=0, o=fake, ws=fake, wn=1 << 40: L.diffattn_extend(q, q, q, bt, width, P, ps, plan, pn, 2, T, H, Hk, d, mx,
                                                               q, 0.5, q, eps, mode, o, ws, wn, nul)
    assert ex(q=nul) == INV and ex(bt=nul) == INV and ex(o=nul) == INV and ex(width=0) == INV and ex(P=0) == INV
    assert ex(ps=0) == INV and ex(ps=8) == UNS and ex(ps=48) == UNS and ex(ps=512) == UNS and ex(P=1 << 28) == INV
    assert ex(eps=-1.0) == INV and ex(eps=float("nan")) == INV and ex(mode=3) == INV and ex(q=odd) == INV
    assert ex(plan=nul) == WS and ex(pn=16) == WS and ex(Hk=3) == INV and ex(d=96) == UNS
    assert ex(T=0) == api.OK and ex(mx=0) == api.OK
    if size()[1]:
        assert ex(ws=nul) == WS and ex(wn=8) == WS


def test_overlapping_buffers_are_refused(L):
    """Every buffer has a megabyte (a plan or a workspace 256) of its own; one that is moved into another's is refused
    before anything is launched."""
    at = lambda i, off=0: ctypes.c_void_p((i + 1 << 28) + off)
    step = lambda **m: L.diffattn_paged_step(*(m.get(n, at(i)) for i, n in enumerate(("ctx", "new"))), 2,
                                             m.get("bt", at(2)), 3, m.get("ring", at(3)), 9, m.get("pool", at(4)),
                                             m.get("po", at(5)), 16, 4,
                                             *(m.get(n, at(6 + i)) for i, n in enumerate(("cu", "kv", "pos", "sl", "info"))),
                                             nul)
    for m in (dict(kv=at(0)), dict(kv=at(0, 4)), dict(cu=at(1, -8)), dict(bt=at(0)), dict(ring=at(2, 20)),
              dict(po=at(0)), dict(sl=at(8)), dict(info=at(4)), dict(pos=at(1, 4)), dict(ctx=at(2, 20))):
        assert step(**m) == INV, m
    rope = lambda Hk=2, q=at(0), k=at(1), qo=at(4), ko=at(5), pos=at(2), tab=at(3): L.diffattn_rope(
        q, k, pos, tab, 8, 4, 2, Hk, 64, 64, 1, 0, 0, qo, ko, nul)
    # 4 rows x 2 heads x 2 x 64 bf16: 2048 bytes
    for m in (dict(qo=at(0, 16)), dict(qo=at(0, -2032)), dict(ko=at(0)), dict(qo=at(1)), dict(ko=at(4)),
              dict(ko=at(4, 2032)), dict(qo=at(2)), dict(ko=at(3, 16)), dict(Hk=0, qo=at(0, 16))):
        assert rope(**m) == INV, m
    app = lambda q=at(0), k=at(1), v=at(2), qo=at(6), kc=at(7), vc=at(8): L.diffattn_kv_append(
        q, k, v, at(3), at(4), at(5), 8, 4, 2, 2, 64, 64, 0, 3, 16, qo, kc, vc, nul)
    for m in (dict(qo=at(0, 16)), dict(k=at(7)), dict(v=at(8, 512)), dict(vc=at(7)), dict(qo=at(1)), dict(q=at(7, 16))):
        assert app(**m) == INV, m
    ext = lambda q=at(0), kc=at(1), vc=at(2), bt=at(3), plan=at(4), lam=at(5), w=at(6), o=at(7), ws=at(8): \
        L.diffattn_extend(q, kc, vc, bt, 3, 5, 16, plan, 1 << 28, 2, 8, 4, 2, 64, 4, lam, 0.5, w, 1e-5, 0, o, ws,
                          1 << 28, nul)
    for m in (dict(o=at(0)), dict(o=at(0, 16)), dict(o=at(2)), dict(o=at(4)), dict(ws=at(4)), dict(ws=at(0)),
              dict(ws=at(7)), dict(o=at(8, 64)), dict(lam=at(7)), dict(w=at(8, 16)), dict(bt=at(7))):
        assert ext(**m) == INV, m
    n = L.diffattn_extend_plan_size(2, 8, 4, 2, 64, 4)
    for cu, kv in ((at(0), at(1)), (at(1), at(0, 16)), (at(1), at(0, n - 4))):
        assert L.diffattn_extend_plan(cu, kv, 2, 8, 4, 2, 64, 4, 1, at(0), 1 << 28, nul) == INV


def _rejects(match, fn, *a, **k):
    with pytest.raises(ValueError, match=match):
        fn(*a, **k)


def test_binding_refusals():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    dev = "must be CUDA tensors"
    _rejects(dev, api.paged_step, i(2), i(2), i(2, 3), i(9), i(2), 16, 4)
    _rejects("new_lens", api.paged_step, i(2), i(3), i(2, 3), i(9), i(2), 16, 4)
    _rejects("ctx_lens", api.paged_step, i(2).long(), i(2), i(2, 3), i(9), i(2), 16, 4)
    _rejects("pool", api.paged_step, i(2), i(2), i(2, 3), i(9), i(3), 16, 4)
    _rejects("info", api.paged_step, i(2), i(2), i(2, 3), i(9), i(2), 16, 4, out=(i(3), i(2), i(4), i(4), i(3)))
    bf = dict(dtype=torch.bfloat16)
    q, k, v = torch.zeros(4, 4, 2, 64, **bf), torch.zeros(4, 2, 2, 64, **bf), torch.zeros(4, 2, 128, **bf)
    tab, kc, vc = torch.zeros(9, 16, 2), torch.zeros(3, 16, 2, 2, 64, **bf), torch.zeros(3, 16, 2, 128, **bf)
    _rejects(dev, api.rope, q, k, i(4), tab)
    _rejects(dev, api.rope, q, None, i(4), tab, inverse=True)
    _rejects("positions", api.rope, q, k, i(3), tab)
    _rejects("k must be", api.rope, q, k.float(), i(4), tab)
    _rejects("table", api.rope, q, k, i(4), torch.zeros(9, 33, 2))
    _rejects("dtype", api.rope, q.half(), None, i(4), tab)
    _rejects(dev, api.kv_append, q, k, v, i(4), i(4), tab, kc, vc)
    _rejects(dev, api.kv_append, q, k, v, None, i(4), None, kc, vc)
    _rejects("slots", api.kv_append, q, k, v, i(4), i(5), tab, kc, vc)
    _rejects("positions", api.kv_append, q, k, v, None, i(4), tab, kc, vc)
    _rejects("v_cache", api.kv_append, q, k, v, i(4), i(4), tab, kc, vc[:2])
    _rejects("k must be", api.kv_append, q, k[:, :1], v, i(4), i(4), tab, kc, vc)
    _rejects(dev, api.extend_plan, i(3), i(2), 4, 4, 2, 64, 4)
    _rejects("cu_q", api.extend_plan, i(2), i(2), 4, 4, 2, 64, 4)
    plan = api.ExtendPlan(torch.zeros(1 << 16, dtype=torch.uint8), 2, 4, 4, 2, 64, 4)
    lam, w = torch.zeros(1), torch.ones(128)
    _rejects(dev, api.diffattn_extend, q, kc, vc, i(2, 3), plan, lam, 0.5, w)
    _rejects("other sizes", api.diffattn_extend, q[:3], kc, vc, i(2, 3), plan, lam, 0.5, w)
    _rejects("block_table", api.diffattn_extend, q, kc, vc, i(3, 3), plan, lam, 0.5, w)
    _rejects("rms_w", api.diffattn_extend, q, kc, vc, i(2, 3), plan, lam, 0.5, w[:64])


def test_marshalling_module_leaves_what_is_not_plain(L):
    """Whatever is not plainly right (here: tensors that are not on a GPU, wrong counts, other objects) is left to the
    binding's checks: the module has done nothing and says so."""
    m = _lib.marshal()
    assert m
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    none = (None,) * 5
    step = (i(2), i(2), i(2, 3), i(9), i(2), i(2), 16, 4)
    q, k, v, tab = bf(4, 4, 2, 64), bf(4, 2, 2, 64), bf(4, 2, 128), torch.zeros(9, 32, 2)
    kc, vc = bf(3, 16, 2, 2, 64), bf(3, 16, 2, 128)
    plan = (torch.zeros(64, dtype=torch.uint8), 2, 4, 4, 2, 64, 4)
    ext = (q, kc, vc, i(2, 3), *plan, torch.zeros(1), 0.5, torch.ones(128), 1e-5, 0, plan[0], bf(4, 4, 128))
    for f, args in ((m.paged_step, step + none), (m.paged_step, step), (m.paged_step, (1,) * 13),
                    (m.paged_step, step[:6] + ("16", 4) + none), (m.rope, (q, k, i(4), tab, 0, 0, q, k)),
                    (m.rope, (q, None, i(4), tab, 0, 0, q, None)), (m.rope, (None,) * 8), (m.rope, ()),
                    (m.kv_append, (q, k, v, i(4), i(4), tab, kc, vc, 0, q)), (m.kv_append, (None,) * 10),
                    (m.extend, ext), (m.extend, (None,) * 18), (m.extend, ext[:-1]),
                    (m.extend, ext[:5] + (2 ** 70,) + ext[6:])):
        assert f(*args) == -1
    with pytest.raises(TypeError):
        m.bind(1, 2)
