"""The paged serving calls under the bounds-checked build: its checks pass and change no bit of any form, and a plan
whose entries were overwritten is reported, with every access that would leave a buffer skipped.  (Such a plan is only
ever given to the checked build, whose kernels turn each bad entry into an error before they use it.)"""
import numpy as np
import pytest
import torch

from differential_attention_04_b200 import _lib, api

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from differential_attention_04_b200.build import build
    build()
    build(debug=True)
    torch.cuda.set_device(0)
    api.device_status()
    yield
    _lib.use_debug_library(False)
    assert api.device_status() == api.OK


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


class _Checked:
    def __enter__(self):
        _lib.use_debug_library(True)

    def __exit__(self, *e):
        _lib.use_debug_library(False)


class Step:
    """Inputs of one attention call, and an output with a row of others in front and behind."""

    def __init__(self, new, kv, H, Hkv, d, page=16, causal=True):
        g = torch.Generator(device=DEV).manual_seed(sum(kv))
        bf = lambda *s: torch.randn(*s, generator=g, device=DEV).bfloat16()
        held = [-(-x // page) for x in kv]
        table, at = np.full((len(kv), max(held)), -1), 0
        for s, n in enumerate(held):
            table[s, :n] = np.arange(at, at + n)[::-1]
            at += n
        T = sum(new)
        self.q, self.kc, self.vc = bf(T, H, 2, d), bf(at, page, Hkv, 2, d), bf(at, page, Hkv, 2 * d)
        self.lam, self.w, self.bt = torch.tensor([0.3], device=DEV), torch.ones(2 * d, device=DEV), i32(table)
        self.cu, self.kv = i32(np.concatenate([[0], np.cumsum(new)])), i32(kv)
        self.shape, self.causal = (len(new), T, H, Hkv, d, max(new)), causal
        self.all = torch.empty(T + 2, H, 2 * d, device=DEV, dtype=torch.bfloat16)
        self.ws = torch.empty(max(16, api.extend_workspace_size(api.ExtendPlan(self.q, *self.shape))),
                              dtype=torch.uint8, device=DEV)

    def plan(self):
        return api.extend_plan(self.cu, self.kv, *self.shape[1:], causal=self.causal)

    def run(self, plan):
        self.all.fill_(7.0)
        api.diffattn_extend(self.q, self.kc, self.vc, self.bt, plan, self.lam, 0.4, self.w, workspace=self.ws,
                            out=self.all[1:-1])
        assert bool((self.all[0] == 7).all()) and bool((self.all[-1] == 7).all())
        return self.all[1:-1].clone()


FORMS = [([1, 1, 3], [5000, 40, 700], 6, 3, 128), ([1, 1, 3], [5000, 40, 700], 6, 3, 64), ([9, 16], [600, 300], 2, 2, 128),
         ([9, 16], [600, 300], 2, 2, 64), ([1] * 400, [40] * 400, 2, 2, 64), ([1, 200, 40], [900, 1500, 40], 6, 3, 64),
         ([1, 200, 40], [900, 1500, 40], 6, 3, 128), ([128] * 40, [300] * 40, 16, 16, 128), ([128] * 40, [300] * 40, 16, 16, 64),
         ([4, 150], [0, 60], 2, 2, 128), ([4, 150], [0, 60], 10, 1, 64)]


@pytest.mark.parametrize("new,kv,H,Hkv,d", FORMS)
@pytest.mark.parametrize("causal", [True, False])
def test_attention_passes_every_check(new, kv, H, Hkv, d, causal):
    s = Step(new, kv, H, Hkv, d, causal=causal)
    plan = s.plan()
    want = s.run(plan)
    with _Checked():
        mine = s.plan()
        got = s.run(mine)
        assert api.device_status() == api.OK
    assert torch.equal(got, want) and torch.equal(plan.buf[:64], mine.buf[:64])


@pytest.mark.parametrize("rot,half", [(128, False), (128, True), (64, True), (112, True), (6, False), (6, True), (0, False)])
def test_rows_pass_every_check(rot, half):
    T, H, Hkv, d, page = 77, 5, 2, 128, 16
    g = torch.Generator(device=DEV).manual_seed(rot)
    bf = lambda *s: torch.randn(*s, generator=g, device=DEV).bfloat16()
    q, k, v, kc, vc = bf(T, H, 2, d), bf(T, Hkv, 2, d), bf(T, Hkv, 2 * d), bf(6, page, Hkv, 2, d), bf(6, page, Hkv, 2 * d)
    pos, slots = i32(np.arange(T) * 3), i32(np.random.default_rng(1).permutation(6 * page)[:T])
    table = api.rope_table_scaled(300, rot) if rot else None
    lay = api.ROPE_HALF if half else api.ROPE_INTERLEAVED

    def run():
        a, b = kc.clone(), vc.clone()
        res = [api.kv_append(q, k, v, pos, slots, table, a, b, lay), a, b]
        if rot:
            res += [*api.rope(q, k, pos, table, lay, True), api.rope(q.float(), None, pos, table, lay)[0]]
        return res

    want = run()
    with _Checked():
        got = run()
        assert api.device_status() == api.OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("S,page", [(1, 16), (300, 1), (700, 24)])
def test_page_step_passes_every_check(S, page):
    r = np.random.default_rng(S)
    ctx, new = r.integers(0, 500, S), r.integers(-1, 60, S)
    held, want = -(-ctx // page), -(-(ctx + np.maximum(new, 0)) // page)
    total, width = int(held.sum() + want.sum()) + 3, int(want.max(initial=1)) + int(held.max())
    table, at = np.full((S, width), -1), 0
    for s, n in enumerate(held):
        table[s, :n] = np.arange(at, at + n)
        at += n
    ring = np.full(total, -1)
    ring[(total - 5 + np.arange(total - at)) % total] = np.arange(at, total)
    T = int(np.maximum(new, 0).sum()) + 9

    def run():
        bt, rg, pool = i32(table), i32(ring), i32([total - 5, total - at])
        return [*api.paged_step(i32(ctx), i32(new), bt, rg, pool, page, T), bt, rg, pool]

    a = run()
    assert a[4].tolist()[3] == 0
    with _Checked():
        b = run()
        assert api.device_status() == api.OK
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def _sections(S, T, H, Hkv, d, max_new):
    """Where a plan's parts begin, in words: the workers' starts and tails of both classes, requests, items."""
    wide = 148 if d == 64 else 74
    at, where = 16, {}
    for c, w in (("narrow", 296), ("wide", wide)):
        where["start_" + c], where["tail_" + c] = at, at + 8 * w
        at += 12 * w
    where["requests"] = at
    tiles = T // (128 // (H // Hkv)) + min(S, T) if max_new * (H // Hkv) > 16 else 0
    at += 4 * S + 8 * tiles + 2 * (S + 1) + 2 * (tiles + 1)
    where["items"] = -(-at // 4) * 4
    return where


# what, the words of an entry that are overwritten, and with what
BAD = [("requests", 0, 10 ** 9), ("requests", 0, -1), ("requests", 1, 10 ** 6), ("requests", 1, -1),
       ("requests", 2, 2 ** 31 - 1), ("requests", 2, -2), ("requests", 3, 10 ** 8), ("requests", 3, -1),
       ("start_narrow", 0, 10 ** 7), ("start_narrow", 1, 10 ** 7), ("start_narrow", 2, 10 ** 7), ("start_narrow", 2, -9),
       ("start_narrow", 4, 10 ** 9), ("tail_narrow", 0, 10 ** 9), ("tail_narrow", 1, 10 ** 7), ("tail_narrow", 2, 10 ** 6),
       ("tail_narrow", 3, -7), ("start_wide", 0, 10 ** 7), ("start_wide", 0, -1), ("start_wide", 2, 10 ** 7),
       ("start_wide", 2, -9), ("tail_wide", 0, 10 ** 9), ("tail_wide", 2, 10 ** 6), ("tail_wide", 3, -7),
       ("items", 0, 10 ** 9), ("items", 0, -1), ("items", 1, 129), ("items", 1, -1), ("items", 3, 2 ** 31 - 1),
       ("items", 3, 0), ("items", 4, -1), ("items", 5, 10 ** 8), ("items", 6, 10 ** 7), ("items", 6, -1), ("head", 3, 10 ** 8),
       ("head", 0, 10 ** 6), ("head", 1, 10 ** 6), ("head", 11, 10 ** 7), ("head", 11, -1)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("part,word,value", BAD)
def test_overwritten_plans_are_reported(part, word, value, d):
    narrow = part.endswith("narrow") or part == "requests"
    s = Step(*(([1, 3] * 200 + [2], [90, 300] * 200 + [9000]) if narrow else ([300, 1, 600], [800, 700, 600])), 4, 2, d)
    plan = s.plan()
    want = s.run(plan)
    words = plan.buf.view(torch.int32).clone()
    where = {**_sections(*s.shape), "head": 0}
    size = {"requests": 4, "items": 8, "start": 8, "tail": 4, "head": 16}[part.split("_")[0]]
    lo = where[part]
    count = 1 if part == "head" else 148 if d == 64 else 74
    hit = 0
    for e in range(0, count, 1 if part == "head" else 5):
        old = words[lo + e * size:lo + (e + 1) * size].tolist()
        if part.startswith("start") and old[3] == 0 or part.startswith("tail") and old[2] == 0:
            continue  # a worker without work, or without a split item
        if part == "items" and e >= 3 * 2:
            break
        words[lo + e * size + word] = value
        hit += 1
    assert hit
    bad = plan._replace(buf=words.view(torch.uint8))
    with _Checked():
        s.run(bad)  # (asserts that the rows around the output are as they were)
        assert api.device_status() == api.ERR_BOUNDS
        assert torch.equal(s.run(plan), want) and api.device_status() == api.OK
