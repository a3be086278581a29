"""The paged serving calls at the ends of their ranges."""
import numpy as np
import pytest
import torch

import oracle.paged_ref as pr
from differential_attention_04_b200 import api

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from differential_attention_04_b200.build import build
    build()
    torch.cuda.set_device(0)
    api.device_status()
    yield
    assert api.device_status() == api.OK


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("T", [2 ** 31 - 1, 2 ** 31 - 5000])
def test_step_with_as_many_rows_as_an_index_can_count(T):
    """The last rows of positions and slots: the index behind them passes 2^31."""
    ctx, new, page = [5, 40, 0], [3, 1, 20], 16
    table, ring = np.array([[7, -1, -1], [1, 2, 3], [-1, -1, -1]]), np.array([4, 5, 6, 0, -1, -1, -1, -1])
    want = pr.paged_step(ctx, new, table, ring, [0, 4], page, 24)
    bt, po = i32(table), i32([0, 0])
    cu, kv, pos, slots, info = api.paged_step(i32(ctx), i32(new), bt, i32(ring), i32([0, 4]), page, T, pool_out=po)
    assert info.tolist() == list(want[7]) and po.tolist() == list(want[2]) and np.array_equal(bt.cpu(), want[0])
    assert cu.tolist() == list(want[3]) and kv.tolist() == list(want[4])
    for got, w in ((pos, want[5]), (slots, want[6])):
        assert got.numel() == T and got[:24].tolist() == list(w)
        assert all(bool((x == -1).all()) for x in got[24:].split(1 << 28))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,kv,H,G", [
    ([4, 1, 1], [0, 0, 30], 2, 1),          # few rows
    ([7, 2], [2, 150], 4, 2),               # up to 14 rows: both forms of the few-row kernel
    ([300, 20], [170, 20], 2, 1),           # many rows, some of them blind
    ([260], [0], 2, 1),                     # and all of them
    ([3000], [1500], 1, 1), ([40], [6000], 1, 1), ([6], [20000], 1, 1)])  # rows whose keys are split among workers
@pytest.mark.parametrize("causal", [True, False])
def test_extend_without_an_epsilon(d, new, kv, H, G, causal):
    """eps = 0: rows that see no key are zeros, the others are normalised to their mean square alone."""
    page, T, Hkv = 16, sum(new), H // G
    held = [-(-x // page) for x in kv]
    table, at = np.full((len(kv), max(max(held), 1)), -1), 0
    for s, n in enumerate(held):
        table[s, :n] = np.arange(at, at + n)[::-1]
        at += n
    g = torch.Generator(device=DEV).manual_seed(T)
    bf = lambda *s: torch.randn(*s, generator=g, device=DEV).bfloat16()
    q, kc, vc = bf(T, H, 2, d), bf(at + 1, page, Hkv, 2, d), bf(at + 1, page, Hkv, 2 * d)
    lam, w = torch.tensor([0.3], device=DEV), torch.linspace(0.5, 1.5, 2 * d, device=DEV)
    cu = np.concatenate([[0], np.cumsum(new)])
    plan = api.extend_plan(i32(cu), i32(kv), T, H, Hkv, d, max(new), causal)
    out = api.diffattn_extend(q, kc, vc, i32(table), plan, lam, 0.4, w, 0.0)
    assert bool(torch.isfinite(out.float()).all())
    # (mean of (y / w)^2: (1 - 0.4)^2 where there are keys; the rounding to bf16 is at most 2^-8 of each y)
    ms = (out.double() / w.double()).square().mean(-1)
    for s, (n, L) in enumerate(zip(new, kv)):
        rows = ms[cu[s]:cu[s + 1]]
        blind = n if L == 0 else max(0, n - L) if causal else 0
        assert bool((out[cu[s]:cu[s] + blind] == 0).all())
        # float32 sums of 2d squares and their rsqrt: below 2^-12
        assert bool(((rows[blind:] / 0.36 - 1).abs() <= 2 * 2.0 ** -8 + 2.0 ** -16 + 2.0 ** -12).all())


def test_public_getters_make_the_same_calls(monkeypatch):
    """The binding on a torch without the raw getters: the current stream and device are still those of the call."""
    class Bare:
        pass

    q = torch.randn(64, 4, 2, 128, device=DEV)
    pos, table = i32(np.arange(64)), api.rope_table(64, 128)
    want = api.rope(q, None, pos, table)[0]
    device, stream = api._getters(Bare())
    monkeypatch.setattr(api, "_current_device", device)
    monkeypatch.setattr(api, "_raw_stream", stream)
    side = torch.cuda.Stream()
    assert stream(0) == torch.cuda.current_stream().cuda_stream
    with torch.cuda.stream(side):
        assert stream(0) == side.cuda_stream
        side.wait_stream(torch.cuda.default_stream())
        got = torch.zeros_like(q)
        api._launch("diffattn_rope", (q, pos, table, got), q.data_ptr(), None, pos.data_ptr(), table.data_ptr(), 64, 64, 4,
                    0, 128, 128, api.F32, 0, 0, got.data_ptr(), None)
    side.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("d,rot,dtype", [(128, 128, torch.bfloat16), (128, 64, torch.float32), (64, 22, torch.bfloat16),
                                         (256, 2, torch.float32), (64, 64, torch.bfloat16)])
@pytest.mark.parametrize("half", [False, True])
def test_rows_without_a_position_are_zeros_in_a_new_output(d, rot, dtype, half):
    """Whatever the allocation held before: a padded batch goes on into products where a NaN would not stay alone."""
    T, H, Hkv, n_pos = 301, 5, 2, 50
    pos = np.random.default_rng(d).integers(0, n_pos, T)
    pos[::3], pos[7] = -1, n_pos
    table, lay = api.rope_table_scaled(n_pos, rot), api.ROPE_HALF if half else api.ROPE_INTERLEAVED
    g = torch.Generator(device=DEV).manual_seed(rot)
    q, k, v = (torch.randn(T, h, *s, generator=g, device=DEV).to(dtype) for h, s in ((H, (2, d)), (Hkv, (2, d)), (Hkv, (2 * d,))))
    live = torch.as_tensor((pos >= 0) & (pos < n_pos))
    slots = i32(np.arange(T))
    kc, vc = (torch.full((10, 32, Hkv, *s), 3.0, device=DEV).bfloat16() for s in ((2, d), (2 * d,)))

    def calls(out):
        res = list(api.rope(q, k, i32(pos), table, lay, out=out and (out[0].clone(), out[1].clone())))
        if dtype == torch.bfloat16:
            res.append(api.kv_append(q, k, v, i32(pos), slots, table, kc, vc, lay, out=out and out[0].clone()))
        return res

    kept = calls((torch.full_like(q, 5.0), torch.full_like(k, 5.0)))
    for _ in range(4):  # the next allocations of these sizes would get these blocks
        del [torch.full_like(x, float("nan")) for x in (q, k, q)][:]
    zeroed = calls(None)
    for a, b in zip(kept, zeroed):
        assert torch.equal(a[live], b[live]) and bool((a[~live] == 5).all()) and bool((b[~live] == 0).all())
    if dtype == torch.bfloat16:  # the caches' rows of padding are left in both
        rows = kc.view(-1, Hkv, 2, d)[:T]
        assert bool((rows[~live] == 3).all()) and torch.equal(rows[live], zeroed[1][live])
    assert api.device_status() == api.ERR_BOUNDS  # (the position behind the table)
    qo = torch.full_like(q, 5.0)
    api.rope(q, None, i32(np.where(pos == n_pos, 0, pos)), table, lay | api.ROPE_PAD_ZERO, out=(qo, None))
    assert bool((qo[::3] == 0).all()) and api.device_status() == api.OK


@pytest.mark.parametrize("missing", range(5))
def test_step_with_a_missing_output_does_nothing(missing):
    out = [i32([9] * n) for n in (2, 1, 3, 3, 4)]
    kept, out[missing] = out[missing], None
    bt, ring, pool = i32([[-1, -1]]), i32([0, 1]), i32([0, 2])
    with pytest.raises(ValueError, match="out must hold"):
        api.paged_step(i32([0]), i32([3]), bt, ring, pool, 16, 3, out=out)
    assert bt.tolist() == [[-1, -1]] and pool.tolist() == [0, 2]
    out[missing] = kept
    assert api.paged_step(i32([0]), i32([3]), bt, ring, pool, 16, 3, out=out)[0] is out[0]
    assert out[2].tolist() == [0, 1, 2] and pool.tolist() == [1, 1]


def test_attention_without_buffers_is_marshalled_too(monkeypatch):
    """The short form makes the buffers and then the same compiled call as the one that is given them."""
    q, kc, vc = (torch.randn(*s, device=DEV).bfloat16() for s in ((5, 2, 2, 64), (4, 16, 2, 2, 64), (4, 16, 2, 128)))
    plan = api.extend_plan(i32([0, 3]), i32([40]), 5, 2, 2, 64, 3)
    ws = torch.empty(api.extend_workspace_size(plan), dtype=torch.uint8, device=DEV)
    lam, w, bt, made = torch.tensor([0.3], device=DEV), torch.ones(128, device=DEV), i32([[2, 0, 3]]), []
    real = api._made
    monkeypatch.setattr(api, "_made", lambda name, status: made.append(status) or real(name, status))
    outs = [api.diffattn_extend(q, kc, vc, bt, plan, lam, 0.4, w, **k) for k in (
        dict(), dict(workspace=ws), dict(out=torch.zeros(5, 2, 128, device=DEV).bfloat16()),
        dict(workspace=ws, out=torch.zeros(5, 2, 128, device=DEV).bfloat16()))]
    assert made == [0] * 4 and all(torch.equal(o, outs[0]) for o in outs) and bool((outs[0][3:] == 0).all())


def test_calls_from_several_threads():
    """Host threads with a stream and buffers of their own, over one plan and one cache."""
    import threading

    new, kv, H, Hkv, d, page = [1, 5, 140], [700, 90, 300], 4, 2, 128, 16
    held = [-(-x // page) for x in kv]
    table = np.full((3, max(held)), -1)
    for s, n in enumerate(held):
        table[s, :n] = np.arange(n) + sum(held[:s])
    g = torch.Generator(device=DEV).manual_seed(1)
    bf = lambda *s: torch.randn(*s, generator=g, device=DEV).bfloat16()
    T = sum(new)
    q, kc, vc, bt = bf(T, H, 2, d), bf(sum(held), page, Hkv, 2, d), bf(sum(held), page, Hkv, 2 * d), i32(table)
    lam, w, cos = torch.tensor([0.3], device=DEV), torch.ones(2 * d, device=DEV), api.rope_table(T, d)
    plan = api.extend_plan(i32(np.concatenate([[0], np.cumsum(new)])), i32(kv), T, H, Hkv, d, max(new))
    pos = i32(np.arange(T))
    want = [api.diffattn_extend(q, kc, vc, bt, plan, lam, 0.4, w), api.rope(q, None, pos, cos)[0]]
    torch.cuda.synchronize()
    bad = []

    def work():
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                ws = torch.empty(api.extend_workspace_size(plan), dtype=torch.uint8, device=DEV)
                for _ in range(40):
                    got = [api.diffattn_extend(q, kc, vc, bt, plan, lam, 0.4, w, workspace=ws),
                           api.rope(q, None, pos, cos)[0]]
                    if not all(torch.equal(a, b) for a, b in zip(got, want)):
                        bad.append("a result differs")
        except Exception as e:  # an assertion in a thread would pass unseen
            bad.append(repr(e))

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad
