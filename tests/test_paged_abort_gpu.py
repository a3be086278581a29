"""The many-row kernels of the paged attention after a wait that ran out: each launch ends, says so, and leaves nothing
behind that a later launch could meet.  Nothing faults or hangs here: the waits are the library's bounded ones, with a
short limit, and the limits range from one that no wait survives to ones that run out in the middle of a row's keys."""
import numpy as np
import pytest
import torch

from differential_attention_04_b200 import api

pytestmark = pytest.mark.gpu

DEV = "cuda"
LIMITS = (1, 700, 1500, 3000, 6000, 12000)


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
    api.set_wait_limit_ns(0)
    assert api.device_status() == api.OK


def _call(new, kv, H, Hkv, d, page):
    """A function that makes one call into a fresh output, and the plan."""
    i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(sum(kv) + d)
    bf = lambda *s: torch.randn(*s, generator=g, device=DEV).bfloat16()
    held = -(-np.asarray(kv) // page)
    table = np.full((len(kv), int(held.max())), -1)
    ids, at = np.random.default_rng(d).permutation(int(held.sum())), 0
    for s, n in enumerate(held):
        table[s, :n] = ids[at:at + n]
        at += n
    T = sum(new)
    q, kc, vc = bf(T, H, 2, d), bf(at, page, Hkv, 2, d), bf(at, page, Hkv, 2 * d)
    lam, w, bt = torch.tensor([0.3], device=DEV), torch.linspace(0.5, 1.5, 2 * d, device=DEV), i32(table)
    plan = api.extend_plan(i32(np.concatenate([[0], np.cumsum(new)])), i32(kv), T, H, Hkv, d, max(new))
    ws = torch.empty(max(16, api.extend_workspace_size(plan)), dtype=torch.uint8, device=DEV)
    outs = [torch.zeros(T, H, 2 * d, device=DEV).bfloat16() for _ in range(2)]

    def run(i=0):
        return api.diffattn_extend(q, kc, vc, bt, plan, lam, 0.4, w, workspace=ws, out=outs[i])

    return run, plan


def _aborts(run, limits=LIMITS, repeats=2):
    """Calls that give up, each with a normal one right behind it: that one's result is the undisturbed call's."""
    want = run().clone()
    assert api.device_status() == api.OK and bool(torch.isfinite(want.float()).all())
    for limit in limits:
        for _ in range(repeats):
            api.set_wait_limit_ns(limit)
            try:
                run(0)
            finally:
                api.set_wait_limit_ns(0)
            got = run(1)
            status = api.device_status()
            assert status == api.ERR_TIMEOUT or (limit > 1 and status == api.OK), (limit, status)
            assert torch.equal(got, want), limit
    return want


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,kv", [([200, 64, 300], [700, 300, 300]), ([40], [9000])])
def test_split_rows(d, new, kv):
    run, plan = _call(new, kv, 3, 3, d, 16)
    _aborts(run)


@pytest.mark.parametrize("d", [64, 128])
def test_limits_that_run_out_anywhere(d):
    """A wait may end in some lanes of a warp and run out in others: the warp has to leave as one."""
    run, plan = _call([130], [6000], 2, 2, d, 64)
    _aborts(run, range(150, 9000, 150), 1)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,kv,limits", [([128] * 60, [128] * 60, (1, 2000, 10000, 40000)),
                                           ([100, 256, 7] * 20, [260, 700, 90] * 20, (1, 5000, 20000))])
def test_several_whole_items_a_worker(d, new, kv, limits):
    """Items that are combined, exchanged between two blocks (d 128) and handed over one behind the other: a worker
    that gives up has several of them left."""
    run, plan = _call(new, kv, 16, 16, d, 64)
    head = plan.buf[:64].view(torch.int32).tolist()
    assert head[1] == (148 if d == 64 else 74) and head[11] >= 3, head  # workers, and the whole items of each
    _aborts(run, limits)
