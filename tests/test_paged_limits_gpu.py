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
