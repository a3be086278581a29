"""What the binding of the paged serving calls makes of its arguments, before any CUDA call (no GPU needed)."""
import types

import pytest
import torch

from differential_attention_04_b200 import _lib, api
from differential_attention_04_b200.build import build


@pytest.fixture(scope="module", autouse=True)
def _library():
    build()


def _i(*s):
    return torch.zeros(s, dtype=torch.int32)


BF = dict(dtype=torch.bfloat16)
Q, K, V = torch.zeros(4, 4, 2, 64, **BF), torch.zeros(4, 2, 2, 64, **BF), torch.zeros(4, 2, 128, **BF)
TAB, KC, VC = torch.zeros(9, 16, 2), torch.zeros(3, 16, 2, 2, 64, **BF), torch.zeros(3, 16, 2, 128, **BF)
PLAN = api.ExtendPlan(torch.zeros(1 << 16, dtype=torch.uint8), 2, 4, 4, 2, 64, 4)

WIDE = [
    ("num_tokens", lambda x: api.paged_step(_i(2), _i(2), _i(2, 3), _i(9), _i(2), 16, x)),
    ("page_size", lambda x: api.paged_step(_i(2), _i(2), _i(2, 3), _i(9), _i(2), x, 4)),
    ("N", lambda x: api.rope_table_scaled(x, 64, device="cpu")),
    ("rot", lambda x: api.rope_table_scaled(8, x, device="cpu")),
    ("scaling", lambda x: api.rope_table_scaled(8, 64, scaling=x, device="cpu")),
    ("orig_len", lambda x: api.rope_table_scaled(8, 64, scaling=api.ROPE_YARN, factor=2.0, orig_len=x, device="cpu")),
    ("layout", lambda x: api.rope(Q, K, _i(4), TAB, x)),
    ("layout", lambda x: api.kv_append(Q, K, V, _i(4), _i(4), TAB, KC, VC, x)),
    ("num_tokens", lambda x: api.extend_plan(_i(3), _i(2), x, 4, 2, 64, 4)),
    ("H", lambda x: api.extend_plan(_i(3), _i(2), 4, x, 2, 64, 4)),
    ("H_kv", lambda x: api.extend_plan(_i(3), _i(2), 4, 4, x, 64, 4)),
    ("d", lambda x: api.extend_plan(_i(3), _i(2), 4, 4, 2, x, 4)),
    ("max_new", lambda x: api.extend_plan(_i(3), _i(2), 4, 4, 2, 64, x)),
    ("max_new", lambda x: api.extend_workspace_size(PLAN._replace(max_new=x))),
    ("max_new", lambda x: api.diffattn_extend(Q, KC, VC, _i(2, 3), PLAN._replace(max_new=x), torch.zeros(1), 0.5,
                                              torch.ones(128))),
    ("mode", lambda x: api.diffattn_extend(Q, KC, VC, _i(2, 3), PLAN, torch.zeros(1), 0.5, torch.ones(128), mode=x)),
]


@pytest.mark.parametrize("name,call", WIDE, ids=[f"{i}-{n}" for i, (n, _) in enumerate(WIDE)])
@pytest.mark.parametrize("x", [2 ** 32, 2 ** 32 + 64, 2 ** 31, -2 ** 31 - 1])
def test_numbers_beyond_32_bits_are_refused(name, call, x):
    """(A bound of 2^32 new tokens would otherwise reach the library as 0, and nothing would be computed.)"""
    with pytest.raises(ValueError, match=f"^{name} must fit 32 bits"):
        call(x)


def test_binding_has_the_public_getters_to_fall_back_on():
    raw = types.SimpleNamespace(_cuda_getDevice=object(), _cuda_getCurrentRawStream=object())
    assert api._getters(raw) == (raw._cuda_getDevice, raw._cuda_getCurrentRawStream)
    device, stream = api._getters(types.SimpleNamespace())
    assert device is torch.cuda.current_device and callable(stream)


@pytest.mark.parametrize("missing", range(5))
def test_step_outputs_come_whole_or_not_at_all(missing):
    out = [_i(3), _i(2), _i(4), _i(4), _i(4)]
    out[missing] = None
    with pytest.raises(ValueError, match="out must hold"):
        api.paged_step(_i(2), _i(2), _i(2, 3), _i(9), _i(2), 16, 4, out=out)
