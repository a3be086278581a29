"""The tensor-core backward repeats bit for bit, its sums over all rows (dlambda and the norm weight's gradient)
included; their values are held against the oracle elsewhere."""
import pytest
import torch

from differential_attention_04_b200 import api
from differential_attention_04_b200 import workloads as wl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from differential_attention_04_b200.build import build
    build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("B,N,H,d", [(1, 1, 1, 64), (1, 9, 1, 128), (2, 517, 3, 128), (1, 2000, 12, 64),
                                     (2, 4096, 12, 128)])
def test_every_gradient_repeats(B, N, H, d):
    inp = wl.make_prefill(B, N, H, d, causal=True, dtype="bf16", seed=N + d, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    dy = torch.randn(inp.v.shape, generator=g, device="cuda").to(torch.bfloat16)
    lam = api.diffattn_lambda(inp.lq1, inp.lk1, inp.lq2, inp.lk2, inp.lambda_init)
    args = (inp.q, inp.k, inp.v, dy, lam, inp.lambda_init, inp.rms_w, inp.eps, True)
    want = api.diffattn_bwd_tc(*args)
    assert all(bool(torch.isfinite(x).all()) for x in want)
    for _ in range(4):
        assert all(torch.equal(a, b) for a, b in zip(want, api.diffattn_bwd_tc(*args)))
    _, ws = api.diffattn_fwd_train(inp.q, inp.k, inp.v, lam, inp.lambda_init, inp.rms_w, inp.eps, True)
    for _ in range(2):  # the saved statistics serve any number of backward calls
        got = api.diffattn_bwd_tc_saved(inp.q, inp.k, inp.v, dy, lam, inp.lambda_init, inp.rms_w, inp.eps, True,
                                        api.MODE_DIFF, ws)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert api.device_status() == api.OK


def test_a_captured_backward_repeats():
    inp = wl.make_prefill(1, 700, 3, 64, causal=True, dtype="bf16", seed=8, device="cuda")
    dy = torch.randn_like(inp.v)
    lam = api.diffattn_lambda(inp.lq1, inp.lk1, inp.lq2, inp.lk2, inp.lambda_init)
    ws = torch.empty(api.bwd_tc_workspace_size(1, 700, 3, 64), dtype=torch.uint8, device="cuda")
    f32 = dict(dtype=torch.float32, device="cuda")
    out = tuple(torch.empty(s, **f32) for s in (inp.q.shape, inp.k.shape, inp.v.shape, 1, 128))
    run = lambda: api.diffattn_bwd_tc(inp.q, inp.k, inp.v, dy, lam, inp.lambda_init, inp.rms_w, inp.eps, True,
                                      workspace=ws, out=out)
    want = [x.clone() for x in run()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        for x in out:
            x.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    del graph
