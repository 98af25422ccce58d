"""AdaptedLinear on the GPU where the framework's other calls do not come before it: streams."""
import pytest
import torch

from adapter_reference import check, inputs, reference

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import int8_mixed_precision_gb300 as dit  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


def test_backward_on_another_stream_starts_from_zeros():
    """Without the frozen weight dx is the adapters' part alone, whatever it held: cleared on the call's stream,
    not on the current one, which is kept busy meanwhile."""
    T, K, N, G, r = 600, 256, 512, 2, 16
    c = inputs([400, 200], [1, 0], G, r, K, N, F32, seed=21)
    c["dx"].zero_()
    want, off = reference(c)
    d = {k: v.cuda() for k, v in c.items() if torch.is_tensor(v)}
    ws = dit.workspace()
    projection = dit.RoutedLinear(dit.QuantizedWeight(torch.randn(N, K, device="cuda"), 64, ws), T, ws)
    bank = dit.AdapterBank(d["a"], d["b"], d["scale"])
    layer = dit.AdaptedLinear(projection, bank)
    plan = dit.AdapterPlan(c["lengths"], c["adapters"], G, training=True)
    scratch, saved = dit.adapter_scratch(plan, bank), dit.adapter_saved(plan, bank)
    da, db = torch.empty_like(d["a"], dtype=F32), torch.empty_like(d["b"], dtype=F32)
    y, dx = torch.zeros(T, N, device="cuda"), torch.full((T, K), 3.0, device="cuda")
    dit.lora_forward(plan, bank, d["x"], y, scratch, ws, saved=saved)
    busy = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for _ in range(20):
        busy = busy @ busy
    st = torch.cuda.Stream()
    layer.backward(d["x"], d["dy"], plan, saved, da, db, dx, scratch, stream=st)
    torch.cuda.synchronize()
    check(dx, want["dx"], off["dx"], "dx")
    check(da, want["da"], off["da"], "da")
    check(db, want["db"], off["db"], "db")
    assert dit.device_status(ws) == 0
