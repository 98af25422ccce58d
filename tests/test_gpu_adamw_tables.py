"""AdamW's chunk table: entries past a tensor's end are skipped and reported by every kernel that reads the table."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import int8_mixed_precision_gb300 as dit  # noqa: E402

BF16 = torch.bfloat16


@pytest.mark.parametrize("chunk", [3, 1000])
@pytest.mark.parametrize("bits", [32, 8])
def test_a_chunk_past_the_end_is_reported(bits, chunk):
    n = 10000                                           # chunks 0, 1 and 2
    p, g = torch.ones(n, device="cuda"), torch.ones(n, device="cuda")
    values = {} if bits == 32 else {k: [torch.full((n,), 7.0, dtype=BF16, device="cuda")] for k in ("m_values", "v_values")}
    opt = dit.AdamW([p], [g], **dit.adamw_moments([p], bits), **values)
    opt._chunks[1, 1] = chunk
    opt.step()
    torch.cuda.synchronize()
    assert dit.device_status(opt.ws) == 1 << 1
    assert bool((p[4096:8192] == 1).all()) and bool((p[:4096] != 1).all()) and bool((p[8192:] != 1).all())
    if bits == 8:
        dit.clear_device_status(opt.ws)
        opt.export_moments()
        torch.cuda.synchronize()
        assert dit.device_status(opt.ws) == 1 << 1
        m = values["m_values"][0]
        assert bool((m[4096:8192] == 7).all()) and bool((m[:4096] != 7).all()) and bool((m[8192:] != 7).all())


def test_right_tables_are_not_reported():
    sizes = [0, 1, 4096, 4097, 12288]
    p, g = [torch.ones(n, device="cuda") for n in sizes], [torch.ones(n, device="cuda") for n in sizes]
    for bits in (8, 32):
        opt = dit.AdamW(p, g, **dit.adamw_moments(p, bits))
        opt.step()
        assert dit.device_status(opt.ws) == 0
