"""AdamW's tables hold addresses: what they point to lives as long as the optimiser, whatever becomes of the tensors."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import int8_mixed_precision_gb300 as dit  # noqa: E402


def test_memory_that_the_tables_point_to_is_not_given_away():
    """Storages exchanged under the tensors (``.data = ...``): a step still writes to those it was made with and not
    to tensors made since."""
    n = 3 << 20                                          # a block of the allocator's own
    p, g = torch.ones(n, device="cuda"), torch.ones(n, device="cuda")
    opt = dit.AdamW([p], [g], **dit.adamw_moments([p], 32))
    at = {t.data_ptr() for t in (p, g, opt._lists["m"][0], opt._lists["v"][0])}
    for t in (p, g, opt._lists["m"][0], opt._lists["v"][0]):
        t.data = torch.zeros(n, device="cuda")
    since = [torch.full((n,), 7.0, device="cuda") for _ in range(8)]
    assert not at & {t.data_ptr() for t in since}        # the step would write over them
    opt.step()
    torch.cuda.synchronize()
    assert all(bool((t == 7).all()) for t in since) and not p.any()
