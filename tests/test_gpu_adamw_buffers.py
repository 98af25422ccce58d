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


def test_states_that_do_not_fit_are_refused_before_anything_is_copied():
    p, g = [torch.ones(300, device="cuda"), torch.ones(700, device="cuda")], [torch.ones(300, device="cuda"), torch.ones(700, device="cuda")]
    opt = dit.AdamW(p, g, **dit.adamw_moments(p, 8))
    opt.step()
    good = opt.state_dict()
    other = dit.AdamW(p, g, **dit.adamw_moments(p, 8))
    short = lambda name, ts: {**good, name: ts}  # noqa: E731
    for bad in (short("m_scale", good["m_scale"][:1]), short("v_scale", []), {k: v for k, v in good.items() if k != "v_scale"},
                short("v", good["v"][:1]), short("m", [t.float() for t in good["m"]]), short("bits", 32), short("step", -1),
                short("v_scale", [t[:1] for t in good["v_scale"]]), short("m_scale", [t.double() for t in good["m_scale"]])):
        with pytest.raises(dit.DitError):
            other.load_state_dict(bad)
        assert other.step_count == 0 and not any(t.float().any() for name in ("m", "v", "m_scale", "v_scale") for t in other._lists[name])
    other.load_state_dict(good)
    assert other.step_count == 1
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for n in ("m", "v") for a, b in zip(opt._lists[n], other._lists[n]))
