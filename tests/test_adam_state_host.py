"""Checks of a list update's state on the CPU: its buffers may have been exchanged for others,
which a list must not take by their address alone."""
import pytest

torch = pytest.importorskip("torch")


class _State:
    """An AdamState's fields, on the CPU."""

    def __init__(self, bits):
        self.numels, self.bits, self.device = [130, 0, 5], bits, torch.device("cpu")
        wide = torch.float32 if bits == 32 else torch.uint8
        self.m, self.v = torch.zeros(384, dtype=wide), torch.zeros(384, dtype=wide)
        self.m_exp = self.v_exp = None
        if bits == 8:
            self.m_exp, self.v_exp = (torch.zeros(3, dtype=torch.uint8) for _ in range(2))


@pytest.mark.parametrize("bits", [32, 8])
def test_buffers_of_a_state(bits):
    from zero_sharded_optimizer_rank_amd.adam import MOMENTS, _moments_of
    s = _State(bits)
    assert all(a is getattr(s, name) for a, name in zip(_moments_of(s), MOMENTS))
    for name in MOMENTS if bits == 8 else MOMENTS[:2]:
        t = getattr(s, name)
        for bad in (None, t[:-1], t.double(), t.to("meta"), torch.cat([t, t])[::2]):
            setattr(s, name, bad)
            with pytest.raises(ValueError, match=f"the state's {name} "):
                _moments_of(s)
        setattr(s, name, t)
    _moments_of(s)
