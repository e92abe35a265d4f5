"""GPU: a call whose tensors are not on the current device makes theirs current
for its launch (shown with a stand-in for the device's number, on one GPU)."""
import pytest
import torch

import linear_exl3_input_amd as ex
from linear_exl3_input_amd import attention as at

pytestmark = pytest.mark.gpu


class Devices:
    """Counts as device 1 being current; `torch.cuda.device` switches the count."""

    def __init__(self, monkeypatch):
        self.current, self.entered = 1, []
        outer = self

        class Switch:
            def __init__(self, device):
                self.device = torch.device(device)

            def __enter__(self):
                self.before, outer.current = outer.current, self.device.index
                outer.entered.append(self.device.index)

            def __exit__(self, *exc):
                outer.current = self.before

        monkeypatch.setattr(at, "_current_device", lambda: self.current)
        monkeypatch.setattr(torch.cuda, "device", Switch)


def test_calls_switch_to_their_tensors_device(monkeypatch):
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(5, h, 64, generator=g).bfloat16().cuda() for h in (4, 2, 2))
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    r, cache = ex.Rope.make(64, 1e4, 32), ex.KvCache.empty(2, 16, 2, 64, 8)
    pos, slots, cu, lens, table = ints(0, 1, 2, 3, 4), ints(16, 17, 18, 19, 20), ints(0, 5), ints(5), ints(1).view(1, 1)
    calls = [lambda: ex.rope(r, pos, q, k), lambda: ex.rope(r, positions=pos, q=q),
             lambda: ex.cache_write(cache, k, v, slots), lambda: ex.cache_read(cache, slots),
             lambda: ex.rope_cache_write(cache, r, pos, slots, q, k, v), lambda: ex.cache_read(cache, slots),
             lambda: ex.paged_attention(cache, q, cu, lens, table), lambda: ex.paged_attention(cache, q, cu, lens, table, 0.3, 2),
             lambda: ex.prompt_attention(q, k, v, cu), lambda: ex.prompt_attention(q, k, v, cu, False, scale=0.2)]

    def results():
        out = []
        for c in calls:
            y = c()
            out += [] if y is None else [y] if torch.is_tensor(y) else list(y)
        return [t.clone() for t in out]

    want = results()
    devices = Devices(monkeypatch)
    got = results()
    assert devices.entered == [0] * len(calls) and devices.current == 1
    assert len(got) == len(want) and all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(got, want))
    devices.current, devices.entered = 0, []
    results()
    assert devices.entered == []
