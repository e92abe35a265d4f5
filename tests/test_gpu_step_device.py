"""GPU: the step's calls make their tensors' device current for their launch
(shown with a stand-in for the device's number, on one GPU)."""
import pytest
import torch

import linear_exl3_input_amd as ex
from test_gpu_attention_device import Devices

pytestmark = pytest.mark.gpu


def test_calls_switch_to_their_tensors_device(monkeypatch):
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(5, h, 64, generator=g).bfloat16().cuda() for h in (4, 2, 2))
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    r, cache = ex.Rope.make(64, 1e4, 32, sections=(16, 16)), ex.KvCache.empty(2, 16, 2, 64, 8)
    norm = ex.HeadNorm(torch.ones(64, device="cuda"), torch.ones(64, device="cuda"))
    pos, slots, cu, lens, table = ints(*range(10)).view(2, 5), ints(16, 17, 18, 19, 20), ints(0, 2, 5), ints(5, 5), ints(1, 1).view(2, 1)
    calls = [lambda: ex.rope(r, pos, q, k, norm=norm), lambda: ex.rope_cache_write(cache, r, pos, slots, q, k, v, norm=norm),
             lambda: ex.cache_read(cache, slots), lambda: ex.paged_attention(cache, q, cu, lens, table, window=2, sinks=1),
             lambda: ex.prompt_attention(q, k, v, cu, window=1, sinks=1),
             lambda: ex.prefix_attention(cache, q, cu, lens, table, ints(0, 2), ints(3)),
             lambda: ex.cache_extend(cache, ints(1, 2), lens, table, ints(0), 4)]

    def results():
        out = []
        for c in calls:
            y = c()
            out += [y] if torch.is_tensor(y) else list(y)
        return [t.clone() for t in out]

    want = results()
    devices = Devices(monkeypatch)
    got = results()
    assert devices.entered == [0] * len(calls) and devices.current == 1
    assert len(got) == len(want) and all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(got, want))


def test_tensors_of_different_devices_are_refused():
    cache, r = ex.KvCache.empty(2, 16, 2, 64, 8), ex.Rope.make(64, 1e4, 32, sections=(16, 16))
    q = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    ints = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    with pytest.raises(ValueError, match="positions must be int32"):
        ex.rope(r, pos.cpu(), q)
    with pytest.raises(ValueError, match="positions must be int32"):
        ex.rope(r, pos[0], q)
    with pytest.raises(ValueError, match="positions must be int32"):
        ex.rope(r, pos.T.contiguous().T, q)
    with pytest.raises(ValueError, match="norms are of 128-value heads"):
        ex.rope(r, pos, q, norm=ex.HeadNorm(torch.ones(128, device="cuda")))
    with pytest.raises(ex.Exl3Error, match="norm k is NULL"):
        ex.rope(r, pos, q, q, norm=ex.HeadNorm(torch.ones(64, device="cuda")))
    with pytest.raises(ValueError, match="k_weight"):
        ex.HeadNorm(torch.ones(64, device="cuda"), torch.ones(128, device="cuda"))
    table = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="dense int32"):
        ex.cache_extend(cache, ints(2).cpu(), ints(2), table, ints(3), 4)
    with pytest.raises(ValueError, match="page_table must be int32"):
        ex.cache_extend(cache, ints(2), ints(2), table[:1], ints(3), 4)
    with pytest.raises(ValueError, match="tokens=-1"):
        ex.cache_extend(cache, ints(2), ints(2), table, ints(3), -1)
    kv = ints(2)
    with pytest.raises(ex.Exl3Error, match="kv_len and kv_out overlap"):
        ex.cache_extend(cache, ints(2), kv, table, ints(3), 4, out=ex.CacheStep(ints(3), kv, ints(4), ints(4), ints(2)))
    with pytest.raises(ValueError, match="slots must be"):
        ex.cache_extend(cache, ints(2), kv, table, ints(3), 4, out=ex.CacheStep(ints(3), ints(2), ints(4), ints(5), ints(2)))
    with pytest.raises(ValueError, match="group_cu must be"):
        ex.prefix_attention(cache, q, ints(3), kv, table, ints(2).cpu(), ints(1))
    with pytest.raises(ex.Exl3Error, match="groups=3"):
        ex.prefix_attention(cache, q, ints(3), kv, table, ints(4), ints(3))
