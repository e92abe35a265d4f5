"""GPU: two host threads on one stream, whose calls share its workspace: shared
prefixes (two launches and more, with results in the workspace between them)
beside attention in parts, give the bits that each gives alone."""
import threading

import pytest
import torch

import linear_exl3_input_amd as ex
from gpu_util import banner
from test_gpu_step_prefix import Shared
from test_gpu_step_sinks import BF16, Paged, same_bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sequences", [8, 270])
def test_two_threads_on_one_stream(sequences):
    banner(f"two threads, {sequences} sequences")
    x = Shared([(640, [(1, 50 + i % 40) for i in range(sequences)])], 8, 2, 128, BF16, 8, 64, seed=40)
    cache, q, cu, kv, table = x.args()
    more = (x.group_cu.cuda(), torch.tensor(x.shared, dtype=torch.int32).cuda())
    y = Paged([1, 1, 2], [9000, 50, 7000], 8, 2, 128, BF16, 8, 64, seed=41)
    y_args = (y.cache, y.q.cuda(), y.cu.cuda(), torch.tensor(y.kv_lens, dtype=torch.int32).cuda(), y.table.cuda())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    calls = (lambda out: ex.prefix_attention(cache, q, cu, kv, table, *more, out=out),
             lambda out: ex.paged_attention(*y_args, out=out))
    with torch.cuda.stream(side):
        want = [calls[0](None), calls[1](None)]
        outs = [[torch.zeros_like(w) for _ in range(40)] for w in want]
    side.synchronize()
    failed = []
    start = threading.Barrier(2)

    def run(i):
        try:
            with torch.cuda.stream(side):
                start.wait(20)
                for out in outs[i]:
                    calls[i](out)
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    side.synchronize()
    assert not failed, failed
    for w, each in zip(want, outs):
        assert all(same_bits(o, w) for o in each)
