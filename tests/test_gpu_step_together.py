"""GPU: a server's steps with all of the step's operators together: tables from
lengths, norms and rotation over three axes with the cache write, attention with
shared prefixes and attention with first tokens beside a window, eagerly and from
a captured graph, each step against the definitions in 64 bits."""
import pytest
import torch

import attn_reference as ref
import linear_exl3_input_amd as ex
import step_reference as step
from gpu_util import banner
from test_gpu_step_prefix import widened
from test_gpu_step_sinks import seen_of

pytestmark = pytest.mark.gpu

HQ, HKV, PAGE, ROWS = 4, 2, 16, 24  # a step has room for ROWS tokens


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Server:
    """Requests in groups that start with the same tokens, and on the CPU what each has in the cache."""

    def __init__(self, d, dtype, bits, window, sinks):
        g = torch.Generator().manual_seed(d + bits)
        self.g, self.d, self.dtype, self.window, self.sinks = g, d, dtype, window, sinks
        self.cache = ex.KvCache.empty(60, PAGE, HKV, d, bits, dtype)
        nan = torch.full((60 * PAGE, HKV, d), float("nan"), dtype=dtype, device="cuda")
        ex.cache_write(self.cache, nan, nan, torch.arange(60 * PAGE, dtype=torch.int32, device="cuda"))
        self.rope = ex.Rope.make(d // 2, 1e4, 400, sections=(d // 8, d // 16, d // 16), in_turn=True)
        self.wq, self.wk = (1 + 0.3 * torch.randn(d, generator=g) for _ in range(2))
        self.norm = ex.HeadNorm(self.wq.cuda(), self.wk.cuda(), 1e-5)
        self.group_cu, self.prefix = [0, 3, 5], [96, 64]
        B = 6  # the last one shares nothing
        self.table = widened(self.cache, torch.full((B, 20), -1, dtype=torch.int32, device="cuda"))
        self.free = torch.randperm(60, generator=g).int().cuda()
        self.taken = ints([0])
        self.kv_len = ints([0] * B)
        self.keys, self.values = [torch.zeros(0, HKV, d) for _ in range(B)], [torch.zeros(0, HKV, d) for _ in range(B)]
        self.q, self.k, self.v, self.out, self.low, self.k_out = (
            torch.zeros(ROWS, h, d, dtype=dtype, device="cuda") for h in (HQ, HKV, HKV, HQ, HQ, HKV))
        self.q_len, self.groups, self.lens = ints([0] * B), ints(self.group_cu), ints(self.prefix)
        self.fill()

    def fill(self):
        """The groups' first tokens, by way of their first sequences."""
        kv = [0] * 6
        for lead, n in zip(self.group_cu, self.prefix):
            for start in range(0, n, ROWS):
                want = [min(ROWS, n - start) if b == lead else 0 for b in range(6)]
                self.inputs(want)
                self.forward()
                self.follow(want)
                self.advance()
        for g, n in enumerate(self.prefix):
            lead = self.group_cu[g]
            for b in range(lead + 1, self.group_cu[g + 1]):
                self.table[b] = self.table[lead]
                self.kv_len[b] = n
                self.keys[b], self.values[b] = self.keys[lead].clone(), self.values[lead].clone()

    def inputs(self, q_len):
        for t, h in ((self.q, HQ), (self.k, HKV), (self.v, HKV)):
            t.copy_((2 * torch.randn(ROWS, h, self.d, generator=self.g)).to(self.dtype))
        self.q_len.copy_(ints(q_len))

    def forward(self):
        self.step = s = ex.cache_extend(self.cache, self.q_len, self.kv_len, self.table, self.free, ROWS, self.taken)
        self.pos = torch.stack((s.positions, s.positions // 7, s.positions % 7))
        q = ex.rope_cache_write(self.cache, self.rope, self.pos, s.slots, self.q, self.k, self.v, k_out=self.k_out, norm=self.norm)
        ex.prefix_attention(self.cache, q, s.cu_q, s.kv_len, self.table, self.groups, self.lens, out=self.out)
        ex.paged_attention(self.cache, q, s.cu_q, s.kv_len, self.table, window=self.window, sinks=self.sinks, out=self.low)
        self.turned = q

    def advance(self):
        self.kv_len.copy_(self.step.kv_len)
        self.taken.add_(self.step.counts[1:])

    def follow(self, q_len):
        """Adds the step's tokens to what the requests have here."""
        at = 0
        for b, n in enumerate(q_len):
            for to, x in ((self.keys, self.k_out), (self.values, self.v)):
                to[b] = torch.cat((to[b], ref.quantise(x[at:at + n].cpu(), self.cache.bits).float()))
            at += n

    def check(self, q_len, what):
        self.follow(q_len)
        s, total = self.step, sum(q_len)
        assert s.cu_q.tolist() == [sum(q_len[:b]) for b in range(7)], what
        assert s.kv_len.tolist() == [len(k) for k in self.keys], what
        # rows that no request has: no slot, and results as they were
        assert (s.slots[total:] == -1).all() and (s.positions[total:] == 0).all(), what
        assert (self.out[total:] == 7).all() and (self.low[total:] == 7).all(), what
        axes = self.rope.axes
        for x, y, w in ((self.q, self.turned, self.wq), (self.k, self.k_out, self.wk)):
            n, err = step.normed(x.cpu(), w, 1e-5)
            ref.check(y[:total], *(t[:total] for t in step.turned(n, err, self.rope.table.cpu(), self.pos.cpu(), axes, False, self.dtype)), what)
        at = 0
        for b, n in enumerate(q_len):
            if n == 0:
                continue
            k, v, q = self.keys[b].double(), self.values[b].double(), self.turned[at:at + n].cpu().double()
            m = len(k)
            ref.check(self.out[at:at + n], *ref.attend(q, k, v, ref.mask(n, m), self.d ** -0.5, self.dtype), f"{what}, request {b}")
            ref.check(self.low[at:at + n], *ref.attend(q, k, v, seen_of(n, m, self.window, self.sinks), self.d ** -0.5, self.dtype),
                      f"{what}, request {b}, window")
            at += n

    def clear(self):
        self.out.fill_(7)
        self.low.fill_(7)


@pytest.mark.parametrize("d,dtype,bits,window,sinks", [(64, torch.float16, 16, 20, 3), (128, torch.bfloat16, 8, 70, 17),
                                                       (256, torch.bfloat16, 4, 33, 40)])
def test_steps_of_a_server(d, dtype, bits, window, sinks):
    banner(f"a server's steps, {bits} bits, heads of {d}")
    x = Server(d, dtype, bits, window, sinks)
    for q_len in ([5, 1, 9, 2, 0, 7], [1, 0, 1, 1, 1, 1], [0, 8, 0, 0, 8, 8]):
        x.inputs(q_len)
        x.clear()
        x.forward()
        torch.cuda.synchronize()
        x.check(q_len, f"eager {q_len}")
        x.advance()
    # one token each from a graph, twice over a page
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ex.reserve_workspace(max(ex.prefix_attention_workspace_bytes(6, ROWS, 2, HQ, HKV, d),
                                 ex.attention_workspace_bytes(6, ROWS, HQ, HKV, d)))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    q_len = [1, 1, 1, 0, 1, 1]
    x.inputs(q_len)
    with torch.cuda.graph(graph, stream=side):
        x.forward()
        x.advance()
    for i in range(18):
        x.inputs(q_len)
        x.clear()
        graph.replay()
        torch.cuda.synchronize()
        x.check(q_len, f"replay {i}")
    used = int(x.taken)
    held = {p for b in range(6) for p in x.table[b, :-(-len(x.keys[b]) // PAGE)].tolist()}
    assert -1 not in held and len(held) == used  # every page taken is in some table, and none twice but the shared ones
