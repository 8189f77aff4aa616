"""Workgroups of lora_add that give up waiting for v and make it themselves
(moe_lora_add_polls): every kernel ends, and the results have the bits of the
call that waits, whether none, some or all of them gave up."""

import pytest
import torch

import batch_ref as B
import quantized_routed_moe_amd as qm
from batch_ref import gen

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class Case:
    def __init__(self, T, K, N, r, L, dtype, run=1):
        g = gen(T + K + N + r)
        self.size, self.dtype = (T, K, N, r, L), dtype
        self.x, self.a, self.b, self.base, self.s = B.lora_case(g, T, K, N, r, L, dtype)
        self.ids = torch.randint(-1, L, (T // run + 1,), generator=g, device="cuda", dtype=I32).repeat_interleave(run)[:T].contiguous()
        self.plan = qm.lora_plan(self.ids, L)
        n = qm.lib().moe_lora_add_workspace_bytes(*self.size)
        assert n > 0                    # v is handed over
        self.ws = torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")

    def run(self, polls, base=None, out=None):
        T, K, N, r, L = self.size
        base = self.base if base is None else base
        out = torch.full_like(base, 7.0) if out is None else out
        rc = qm.lib().moe_lora_add_polls(
            T, K, N, r, L, self.x.data_ptr(), K, self.a.data_ptr(), self.b.data_ptr(), self.s.data_ptr(), self.plan.perm_addr,
            self.plan.items_addr, base.data_ptr(), N, out.data_ptr(), N, qm.MOE_TYPE_BF16 if self.dtype == BF16 else qm.MOE_TYPE_F32,
            self.ws.data_ptr(), self.ws.numel(), polls, torch.cuda.current_stream().cuda_stream)
        assert rc == qm.MOE_OK
        return out


# steps of ranks 1 / 2 / 4 / 8, whole 16 bytes of columns or not, runs of up to 16 and 32 tokens and of several parts of K
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N", [520, 1111])
@pytest.mark.parametrize("r", [8, 24, 40, 64, 104, 256])
@pytest.mark.parametrize("T,K,L,run", [(5, 96, 2, 1), (41, 4096, 3, 1), (200, 1056, 5, 40)])
def test_the_same_bits_without_waiting(T, K, N, r, L, run, dtype):
    c = Case(T, K, N, r, L, dtype, run)
    want = qm.lora_add(c.base, c.x, c.a, c.b, c.plan, scales=c.s)
    ref, bound = B.lora(c.base, c.x, c.a, c.b, c.ids, c.s)
    B.check_rounded(want, ref, bound, dtype)
    for polls in (0, 1, 2, 1 << 18):
        c.ws.fill_(0xff if polls else 0)
        assert torch.equal(c.run(polls), want), polls
        again = c.base.clone()          # in place: what was given up has not been touched
        assert torch.equal(c.run(polls, again, again), want), polls


def test_many_tokens_without_waiting():
    c = Case(2048, 4096, 1024, 128, 16, BF16, 256)
    want = c.run(1 << 14)
    for polls in (0, 1, 4, 16):
        assert torch.equal(c.run(polls), want), polls


def test_some_wait_and_others_do_not_on_two_streams():
    cases = [Case(300, 2048, 2048, 72, 5, F32, 60), Case(64, 2048, 2048, 16, 64, BF16)]
    want = [c.run(1 << 14) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for polls in (0, 3, 1 << 14):
        got = []
        for c, st in zip(cases, streams):
            with torch.cuda.stream(st):
                got.append(c.run(polls))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w), polls


def test_captured_without_waiting():
    c = Case(70, 512, 640, 40, 6, BF16)
    want = c.run(0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = c.run(0)
    for _ in range(4):
        got.zero_()
        c.ws.random_(0, 256)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
