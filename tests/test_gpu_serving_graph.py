"""A whole serving step -- release, plan, rotary append, attention -- captured in one graph and replayed
while lengths, new tokens and inputs change on the device: the same bits as the calls made one by one."""

import pytest
import torch

import paged_kv_cache_page_gb300 as pa

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HQ, HKV, D, PAGE, B, POOL, CAP = 8, 2, 64, 16, 4, 40, 96


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Server:
    """The buffers of one server, and one step of it."""

    def __init__(self):
        self.caches = [torch.zeros((POOL, PAGE, HKV, D), device=DEV).to(torch.float8_e4m3fn) for _ in range(2)]
        self.scale = [torch.full((HKV,), s, device=DEV) for s in (0.02, 0.01)]
        self.lens, self.new, self.keep = i32([0] * B), i32([0] * B), i32([0] * B)
        self.table, self.pool, self.count = i32([[-1] * 20] * B), i32(list(range(POOL))), i32([POOL])
        self.cu, self.pos = i32([0] * (B + 1)), i32([0] * CAP)
        self.slots = torch.zeros(CAP, dtype=torch.int64, device=DEV)
        self.qkv = torch.zeros((CAP, HQ + 2 * HKV, D), dtype=torch.bfloat16, device=DEV)
        self.q = torch.zeros((CAP, HQ, D), dtype=torch.bfloat16, device=DEV)
        self.out, self.lse = torch.zeros_like(self.q), torch.zeros((HQ, CAP), device=DEV)
        ang = torch.arange(400).double()[:, None] * 100.0 ** (-torch.arange(0, D, 2).double() / D)
        self.cos, self.sin = ang.cos().float().to(DEV), ang.sin().float().to(DEV)
        self.workspace = torch.full((pa.fwd_varlen_e4m3_workspace_size(B, CAP, CAP, HQ, HKV, D, 320),), 0xff,
                                    dtype=torch.uint8, device=DEV)
        self.err = pa.new_err_word(DEV)

    def step(self):
        pa.pa_release_pages(self.lens, self.keep, self.table, self.pool, self.count, PAGE, err=self.err)
        pa.pa_plan_step(self.lens, self.new, self.table, self.pool, self.count, PAGE, self.cu, self.lens,
                        self.slots, self.pos, err=self.err)
        q, k, v = self.qkv[:, :HQ], self.qkv[:, HQ:HQ + HKV], self.qkv[:, HQ + HKV:]
        pa.pa_rotary_append_varlen(q, k, v, *self.caches, self.slots, positions=self.pos, rotary_cos=self.cos,
                                   rotary_sin=self.sin, k_scale=self.scale[0], v_scale=self.scale[1],
                                   q_out=self.q, err=self.err)
        pa.pa_fwd_varlen_e4m3(self.q, *self.caches, self.cu, self.lens, self.table, CAP, 320,
                              k_scale=self.scale[0], v_scale=self.scale[1], out=self.out, lse=self.lse,
                              workspace=self.workspace, err=self.err)


def test_a_captured_step_replayed():
    eager, graphed = Server(), Server()
    # (calls outside the capture first, as a server makes them; a step without requests changes nothing)
    graphed.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.step()
    steps = [([30, 0, 1, 40], [999] * B), ([1, 20, 1, 1], [999] * B), ([1, 1, 50, 1], [32, 21, 0, 40]),
             ([1, 1, 0, 1], [999] * B), ([9, 60, 1, 3], [0, 22, 50, 43]), ([1, 1, 1, 1], [999] * B),
             ([90, 0, 0, 0], [0, 0, 0, 0])]
    g = torch.Generator().manual_seed(6)
    for new, keep in steps:
        x = torch.randn(eager.qkv.shape, generator=g).bfloat16()
        for s in (eager, graphed):
            s.new.copy_(i32(new))
            s.keep.copy_(i32(keep))
            s.qkv.copy_(x)
        eager.step()
        graph.replay()
        torch.cuda.synchronize()
        rows = sum(new)
        assert eager.cu.tolist()[-1] == rows and eager.err.tolist() == graphed.err.tolist() == [0] * 4
        for name in ("lens", "table", "pool", "count", "cu", "slots", "pos"):
            assert torch.equal(getattr(eager, name), getattr(graphed, name)), name
        assert torch.equal(eager.q, graphed.q)
        for a, b in zip(eager.caches, graphed.caches):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert torch.equal(eager.out[:rows], graphed.out[:rows])
        assert torch.equal(eager.lse[:, :rows], graphed.lse[:, :rows])
        assert torch.isfinite(eager.out).all()
