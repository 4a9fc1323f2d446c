"""Serving steps back to back in one graph: reserve, append by slots and attention with nothing between them, so that every
kernel is resident while the ones that write its page table, lengths, rows and scales still run."""
import numpy as np
import pytest
import torch

from decode_attention_mfa_gb300 import capi

pytestmark = pytest.mark.gpu
PAGE, HEADS, DIM = 64, 64, 256
SCALE = 1.0 / 16.0
KV = pytest.mark.parametrize("fp8", [False, True])


class Server:
    """Two groups of requests behind prompts of three and two pages, and the tokens that `steps` steps bring."""
    sizes, pages, cols, num_pages, most = [3, 4], [3, 2], 14, 160, 24

    def __init__(self, fp8, steps, seed):
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.fp8, self.steps, self.B = fp8, steps, sum(self.sizes)
        self.rows = self.B * self.most
        self.counts = rng.integers(0, self.most + 1, (steps, self.B))
        self.counts[3] = 0  # a step without a token
        self.prefix = np.repeat(self.pages, self.sizes)
        self.new = torch.from_numpy(self.counts).int().cuda()
        self.kv_new = torch.randn((steps, self.rows, 2 * DIM), generator=gen, device="cuda").bfloat16()
        self.q = torch.randn((steps, self.B, HEADS, DIM), generator=gen, device="cuda").bfloat16()
        prompt = torch.randn((2, sum(self.pages), PAGE, DIM), generator=gen, device="cuda")
        if fp8:
            self.prompt_scales = prompt.abs().amax(-1) / 448.0
            self.prompt = (prompt / self.prompt_scales.unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            self.prompt = prompt.bfloat16()
        self.kv = torch.empty((2, self.num_pages, PAGE, DIM), dtype=self.prompt.dtype, device="cuda")
        self.scales = torch.empty((2 * fp8, self.num_pages, PAGE), device="cuda")
        self.table = torch.empty((self.B, self.cols), **i32)
        self.free, self.n_free, self.lens = torch.empty(self.num_pages, **i32), torch.empty(1, **i32), torch.empty(self.B, **i32)
        self.starts = torch.empty(self.B + 1, **i32)
        self.slots = torch.empty(self.rows, dtype=torch.int64, device="cuda")
        self.group_starts = torch.tensor([0, 3, 7], **i32)
        self.group_pages = torch.tensor(self.pages, **i32)
        self.out = torch.empty((2, steps, self.B, HEADS, DIM), dtype=torch.bfloat16, device="cuda")
        self.lse = torch.empty((2, steps, self.B, HEADS), device="cuda")
        self.hints = (max(self.pages) * PAGE, steps * self.most)
        self.length = max(self.pages) * PAGE + steps * self.most
        need = max(capi.mfa_decode_prefix_workspace_bytes(self.B, 2, *self.hints),
                   capi.mfa_decode_workspace_bytes(self.B, self.length))
        self.ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        capi.mfa_workspace_init(self.ws, need)

    def reset(self, seed):
        """The state before the first step, with pages in another order; what no token has reached yet is poisoned."""
        ids = torch.randperm(self.num_pages, generator=torch.Generator().manual_seed(seed)).int().cuda()
        self.kv.fill_(0x7F if self.fp8 else float("nan"))
        self.scales.fill_(float("nan"))
        own = ids[:sum(self.pages)].long()
        self.kv[:, own] = self.prompt
        if self.fp8:
            self.scales[:, own] = self.prompt_scales
        self.table.fill_(-1)
        self.table[:3, :3] = ids[:3]
        self.table[3:, :2] = ids[3:5]
        left = ids[sum(self.pages):]
        self.free.fill_(-1)
        self.free[:len(left)] = left
        self.n_free.fill_(len(left))
        self.lens.copy_(torch.from_numpy(self.prefix * PAGE))
        self.out.fill_(7.0)
        self.lse.fill_(7.0)
        torch.cuda.synchronize()

    def step(self, s, between=lambda: None):
        caches, scales = list(self.kv), list(self.scales)
        capi.mfa_reserve_pages(self.new[s], self.lens, self.table, self.free, self.n_free, self.B, self.cols, self.num_pages,
                               self.rows, self.starts, self.slots, self.lens, self.n_free, self.ws)
        between()
        append = capi.mfa_kv_append_slots_fp8 if self.fp8 else capi.mfa_kv_append_slots
        append(self.kv_new[s], self.kv_new[s][:, DIM:], 2 * DIM, 2 * DIM, self.slots, self.rows, *caches, *scales,
               self.num_pages, self.ws)
        between()
        size = self.ws.numel()
        for i in ((0, 1) if s % 2 else (1, 0)):
            if i == 0:
                f = capi.mfa_decode_attention_prefix_fp8 if self.fp8 else capi.mfa_decode_attention_prefix
                f(self.q[s], *caches, *scales, self.table, self.lens, self.group_starts, self.group_pages, 2, self.out[0, s],
                  self.lse[0, s], SCALE, self.B, self.cols, self.num_pages, *self.hints, self.ws, size)
            else:
                f = capi.mfa_decode_attention_fp8 if self.fp8 else capi.mfa_decode_attention
                f(self.q[s], *caches, *scales, self.table, self.lens, self.out[1, s], self.lse[1, s], SCALE, self.B, self.cols,
                  self.num_pages, self.length, self.ws, size)
            between()

    def reference(self, s, b):
        """Attention of step s for request b in 64 bits, from the cache as it stands at the end: rows are only added."""
        n = int(self.prefix[b] * PAGE + self.counts[:s + 1, b].sum())
        ids = self.table[b, :-(-n // PAGE)].long()
        k, v = (c[ids].view(torch.float8_e4m3fn).double() * self.scales[i][ids].double().unsqueeze(-1) if self.fp8
                else c[ids].double() for i, c in enumerate(self.kv))
        k, v = k.reshape(-1, DIM)[:n], v.reshape(-1, DIM)[:n]
        logits = self.q[s, b].double() @ k.T * SCALE
        lse = torch.logsumexp(logits, 1)
        return torch.exp(logits - lse[:, None]) @ v, lse, v.abs().max()


@KV
def test_steps_back_to_back_in_one_graph(fp8):
    """Twenty steps in a graph, replayed with pages in other orders, give bit for bit what the same calls give one after the
    other, and the first and last steps are held against 64 bits. Both attentions have the bounds of their own tests: a weight
    is off by 2^-8 of itself, the output's rounding by 2^-8, an 8-bit cache by as much again."""
    server = Server(fp8, 20, seed=31)
    server.reset(0)
    for s in range(server.steps):
        server.step(s, between=torch.cuda.synchronize)
    capi.mfa_check_device_errors(server.ws)
    want = server.out.clone(), server.lse.clone()
    assert server.lens.tolist() == (server.prefix * PAGE + server.counts.sum(0)).tolist()
    for s in (0, 1, 2, 9, 18, 19):
        for b in range(server.B):
            out, lse, top = server.reference(s, b)
            for i in range(2):
                assert ((server.out[i, s, b].double() - out).abs() <= 2 ** -8 * (2 * (1 + fp8) * top + out.abs())).all(), (s, b, i)
                assert float((server.lse[i, s, b].double() - lse).abs().max()) <= 1e-3, (s, b, i)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            for s in range(server.steps):
                server.step(s)
    for turn in range(1, 13):
        server.reset(turn)
        with torch.cuda.stream(stream):
            graph.replay()
        stream.synchronize()
        capi.mfa_check_device_errors(server.ws)
        assert torch.equal(server.lse, want[1]) and torch.equal(server.out, want[0]), turn


@KV
def test_steps_back_to_back_without_a_graph(fp8):
    server = Server(fp8, 20, seed=32)
    server.reset(0)
    for s in range(server.steps):
        server.step(s, between=torch.cuda.synchronize)
    want = server.out.clone(), server.lse.clone()
    for turn in range(1, 5):
        server.reset(turn)
        for s in range(server.steps):
            server.step(s)
        torch.cuda.synchronize()
        capi.mfa_check_device_errors(server.ws)
        assert torch.equal(server.lse, want[1]) and torch.equal(server.out, want[0]), turn
