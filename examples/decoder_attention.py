"""A decoder's attention block served with 4-bit weights: requests of different
lengths, each with its own low-rank adapter, share the projections and a paged
cache of keys and values.

    python examples/decoder_attention.py

The prompts go through in chunks, mixed with single tokens of requests that are
further on; the decode steps are one captured graph, whose lengths and positions
advance on the device. Weights and inputs are random.
"""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gptq_bit_weight_amd as q4  # noqa: E402


def random_layer(K, N, group, g):
    """Packed weights, zero points and scales of a [K, N] layer."""
    words = lambda shape: torch.randint(-2 ** 31, 2 ** 31, shape, generator=g, device="cuda").int()  # noqa: E731
    scales = (torch.rand((K // group, N), generator=g, device="cuda") * 0.1 + 0.05) * K ** -0.5
    return words((K // 8, N)), words((K // group, N // 8)), scales.half()


class AttentionBlock:
    """x + o_proj(attention(q, k, v)), with q/k/v as one fused projection. The
    residual is in the activations' type; layers and adapters are kept for a
    caller that wants to check the block."""

    def __init__(self, hidden=1024, heads=8, kv_heads=2, dim=128, *, group=128, pages=512, page_size=16, adapters=4,
                 rank=16, dtype=torch.float16, scaling=None, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.kv_heads, self.dim, self.dtype = heads, kv_heads, dim, dtype
        sizes = [heads * dim, kv_heads * dim, kv_heads * dim]
        self.qkv_layers = [random_layer(hidden, n, group, g) for n in sizes]
        self.o_layer = random_layer(heads * dim, hidden, group, g)
        self.qkv = q4.Q4Matrix.concat(self.qkv_layers, groupsize=group)
        self.o = q4.Q4Matrix(*self.o_layer, groupsize=group)
        self.qkv_bank = q4.Q4Adapters(self.qkv, slots=adapters, rank=rank, dtype=dtype)
        self.o_bank = q4.Q4Adapters(self.o, slots=adapters, rank=rank, dtype=dtype)
        normal = lambda *s: (torch.randn(*s, generator=g, device="cuda") * 0.03).to(dtype)  # noqa: E731
        self.adapters = []
        for i in range(adapters):
            a = (normal(3, rank, hidden), normal(sum(sizes), rank), normal(1, rank, heads * dim), normal(hidden, rank))
            self.qkv_bank.load(i, a[0], a[1], 2.0)
            self.o_bank.load(i, a[2], a[3], 2.0)
            self.adapters.append(a)
        self.rotary = q4.Rotary(dim, scaling=scaling)
        store = torch.zeros(2, pages, kv_heads, page_size, dim, dtype=dtype, device="cuda")
        self.cache = q4.PagedCache(store[0], store[1])

    def __call__(self, x, positions, slots, starts, lengths, table, adapter):
        """x [tokens, hidden]; adapter: each token's slot in the banks, or -1."""
        T, n, m = x.shape[0], self.heads * self.dim, self.kv_heads * self.dim
        y = self.qkv.matmul_adapters(x, self.qkv_bank, adapter)
        q, k, v = (t.view(T, -1, self.dim) for t in y.split([n, m, m], 1))
        q = self.cache.append(k, v, slots, rotary=self.rotary, positions=positions, q=q)
        o = self.cache.attend(q, starts, lengths, table)
        return x + self.o.matmul_adapters(o.view(T, n), self.o_bank, adapter)


class Requests:
    """Which pages each request has, and the arrays of a step."""

    def __init__(self, cache, width):
        self.page_size, self.width = cache.page_size, width
        self.free = list(range(cache.pages - 1, -1, -1))
        self.pages, self.length, self.adapter = [], [], []

    def add(self, adapter):
        self.pages.append([])
        self.length.append(0)
        self.adapter.append(adapter)
        return len(self.pages) - 1

    def reserve(self, r, length):
        while len(self.pages[r]) * self.page_size < length:
            self.pages[r].append(self.free.pop())

    def arrays(self, news):
        """The arrays of a step in which request r gets news[r] tokens."""
        positions, slots, adapter, starts = [], [], [], [0]
        for r, n in enumerate(news):
            self.reserve(r, self.length[r] + n)
            for p in range(self.length[r], self.length[r] + n):
                positions.append(p)
                slots.append(self.pages[r][p // self.page_size] * self.page_size + p % self.page_size)
                adapter.append(self.adapter[r])
            self.length[r] += n
            starts.append(starts[-1] + n)
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        table = [p[:self.width] + [0] * (self.width - len(p)) for p in self.pages]
        return ints(positions), ints(slots), ints(starts), ints(self.length), ints(table), ints(adapter)


def serve(block, prompts, adapters, chunk, steps):
    """Prompts [tokens, hidden] in chunks, then `steps` decode steps that feed
    each request its own last output. Returns the prompts' outputs, the decode
    steps' [steps, requests, hidden], and the seconds of a decode step."""
    R = len(prompts)
    ps = block.cache.page_size
    reqs = Requests(block.cache, max(len(p) + steps for p in prompts) // ps + 1)
    for a in adapters:
        reqs.add(a)
    done, outs = [0] * R, [[] for _ in range(R)]
    while any(d < len(p) for d, p in zip(done, prompts)):
        news = [min(chunk, len(p) - d) for d, p in zip(done, prompts)]
        x = torch.cat([p[d:d + n] for p, d, n in zip(prompts, done, news)])
        positions, slots, starts, lengths, table, adapter = reqs.arrays(news)
        y = block(x, positions, slots, starts, lengths, table, adapter)
        for r, part in enumerate(y.split(news)):
            outs[r].append(part)
            done[r] += news[r]
    outs = [torch.cat(o) for o in outs]
    # ---- decode: everything that changes from step to step is on the device
    for r in range(R):
        reqs.reserve(r, reqs.length[r] + steps + 1)
    positions, slots, starts, lengths, table, adapter = reqs.arrays([1] * R)
    x = torch.stack([o[-1] for o in outs])
    history = torch.zeros(steps, *x.shape, dtype=x.dtype, device="cuda")
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    first = (positions.clone(), lengths.clone(), x.clone())

    def decode():
        torch.add(table.gather(1, (positions // ps).long()[:, None])[:, 0] * ps, positions % ps, out=slots)
        y = block(x, positions, slots, starts, lengths, table, adapter)
        history.index_copy_(0, step, y[None])
        x.copy_(y)
        positions.add_(1)
        lengths.add_(1)
        step.add_(1)

    decode()                     # (workspaces grow outside the capture)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        decode()
    for t, f in zip((positions, lengths, x), first):
        t.copy_(f)
    step.zero_()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(steps):
        graph.replay()
    torch.cuda.synchronize()
    return outs, history, (time.perf_counter() - t) / steps


def main():
    block = AttentionBlock(hidden=4096, heads=32, kv_heads=8, adapters=4, pages=1024)
    g = torch.Generator(device="cuda").manual_seed(1)
    prompts = [torch.randn(n, 4096, generator=g, device="cuda").half() for n in (700, 33, 5, 1200)]
    outs, history, seconds = serve(block, prompts, [0, 1, -1, 3], chunk=256, steps=32)
    whole, _, _ = serve(block, prompts, [0, 1, -1, 3], chunk=4096, steps=1)
    off = max((a.float() - b.float()).abs().max().item() for a, b in zip(outs, whole))
    print(f"4 requests, prompts of {[len(p) for p in prompts]} tokens in chunks of 256: outputs {off:.2g} from those of whole "
          f"prompts; a decode step of 4 tokens {seconds * 1e6:.1f} us; last values finite: {bool(history.isfinite().all())}")


if __name__ == "__main__":
    main()
