"""Adapters of many requests beside the quantized product on the GPU, against
the definition in 64 bits.

Tolerance: the product's own acceptance rule (tests/gpu_util.py: REL_A A + REL_Y
|y|, for bfloat16 its terms), whose |y| term covers the one rounding of the whole
sum, plus what the adapter's part adds, derived: c A x is a fp32 sum of K exact products
(K 2^-24 c sum |A x|) and is kept in fp32 or in two halves (2^-16 of it at
most); B's products are summed in fp32 (rank 2^-24, below the same 2^-16).
"""
import math

import numpy as np
import pytest

import synth
from tests.gpu_util import BF16_GEMM_REL_A, BF16_REL_Y, REL_A, REL_Y, announce, device_tensors, torch_mod

torch = torch_mod()
pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gptq_bit_weight_amd as q4
    q4.load_library()
    yield


class Case:
    """A matrix of parts, a bank, activations, and the definition's result."""

    def __init__(self, K, parts, G, fmt="f16", slots=5, rank=8, act=False, bits=4, seed=0, ranks=None):
        import gptq_bit_weight_amd as q4
        self.K, self.N, self.fmt, self.dt = K, sum(parts), fmt, DT[fmt]
        self.bits, self.parts, self.slots, self.rank = bits, parts, slots, rank
        L = [synth.make_layer(K, n, G, 1, seed=synth.layer_seed("adapters", K, n, i, seed), act_order=act, bits=bits)
             for i, n in enumerate(parts)]
        if act:
            for part in L[1:]:
                part.g_idx = L[0].g_idx
        T = [device_tensors(part) for part in L]
        self.W = q4.Q4Matrix.concat([(t["qweight"], t["qzeros"], t["scales"]) for t in T], T[0]["g_idx"],
                                    groupsize=-1 if G == K else G, bits=bits)
        g = self.gen = torch.Generator(device="cuda").manual_seed(seed + 17)
        self.bank = q4.Q4Adapters(self.W, slots, rank, self.dt)
        self.A, self.B, self.c = [], [], []
        for s in range(slots):
            r = rank if ranks is None else ranks[s]
            self.A.append((torch.randn(len(parts), r, K, generator=g, device="cuda") * K ** -0.5).to(self.dt))
            self.B.append((torch.randn(self.N, r, generator=g, device="cuda") * 0.2).to(self.dt))
            self.c.append(0.5 + s * 0.25)
            self.bank.load(s, self.A[s], self.B[s], self.c[s])
        # the weights in 64 bits, by the definition
        per, cols = 32 // bits, []
        for t in T:
            sh = torch.arange(per, device="cuda") * bits
            m = (1 << bits) - 1
            q = ((t["qweight"].long()[:, None] >> sh[None, :, None]) & m).reshape(K, -1)
            z = ((t["qzeros"].long()[:, :, None] >> sh) & m).reshape(t["qzeros"].shape[0], -1)
            grp = T[0]["g_idx"].long() if act else torch.arange(K, device="cuda") // G
            cols.append((q - z[grp]).double() * t["scales"].double()[grp])
        self.w = torch.cat(cols, 1)

    def inputs(self, M, index=None, bias=True):
        x = torch.randn(M, self.K, generator=self.gen, device="cuda").to(self.dt)
        b = (torch.randn(self.N, generator=self.gen, device="cuda") * 0.1).to(self.dt) if bias else None
        if index is None:
            index = torch.randint(-1, self.slots, (M,), generator=self.gen, device="cuda")
        return x, b, index.int().cuda()

    def check(self, y, x, b, index, what="", skip=None):
        xd = x.double()
        ref = xd @ self.w + (b.double() if b is not None else 0)
        A = xd.abs() @ self.w.abs()
        extra = torch.zeros_like(ref)
        for s in range(self.slots):
            rows = (index == s).nonzero()[:, 0]
            if not rows.numel():
                continue
            at = 0
            for p, n in enumerate(self.parts):
                a, bb = self.A[s][p].double(), self.B[s][at:at + n].double()
                t, ta = xd[rows] @ a.t() * self.c[s], xd[rows].abs() @ a.abs().t() * self.c[s]
                ref[rows, at:at + n] += t @ bb.t()
                extra[rows, at:at + n] = (self.K * 2.0 ** -24 * ta + 2.0 ** -16 * t.abs()) @ bb.abs().t()
                at += n
        bf = self.fmt == "bf16"
        ra = BF16_GEMM_REL_A if bf and x.shape[0] > 32 else REL_A
        tol = ra * A + (BF16_REL_Y if bf else REL_Y) * ref.abs() + extra
        err = (y.double() - ref).abs()
        bad = ~(err <= tol)
        if skip is not None:
            bad[skip] = False
        assert not bad.any(), f"{what}: {int(bad.sum())} outside, first {bad.nonzero()[0].tolist()}, worst {(err / tol)[bad].max().item()}"

    def run(self, M, index=None, bias=True):
        announce(f"adapters {self.fmt} K={self.K} parts={self.parts} M={M} slots={self.slots} rank={self.rank}")
        x, b, index = self.inputs(M, index, bias)
        y = self.W.matmul_adapters(x, self.bank, index, b)
        self.check(y, x, b, index, f"M={M}")
        return y


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("K,parts,G,rank,act", [
    (512, [512], 128, 16, False), (1024, [264], 32, 4, True), (160, [72], -1, 24, False), (960, [136, 8, 40], 64, 8, False),
    (512, [128, 256], 128, 12, True), (2048, [1000], 128, 64, False), (256, [16, 24, 8, 400], 64, 1, False), (128, [64], 128, 100, False)])
def test_shapes(fmt, K, parts, G, rank, act):
    c = Case(K, parts, G if G > 0 else K, fmt, rank=rank, act=act)
    for M in (1, 2, 4, 5, 8, 9, 16, 17, 32, 33, 64, 77, 130, 300, 513, 700):
        c.run(M, bias=M % 2 == 0)


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
def test_eight_bit_weights(fmt):
    c = Case(512, [264, 64], 64, fmt, rank=16, bits=8)
    for M in (1, 7, 20, 40, 600):
        c.run(M)


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
def test_orders_of_rows(fmt):
    """Runs, all one slot, none at all, indexes outside the slots, one row each."""
    c = Case(512, [520], 128, fmt, slots=70, rank=16)
    for M in (3, 32, 33, 100, 600):
        a = torch.arange(M)
        for index in (a // 7 % 70, torch.full((M,), 69), torch.full((M,), -1), a % 70, (a * 37) % 70, 70 + a, -a - 1,
                      torch.where(a % 3 == 0, a % 70, torch.tensor(2 ** 31 - 1)), torch.where(a == M - 1, 3, -1)):
            c.run(M, index)


def test_many_slots():
    c = Case(128, [64], 128, slots=1500, rank=4)
    for M in (20, 200, 2500):
        c.run(M)


@pytest.mark.parametrize("K,parts,M", [(4096, [4096], 1), (4096, [4096, 4096, 4096], 32), (4096, [11008], 77), (11008, [4096], 33),
                                       (4096, [11008], 1200)])
def test_layer_sizes(K, parts, M):
    c = Case(K, parts, 128, "bf16" if M > 40 else "f16", slots=9, rank=16)
    c.run(M)


def test_split_k_and_stream_k():
    """Narrow layers, whose K is split between workgroups in both kernels."""
    c = Case(11008, [64], 128, rank=8)
    for M in (1, 30, 60, 300):
        c.run(M)
    c = Case(8192, [128, 8], 128, "bf16", rank=16)
    for M in (2, 32, 70, 600):
        c.run(M)


def test_ranks_below_the_banks_and_clear():
    c = Case(256, [72, 56], 64, "f16", slots=4, rank=20, ranks=[20, 1, 7, 16])
    for M in (5, 90):
        c.run(M)
    c.bank.load(0, c.A[2], c.B[2], -1.5)        # a smaller one over a larger
    c.A[0], c.B[0], c.c[0] = c.A[2], c.B[2], -1.5
    c.bank.clear(3)
    c.A[3], c.B[3], c.c[3] = c.A[3][:, :0], c.B[3][:, :0], 0.0
    for M in (5, 90):
        c.run(M)


def test_without_adapters_it_is_the_product():
    """Rows of no adapter have the product's own bits on the skinny kernel (the
    same kernel and plan), whatever other rows have. (The GEMM takes rows in
    another order, so a row's K may be split elsewhere.)"""
    c = Case(1024, [512], 128, rank=16)
    for M in (1, 8, 20, 32):
        x, b, index = c.inputs(M)
        index[::2] = -1
        y = c.W.matmul_adapters(x, c.bank, index, b)
        assert torch.equal(y[::2], c.W.matmul(x, b)[::2])


def test_what_is_not_finite_stays_with_its_rows():
    for M in (6, 32, 50, 600):
        for fmt in ("f16", "bf16"):
            c = Case(256, [72, 64], 64, fmt, slots=4, rank=8)
            bad_b, bad_a = c.B[1].clone(), c.A[2].clone()
            bad_b[5, 2] = float("inf")
            bad_b[75, 0] = float("nan")
            bad_a[0, 3, 9] = float("nan")
            c.bank.load(1, c.A[1], bad_b, c.c[1])
            c.bank.load(2, bad_a, c.B[2], c.c[2])
            x, b, index = c.inputs(M)
            x[3] = float("nan")
            y = c.W.matmul_adapters(x, c.bank, index, b)
            skip = torch.zeros(M, 136, dtype=torch.bool, device="cuda")
            skip[3] = True
            skip[index == 1, 5] = True
            skip[index == 1, 75] = True
            skip[(index == 2).nonzero()[:, 0], :72] = True      # (its second part's columns hold)
            xc = x.clone()
            xc[3] = 0
            c.check(torch.where(skip, torch.zeros_like(y), y), xc, b, index, f"M={M}", skip)
            assert y[3].isnan().all()


def test_a_slot_loaded_again_is_as_new():
    """Values that are not finite leave nothing behind when their slot is loaded
    or cleared."""
    for M in (8, 50, 600):
        c = Case(256, [72, 64], 64, "f16", slots=3, rank=8)
        c.bank.load(1, c.A[1], torch.full_like(c.B[1], math.nan), c.c[1])
        x, b, index = c.inputs(M)
        assert c.W.matmul_adapters(x, c.bank, index, b)[index == 1].isnan().all()
        c.bank.load(1, c.A[1], c.B[1], c.c[1])
        c.check(c.W.matmul_adapters(x, c.bank, index, b), x, b, index, f"M={M}")
        c.bank.load(0, c.A[0], torch.full_like(c.B[0], math.inf), c.c[0])
        c.bank.clear(0)
        c.check(c.W.matmul_adapters(x, c.bank, torch.where(index == 0, -1, index), b), x, b, torch.where(index == 0, -1, index), "cleared")
        zero = c.W.matmul_adapters(x, c.bank, index, b)
        c.check(zero, x, b, torch.where(index == 0, -1, index), "empty")


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("rank", [72, 150, 200])
def test_ranks_of_several_stretches(fmt, rank):
    """Ranks past the 64 values that are in LDS at a time, over several parts
    whose borders lie inside a wave's columns."""
    c = Case(512, [72, 64, 120], 128, fmt, slots=3, rank=rank)
    for M in (5, 33, 70, 600):
        c.run(M)


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("K,G", [(4096, 128), (4128, 32), (288, 32)])
def test_shared_k(fmt, K, G):
    """Few tiles, whose K several workgroups share; K that ends inside a stage."""
    c = Case(K, [264], G, fmt, slots=6, rank=40)
    for M in (33, 77, 200):
        c.run(M)
        c.run(M, index=torch.full((M,), 4))


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
def test_more_rows_than_stay_in_registers(fmt):
    c = Case(256, [136], 128, fmt, slots=37, rank=20)
    for M in (2049, 5003):
        c.run(M)
        c.run(M, index=torch.sort(torch.randint(-1, 37, (M,), generator=torch.Generator().manual_seed(M))).values)
        c.run(M, index=torch.arange(M) % 40 - 1)


def test_largest_bank():
    c = Case(128, [64], 128, slots=4096, rank=1)
    for M in (100, 5000):
        c.run(M)


def test_graph_and_repeats():
    c = Case(512, [256, 64], 128, "bf16", rank=16)
    for M in (4, 200):
        x, b, index = c.inputs(M)
        first = c.W.matmul_adapters(x, c.bank, index, b)        # (the workspace's first size)
        for _ in range(3):
            assert torch.equal(first, c.W.matmul_adapters(x, c.bank, index, b))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = c.W.matmul_adapters(x, c.bank, index, b)
        for i in range(3):
            x.normal_()
            index.copy_(torch.randint(-1, 5, (M,), generator=torch.Generator().manual_seed(i)))
            graph.replay()
            torch.cuda.synchronize()
            c.check(y, x, b, index, f"replay {i}")


def test_growth_under_capture_is_refused():
    c = Case(256, [64], 64, rank=8)
    x, b, index = c.inputs(40)
    c.W.matmul_adapters(x, c.bank, index, b)
    x, b, index = c.inputs(400)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z = x * 1
        with pytest.raises(ValueError, match="must grow"):
            c.W.matmul_adapters(x, c.bank, index, b)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(z, x)


def test_other_stream():
    c = Case(512, [256], 128, rank=16)
    for M in (3, 100):
        x, b, index = c.inputs(M)
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        y = c.W.matmul_adapters(x, c.bank, index, b, stream=s)
        s.synchronize()
        c.check(y, x, b, index)


def test_refusals():
    import gptq_bit_weight_amd as q4
    c = Case(256, [64, 72], 64, rank=8)
    d = Case(256, [136], 64, rank=8)
    x, b, index = c.inputs(4)
    W, bank = c.W, c.bank
    A, B = c.A[0], c.B[0]
    bad = [
        lambda: W.matmul_adapters(x.bfloat16(), bank, index), lambda: W.matmul_adapters(x, d.bank, index),
        lambda: W.matmul_adapters(x, bank, index.long()), lambda: W.matmul_adapters(x, bank, index[:3]),
        lambda: W.matmul_adapters(x, bank, index.cpu()), lambda: W.matmul_adapters(x[:, :128], bank, index),
        lambda: W.matmul_adapters(x, bank, index, b[:7]), lambda: W.matmul_adapters(x, bank, index, out=x),
        lambda: bank.load(5, A, B), lambda: bank.load(-1, A, B), lambda: bank.load(0, A[:1], B), lambda: bank.load(0, A, B[:9]),
        lambda: bank.load(0, A.bfloat16(), B.bfloat16()), lambda: bank.load(0, A, B[:, :4]), lambda: bank.load(0, A.cpu(), B),
        lambda: bank.clear(99), lambda: q4.Q4Adapters(W, 0, 8), lambda: q4.Q4Adapters(W, 3, 0),
        lambda: q4.Q4Adapters(W, 3, 8, torch.float32), lambda: bank.load(0, A.repeat(1, 2, 1), B.repeat(1, 2)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"case {i} was taken")
    with pytest.raises(NotImplementedError):
        q4.Q4Adapters(W, 5000, 8)
    assert W.matmul_adapters(x[:0], bank, index[:0]).shape == (0, 136)
    bank.close()
    with pytest.raises(ValueError, match="closed"):
        W.matmul_adapters(x, bank, index)


def test_growth_row_by_row_keeps_little_memory():
    """A bank's workspace grows by doubling: calls of one row more each time do not
    allocate each time, and what is outgrown is no more than what is held."""
    c = Case(128, [64], 128, slots=3, rank=16)
    x, b, index = c.inputs(700)
    c.W.matmul(x, b)
    c.W.matmul_adapters(x[:2], c.bank, index[:2], b)
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    least = free
    for M in range(33, 700):
        y = c.W.matmul_adapters(x[:M], c.bank, index[:M], b)
        if M % 97 == 0:
            c.check(y, x[:M], b, index[:M], f"M={M}")
        least = min(least, torch.cuda.mem_get_info()[0])
    torch.cuda.synchronize()
    # 2 MiB of sums, 1024 rows of 80 bytes and as much outgrown, each allocation up to 2 MiB; and the checks' own
    assert free - least < 100 << 20, (free - least) / 2 ** 20


def test_two_threads_on_one_bank_and_stream():
    """A call's launches hand c A x over in the bank: another thread's on the same
    stream do not come between them."""
    import threading
    c = Case(512, [264, 64], 64, "bf16", slots=6, rank=16)
    work, errors = [], []
    for M in (5, 70, 31, 300):
        x, b, index = c.inputs(M)
        y = c.W.matmul_adapters(x, c.bank, index, b)
        c.check(y, x, b, index, f"M={M}")
        work.append((x, b, index, y, []))
    torch.cuda.synchronize()

    def run(x, b, index, y, outs):
        try:
            for _ in range(200):
                outs.append(c.W.matmul_adapters(x, c.bank, index, b))
        except Exception as e:      # reported below
            errors.append(repr(e))

    threads = [threading.Thread(target=run, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for x, _, _, y, outs in work:
        assert len(outs) == 200
        for i, o in enumerate(outs):
            assert torch.equal(o, y), (x.shape[0], i)


def test_out_that_meets_an_input_is_refused():
    c = Case(128, [128], 128, rank=8)
    for M in (4, 40):
        x, b, index = c.inputs(M)
        own = torch.zeros(3 * M * 128, dtype=c.dt, device="cuda")
        out, ints = own[:M * 128].view(M, 128), own[M * 128 - 2 * M:M * 128].view(torch.int32)
        ints.copy_(index)
        for args, kw in (((x, c.bank, index, b), dict(out=x)), ((x, c.bank, ints, b), dict(out=out)),
                         ((x, c.bank, index, own[64:192]), dict(out=out))):
            with pytest.raises(ValueError, match="overlaps"):
                c.W.matmul_adapters(*args, **kw)
        y = c.W.matmul_adapters(x, c.bank, index, own[M * 128:M * 128 + 128], out=out)
        c.check(y, x, own[M * 128:M * 128 + 128], index)


def test_activations_off_sixteen_bytes_are_refused():
    c = Case(128, [128], 128, rank=8)
    for M in (4, 40):
        x, b, index = c.inputs(M)
        odd = torch.zeros(x.numel() + 1, dtype=c.dt, device="cuda")[1:].view(x.shape)
        odd.copy_(x)
        with pytest.raises(ValueError, match="16-byte aligned"):
            c.W.matmul_adapters(odd, c.bank, index, b)


def test_out_is_told_to_autograd():
    c = Case(128, [128], 128, rank=8)
    x, b, index = c.inputs(4)
    out = torch.zeros(4, 128, dtype=c.dt, device="cuda")
    y = (torch.ones_like(out, requires_grad=True) * out).sum()      # saves out
    c.W.matmul_adapters(x, c.bank, index, b, out=out)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    c.check(out, x, b, index)
    with pytest.raises(ValueError, match="requires a gradient"):
        c.W.matmul_adapters(x, c.bank, index, b, out=out.clone().requires_grad_())
    with torch.no_grad():
        c.check(c.W.matmul_adapters(x, c.bank, index, b, out=out.clone().requires_grad_()), x, b, index)


def test_a_bank_of_other_parts_is_refused_by_the_c_call():
    """The same K, N and number of parts, other widths: another matrix, for callers
    of the C call too (the binding compares them itself)."""
    import gptq_bit_weight_amd as q4
    c, d = Case(128, [64, 128], 128, rank=8), Case(128, [128, 64], 128, rank=8)
    lib = q4.load_library()
    for M in (4, 40):
        x, b, index = c.inputs(M)
        out = torch.zeros(M, 192, dtype=c.dt, device="cuda")
        args = (x.data_ptr(), b.data_ptr(), index.data_ptr(), out.data_ptr(), M, 0, torch.cuda.current_stream().cuda_stream)
        assert lib.q4_matmul_adapters(c.W._handle(), d.bank._handle(), *args) == 1
        assert b"another matrix" in lib.q4_last_error()
        assert lib.q4_matmul_adapters(c.W._handle(), c.bank._handle(), *args) == 0
        c.check(out, x, b, index)


def scaled_reference(c, x, b, index):
    """(result, tolerance) where c A x may lie far from 1: as in Case.check, but for a part's
    c A x off by 2^-16 of its row's largest in place of 2^-16 of itself."""
    xd = x.double()
    ref = xd @ c.w + b.double()
    tol = (BF16_GEMM_REL_A if c.fmt == "bf16" and x.shape[0] > 32 else REL_A) * (xd.abs() @ c.w.abs())
    for s in range(c.slots):
        rows, at = (index == s).nonzero()[:, 0], 0
        for p, n in enumerate(c.parts):
            a, bb = c.A[s][p].double(), c.B[s][at:at + n].double()
            t, ta = xd[rows] @ a.t() * c.c[s], xd[rows].abs() @ a.abs().t() * abs(c.c[s])
            off = c.K * 2.0 ** -24 * ta + 2.0 ** -16 * t.abs().amax(1, keepdim=True)
            ref[rows, at:at + n] += t @ bb.t()
            tol[rows, at:at + n] += off @ bb.abs().t()
            at += n
    return ref, tol + (BF16_REL_Y if c.fmt == "bf16" else REL_Y) * ref.abs()


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("parts,rank", [([264], 16), ([72, 64, 120], 8), ([72, 64, 120], 40), ([200, 64], 150)])
@pytest.mark.parametrize("size", [1e-9, 1e-5, 1e-3, 1.0, 3e4, 1e6, 1e9])
def test_sizes_of_the_adapters_product(fmt, parts, rank, size):
    """c A x from far below to far above the reach of binary16 and B the other way,
    alone (the matrix is zero): the same at 32 rows and more. Slot 0 has c A x of 1; of
    slot 1's parts, the last has 2^20 times less than the others."""
    import gptq_bit_weight_amd as q4
    announce(f"adapters' product {fmt} {parts} rank={rank} of {size}")
    c = Case(256, parts, 64, fmt, slots=3, rank=rank)
    words = lambda *shape: torch.full(shape, -0x77777778, dtype=torch.int32, device="cuda")  # noqa: E731  (codes and zeros of 8)
    c.W = q4.Q4Matrix.concat([(words(32, n), words(4, n // 8), torch.ones(4, n, dtype=torch.float16, device="cuda"))
                              for n in parts], groupsize=64)
    c.w = torch.zeros_like(c.w)
    for s in range(c.slots):
        c.c[s] = 1.0 if s == 0 else float(torch.tensor(size))
        if s == 1:
            c.A[s][-1] *= 2.0 ** -20
        c.B[s] = (c.B[s].sign() * min(max(1.0 / c.c[s], 2.0 ** -13), 2.0 ** 12)).to(c.dt)
        c.bank.load(s, c.A[s], c.B[s], c.c[s])
    for M in (32, 33, 77, 300, 600):
        x, b, index = c.inputs(M)
        if size > 1e6:
            x = x * 2.0 ** -9
        b = b * 0
        y = c.W.matmul_adapters(x, c.bank, index, b)
        ref, tol = scaled_reference(c, x, b, index)
        if fmt == "f16":
            assert (ref.abs() < 6e4).all()
            tol = tol + 2.0 ** -25                          # (half a step of the result's subnormals)
        bad = ~((y.double() - ref).abs() <= tol)
        assert not bad.any(), (M, int(bad.sum()), bad.nonzero()[0].tolist(), ((y.double() - ref).abs() / tol)[bad].max().item())
