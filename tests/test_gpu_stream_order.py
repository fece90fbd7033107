"""Kernel-level entries right after a kernel that writes their operands, on one stream.

Launches overlap (a kernel may start while its predecessor still runs), so an
entry that fetched an operand before waiting would take rows from before the
writer.  The writers here are large and the readers' operands are the last
rows that they write; the buffers hold other values before every round.  Each
reader's result has to equal, to the bit, the result of the same call after
the device was waited for.
"""
import pytest
import torch

import hierarchical_autoregressive_lm_b200 as hal

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
ROUNDS = 12


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, dtype, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(DT[dtype])


class Writers:
    """Three ways to fill k, v [G, H, cap, dim] (views of the writers' outputs) from new rows in one launch."""

    def __init__(self, g, dtype, G, H, cap, dim):
        self.g, self.dtype, self.n, self.H, self.dim = g, dtype, G * cap, H, dim
        self.k, self.v = (torch.empty(G, H, cap, dim, device="cuda", dtype=DT[dtype]) for _ in range(2))
        # rows [tokens, heads, dim] of one group's buffer; groups are sequences with one page each
        self.pages = hal.KVPages(self.k, self.v)
        self.source = hal.KVPages(torch.empty_like(self.k), torch.empty_like(self.v))
        self.table = torch.arange(G, device="cuda", dtype=torch.int32).view(G, 1)
        self.seq = torch.arange(G, device="cuda", dtype=torch.int32).repeat_interleave(cap)
        self.pos = torch.arange(cap, device="cuda", dtype=torch.int32).repeat(G)
        self.rope = hal.Rope(dim)
        self.rows = [torch.empty(G * cap, H, dim, device="cuda", dtype=DT[dtype]) for _ in range(2)]

    def renew(self):
        for t in (*self.rows, self.source.k, self.source.v, self.k, self.v):
            t.copy_(randn(self.g, self.dtype, *t.shape))

    def write(self):
        hal.kv_write(self.pages, self.table, self.pos, *self.rows, seq=self.seq, rope=self.rope)

    def read(self):
        # one group: its buffer as rows of any strides
        hal.kv_read(self.source, self.table, self.pos, self.k[0].transpose(0, 1), self.v[0].transpose(0, 1), seq=self.seq)

    def rotate(self):
        k, v = self.k[0].transpose(0, 1), self.v[0].transpose(0, 1)
        hal.rope(self.rope, self.pos, k, k, v, v)


def check(w, writer, reader, out):
    for _ in range(ROUNDS):
        w.renew()
        before = [t.clone() for t in (w.k, w.v)]
        torch.cuda.synchronize()
        out.fill_(7)
        torch.cuda.synchronize()
        writer()
        reader()
        torch.cuda.synchronize()
        got = out.clone()
        assert not torch.equal(before[0], w.k) and not torch.equal(before[1], w.v)
        reader()  # the operands are in place now
        torch.cuda.synchronize()
        assert torch.equal(got, out)


@pytest.mark.parametrize("entry", ["attn_decode", "attn_decode_noalloc"])
@pytest.mark.parametrize("writer", ["write", "read", "rotate"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("q_len,p0", [(1, None), (1, 300), (2, None)])
def test_decode_attention_after_a_writer(entry, writer, dtype, q_len, p0):
    g = gen(3)
    H, cap, dim = 16, 8192, 64
    w = Writers(g, dtype, 1, H, cap, dim)
    p0 = cap - q_len if p0 is None else p0
    q, out = (torch.empty(q_len, H * dim, device="cuda", dtype=DT[dtype]) for _ in range(2))
    q.copy_(randn(g, dtype, q_len, H * dim))
    if entry == "attn_decode_noalloc" and hal.attn_decode_scratch_bytes(int(dtype == "bf16"), 1, H, dim, cap, q_len, p0) > 256 << 10:
        cap = 1024
        w = Writers(g, dtype, 1, H, cap, dim)
        p0 = min(p0, cap - q_len)
    call = getattr(hal, entry)
    check(w, getattr(w, writer), lambda: call(q, w.k, w.v, q_len, p0, out), out)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_decode_attention_of_groups_after_the_cache_write(dtype):
    # a page a sequence, each a group of the decode attention
    g = gen(5)
    G, H, cap, dim = 64, 8, 512, 64
    w = Writers(g, dtype, G, H, cap, dim)
    q, out = randn(g, dtype, G, H * dim), torch.empty(G, H * dim, device="cuda", dtype=DT[dtype])
    check(w, w.write, lambda: hal.attn_decode(q, w.k, w.v, 1, cap - 1, out), out)


@pytest.mark.parametrize("writer", ["write", "read", "rotate"])
@pytest.mark.parametrize("M,rows,path,splits,swap", [(1, 8192, 0, 0, -1), (64, 4096, 0, 0, -1), (64, 8192, 2, 0, 1), (64, 8192, 2, 4, 1),
                                                     (128, 1024, 2, 2, 0), (512, 8192, 0, 0, -1), (16, 1024, 1, 0, -1)])
def test_gemm_after_a_writer(writer, M, rows, path, splits, swap):
    # scores of queries against keys that were written, read back or rotated just before: W is the last head's rows
    g = gen(7)
    H, dim = 8, 128
    w = Writers(g, "bf16", 1, H, rows, dim)
    A, out = randn(g, "bf16", M, dim), torch.empty(M, rows, device="cuda")
    check(w, getattr(w, writer), lambda: hal.gemm(A, w.k[0, H - 1], out, path=path, splits=splits, swap=swap), out)


@pytest.mark.parametrize("writer", ["write", "read", "rotate"])
@pytest.mark.parametrize("M", [1, 64, 300])
def test_gemm_rmsnorm_after_a_writer(writer, M):
    g = gen(11)
    H, rows, dim = 8, 4096, 256
    w = Writers(g, "bf16", 1, H, rows, dim)
    x, gain, out = randn(g, "fp32", M, dim), randn(g, "fp32", dim), torch.empty(M, rows, device="cuda")
    check(w, getattr(w, writer), lambda: hal.gemm_rmsnorm(x, gain, w.k[0, H - 1], out), out)


@pytest.mark.parametrize("writer", ["write", "read", "rotate"])
def test_decode_attention_after_a_writer_and_a_product(writer):
    # a kernel between the two that reads nothing of the first may start, and let the third start, before the first ends
    g = gen(17)
    H, cap, dim = 16, 8192, 64
    w = Writers(g, "bf16", 1, H, cap, dim)
    q, out = randn(g, "bf16", 1, H * dim), torch.empty(1, H * dim, device="cuda", dtype=torch.bfloat16)
    A, W, C = randn(g, "bf16", 16, 256), randn(g, "bf16", 128, 256), torch.empty(16, 128, device="cuda")

    def write():
        getattr(w, writer)()
        hal.gemm(A, W, C)

    check(w, write, lambda: hal.attn_decode(q, w.k, w.v, 1, cap - 1, out), out)


@pytest.mark.parametrize("writer", ["write", "read", "rotate"])
@pytest.mark.parametrize("entry", ["attn_decode", "gemm"])
def test_captured_pairs(writer, entry):
    g = gen(19)
    H, cap, dim = 16, 8192, 64
    w = Writers(g, "bf16", 1, H, cap, dim)
    if entry == "gemm":
        A, out = randn(g, "bf16", 64, dim), torch.empty(64, cap, device="cuda")
        reader = lambda: hal.gemm(A, w.k[0, H - 1], out)  # noqa: E731
    else:
        q, out = randn(g, "bf16", 1, H * dim), torch.empty(1, H * dim, device="cuda", dtype=torch.bfloat16)
        reader = lambda: hal.attn_decode(q, w.k, w.v, 1, cap - 1, out)  # noqa: E731
    w.renew()
    getattr(w, writer)(), reader()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        getattr(w, writer)()
        reader()
    for _ in range(ROUNDS):
        w.renew()
        out.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        reader()
        torch.cuda.synchronize()
        assert torch.equal(got, out)
    del graph


def test_decode_attention_after_a_product():
    # fp32 keys and values that are the library's own products
    g = gen(13)
    H, cap, dim = 4, 2048, 64
    k, v = (torch.empty(1, H, cap, dim, device="cuda") for _ in range(2))
    q, out = randn(g, "fp32", 1, H * dim), torch.empty(1, H * dim, device="cuda")
    for _ in range(ROUNDS):
        x, wk, wv = randn(g, "fp32", H * cap, 256), randn(g, "fp32", dim, 256), randn(g, "fp32", dim, 256)
        k.copy_(randn(g, "fp32", *k.shape)), v.copy_(randn(g, "fp32", *v.shape))
        torch.cuda.synchronize()
        hal.gemm(x, wv, v.view(-1, dim))
        hal.gemm(x, wk, k.view(-1, dim))
        hal.attn_decode(q, k, v, 1, cap - 1, out)
        torch.cuda.synchronize()
        got = out.clone()
        hal.attn_decode(q, k, v, 1, cap - 1, out)
        torch.cuda.synchronize()
        assert torch.equal(got, out)
