"""The operators around a caller's paged cache against plain 64-bit forms.

Tolerances count roundings.  u = 2^-24 is half a step of fp32, relative to the
value; a result stored as bf16 is off by another 2^-8 of itself.

* Rotation: sincospif's argument is off by 2^-25 half-turns (its rounding to
  fp32) and 2^-32 turns (the dropped bits), so the angle by 1.6 u + 0.03 u; sine
  and cosine are within 2 u, their scale, the product and the sum add 3 u: below
  8 u (|a| + |b|) * scale for a pair (a, b).
* Attention: a score of D products is off by (D + 8) u sum|q k| |scale|, which is
  the relative error of its weight (with exp's own 4 u and the weight's rounding,
  2^-16); a sum over n positions adds at most (n + 64) u.  A weight below 2^-126
  of the largest may vanish: exp's result is then below fp32's normal range, and
  the sum that it is divided by is at least one, so an output loses at most
  2^-126 sum|v|.
* Over 8-bit pages the weight of a position times its scale of V, c_t = w_t s_t, is
  the sum of two fp16 numbers, c_t 2^15 / C = a + b with C a power of two at most
  twice max(c).  fp16's smallest step is 2^-24, so b is off by 2^-25 at most where it
  is too small for its 11 bits, and c_t by 2^-40 C: an output by 2^-39 max(c)
  sum|code|.
"""
import ctypes
import math
import os
import subprocess
import sys
import threading
from decimal import Decimal, localcontext

import pytest
import torch

import hierarchical_autoregressive_lm_b200 as hal

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
HALF = {"fp32": U, "bf16": 2.0 ** -8}
TOP = {"e4m3": 448.0, "int8": 127.0}
KINDS = [("fp32", "fp32"), ("fp32", "e4m3"), ("fp32", "int8"), ("bf16", "bf16"), ("bf16", "e4m3"), ("bf16", "int8")]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def off(got, want, bound):
    """Largest |got - want| over its bound (equal values, infinities and NaN among them, are off by nothing)."""
    got, want = got.double(), want.double()
    same = (got == want) | (got.isnan() & want.isnan())
    ratio = torch.where(same, 0.0, (got - want).abs() / bound)
    return torch.where(ratio.isnan(), math.inf, ratio).max().item() if ratio.numel() else 0.0


def turned(x, pos, r, back=False):
    """64-bit rotation of x [tokens, heads, dim] and the bound of its fp32 error."""
    # turns modulo one in whole numbers: angles are right at any position
    frac = torch.tensor([[(p * f) % (1 << 64) / 2.0 ** 64 for f in r.turns] for p in pos.tolist()], dtype=torch.float64, device="cuda")
    ang = 2 * math.pi * frac[:, None, :]
    c, s = ang.cos() * r.scale, ang.sin() * r.scale * (-1 if back else 1)
    x = x.double()
    y, rot, bound = x.clone(), r.rot_dim, torch.zeros_like(x)
    i0 = slice(0, rot, 2) if r.interleaved else slice(0, rot // 2)
    i1 = slice(1, rot, 2) if r.interleaved else slice(rot // 2, rot)
    a, b = x[..., i0], x[..., i1]
    y[..., i0], y[..., i1] = a * c - b * s, a * s + b * c
    bound[..., i0] = bound[..., i1] = 8 * U * (a.abs() + b.abs()) * r.scale
    return y, bound


# ------------------------------------------------------------------ rotation

@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("n,h,h2,dim,rot,kw", [
    (1, 1, 0, 64, 64, {}), (1, 32, 8, 128, 128, {}), (37, 3, 1, 64, 64, dict(scaling="ntk", factor=4.0)),
    (5, 2, 2, 128, 64, dict(scaling="yarn", factor=32.0, original_len=4096)), (3, 5, 0, 48, 20, dict(scaling="linear", factor=2.5)),
    (2, 1, 1, 2, 2, {}), (9, 2, 1, 512, 512, {}), (257, 7, 3, 96, 96, {}), (2, 1, 0, 80, 6, dict(attn_scale=0.5)),
    (1500, 40, 8, 64, 32, {}), (1, 600, 0, 64, 64, {})])
def test_rope(dtype, inter, n, h, h2, dim, rot, kw):
    g = gen(n * 1000 + dim)
    r = hal.Rope(rot, interleaved=inter, **kw)
    pos = torch.randint(-50, 1 << 20, (n,), generator=g, device="cuda").int()
    pos[0] = 2 ** 31 - 1
    x, x2 = randn(g, n, h, dim).to(DT[dtype]), randn(g, n, h2, dim).to(DT[dtype]) if h2 else None
    for back in (False, True):
        y, y2 = torch.full_like(x, 7), torch.full_like(x2, 7) if h2 else None
        hal.rope(r, pos, x, y, x2, y2, backward=back)
        for i, o in ((x, y), (x2, y2))[: 1 + bool(h2)]:
            want, bound = turned(i, pos, r, back)
            assert off(o, want, bound + HALF[dtype] * want.abs()) <= 1
            assert torch.equal(o[..., rot:], i[..., rot:])
            z = i.clone()
            hal.rope(r, pos, z, z, backward=back)  # in place, one tensor
            assert torch.equal(z, o)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shift", [0, 1, 8])
def test_rope_strided(dtype, shift):
    # q and k as columns of one projection's rows, at any alignment
    g = gen(3)
    n, h, h2, dim = 33, 4, 2, 64
    r = hal.Rope(64)
    pos = torch.arange(n, device="cuda", dtype=torch.int32)
    row = randn(g, n, (h + 2 * h2) * dim + 24).to(DT[dtype])
    q = row[:, shift:shift + h * dim].view(n, h, dim)
    k = row[:, shift + h * dim:shift + (h + h2) * dim].view(n, h2, dim)
    out = torch.zeros(h, n, dim, device="cuda", dtype=DT[dtype]).transpose(0, 1)
    before = row.clone()
    hal.rope(r, pos, q, out, k, k)
    want, bound = turned(q, pos, r)
    assert off(out, want, bound + HALF[dtype] * want.abs()) <= 1
    want, bound = turned(before[:, shift + h * dim:shift + (h + h2) * dim].view(n, h2, dim), pos, r)
    assert off(k, want, bound + HALF[dtype] * want.abs()) <= 1
    k.zero_(), before[:, shift + h * dim:shift + (h + h2) * dim].zero_()
    assert torch.equal(row, before)  # nothing else of the rows was written
    one = q[:1, :1].expand(n, h, dim)  # a broadcast input
    hal.rope(r, pos, one, out)
    want, bound = turned(one, pos, r)
    assert off(out, want, bound + HALF[dtype] * want.abs()) <= 1


@pytest.mark.parametrize("rot,theta", [(64, 10000.0), (128, 500000.0)])
def test_rope_at_the_last_positions(rot, theta):
    """Angles from the formula in 60 digits, not from the library's fractions.

    These may be off by 2^-29 turns, 0.2 u radians, at position 2^31: within the 8 u of a pair, of which the other errors
    take 6.63.
    """
    with localcontext() as ctx:
        ctx.prec = 60
        two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494")
        turns = [Decimal(theta) ** (Decimal(-2 * i) / rot) / two_pi for i in range(rot // 2)]
        at = [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 30, 2 ** 30 + 12345, 1999999999, -2 ** 31, 1 << 20, 1]
        ang = torch.tensor([[float(p * f % 1) for f in turns] for p in at], dtype=torch.float64, device="cuda")[:, None, :] * (2 * math.pi)
    x = randn(gen(83), len(at), 64, rot)
    out = torch.empty_like(x)
    hal.rope(hal.Rope(rot, theta=theta), ints(at), x, out)
    a, b = x.double().chunk(2, -1)
    want = torch.cat([a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()], -1)
    bound = 8 * U * (a.abs() + b.abs()).repeat(1, 1, 2)
    assert off(out, want, bound + U * want.abs()) <= 1


@pytest.mark.parametrize("inter", [False, True])
def test_rope_gradient_against_differences(inter):
    # y is linear in x, so L(x + e d) - L(x - e d) over 2e is the derivative itself
    g = gen(5)
    r = hal.Rope(32, interleaved=inter, scaling="yarn", factor=8.0, original_len=256)
    n, h, dim = 6, 2, 48
    pos = torch.arange(n, device="cuda", dtype=torch.int32) * 1001
    x, w, d = randn(g, n, h, dim), randn(g, n, h, dim), randn(g, n, h, dim)
    out, grad = torch.empty_like(x), torch.empty_like(x)
    hal.rope(r, pos, w, grad, backward=True)
    loss = []
    for e in (0.5, -0.5):
        hal.rope(r, pos, x + e * d, out)
        loss.append((out.double() * w.double()).sum())
    # every output is off by 8 u (|a| + |b|) scale, times its weight, and x +- e d by u: n h dim terms below 4^2 each
    bound = 16 * U * r.scale * n * h * dim * 16
    assert abs((loss[0] - loss[1]) - (grad.double() * d.double()).sum()).item() <= bound


# ------------------------------------------------------------ write and read

def pool(pages, heads, rows, dim, kind, order="phrd", fill=None):
    """A pool in either order of heads and rows."""
    def make(*shape, dtype):
        x = torch.zeros(*shape, device="cuda", dtype=dtype)
        return x if fill is None else (x.view(torch.int8) if dtype.itemsize == 1 else x).fill_(fill).view(dtype)

    out = []
    for d, t in (((dim,), DT[kind]), ((), torch.float32)):
        for _ in range(2):
            if order == "phrd":
                out.append(make(pages, heads, rows, *d, dtype=t))
            else:
                out.append(make(pages, rows, heads, *d, dtype=t).transpose(1, 2))
    return hal.KVPages(*out[:2], *(out[2:] if kind in TOP else ()))


def bytes_of(t):
    return t.contiguous().view(torch.uint8)


def same(a, b):
    """Equal codes, or equal values (any NaN equals any other)."""
    if a.itemsize == 1:
        return torch.equal(bytes_of(a), bytes_of(b))
    return torch.equal(torch.where(a.isnan(), 123.0, a), torch.where(b.isnan(), 123.0, b))


def quantised(x, kind):
    """The documented codes and scales of fp32 rows, each operation rounded once."""
    amax = x.abs().amax(-1)
    fine = amax.isfinite()
    held = torch.where(fine, amax, 1.0).clamp(min=1e-30)
    top = torch.full_like(held, TOP[kind])
    y = torch.where(fine[..., None], x * (top / held)[..., None], 0.0)
    code = y.to(DT["e4m3"]) if kind == "e4m3" else y.round().to(torch.int8)
    return code, torch.where(fine, held / top, math.nan)


def places(g, seqs, n, width, rows):
    """n distinct (seq, pos) in any order."""
    at = torch.randperm(seqs * width * rows, generator=g, device="cuda")[:n]
    return (at // (width * rows)).int(), (at % (width * rows)).int()


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("n,heads,rows,dim,order", [
    (1, 1, 1, 32, "phrd"), (29, 3, 5, 64, "prhd"), (200, 2, 16, 128, "phrd"), (17, 9, 7, 256, "prhd"), (2100, 8, 64, 128, "prhd")])
def test_write_and_read(dtype, kind, n, heads, rows, dim, order):
    g = gen(n + heads)
    seqs = min(n, 5)
    width = -(-n // (seqs * rows)) + 2
    p = pool(seqs * width + 4, heads, rows, dim, kind, order, fill=3)
    table = torch.randperm(p.pages, generator=g, device="cuda")[: seqs * width].int().view(seqs, width)
    seq, pos = places(g, seqs, n, width, rows)
    k, v = (randn(g, n, heads, dim).mul_(3).to(DT[dtype]) for _ in range(2))
    special = [0.0, 1e-38, 1e-35, 2e38, math.inf, -math.inf, math.nan]
    for i, x in enumerate(special[: max(0, n - 1)]):  # rows of one value, or with one in them
        k[i + 1, 0] = x
        v[i + 1, heads - 1, dim // 2] = x
    if n > 20:
        pos[10::7] = -1  # padding
    real = pos >= 0
    page, row = table[seq.long(), (pos.clamp(min=0) // rows).long()].long()[real], (pos % rows).long()[real]
    want_k, want_v, want_ks, want_vs = (None if t is None else t.clone() for t in (p.k, p.v, p.k_scale, p.v_scale))
    for t, s, x in ((want_k, want_ks, k), (want_v, want_vs, v)):
        if kind in TOP:
            code, scale = quantised(x.float(), kind)
            s[page, :, row] = scale[real]
        else:
            code = x
        t.view(torch.int8 if t.itemsize == 1 else t.dtype)[page, :, row] = code.view(torch.int8 if t.itemsize == 1 else t.dtype)[real]
    err = ints([0])
    hal.kv_write(p, table, pos, k, v, seq=seq, err=err)
    assert err.item() == 0
    for got, want in ((p.k, want_k), (p.v, want_v), (p.k_scale, want_ks), (p.v_scale, want_vs)):
        if got is not None:
            assert same(got, want)
    # and back, twice the same place among them, padding rows left as they were
    pos2, seq2 = torch.cat([pos, pos[:1]]), torch.cat([seq, seq[:1]])
    out = [torch.full((n + 1, heads, dim), 9, device="cuda", dtype=DT[dtype]) for _ in range(2)]
    hal.kv_read(p, table, pos2, *out, seq=seq2, err=err)
    assert err.item() == 0
    for o, t, s in ((out[0], want_k, want_ks), (out[1], want_v, want_vs)):
        x = t[page, :, row] if t.itemsize > 1 else t.view(torch.int8)[page, :, row].view(t.dtype)
        x = x.float() if s is None else x.float() * s[page, :, row][..., None]
        x = x.to(DT[dtype])
        assert same(o[:n][real], x) and same(o[n], o[0])
        assert (o[:n][~real] == 9).all()


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("dim,rot,inter", [(64, 64, False), (128, 64, True), (128, 96, False), (32, 20, False), (32, 6, True), (256, 256, False)])
def test_write_rotated(dtype, kind, dim, rot, inter):
    g = gen(dim + rot)
    n, heads, hq, rows = 41, 2, 6, 5
    r = hal.Rope(rot, interleaved=inter)
    for shift in (0, 3):  # rows at a 16-byte boundary, and not
        p = pool(20, heads, rows, dim, kind)
        table = torch.randperm(20, generator=g, device="cuda").int().view(2, 10)
        seq, pos = places(g, 2, n, 10, rows)
        pos[5] = -1
        real = pos >= 0
        width = (hq + 2 * heads) * dim
        row = randn(g, n, width + 8).to(DT[dtype])
        q, k, v = (x.view(n, -1, dim) for x in row[:, shift:shift + width].split([hq * dim, heads * dim, heads * dim], 1))
        q_in, k_in, v_in = q.clone(), k.clone(), v.clone()
        hal.kv_write(p, table, pos, k, v, seq=seq, rope=r, q=q, q_out=q)
        want, bound = turned(q_in, pos.clamp(min=0), r)
        assert off(q[real], want[real], (bound + HALF[dtype] * want.abs())[real]) <= 1
        assert torch.equal(q[~real], q_in[~real]) and torch.equal(k, k_in) and torch.equal(v, v_in)
        page, at = table[seq.long(), (pos.clamp(min=0) // rows).long()].long()[real], (pos % rows).long()[real]
        want, bound = turned(k_in, pos.clamp(min=0), r)
        want, bound = want[real], bound[real]
        got = (p.k.view(torch.int8)[page, :, at].view(p.k.dtype) if kind in TOP else p.k[page, :, at]).double()
        if kind in TOP:
            scale = p.k_scale[page, :, at].double()[..., None]
            got = got * scale
            # half a step of the code (e4m3: 2^-4 of the value, at least 2^-10; int8: a half), the scaled
            # value's own roundings (3 u), and the scale's share of the amax's error
            step = (want.abs() * 2.0 ** -4).clamp(min=2.0 ** -10 * scale) if kind == "e4m3" else 0.5 * scale
            bound = 1.1 * bound + step * (1 + 2.0 ** -12) + 4 * U * want.abs() + bound.amax(-1, keepdim=True)
            amax = want.abs().amax(-1, keepdim=True)
            assert off(scale * TOP[kind], amax, bound.amax(-1, keepdim=True)) <= 1
        else:
            bound = bound + HALF[dtype] * want.abs()
        assert off(got, want, bound) <= 1
        # the values are stored as without a rotation
        p2 = pool(20, heads, rows, dim, kind)
        hal.kv_write(p2, table, pos, k, v, seq=seq)
        assert torch.equal(bytes_of(p.v), bytes_of(p2.v))


def test_bad_places_are_left_out_and_reported():
    g = gen(1)
    p = pool(6, 2, 4, 32, "int8", fill=5)
    table = ints([[0, 1], [2, 77], [-1, 3]])
    k, v = randn(g, 6, 2, 32), randn(g, 6, 2, 32)
    before = p.k.clone()
    err = ints([0])
    #         no such sequence, beyond the table, page 77, page -1, sequence -1, beyond the table by far
    hal.kv_write(p, table, ints([0, 8, 5, 2, 0, 2 ** 31 - 1]), k, v, seq=ints([3, 0, 1, 2, -1, 0]), err=err)
    assert err.item() != 0 and torch.equal(p.k, before)
    err.zero_()
    out = torch.full_like(k, 4), torch.full_like(v, 4)
    hal.kv_read(p, table, ints([0, 8, 5, 2, 0, 2 ** 31 - 1]), *out, seq=ints([3, 0, 1, 2, -1, 0]), err=err)
    assert err.item() != 0 and (out[0] == 4).all() and (out[1] == 4).all()
    hal.kv_write(p, table, ints([0, 8, 2]), k[:3], v[:3])  # without an error word; token 0 is good
    assert not torch.equal(p.k[0], before[0]) and torch.equal(p.k[1:], before[1:])


# ------------------------------------------------------------------ attention

def attended(p, table, lens, q, window, scale):
    """64-bit outputs, log-sum-exps, and the bounds of their errors before the last rounding."""
    B, Hq, D = q.shape
    G = Hq // p.heads
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    bound, lse_bound = torch.zeros_like(out), torch.zeros_like(lse)
    for b, n in enumerate(lens):
        t = torch.arange(max(0, n - window) if window else 0, n, device="cuda")
        if n == 0:
            continue
        page, row = table[b].long()[t // p.page_rows], t % p.page_rows

        def rows(x, s):
            x = x.view(torch.int8)[page, :, row].view(x.dtype) if x.itemsize == 1 else x[page, :, row]
            return x.double() if s is None else x.double() * s[page, :, row].double()[..., None]

        K, V = (rows(x, s).repeat_interleave(G, 1) for x, s in ((p.k, p.k_scale), (p.v, p.v_scale)))
        a = torch.einsum("hd,nhd->hn", q[b].double(), K) * scale
        size = torch.einsum("hd,nhd->hn", q[b].double().abs(), K.abs()) * abs(scale)
        lse[b] = a.logsumexp(-1)
        w = (a - lse[b][:, None]).exp()
        out[b] = torch.einsum("hn,nhd->hd", w, V)
        ds = (D + 8) * U * size.amax(-1)[:, None]
        sums = (len(t) + 64) * U
        bound[b] = (2.0 ** -16 + 2 * (ds + 4 * U) + 2 * sums) * torch.einsum("hn,nhd->hd", w, V.abs()) + 2.0 ** -126 * V.abs().sum(0)
        if p.k_scale is not None:
            vs = p.v_scale[page, :, row].double().T.repeat_interleave(G, 0)
            codes = V.abs() / vs.T.clamp(min=1e-300)[..., None]
            bound[b] += 2.0 ** -39 * (w * vs).amax(-1)[:, None] * codes.sum(0)
        # log2 and its factor: 4 u of the larger of the maximum and the logarithm
        lse_bound[b] = ds[:, 0] + 4 * U + sums + 4 * U * (a.abs().amax(-1) + math.log(len(t)) + 1)
    return out, lse, bound, lse_bound


def filled(g, pages, heads, rows, dim, kind, order="phrd"):
    p = pool(pages, heads, rows, dim, kind, order)
    for t, s in ((p.k, p.k_scale), (p.v, p.v_scale)):
        x = randn(g, pages, heads, rows, dim) * (0.5 + torch.rand(dim, generator=g, device="cuda"))
        if kind in TOP:
            x *= 2 ** randn(g, pages, heads, rows, 1)
            code, scale = quantised(x, kind)
            t.view(torch.int8).copy_(code.view(torch.int8)), s.copy_(scale)
        else:
            t.copy_(x)
    return p


def paged(g, lens, rows, heads, dim, kind, order="phrd", width=None, spare=3):
    """A pool whose only read rows hold numbers: every other row holds NaN."""
    width = width or max(1, max(-(-n // rows) for n in lens))
    used = [-(-n // rows) for n in lens]
    p = filled(g, sum(used) + spare, heads, rows, dim, kind, order)
    ids = torch.randperm(p.pages, generator=g, device="cuda").int()
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    dead = torch.ones(p.pages, rows, dtype=torch.bool, device="cuda")
    i = 0
    for b, n in enumerate(lens):
        table[b, : used[b]] = ids[i:i + used[b]]
        i += used[b]
        t = torch.arange(n, device="cuda")
        dead[table[b].long()[t // rows], t % rows] = False
    page, row = dead.nonzero(as_tuple=True)
    for t, s in ((p.k, p.k_scale), (p.v, p.v_scale)):
        if kind in TOP:
            s[page, :, row] = math.nan
        else:
            t[page, :, row] = math.nan
    return p, table


def check_attention(p, table, lens, q, window=0, scale=None, dtype="bf16", out=None):
    out = torch.full_like(q, 7) if out is None else out
    lse, err = torch.full(q.shape[:2], 7.0, device="cuda"), ints([0])
    hal.attn_decode_paged(p, table, ints(lens), q, out, window=window, scale=scale, lse=lse, err=err)
    assert err.item() == 0
    want, want_lse, bound, lse_bound = attended(p, table, lens, q, window, p.head_dim ** -0.5 if scale is None else scale)
    assert off(lse, want_lse, lse_bound) <= 1
    assert off(out, want, bound + HALF[dtype] * want.abs() * (1 + 2.0 ** -8)) <= 1
    for b, n in enumerate(lens):
        if n == 0:
            assert (out[b] == 0).all() and (lse[b] == -math.inf).all()
    return out, lse


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("dim", [32, 64, 128, 256])
@pytest.mark.parametrize("lens,rows,heads,group", [
    ([1], 1, 1, 1), ([0, 17, 3], 5, 2, 3), ([257], 16, 4, 1), ([100, 0, 1, 640, 333], 7, 3, 4), ([129, 64], 64, 2, 8), ([65, 1000], 16, 1, 12)])
def test_attention(dtype, kind, dim, lens, rows, heads, group):
    g = gen(dim + len(lens))
    p, table = paged(g, lens, rows, heads, dim, kind)
    check_attention(p, table, lens, randn(g, len(lens), heads * group, dim).to(DT[dtype]), dtype=dtype)


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("lens,rows,heads,group,dim,window", [
    ([9000], 16, 2, 4, 128, 0), ([5000, 1, 0, 12345], 64, 1, 8, 64, 0), ([3000, 2999, 100, 333, 5], 32, 4, 2, 64, 333),
    ([20000], 128, 1, 1, 32, 0), ([4096] * 3, 16, 8, 4, 128, 1), ([700] * 70, 16, 2, 1, 64, 100), ([6007], 1, 2, 16, 128, 5000),
    ([40] * 600, 16, 1, 4, 64, 0), ([33] * 1300, 8, 4, 2, 32, 0)])
def test_attention_long(dtype, kind, lens, rows, heads, group, dim, window):
    g = gen(len(lens) + rows)
    p, table = paged(g, lens, rows, heads, dim, kind, order="prhd")
    check_attention(p, table, lens, randn(g, len(lens), heads * group, dim).to(DT[dtype]), window, dtype=dtype)


@pytest.mark.parametrize("dtype,kind", [("fp32", "fp32"), ("bf16", "bf16"), ("bf16", "int8"), ("bf16", "e4m3")])
def test_attention_strides_scale_and_size(dtype, kind):
    g = gen(7)
    lens, heads, group, dim = [70, 300, 12], 2, 3, 64
    p, table = paged(g, lens, 5, heads, dim, kind, width=80)
    wide = torch.full((3, 200), 99, dtype=torch.int32, device="cuda")
    wide[:, :80] = table
    row = randn(g, 3, heads * group * dim * 2 + 5).to(DT[dtype])
    q = row[:, 5:5 + heads * group * dim].view(3, heads * group, dim)  # rows at odd offsets
    out = torch.zeros(heads * group, 3, dim, device="cuda", dtype=DT[dtype]).transpose(0, 1)
    check_attention(p, wide[:, :80], lens, q, dtype=dtype, out=out)
    check_attention(p, table, lens, q, scale=-1.5, dtype=dtype)
    check_attention(p, table, lens, q, scale=0.0, dtype=dtype)
    check_attention(p, table, lens, q[:1, :1].expand(3, heads * group, dim), dtype=dtype)  # a broadcast query
    check_attention(p, table, lens, q * 1e-30, scale=1e28, dtype=dtype)  # far below fp16's range
    check_attention(p, table, lens, q * 64, dtype=dtype)  # one position takes it all


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_attention_unusual_values(dtype, kind):
    g = gen(11)
    lens, dim = [50, 50, 50, 1500, 50], 64
    p, table = paged(g, lens, 16, 1, dim, kind)
    q = randn(g, 5, 2, dim).to(DT[dtype])
    base, base_lse = check_attention(p, table, lens, q, dtype=dtype)
    poison = [(0, p.v, math.nan), (1, p.k, math.nan), (2, p.v, math.inf)]
    for b, t, x in poison:  # one row within the length
        if kind in TOP:
            (p.k_scale if t is p.k else p.v_scale)[table[b, 0].long(), 0, 3] = x
        else:
            t[table[b, 0].long(), 0, 3] = x
    q[4, 1, 0] = math.nan
    out, lse = torch.empty_like(q), torch.empty(5, 2, device="cuda")
    hal.attn_decode_paged(p, table, ints(lens), q, out, lse=lse)
    assert out[0].isnan().all() and torch.equal(lse[0], base_lse[0])
    assert out[1].isnan().all() and lse[1].isnan().all()
    assert not out[2].isfinite().any()
    assert torch.equal(out[3], base[3]) and torch.equal(lse[3], base_lse[3])  # another sequence's rows change nothing
    assert torch.equal(out[4, 0], base[4, 0]) and out[4, 1].isnan().all()


# NaNs by their bits: what GPU arithmetic makes, the same with a sign, others whose payload is all in the upper or in the lower bits
NANS = [0x7fffffff, 0xffffffff, 0x7ffff000, 0xfffff000, 0x7fc00000, 0x7f800001, 0xff801fff]


@pytest.mark.parametrize("dim", [32, 64, 128, 256])
@pytest.mark.parametrize("bits", NANS)
def test_attention_keeps_every_nan(dim, bits):
    g = gen(61)
    lens = [50, 50, 50, 1500, 1500]
    p, table = paged(g, lens, 16, 1, dim, "fp32")
    q = randn(g, 5, 3, dim)
    base, base_lse = check_attention(p, table, lens, q, dtype="fp32")

    def poison(t):
        t.view(torch.int32).fill_(bits - (1 << 32) if bits >> 31 else bits)

    poison(p.k[table[0, 1].item(), 0, 3, 5:6])
    poison(p.v[table[1, 1].item(), 0, 3, 5:6])
    poison(q[2, 1, 7:8])
    poison(p.k[table[3, 70].item(), 0, 2, 9:10])
    out, lse = torch.empty_like(q), torch.empty(5, 3, device="cuda")
    hal.attn_decode_paged(p, table, ints(lens), q, out, lse=lse)
    assert out[0].isnan().all() and lse[0].isnan().all() and out[3].isnan().all() and lse[3].isnan().all()
    assert out[1, :, 5].isnan().all() and torch.equal(lse[1], base_lse[1])
    assert torch.equal(out[1, :, :5], base[1, :, :5]) and torch.equal(out[1, :, 6:], base[1, :, 6:])
    assert out[2, 1].isnan().all() and lse[2, 1].isnan().all()
    for h in (0, 2):
        assert torch.equal(out[2, h], base[2, h]) and torch.equal(lse[2, h], base_lse[2, h])
    assert torch.equal(out[4], base[4]) and torch.equal(lse[4], base_lse[4])


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("x", [math.nan, math.inf, -math.inf])
def test_a_nan_of_the_rotation_reaches_the_attention(dtype, kind, x):
    # the rotation turns what is not finite into the NaN of GPU arithmetic
    g = gen(67)
    B, H, G, dim, rows, n = 3, 2, 3, 64, 8, 20
    p = pool(B * 4, H, rows, dim, kind)
    table = torch.arange(B * 4, device="cuda", dtype=torch.int32).view(B, 4)
    r = hal.Rope(dim)
    seq, pos = torch.arange(B, device="cuda").repeat_interleave(n).int(), torch.arange(n, device="cuda").repeat(B).int()
    q, k, v = (randn(g, B * n, h, dim).to(DT[dtype]) for h in (H * G, H, H))
    k[2 * n // 3, 0, 1] = k[2 * n // 3, 0, 1 + dim // 2] = x  # a pair of sequence 0, key head 0
    q[2 * n - 1, 1, 2] = q[2 * n - 1, 1, 2 + dim // 2] = x    # the last token of sequence 1, head 1
    out_q = torch.empty_like(q)
    hal.kv_write(p, table, pos, k, v, seq=seq, rope=r, q=q, q_out=out_q)
    last = out_q[n - 1::n]
    out, lse = torch.empty_like(last), torch.empty(B, H * G, device="cuda")
    hal.attn_decode_paged(p, table, ints([n] * B), last, out, lse=lse)
    bad = torch.zeros(B, H * G, dtype=torch.bool, device="cuda")
    bad[0, :G], bad[1, 1] = True, True
    assert out[bad].isnan().all() and lse[bad].isnan().all()
    assert out[~bad].isfinite().all() and lse[~bad].isfinite().all()


@pytest.mark.parametrize("dim", [32, 64, 128, 256])
def test_attention_largest_finite_numbers(dim):
    # next to fp32's largest number a rounding to fewer bits would leave the finite ones
    g = gen(71)
    lens = [1, 40, 1]
    p, table = paged(g, lens, 8, 1, dim, "fp32")
    top = torch.finfo(torch.float32).max
    q = randn(g, 3, 2, dim)
    p.v[table[0, 0].long(), 0, 0, ::2] = top
    p.v[table[0, 0].long(), 0, 0, 1::2] = -top * (1 - 2.0 ** -12)
    p.k[table[1, 2].long(), 0, 3] = -top
    q[1] = 0
    p.k[table[2, 0].long(), 0, 0] = torch.arange(dim, device="cuda") % 3 - 1.0
    q[2] = 0
    q[2, 0, 1], q[2, 1, 2] = 7, top / 4
    check_attention(p, table, lens, q, dtype="fp32", scale=2.0 ** -120)


@pytest.mark.parametrize("kind", ["fp32", "e4m3", "int8"])
@pytest.mark.parametrize("dim", [32, 64, 128, 256])
def test_attention_long_sums_have_no_direction(kind, dim):
    """Even weights over values of one sign, thousands of positions to a sum.

    Sums that cut off where they should round come out too small by half a step a
    position.  A tile's sum (64 positions, two terms each, at most 16 steps of the
    tensor cores) may lose 16 u; the tiles' sums are rounded to nearest, without a
    direction: the errors' mean stays below 16 u, while 4096 / (4 * 8) steps cut off
    would take it to 64 u.
    """
    g = gen(47)
    lens = [4096] * 64
    p, table = paged(g, lens, 64, 8, dim, kind)
    p.v.copy_((p.v.float().abs() + 1).clamp(max=TOP.get(kind, 9.0)).to(p.v.dtype))
    for s in (p.k_scale, p.v_scale):
        if s is not None:
            s.fill_(2.0 ** -7)
    q = randn(g, 64, 8, dim) * 0.01
    out, _ = check_attention(p, table, lens, q, dtype="fp32")
    want = attended(p, table, lens[:4], q[:4], 0, dim ** -0.5)[0]
    assert abs(((out[:4].double() - want) / want).mean().item()) <= 16 * U


@pytest.mark.parametrize("kind", ["fp32", "e4m3", "int8"])
@pytest.mark.parametrize("dim", [32, 64, 128, 256])
@pytest.mark.parametrize("group", [1, 4, 8])
def test_attention_fp32_weights_keep_22_bits(kind, dim, group):
    """Values that are all one: an output is the sum of the weights as the product takes them over the sum that divides it.

    Scores and exponentials cancel.  What is left, in u and for up to four positions: two parts of a weight 2, the tensor
    cores' four terms cut off 8, sums of the parts and of the weights 1 + 2, the quotient 1: below 16.  Weights of 17 bits
    would be up to 47 off, of 11 bits 3600.
    """
    g = gen(89)
    lens = [2, 3, 4, 1] * 64
    p, table = paged(g, lens, 4, 2, dim, kind)
    for b, n in enumerate(lens):
        page = table[b, 0].item()
        p.v.view(torch.int8 if kind in TOP else p.v.dtype)[page, :, :n] = torch.ones((), device="cuda").to(DT[kind]).view(
            torch.int8 if kind in TOP else p.v.dtype)
        if kind in TOP:
            p.v_scale[page, :, :n] = 1
    q, out = randn(g, len(lens), 2 * group, dim), torch.empty(len(lens), 2 * group, dim, device="cuda")
    hal.attn_decode_paged(p, table, ints(lens), q, out)
    assert (out.double() - 1).abs().max().item() <= 16 * U


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_attention_weights_far_apart(kind):
    # a position that takes nearly all the weight with small values, beside others with large ones
    g = gen(13)
    lens, dim = [2000], 64
    p, table = paged(g, lens, 16, 1, dim, kind)
    q = randn(g, 1, 4, dim).bfloat16()
    page = table[0, 0].long()
    key = q[0].float().sum(0) * 2
    if kind in TOP:
        code, scale = quantised(key, kind)
        p.k.view(torch.int8)[page, 0, 0] = code.view(torch.int8)
        p.k_scale[page, 0, 0] = scale
        p.v_scale[page, 0, 0] *= 2.0 ** -12
    else:
        p.k[page, 0, 0] = key.bfloat16()
        p.v[page, 0, 0] *= 2.0 ** -12
    check_attention(p, table, lens, q)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("group", [2, 8])
def test_attention_largest_values_in_narrow_pages(dtype, kind, group):
    # rows near the largest number of their type, as the cache write narrows them, and scales beyond those
    g = gen(73)
    lens, dim = [1, 30, 1], 64
    p, table = paged(g, lens, 16, 1, dim, kind)
    top = torch.finfo(DT[dtype]).max
    k, v = randn(g, 2, 1, dim).to(DT[dtype]), (randn(g, 2, 1, dim).sign() * top).to(DT[dtype])
    v[1, 0, ::3] = top / 3
    k[1] = 30.0
    hal.kv_write(p, table, ints([0, 7]), k, v, seq=ints([0, 1]))
    assert (p.v_scale[table[:2, 0].long(), 0, ints([0, 7]).long()] > 2.0 ** (121 if kind == "int8" else 119)).all()
    code = torch.arange(dim, device="cuda") % 3 - 1.0
    p.v.view(torch.int8)[table[2, 0].item(), 0, 0] = code.to(DT[kind]).view(torch.int8)
    p.v_scale[table[2, 0].item(), 0, 0] = 1.9 * 2.0 ** 126
    q = randn(g, 3, group, dim).to(DT[dtype])
    q[1] = 1.0  # position 7 takes all the weight: its score is 30 * dim / 8, others' below 60
    out = torch.empty_like(q)
    hal.attn_decode_paged(p, table, ints(lens), q, out)
    want, _, bound, _ = attended(p, table, lens, q, 0, dim ** -0.5)
    # A result within the bound of `want` may lie beyond the type's largest number, which rounds to infinity: of int8 rows
    # with fp32's largest number the stored value does so itself, 127 * rn(top / 127) = top (1 + 5.6e-8), and half a step
    # of top is 3.0e-8 of it.
    beyond = (want.abs() + bound > top) & out.isinf() & (out.sign() == want.sign())
    assert off(torch.where(beyond, want, out.double()), want, bound + HALF[dtype] * want.abs() * (1 + 2.0 ** -8)) <= 1
    assert (beyond.sum(-1) < dim)[1:].all()  # a third of row 1 is a third as large, row 2 ends at 1.9 * 2^126


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("kind", ["e4m3", "int8", "wide"])
@pytest.mark.parametrize("size", [2.0 ** 20, 2.0 ** 24, 2.0 ** 26, 2.0 ** 40])
def test_attention_large_scores(dtype, kind, size):
    # the largest score decides alone, whatever its size and the scale of its value
    g = gen(79)
    kind = dtype if kind == "wide" else kind
    lens, dim = [1, 100, 3000], 64
    p, table = paged(g, lens, 16, 2, dim, kind)
    for b, n in enumerate(lens):
        for h in range(2):
            at = table[b, (n - 1) // 16].item(), h, (n - 1) % 16
            if kind in TOP:
                p.k.view(torch.int8)[at] = torch.ones(dim, device="cuda").to(DT[kind]).view(torch.int8)
                p.k_scale[at] = size
            else:
                p.k[at] = size
    q = torch.ones(3, 6, dim, device="cuda", dtype=DT[dtype])
    want = torch.empty(3, 2, dim, dtype=torch.float64, device="cuda")
    for scale in (1.49, 2.8, 1.99 * 2 ** 20, 2.0 ** -40):
        for b, n in enumerate(lens):
            at = table[b, (n - 1) // 16].item(), slice(None), (n - 1) % 16
            if kind in TOP:
                p.v_scale[at] = scale
                want[b] = p.v.view(torch.int8)[at].view(p.v.dtype).double() * float(torch.tensor(scale))
            else:
                want[b] = p.v[at].double()
        out, lse = torch.empty_like(q), torch.empty(3, 6, device="cuda")
        hal.attn_decode_paged(p, table, ints(lens), q, out, scale=1.0, lse=lse)
        full = want.repeat_interleave(3, 1)
        # one weight of 1 in two parts: 2^-17 over bf16 pages, 2^-22 else; the quotient and the rounding
        bound = (2.0 ** -16 + HALF[dtype]) * full.abs() + 2.0 ** -39 * full.abs().amax(-1, keepdim=True)
        assert off(out, full, bound) <= 1
        assert off(lse, torch.full_like(lse, size * dim), 8 * U * size * dim) <= 1


def test_bad_lengths_and_pages():
    g = gen(2)
    p, table = paged(g, [32, 32, 32, 32], 8, 1, 64, "bf16")
    q = randn(g, 4, 2, 64).bfloat16()
    good, _ = check_attention(p, table, [32, 32, 0, 32], q)
    out, err = torch.empty_like(q), ints([0])
    hal.attn_decode_paged(p, table, ints([32, 33, -5, 32]), q, out, err=err)
    assert err.item() != 0 and torch.equal(out, good)
    table[3, 1], table[3, 2] = 10 ** 6, -7  # positions 8..23 have no page
    err.zero_()
    hal.attn_decode_paged(p, table, ints([32, 32, 0, 32]), q, out, err=err)
    assert err.item() != 0 and torch.equal(out[:3], good[:3])
    fewer = table.clone()
    fewer[3, 1] = table[3, 3]
    want, _ = check_attention(p, fewer, [32, 32, 0, 16], q)
    assert (out[3].double() - want[3].double()).abs().max().item() <= 2.0 ** -7 * want[3].abs().max().item()
    hal.attn_decode_paged(p, table, ints([32, 32, 0, 32]), q, out)  # and without an error word


# ---------------------------------------------------------------- as used

@pytest.mark.parametrize("dtype,kind", [("fp32", "fp32"), ("bf16", "bf16"), ("bf16", "e4m3"), ("bf16", "int8"), ("fp32", "int8")])
def test_prompt_then_steps(dtype, kind):
    """A padded ragged prompt is written, then single tokens decode over it; every step against the 64-bit chain."""
    g = gen(17)
    B, H, G, dim, rows, width = 3, 2, 4, 64, 8, 12
    prompt, steps = [21, 0, 40], 9
    p = pool(B * width + 1, H, rows, dim, kind)
    table = torch.randperm(B * width + 1, generator=g, device="cuda")[: B * width].int().view(B, width)
    r = hal.Rope(dim, scaling="ntk", factor=2.0)
    seq = torch.arange(B, device="cuda", dtype=torch.int32).repeat_interleave(max(prompt))
    pos = torch.arange(max(prompt), device="cuda", dtype=torch.int32).repeat(B)
    pos = torch.where(pos < ints(prompt)[seq.long()], pos, -1).int()
    k, v = (randn(g, pos.numel(), H, dim).to(DT[dtype]) for _ in range(2))
    err = ints([0])
    hal.kv_write(p, table, pos, k, v, seq=seq, rope=r, err=err)
    lens = list(prompt)
    for step in range(steps):
        at = ints(lens)
        q, k, v = (randn(g, B, h, dim).to(DT[dtype]) for h in (H * G, H, H))
        want_k, bound = turned(k, at, r)
        hal.kv_write(p, table, at, k, v, rope=r, q=q, q_out=q, err=err)
        k2, v2 = torch.empty_like(k), torch.empty_like(v)
        hal.kv_read(p, table, at, k2, v2, err=err)
        share = {"fp32": U, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -4, "int8": 0.5 / 127}[kind] * 1.01 + HALF[dtype]
        assert off(k2, want_k, bound * 2 + share * want_k.abs().amax(-1, keepdim=True)) <= 1
        lens = [n + 1 for n in lens]
        check_attention(p, table, lens, q, dtype=dtype)
    assert err.item() == 0


def test_offsets_past_32_bits():
    # e4m3 pages beyond element 2^32
    g = gen(19)
    H, rows, dim, pages = 8, 64, 128, 66000
    t = [torch.empty(pages, H, rows, dim, dtype=torch.int8, device="cuda").view(DT["e4m3"]) for _ in range(2)]
    s = [torch.empty(pages, H, rows, device="cuda") for _ in range(2)]
    p = hal.KVPages(*t, *s)
    n = 300
    table = torch.arange(pages - 1, pages - 1 - 6, -1, device="cuda", dtype=torch.int32).view(1, 6)
    seq, pos = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.arange(n, device="cuda", dtype=torch.int32)
    k, v = (randn(g, n, H, dim).bfloat16() for _ in range(2))
    hal.kv_write(p, table, pos, k, v, seq=seq)
    out = torch.empty_like(k), torch.empty_like(v)
    hal.kv_read(p, table, pos, *out, seq=seq)
    for x, y in zip((k, v), out):
        code, scale = quantised(x.float(), "e4m3")
        assert torch.equal((code.float() * scale[..., None]).bfloat16(), y)
    check_attention(p, table, [n], randn(g, 1, 4 * H, dim).bfloat16())


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_largest_tables_and_most_sequences(kind):
    # 2^30 positions of room, a length that ends in the second page of a million rows
    g = gen(53)
    p = filled(g, 3, 1, 1 << 20, 32, kind)
    table = torch.full((2, 1024), -1, dtype=torch.int32, device="cuda")
    table[0, :2], table[1, 0] = ints([2, 0]), 1
    check_attention(p, table, [(1 << 20) + 77, 3], randn(g, 2, 4, 32).bfloat16())
    check_attention(p, table, [(1 << 20) + 77, 1 << 20], randn(g, 2, 4, 32).bfloat16(), window=1000)
    err = ints([0])
    k = randn(g, 2, 1, 32).bfloat16()
    hal.kv_write(p, table, ints([(1 << 20) + 77, (1 << 20) - 1]), k, k.clone(), err=err)
    hal.kv_write(p, table, ints([(1 << 30) - 1, -1]), k, k.clone(), err=err)  # no page there
    assert err.item() != 0
    # thousands of short sequences, some empty, over uneven groups
    lens = torch.randint(0, 70, (3000,), generator=g, device="cuda").tolist()
    p, table = paged(g, lens, 5, 3, 64, kind)
    check_attention(p, table, lens, randn(g, 3000, 15, 64).bfloat16())
    p, table = paged(g, [900], 32, 128, 256, kind)
    check_attention(p, table, [900], randn(g, 1, 128, 256).bfloat16())


def test_no_tokens():
    p = pool(2, 1, 4, 32, "bf16")
    x, i = torch.empty(0, 1, 32, dtype=torch.bfloat16, device="cuda"), ints([])
    hal.rope(hal.Rope(32), i, x, x)
    hal.kv_write(p, ints([[0]]), i, x, x, seq=i)
    hal.kv_read(p, ints([[0]]), i, x, x, seq=i)
    hal.attn_decode_paged(p, torch.empty(0, 1, dtype=torch.int32, device="cuda"), i, x, x)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_graphs_and_streams(kind):
    """Two captured steps replay at the same time, on inputs changed since the capture, beside an eager call."""
    g = gen(23)
    heads, dim, rows = 2, 64, 16
    r = hal.Rope(dim)
    jobs = []
    for lens in ([3000, 10, 0], [4500, 4000]):
        p, table = paged(g, [n + 20 for n in lens], rows, heads, dim, kind)
        for s in (p.k_scale, p.v_scale):
            if s is not None:
                s.nan_to_num_(nan=0.5)
        q, k, v = (randn(g, len(lens), h, dim).bfloat16() for h in (4 * heads, heads, heads))
        jobs.append(dict(p=p, table=table, lens=ints(lens), pos=ints(lens), q=q, k=k, v=v, qr=torch.empty_like(q), out=torch.empty_like(q),
                         lse=torch.empty(len(lens), 4 * heads, device="cuda"), stream=torch.cuda.Stream()))

    def step(j):
        hal.kv_write(j["p"], j["table"], j["pos"], j["k"], j["v"], rope=r, q=j["q"], q_out=j["qr"])
        j["lens"].copy_(j["pos"] + 1)
        hal.attn_decode_paged(j["p"], j["table"], j["lens"], j["qr"], j["out"], lse=j["lse"])

    for j in jobs:
        step(j)
    torch.cuda.synchronize()
    for j in jobs:
        j["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(j["graph"], stream=j["stream"]):
            step(j)
    for i in range(5):
        for j in jobs:
            j["pos"].add_(1)
            for n in ("q", "k", "v"):
                j[n].copy_(randn(g, *j[n].shape))
        torch.cuda.synchronize()
        for j in jobs:
            with torch.cuda.stream(j["stream"]):
                j["graph"].replay()
        torch.cuda.synchronize()
        for j in jobs:
            out, lse = j["out"].clone(), j["lse"].clone()
            step(j)
            torch.cuda.synchronize()
            assert torch.equal(out, j["out"]) and torch.equal(lse, j["lse"])
            want, want_lse, bound, lse_bound = attended(j["p"], j["table"], (j["pos"] + 1).tolist(), j["qr"], 0, dim ** -0.5)
            assert off(out, want, bound + 2.0 ** -8 * want.abs() * (1 + 2.0 ** -8)) <= 1
    for j in jobs:
        del j["graph"]


FIRST = """
import sys, torch, hierarchical_autoregressive_lm_b200 as hal
p = hal.KVPages.alloc(800, 16, 2, 64, torch.bfloat16)
p.k.normal_(), p.v.normal_()
table = torch.arange(800, dtype=torch.int32, device="cuda").view(1, 800)
lens = torch.tensor([12000], dtype=torch.int32, device="cuda")
q = torch.randn(1, 8, 64, device="cuda").bfloat16()
a, b = torch.zeros_like(q), torch.zeros_like(q)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    hal.attn_decode_paged(p, table, lens, q, a)
g.replay()
hal.attn_decode_paged(p, table, lens, q, b)
torch.cuda.synchronize()
assert torch.equal(a, b) and a.abs().max().item() > 0
"""


def test_first_call_is_a_captured_one():
    run = subprocess.run([sys.executable, "-c", FIRST], capture_output=True, text=True, timeout=300,
                         cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert run.returncode == 0, run.stderr


def test_scratch_of_the_library_and_of_the_caller():
    """The C entry with scratch from its own pool (and with none to be had), and with the caller's."""
    g = gen(41)
    lens = [40000]
    p, table = paged(g, lens, 16, 1, 128, "bf16")
    q = randn(g, 1, 4, 128).bfloat16()
    good, _ = check_attention(p, table, lens, q)
    out, n = torch.zeros_like(q), ints(lens)
    fn = hal.load_library().photon_attn_decode_paged

    def call(scratch, size):
        a = hal.photon_attn_paged_args()
        vals = dict(pages=p._ref, d_table=table.data_ptr(), table_stride=table.stride(0), seqs=1, width=table.shape[1], d_len=n.data_ptr(), dtype=1,
                    q_heads=4, window=0, q=hal.photon_rows(q.data_ptr(), 512, 128), o=hal.photon_rows(out.data_ptr(), 512, 128), scale=128 ** -0.5,
                    d_scratch=scratch, scratch_bytes=size)
        for name, v in vals.items():
            setattr(a, name, v)
        rc = fn(ctypes.byref(a), torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        return rc

    hal.debug_fail_alloc(1)
    try:
        assert call(None, 0) == -2 and (out == 0).all()
    finally:
        hal.debug_fail_alloc(0)
    assert call(None, 0) == 0 and torch.equal(out, good)
    out.zero_()
    need = call(None, -1)
    assert 0 < need < 64 << 20 and (out == 0).all()
    buf = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    assert call(buf.data_ptr() + 16, need - 1) == -1 and (out == 0).all()
    assert call(buf.data_ptr() + 16, need) == 0 and torch.equal(out, good)
    assert (buf[:16] == 255).all() and (buf[need + 16:] == 255).all()


def test_one_table_row_for_several_sequences():
    # a shared prompt: the table's rows are one row, the lengths differ
    g = gen(43)
    p, table = paged(g, [500], 16, 2, 64, "e4m3")
    lens = [500, 17, 0, 333]
    q = randn(g, 4, 6, 64).bfloat16()
    shared = table.expand(4, -1)
    check_attention(p, shared, lens, q)
    pos, seq = ints([3, 3, 499, 3]), ints([0, 1, 2, 3])
    k, v = (torch.empty(4, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    hal.kv_read(p, shared, pos, k, v, seq=seq)
    assert torch.equal(k[0], k[1]) and torch.equal(v[0], v[3]) and not torch.equal(k[0], k[2])


def test_calls_from_threads():
    """Eager calls of four threads on four streams give what each gives alone."""
    work = []
    for i in range(4):
        g = gen(31 + i)
        lens = [2500 + 300 * i, 700]
        p, table = paged(g, lens, 16, 2, 128, "bf16")
        q = randn(g, 2, 8, 128).bfloat16()
        out, _ = check_attention(p, table, lens, q)
        work.append((p, table, ints(lens), q, out, torch.empty_like(out), torch.cuda.Stream()))
    torch.cuda.synchronize()

    def call(w):
        for i in range(20):
            hal.attn_decode_paged(*w[:4], w[5], stream=w[6] if i % 2 else w[6].cuda_stream)

    threads = [threading.Thread(target=call, args=(w,)) for w in work]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    for w in work:
        assert torch.equal(w[4], w[5])


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two devices")
def test_tensors_on_another_device():
    with torch.cuda.device(1):
        g = torch.Generator(device="cuda:1").manual_seed(1)
        p = hal.KVPages.alloc(4, 16, 1, 64, torch.bfloat16, device="cuda:1")
        p.k.normal_(generator=g), p.v.normal_(generator=g)
        table = torch.arange(4, dtype=torch.int32, device="cuda:1").view(1, 4)
        q = torch.randn(1, 2, 64, generator=g, device="cuda:1").bfloat16()
        lens, a, b = torch.tensor([60], dtype=torch.int32, device="cuda:1"), torch.empty_like(q), torch.empty_like(q)
        hal.attn_decode_paged(p, table, lens, q, a)
    hal.attn_decode_paged(p, table, lens, q, b)  # the current device is another
    torch.cuda.synchronize(1)
    assert torch.equal(a, b)


def test_binding_refusals():
    p = pool(2, 2, 4, 32, "bf16")
    bf = dict(dtype=torch.bfloat16, device="cuda")
    k, q, table = torch.zeros(3, 2, 32, **bf), torch.zeros(3, 4, 32, **bf), ints([[0], [1], [0]])
    pos = ints([0, 1, 2])
    for kw, match in ((dict(k=k.float()), "as the pages"), (dict(v=k[:2]), "expected shape"), (dict(pos=pos.long()), "int32"),
                      (dict(table=table.long()), "int32"), (dict(seq=pos.cpu()), "CUDA"), (dict(q=q, q_out=q), "needs rope"),
                      (dict(rope=hal.Rope(32), q=q, q_out=q[:, :2]), "expected shape"), (dict(q_out=q), "without q"),
                      (dict(k=k.transpose(1, 2).contiguous().transpose(1, 2)), "contiguous")):
        a = dict(pages=p, table=table, pos=pos, k=k, v=k)
        a.update(kw)
        with pytest.raises(ValueError, match=match):
            hal.kv_write(**a)
    with pytest.raises(ValueError, match="expanded"):
        hal.kv_read(p, table, pos, k, k[:1].expand(3, 2, 32))
    with pytest.raises(ValueError, match="expected shape"):
        hal.attn_decode_paged(p, table, pos, q[:2], q[:2])
    with pytest.raises(hal.PhotonError, match="multiple of heads"):
        hal.attn_decode_paged(p, table, pos, q[:, :3], q[:, :3].clone())
    with pytest.raises(hal.PhotonError, match="must not be q"):
        hal.attn_decode_paged(p, table, pos, q, q)
    with pytest.raises(hal.PhotonError, match="share memory"):
        hal.kv_write(hal.KVPages(p.k, p.k), table, pos, k, k)
    with pytest.raises(hal.PhotonError, match="rot_dim"):
        hal.rope(hal.Rope(64), pos, k, k)
    with pytest.raises(ValueError, match="x2"):
        hal.rope(hal.Rope(32), pos, k, k, out2=k)
    q1 = torch.zeros(3, 4, 32, **bf)
    with pytest.raises(hal.PhotonError, match="in place"):
        hal.rope(hal.Rope(32), pos, q1.view(-1)[: 3 * 2 * 32].view(3, 2, 32), q1[:, :2])
