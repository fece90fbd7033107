"""Host-side checks of the paged-cache operators: frequencies and refusals, without a device.

The entry points check every argument before any CUDA call, so a refused
call needs no GPU; the addresses given here are never dereferenced.
"""
import ctypes
from decimal import Decimal, getcontext

import pytest
import torch

import hierarchical_autoregressive_lm_b200 as hal

getcontext().prec = 60
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494")
A = 1 << 20  # aligned addresses that nothing reads
B = 1 << 21


def _turns(rot, theta=10000.0, scaling="none", factor=1.0, original_len=0, alpha=1.0, beta=32.0):
    """Turns a position of each pair in 60 digits."""
    d, s, base = Decimal(rot), Decimal(factor), Decimal(theta)
    if scaling == "ntk":
        base *= s ** (d / (d - 2))
    out = []
    for i in range(rot // 2):
        f = base ** (Decimal(-2 * i) / d)
        if scaling == "linear":
            f /= s
        if scaling == "yarn":
            g = (Decimal(original_len) * f / (2 * PI) - Decimal(alpha)) / (Decimal(beta) - Decimal(alpha))
            g = min(Decimal(1), max(Decimal(0), g))
            f = f * g + f / s * (1 - g)
        out.append(f / (2 * PI) % 1)
    return out


@pytest.mark.parametrize("kw", [
    dict(rot=64), dict(rot=2), dict(rot=128, theta=500000.0), dict(rot=64, scaling="linear", factor=4.0),
    dict(rot=64, scaling="ntk", factor=8.0), dict(rot=128, scaling="yarn", factor=32.0, original_len=4096),
    dict(rot=96, scaling="yarn", factor=2.5, original_len=2048, alpha=2.0, beta=16.0), dict(rot=4, theta=0.01)])
def test_frequencies(kw):
    kw = dict(kw)
    rot = kw.pop("rot")
    r = hal.Rope(rot, device="cpu", **kw)
    want = _turns(rot, **kw)
    assert len(r.turns) == rot // 2
    for got, w in zip(r.turns, want):
        # pow, the scaling's few operations and 1 / (2 pi), each within 2^-52 of its value, then 2^-65
        off = abs(Decimal(got) / 2 ** 64 - w)
        off = min(off, 1 - off)
        size = max(w, Decimal(1) if kw.get("theta", 1e4) < 1 else w)  # below 1: whole turns were dropped from up to 1/theta
        size *= 100 if kw.get("theta", 1e4) < 1 else 1
        assert off <= size * 8 * Decimal(2) ** -52 + Decimal(2) ** -64, (got, w)
    assert r.scale == pytest.approx(1 + 0.1 * float(Decimal(kw.get("factor", 1.0)).ln()) if kw.get("scaling") == "yarn" else 1.0, rel=1e-6)
    assert hal.Rope(rot, device="cpu", attn_scale=0.75, **kw).scale == 0.75


@pytest.mark.parametrize("kw", [
    dict(rot=64), dict(rot=2), dict(rot=512), dict(rot=128, theta=500000.0), dict(rot=128, theta=1e7), dict(rot=64, scaling="linear", factor=4.0),
    dict(rot=128, theta=500000.0, scaling="linear", factor=2.5), dict(rot=64, scaling="ntk", factor=8.0), dict(rot=4, scaling="ntk", factor=1000.0),
    dict(rot=128, scaling="yarn", factor=32.0, original_len=4096), dict(rot=96, scaling="yarn", factor=2.5, original_len=2048, alpha=2.0, beta=16.0)])
def test_frequencies_are_right_at_the_last_position(kw):
    """Within 2^-60 of a turn, 2^-29 turns at position 2^31 - 1, a sixteenth of the angle's rounding to fp32.

    f of at most one radian is 0.16 turns.  Host arithmetic of 64 bits is off by 2^-64 of each result: the power by its
    exponent's rounding, at most ln(theta factor^2) = 23, and its own 2; the division by 2 pi, the scaling and the blend by
    fewer than 16 more: 41 * 0.16 + 0.5 units of 2^-64, below 2^-61."""
    kw = dict(kw)
    rot = kw.pop("rot")
    for got, want in zip(hal.Rope(rot, device="cpu", **kw).turns, _turns(rot, **kw)):
        off = abs(Decimal(got) / 2 ** 64 - want)
        assert min(off, 1 - off) <= Decimal(2) ** -60


def test_rope_config_refusals():
    for kw in (dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=514), dict(rot_dim=64, theta=0.0), dict(rot_dim=64, theta=float("nan")),
               dict(rot_dim=64, scaling="linear", factor=0.5), dict(rot_dim=2, scaling="ntk", factor=2.0),
               dict(rot_dim=64, scaling="yarn", factor=2.0), dict(rot_dim=64, scaling="yarn", factor=2.0, original_len=4, alpha=2.0, beta=2.0),
               dict(rot_dim=64, attn_scale=float("inf")), dict(rot_dim=64, scaling="linear", factor=float("nan"))):
        with pytest.raises(hal.PhotonError) as e:
            hal.Rope(device="cpu", **kw)
        assert e.value.code == -1
    with pytest.raises(ValueError, match="scaling"):
        hal.Rope(64, scaling="dynamic", device="cpu")
    lib = hal.load_library()
    assert lib.photon_rope_frequencies(None, None, None) == -1


def _pages(**kw):
    d = dict(k=A, v=B, k_scale=A, v_scale=B, page_stride=8 * 16 * 64, head_stride=16 * 64, row_stride=64, scale_page=8 * 16,
             scale_head=16, scale_row=1, kind=2, pages=10, page_rows=16, heads=8, head_dim=64)
    d.update(kw)
    return hal.photon_kv_pages(**d)


BAD_PAGES = [dict(kind=4), dict(kind=-1), dict(kind=0), dict(pages=0), dict(page_rows=0), dict(heads=0), dict(head_dim=48),
             dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None), dict(k=A + 8), dict(page_stride=8 * 16 * 64 + 8),
             dict(row_stride=72), dict(head_stride=-16), dict(k_scale=A + 2), dict(page_stride=1 << 40), dict(page_stride=16 + (1 << 36)),
             dict(row_stride=1 << 62)]


def _call(fn, cls, defaults, kw):
    """fn on a structure with the defaults changed by kw (rows: (address, token stride, head stride))."""
    a = cls()
    for n, v in {**defaults, **kw}.items():
        if isinstance(v, ctypes.Structure):
            v = ctypes.addressof(v)
        setattr(a, n, hal.photon_rows(*v) if isinstance(v, tuple) else v)
    return fn(ctypes.byref(a), None)


ROWS, OUT, NONE = (A, 1024, 64), (B, 1024, 64), (None, 1024, 64)


def _attn(lib, pages, **kw):
    d = dict(pages=pages, dtype=1, d_table=A, table_stride=4, seqs=2, width=4, d_len=A, q=ROWS, q_heads=16, window=0, scale=0.125, o=OUT)
    return _call(lib.photon_attn_decode_paged, hal.photon_attn_paged_args, d, kw)


def test_attention_refusals():
    lib = hal.load_library()
    for kw in BAD_PAGES:
        assert _attn(lib, _pages(**kw)) == -1, kw
        assert lib.photon_last_error() != b""
    for kw in (dict(dtype=2), dict(d_table=None), dict(seqs=-1), dict(width=0), dict(width=1 << 28), dict(width=1 << 40), dict(d_len=None),
               dict(q=NONE), dict(o=NONE), dict(o=ROWS), dict(q_heads=12), dict(q_heads=0), dict(q_heads=1 << 40), dict(window=-1), dict(window=1 << 31),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=1e39), dict(q=(A + 1, 1024, 64)), dict(d_lse=A + 2),
               dict(d_err=A + 1), dict(d_scratch=A + 8, scratch_bytes=1 << 20), dict(scratch_bytes=1 << 20), dict(d_table=A + 1), dict(seqs=1 << 28), dict(seqs=1 << 40)):
        assert _attn(lib, _pages(), **kw) == -1, kw
        assert lib.photon_last_error() != b""
    assert _attn(lib, None) == -1
    assert lib.photon_attn_decode_paged(None, None) == -1
    assert _attn(lib, _pages(), seqs=0, d_table=None) == 0  # nothing to do


def test_write_and_read_refusals():
    lib = hal.load_library()
    rope = hal.photon_rope_table(A, 64, 0, 1.0)

    both = dict(dtype=1, d_table=A, table_stride=4, seqs=2, width=4, d_pos=A, tokens=2, k=ROWS, v=ROWS)
    for fn in (lib.photon_kv_write, lib.photon_kv_read):
        assert fn(None, None) == -1
        for kw in BAD_PAGES:
            assert _call(fn, hal.photon_kv_args, dict(both, pages=_pages(**kw)), {}) == -1, kw
        pages = _pages()
        for kw in (dict(pages=None), dict(dtype=3), dict(d_table=None), dict(seqs=0), dict(seqs=1 << 31), dict(width=-1), dict(d_pos=None),
                   dict(tokens=-1), dict(k=NONE), dict(v=NONE), dict(tokens=1 << 29), dict(tokens=1 << 33), dict(d_pos=A + 1), dict(d_seq=A + 2),
                   dict(d_err=A + 2), dict(k=(A + 1, 512, 64)), dict(q_heads=-1), dict(q_heads=1 << 33), dict(q=ROWS, q_out=ROWS, q_heads=16)):
            assert _call(fn, hal.photon_kv_args, dict(both, pages=pages), kw) == -1, (fn, kw)
            assert lib.photon_last_error() != b""
        assert _call(fn, hal.photon_kv_args, dict(both, pages=pages), dict(tokens=0, d_pos=None, k=NONE, v=NONE, d_table=None)) == 0
    assert _call(lib.photon_kv_read, hal.photon_kv_args, dict(both, pages=pages), dict(rope=rope)) == -1
    for kw in (dict(pages=_pages(v=A)), dict(pages=_pages(v_scale=A)), dict(rope=hal.photon_rope_table(None, 64, 0, 1.0)),
               dict(rope=hal.photon_rope_table(A, 66, 0, 1.0)), dict(rope=hal.photon_rope_table(A, 31, 0, 1.0)), dict(rope=rope, q_heads=16, q=ROWS),
               dict(rope=rope, q_heads=16, q_out=ROWS), dict(rope=rope, q=ROWS, q_out=(A, 2048, 64), q_heads=16)):
        assert _call(lib.photon_kv_write, hal.photon_kv_args, dict(both, pages=pages), kw) == -1, kw


def test_rope_refusals():
    lib = hal.load_library()
    table = hal.photon_rope_table(A, 64, 0, 1.0)
    rows = (A, 128, 64)
    good = dict(rope=table, dtype=0, d_pos=A, tokens=3, head_dim=64, x=rows, heads=2, y=rows)
    assert lib.photon_rope(None, None) == -1
    for kw in (dict(dtype=7), dict(d_pos=None), dict(tokens=-1), dict(head_dim=62), dict(head_dim=65), dict(head_dim=514), dict(x=NONE),
               dict(y=NONE), dict(heads=0), dict(heads=1 << 32), dict(heads2=-1), dict(heads2=2), dict(heads2=2, x2=rows), dict(y=(A, 256, 64)),
               dict(heads2=1, x2=rows, y2=(A, 128, 32)), dict(x=(A + 2, 128, 64)), dict(tokens=1 << 30), dict(rope=None),
               dict(rope=hal.photon_rope_table(A + 4, 64, 0, 1.0))):
        assert _call(lib.photon_rope, hal.photon_rope_args, good, kw) == -1, kw
        assert lib.photon_last_error() != b""
    assert _call(lib.photon_rope, hal.photon_rope_args, good, dict(tokens=0, d_pos=None, x=NONE, y=NONE)) == 0


def test_struct_layouts():
    assert ctypes.sizeof(hal.photon_kv_pages) == 4 * 8 + 6 * 8 + 5 * 4 + 4
    assert ctypes.sizeof(hal.photon_rope_table) == 8 + 3 * 4 + 4
    assert ctypes.sizeof(hal.photon_rope_config) == 3 * 4 + 4 + 5 * 8
    for cls, pack in ((hal.photon_rope_args, hal._pack_rope), (hal.photon_kv_args, hal._pack_kv), (hal.photon_attn_paged_args, hal._pack_attn)):
        n = ctypes.sizeof(cls) // 8
        packed = pack(*range(1, n + 1))
        got, i = cls.from_buffer_copy(packed), 1
        for name, kind in cls._fields_:
            for value in ([getattr(got, name)] if kind is not hal.photon_rows else [getattr(getattr(got, name), f) for f in ("p", "token", "head")]):
                assert value == i, (cls, name)
                i += 1
        assert i == n + 1


def test_binding_refuses_before_the_library():
    k = torch.zeros(4, 2, 16, 64)
    with pytest.raises(ValueError, match="CUDA"):
        hal.KVPages(k, k)
    with pytest.raises(ValueError, match="8-bit"):
        hal.KVPages(k.to(torch.int8), k.to(torch.int8))
    with pytest.raises(ValueError, match="8-bit"):
        hal.KVPages(k, k, torch.zeros(4, 2, 16), torch.zeros(4, 2, 16))
    with pytest.raises(ValueError, match="pages, heads"):
        hal.KVPages(k.half(), k.half())
    with pytest.raises(ValueError, match="of shape"):
        hal.KVPages(k, k[:3])
    with pytest.raises(ValueError, match="last dimension"):
        hal.KVPages(k.transpose(2, 3), k.transpose(2, 3))
    with pytest.raises(ValueError, match="expanded"):
        hal.KVPages(k[:1].expand(4, 2, 16, 64), k[:1].expand(4, 2, 16, 64))
    with pytest.raises(TypeError, match="KVPages"):
        hal.attn_decode_paged(k, torch.zeros(1, 1, dtype=torch.int32), None, None, None)
    r = hal.Rope(64, device="cpu")
    x, pos = torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        hal.rope(r, pos, x, x)
    with pytest.raises(ValueError, match="float32 or"):
        hal.rope(r, pos, x.half(), x.half())
    with pytest.raises(ValueError, match="tokens, heads"):
        hal.rope(r, pos, x[0], x[0])
    with pytest.raises(TypeError, match="Rope"):
        hal.rope(None, pos, x, x)
