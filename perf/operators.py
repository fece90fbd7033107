"""Cases of the operators around a paged key-value cache: rotary positions,
the (quantising) cache write, the read back, and the decode attention over
pages.  Every case runs in a plain form (elementary torch operations in 32
bits, angles in 64) or, with `own`, through the package's entry points.
"""
import math

import torch

own = False

E4M3, I8 = torch.float8_e4m3fn, torch.int8
_DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "e4m3": E4M3, "int8": I8}
_SIZE = {"fp32": 4, "bf16": 2, "e4m3": 1, "int8": 1}
_TOP = {"e4m3": 448.0, "int8": 127.0}
_TINY = 1e-30


def listed():
    return [
        # one decode step's q and k of the 600M-class batch-64 model (16 heads of 64)
        dict(name="rope_step", op="rope", dtype="bf16", tokens=64, heads=16, kv_heads=16, dim=64, rot=64,
             inter=False, scaling="none", factor=1.0, far=4096, back=False),
        # a long prompt with grouped heads, half of the head rotated, positions near a million
        dict(name="rope_prompt", op="rope", dtype="bf16", tokens=8191, heads=32, kv_heads=8, dim=128, rot=64,
             inter=True, scaling="yarn", factor=32.0, far=1 << 20, back=False),
        # gradient of the rotation, fp32, an odd number of tokens
        dict(name="rope_grad", op="rope", dtype="fp32", tokens=2047, heads=16, kv_heads=16, dim=64, rot=64,
             inter=False, scaling="ntk", factor=4.0, far=32768, back=True),
        # one decode step's keys and values into an 8-bit cache, q rotated on the way
        dict(name="write_step", op="write", dtype="bf16", kind="e4m3", seqs=64, tokens=64, heads=16, kv_heads=16,
             dim=64, rot=64, inter=False, page=16, pad=0),
        # ragged prompts, padded, grouped heads, int8 (rotated before)
        dict(name="write_prompt", op="write", dtype="bf16", kind="int8", seqs=13, tokens=32768, heads=32, kv_heads=8,
             dim=128, rot=0, inter=False, page=64, pad=513),
        # a prompt into a bf16 cache with the keys rotated as they are written
        dict(name="write_rotated", op="write", dtype="bf16", kind="bf16", seqs=16, tokens=8192, heads=16, kv_heads=16,
             dim=64, rot=64, inter=False, page=16, pad=0),
        # a long shared context read back for a prefill after it
        dict(name="read_context", op="read", dtype="bf16", kind="e4m3", seqs=4, tokens=65536, kv_heads=8, dim=128, page=64),
        # a few hundred rows of the tiny fp32 model, pages of five
        dict(name="read_small", op="read", dtype="fp32", kind="int8", seqs=3, tokens=777, kv_heads=2, dim=32, page=5),
        # one sequence, a short cache: latency alone
        dict(name="attn_short", op="attn", dtype="bf16", kind="bf16", seqs=1, longest=257, ragged=False, heads=16,
             kv_heads=16, dim=64, page=16, window=0),
        # a serving batch of uneven lengths, grouped heads
        dict(name="attn_batch", op="attn", dtype="bf16", kind="bf16", seqs=64, longest=4096, ragged=True, heads=32,
             kv_heads=8, dim=128, page=16, window=0),
        # two long contexts in an 8-bit cache
        dict(name="attn_long", op="attn", dtype="bf16", kind="e4m3", seqs=2, longest=131072, ragged=False, heads=32,
             kv_heads=8, dim=128, page=64, window=0),
        # fp32 queries over int8 pages of seven, odd lengths, a window
        dict(name="attn_fp32", op="attn", dtype="fp32", kind="int8", seqs=9, longest=2049, ragged=True, heads=12,
             kv_heads=4, dim=32, page=7, window=1000),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "attn", "attn"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    kv = rng.choice([1, 2, 4, 5, 8, 16])
    dim = rng.choice([32, 64, 128])
    heads = kv * rng.choice([1, 2, 4])
    c = dict(op=op, dtype=dtype, dim=dim, kv_heads=kv)
    rot, inter = rng.choice([dim, dim, dim // 2]), rng.random() < 0.5
    if op == "rope":
        return dict(c, tokens=_log(rng, 1, min(16384, 2**26 // ((heads + kv) * dim))), heads=heads, rot=rot, inter=inter,
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]), factor=float(rng.choice([2, 4, 8, 32])),
                    far=_log(rng, 1024, 1 << 20), back=rng.random() < 0.3)
    kind, page = rng.choice([dtype, "e4m3", "int8"]), rng.choice([1, 5, 7, 16, 32, 64, 128])
    c = dict(c, kind=kind, page=page)
    if op == "write":
        tokens = _log(rng, 1, min(16384, 2**27 // ((2 * heads + 4 * kv) * dim)))
        # an int8 code is a whole number: its keys come rotated, so that both forms round the same value
        rot = 0 if kind == "int8" else rng.choice([0, rot])
        return dict(c, tokens=tokens, seqs=rng.randint(1, min(64, tokens)), heads=heads, rot=rot, inter=inter,
                    pad=0 if rot else rng.choice([0, tokens // 9]))
    if op == "read":
        tokens = _log(rng, 1, min(32768, 2**25 // (kv * dim)))
        return dict(c, tokens=tokens, seqs=rng.randint(1, min(64, tokens)))
    seqs = _log(rng, 1, 64)
    longest = _log(rng, 1, min(131072, 2**26 // (kv * dim)) // seqs)
    return dict(c, seqs=seqs, longest=longest, ragged=rng.random() < 0.7, heads=kv * rng.choice([1, 2, 3, 4, 8]),
                window=rng.choice([0, 0, 0, 333]))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _heads(g, n, heads, dim, dtype):
    """Rows of one projection: channels of uneven size, as q and k have them."""
    channel = 0.5 + torch.rand(1, 1, dim, generator=g, device="cuda")
    return (torch.randn(n, heads, dim, generator=g, device="cuda") * channel).to(dtype)


def _quantise(x, kind):
    """Codes and scales of the rows of x (fp32), one scale a row."""
    top = _TOP[kind]
    amax = x.abs().amax(-1)
    fine = torch.isfinite(amax)
    held = torch.where(fine, amax, 1.0).clamp(min=_TINY)
    top = torch.full_like(held, top)  # a quotient of tensors is rounded once, one with a number is not
    y = torch.where(fine.unsqueeze(-1), x * (top / held).unsqueeze(-1), 0.0)
    code = y.to(E4M3) if kind == "e4m3" else y.round().to(I8)
    return code, torch.where(fine, held / top, math.nan)


def _table(g, seqs, width, pages):
    """Each sequence's pages, scattered over the pool."""
    return torch.randperm(pages, generator=g, device="cuda")[: seqs * width].to(torch.int32).view(seqs, width)


def _pool(g, pages, heads, page, dim, kind):
    """K and V pages [pages, heads, page, dim] that hold a cache, with their scales where they are narrow."""
    out = []
    for _ in range(2):
        x = torch.randn(pages, heads, page, dim, generator=g, device="cuda")
        if kind in _TOP:
            out.append(_quantise(x.mul_(0.5 + torch.rand(dim, generator=g, device="cuda")), kind))
        else:
            out.append((x.to(_DT[kind]), None))
        del x
    return dict(k=out[0][0], v=out[1][0], k_scale=out[0][1], v_scale=out[1][1])


def _lengths(g, case):
    """Each sequence's length: ragged ones run from an eighth of the longest to it, with an empty one among four."""
    n = case["seqs"]
    lens = torch.full((n,), case["longest"], device="cuda")
    if case["ragged"]:
        low = max(1, case["longest"] // 8)
        lens = torch.randint(low, case["longest"] + 1, (n,), generator=g, device="cuda")
        lens[0] = case["longest"]
        if n >= 4:
            lens[3] = 0
    return lens.to(torch.int32)


def _places(g, case):
    """(seq, pos) of every token: runs of each sequence's positions, the last `pad` of them padding (-1)."""
    n, seqs = case["tokens"], case["seqs"]
    each = -(-n // seqs)
    at = torch.arange(n, device="cuda")
    seq, pos = at // each, at % each
    start = int(torch.randint(0, 40, (1,), generator=torch.Generator().manual_seed(int(g.initial_seed()))).item())
    pos = pos + start
    pad = case.get("pad", 0)
    if pad:
        pos[n - pad:] = -1
    return seq.to(torch.int32), pos.to(torch.int32), each + 40


def _frequencies(case):
    """Angle a position of each rotated pair, in 64 bits, and the factor on the rotated part."""
    rot, theta, scaling, s = case["rot"], 10000.0, case.get("scaling", "none"), case.get("factor", 1.0)
    i = torch.arange(rot // 2, dtype=torch.float64)
    if scaling == "ntk":
        theta = theta * s ** (rot / (rot - 2))
    f = theta ** (-2.0 * i / rot)
    if scaling == "linear":
        f = f / s
    if scaling == "yarn":
        turns = 4096 * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        f = f * keep + f / s * (1 - keep)
    return f.cuda(), 0.1 * math.log(s) + 1.0 if scaling == "yarn" else 1.0


def _handle(case):
    import hierarchical_autoregressive_lm_b200 as hal
    return hal.Rope(case["rot"], theta=10000.0, interleaved=case["inter"], scaling=case.get("scaling", "none"),
                    factor=case.get("factor", 1.0), original_len=4096)


def prepare(case, seed):
    g, dt = _gen(seed), _DT[case["dtype"]]
    s = dict(case=case)
    if case["op"] == "rope":
        n = case["tokens"]
        first = int(torch.randint(0, max(1, case["far"] - n), (1,), generator=torch.Generator().manual_seed(seed)).item())
        s["pos"] = torch.arange(first, first + n, device="cuda", dtype=torch.int32)
        s["q"], s["k"] = (_heads(g, n, h, case["dim"], dt) for h in (case["heads"], case["kv_heads"]))
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
    elif case["op"] in ("write", "read"):
        s["seq"], s["pos"], longest = _places(g, case)
        width = -(-longest // case["page"])
        pages = case["seqs"] * width + 3
        s["table"] = _table(g, case["seqs"], width, pages)
        s["pool"] = _pool(g, pages, case["kv_heads"], case["page"], case["dim"], case["kind"])
        s["k"], s["v"] = (_heads(g, case["tokens"], case["kv_heads"], case["dim"], dt) for _ in range(2))
        if case.get("rot"):
            s["q"] = _heads(g, case["tokens"], case["heads"], case["dim"], dt)
            s["q_out"] = torch.empty_like(s["q"])
    else:
        s["lens"] = _lengths(g, case)
        width = -(-case["longest"] // case["page"])
        used = -(-s["lens"] // case["page"])
        pages = int(used.sum().item()) + 3
        table = torch.full((case["seqs"], width), -1, dtype=torch.int32, device="cuda")
        table[torch.arange(width, device="cuda") < used[:, None]] = _table(g, 1, pages - 3, pages)[0]
        s["table"] = table
        s["pool"] = _pool(g, pages, case["kv_heads"], case["page"], case["dim"], case["kind"])
        s["q"] = _heads(g, case["seqs"], case["heads"], case["dim"], dt)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(case["seqs"], case["heads"], device="cuda")
    if case.get("rot"):
        s["freq"], s["factor"] = _frequencies(case)
    if own:
        import hierarchical_autoregressive_lm_b200 as hal
        if case.get("rot"):
            s["rope"] = _handle(case)
        if "pool" in s:
            s["pages"] = hal.KVPages(**s["pool"])
    return s


# -------------------------------------------------------------- plain forms

def _plain_rotate(x, pos, s, back=False):
    """x (fp32 [n, heads, dim]) rotated by its positions."""
    rot, inter = s["case"]["rot"], s["case"]["inter"]
    angle = pos.double()[:, None, None] * s["freq"]
    c, d = (angle.cos() * s["factor"]).float(), (angle.sin() * s["factor"]).float()
    d = -d if back else d
    y = x.clone()
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * d, a * d + b * c
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y[..., : rot // 2], y[..., rot // 2: rot] = a * c - b * d, a * d + b * c
    return y


def _plain_rope(s):
    return [_plain_rotate(s[n].float(), s["pos"], s, s["case"]["back"]).to(s[n].dtype) for n in ("q", "k")]


def _plain_slots(s):
    """Page and row of each token; a padding token takes the place of the first real one in `src`."""
    real = s["pos"] >= 0
    src = torch.where(real, torch.arange(real.numel(), device="cuda"), real.int().argmax())
    pos, seq = s["pos"][src].long(), s["seq"][src].long()
    R = s["case"]["page"]
    return src, s["table"][seq, pos // R].long(), pos % R


def _plain_write(s):
    pool, case = s["pool"], s["case"]
    src, page, row = _plain_slots(s)
    k, v = s["k"].float(), s["v"].float()
    out = []
    if case["rot"]:
        k = _plain_rotate(k, s["pos"], s)
        s["q_out"] = _plain_rotate(s["q"].float(), s["pos"], s).to(s["q"].dtype)
        out.append(s["q_out"])
    if case["kind"] in _TOP:
        (k, ks), (v, vs) = _quantise(k, case["kind"]), _quantise(v, case["kind"])
        pool["k_scale"][page, :, row], pool["v_scale"][page, :, row] = ks[src], vs[src]
        out += [pool["k_scale"], pool["v_scale"]]
    else:
        k, v = k.to(_DT[case["kind"]]), v.to(_DT[case["kind"]])
    # codes are moved as bytes: indexing knows no 8-bit floating type
    move = (lambda x: x.view(I8)) if case["kind"] == "e4m3" else (lambda x: x)
    move(pool["k"])[page, :, row], move(pool["v"])[page, :, row] = move(k)[src], move(v)[src]
    return [pool["k"], pool["v"]] + out


def _plain_read(s):
    pool, case = s["pool"], s["case"]
    _, page, row = _plain_slots(s)
    move = (lambda x: x.view(I8)) if case["kind"] == "e4m3" else (lambda x: x)
    out = []
    for n in ("k", "v"):
        x = move(pool[n])[page, :, row].view(pool[n].dtype).float()
        if case["kind"] in _TOP:
            x = x * pool[n + "_scale"][page, :, row].unsqueeze(-1)
        out.append(x.to(_DT[case["dtype"]]))
    return out


def _plain_attn(s):
    pool, case, lens = s["pool"], s["case"], s["lens"].long()
    B, H, D = case["seqs"], case["kv_heads"], case["dim"]
    at = s["table"].clamp(min=0).long()
    move = (lambda x: x.view(I8)) if case["kind"] == "e4m3" else (lambda x: x)

    def rows(n):  # [B, H, positions, D] in fp32
        x = move(pool[n])[at].view(pool[n].dtype).float()
        if case["kind"] in _TOP:
            x = x * pool[n + "_scale"][at].unsqueeze(-1)
        return x.transpose(1, 2).reshape(B, H, -1, D)

    q = s["q"].float().view(B, H, -1, D)
    score = q @ rows("k").transpose(2, 3) / math.sqrt(D)
    pos = torch.arange(score.shape[-1], device="cuda")
    seen = pos < lens[:, None]
    if case["window"]:
        seen = seen & (pos >= lens[:, None] - case["window"])
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = (score - torch.where(top == -math.inf, 0.0, top)).exp()
    total = p.sum(-1, keepdim=True)
    out = (p @ rows("v")) / total.clamp(min=1e-37)
    lse = (top + total.log()).view(B, -1)
    return [out.view(B, -1, D).to(s["q"].dtype), lse]


# -------------------------------------------------------------- both forms

def run(s):
    op = s["case"]["op"]
    if not own:
        return {"rope": _plain_rope, "write": _plain_write, "read": _plain_read, "attn": _plain_attn}[op](s)
    import hierarchical_autoregressive_lm_b200 as hal
    if op == "rope":
        hal.rope(s["rope"], s["pos"], s["q"], s["q_out"], s["k"], s["k_out"], backward=s["case"]["back"])
        return [s["q_out"], s["k_out"]]
    pool = s["pool"]
    if op == "write":
        hal.kv_write(s["pages"], s["table"], s["pos"], s["k"], s["v"], seq=s["seq"], rope=s.get("rope"),
                     q=s.get("q"), q_out=s.get("q_out"))
        more = [s["q_out"]] if "q" in s else []
        more += [pool["k_scale"], pool["v_scale"]] if s["case"]["kind"] in _TOP else []
        return [pool["k"], pool["v"]] + more
    if op == "read":
        hal.kv_read(s["pages"], s["table"], s["pos"], s["k"], s["v"], seq=s["seq"])
        return [s["k"], s["v"]]
    hal.attn_decode_paged(s["pages"], s["table"], s["lens"], s["q"], s["out"], window=s["case"]["window"], lse=s["lse"])
    return [s["out"], s["lse"]]


def work(case):
    e, D, H = _SIZE[case["dtype"]], case["dim"], case["kv_heads"]
    if case["op"] == "rope":
        rows = case["tokens"] * (case["heads"] + H)
        return {"bytes": 2 * rows * D * e + 4 * case["tokens"], "flops": 3 * rows * case["rot"]}
    narrow = case["kind"] in _TOP
    row = D * _SIZE[case["kind"]] + (4 if narrow else 0)  # one cached row: codes and its scale
    if case["op"] in ("write", "read"):
        n = case["tokens"] - case.get("pad", 0)
        q = 2 * n * case["heads"] * D * e if case.get("rot") else 0
        return {"bytes": n * (2 * H * (D * e + row) + 8 + 4) + q,
                "flops": 2 * n * H * D * (2 if narrow else 0) + (3 * n * (H + case["heads"]) * case["rot"] if case.get("rot") else 0)}
    n = case["seqs"] * case["longest"] * (9 / 16 if case["ragged"] else 1)
    if case["window"]:
        n = min(n, case["seqs"] * case["window"])
    io = case["seqs"] * case["heads"] * (2 * D * e + 4)
    return {"bytes": int(n * (2 * H * row) + n / case["page"] * 4 + io), "flops": int(4 * n * case["heads"] * D)}


# ------------------------------------------------------------ in 64 bits

def _exact_turned(x, pos, case):
    """x as complex numbers times exp(i * angle)."""
    rot = case["rot"]
    f, factor = _frequencies(case)
    sign = -1.0 if case.get("back") else 1.0
    turn = torch.polar(torch.full_like(f, factor).expand(pos.numel(), -1).contiguous(), sign * pos.double()[:, None] * f)
    x = x.double()
    pairs = x[..., :rot].unflatten(-1, (rot // 2, 2)) if case["inter"] else x[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None])
    z = z.flatten(-2) if case["inter"] else z.transpose(-1, -2).flatten(-2)
    return torch.cat([z, x[..., rot:]], -1)


def _exact_values(x, scale):
    return x.double() if scale is None else x.double() * scale.double().unsqueeze(-1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return [_exact_turned(s[n], s["pos"], case) for n in ("q", "k")]
    pool = s["pool"]
    if case["op"] == "attn":
        out = torch.zeros(case["seqs"], case["heads"], case["dim"], dtype=torch.float64, device="cuda")
        lse = torch.full(out.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
        for b, n in enumerate(s["lens"].tolist()):
            first = max(0, n - case["window"]) if case["window"] else 0
            if n == 0:
                continue
            t = torch.arange(first, n, device="cuda")
            page, row = s["table"][b].long()[t // case["page"]], t % case["page"]
            group = case["heads"] // case["kv_heads"]
            for h in range(case["kv_heads"]):
                K, V = (_exact_values(pool[m].view(I8)[page, h, row].view(pool[m].dtype) if case["kind"] == "e4m3" else pool[m][page, h, row],
                                      None if pool[m + "_scale"] is None else pool[m + "_scale"][page, h, row]) for m in ("k", "v"))
                a = s["q"][b, h * group:(h + 1) * group].double() @ K.T * case["dim"] ** -0.5
                lse[b, h * group:(h + 1) * group] = a.logsumexp(-1)
                out[b, h * group:(h + 1) * group] = a.softmax(-1) @ V
        return [out, lse]
    n = case["tokens"] - case.get("pad", 0)
    seq, pos = s["seq"][:n].long(), s["pos"][:n].long()
    page, row = s["table"][seq, pos // case["page"]].long(), pos % case["page"]
    if case["op"] == "read":
        return [_exact_values(pool[m].double()[page, :, row], None if pool[m + "_scale"] is None else pool[m + "_scale"][page, :, row])
                for m in ("k", "v")]
    k, v = s["k"][:n].double(), s["v"][:n].double()
    q = []
    if case["rot"]:
        k, q = _exact_turned(k, pos, case), [_exact_turned(s["q"], s["pos"], case)]
    if case["kind"] not in _TOP:
        wide = [pool["k"].double(), pool["v"].double()]
        wide[0][page, :, row], wide[1][page, :, row] = k, v
        return wide + q
    codes, scales = [], []
    for m, x in (("k", k), ("v", v)):
        scale = x.abs().amax(-1) / _TOP[case["kind"]]
        code, all_scales = pool[m].double(), pool[m + "_scale"].double()
        code[page, :, row], all_scales[page, :, row] = x / scale.unsqueeze(-1), scale
        codes.append(code if case["kind"] == "e4m3" else None)
        scales.append(all_scales)
    return codes + q + scales
