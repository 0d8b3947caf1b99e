"""The operators of a speculative decoding step over the KV cache, as measurable cases.

A step drafts a tree of tokens, rotates their queries and keys to the positions of their depth (rope), writes their
keys and values into the cache in its own type (kv_write), attends from every node to the cached past, its ancestors
and itself (attn), and, when a branch is accepted, reads its slots back to move them (kv_read; the same call hands a
quantized cache to code that wants fp32 rows).

``own`` selects the library's kernels; otherwise the operators are computed in their plain form with elementary torch
operations.  Shapes are those of the synthetic models (synth/configs.py).
"""
import math

import torch

own = False

KV_TYPES = ("f32", "f16", "q8_0", "q4_0")
MASK_BYTES = 4
WORKSPACE = 128 << 20  # bytes of scratch a program keeps for its attention calls


def listed():
    return [
        # a 16-node draft of the 8B shape: the q and k heads of the fused projection's rows
        dict(name="rope tree 16x40x128 f32", op="rope", rows=16, heads=40, head_dim=128, rot_dim=128, layout="interleaved",
             dtype="f32", scaling="none", factor=1.0, native_ctx=8192, base=500000.0, pos=4096, spread="tree"),
        # a context shift: the cached fp16 keys of 30720 slots x 8 heads move 512 positions back, scaled long context
        dict(name="rope shift 245760x1x128 f16", op="rope", rows=245760, heads=1, head_dim=128, rot_dim=96, layout="half",
             dtype="f16", scaling="yarn", factor=4.0, native_ctx=8192, base=500000.0, pos=-512, spread="same"),
        # the keys and values of a 16-node draft into free slots, read back as the next layer sees them
        dict(name="write 16 q8_0", op="kv_write", rows=16, kv_heads=8, head_dim=128, kv_dtype="q8_0", ctx=8192,
             slots="list", slot=0),
        # a prompt of the 8B shape written in one go
        dict(name="write 4096 q4_0", op="kv_write", rows=4096, kv_heads=8, head_dim=128, kv_dtype="q4_0", ctx=8192,
             slots="run", slot=37),
        # an accepted branch of a draft read back to be moved (1B shape, odd count)
        dict(name="read 21 q4_0 d64", op="kv_read", rows=21, kv_heads=8, head_dim=64, kv_dtype="q4_0", ctx=4096,
             slots="list", slot=0),
        # a long quantized context handed over as fp32 rows
        dict(name="read 30720 q8_0", op="kv_read", rows=30720, kv_heads=8, head_dim=128, kv_dtype="q8_0", ctx=32768,
             slots="run", slot=0),
        # the smallest call: one token of the tiny decoder
        dict(name="attn 1 tiny f32", op="attn", n=1, heads=8, kv_heads=4, head_dim=64, kv_dtype="f32", ctx=64, past=31,
             mask="kept"),
        # a 16-node draft of the 1B shape after a 1024-token prompt, the mask built from the parents in the same pass
        dict(name="attn 16 1b f16", op="attn", n=16, heads=32, kv_heads=8, head_dim=64, kv_dtype="f16", ctx=4096,
             past=1024, mask="built"),
        # a 64-node draft of the 8B shape after a 4096-token prompt (the mask is kept for all layers)
        dict(name="attn 64 8b f16", op="attn", n=64, heads=32, kv_heads=8, head_dim=128, kv_dtype="f16", ctx=8192,
             past=4096, mask="kept"),
        # an odd draft over a long Q8_0 context
        dict(name="attn 25 8b q8_0 long", op="attn", n=25, heads=32, kv_heads=8, head_dim=128, kv_dtype="q8_0", ctx=32768,
             past=30011, mask="built"),
        # a chain of 4 drafted tokens over a long Q4_0 context
        dict(name="attn 4 8b q4_0 long", op="attn", n=4, heads=32, kv_heads=8, head_dim=128, kv_dtype="q4_0", ctx=32768,
             past=30720, mask="kept"),
        # the largest: a 64-node draft over the long fp32 cache
        dict(name="attn 64 8b f32 long", op="attn", n=64, heads=32, kv_heads=8, head_dim=128, kv_dtype="f32", ctx=32768,
             past=30720, mask="kept"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "kv_write", "kv_read", "attn", "attn"))
    if op == "rope":
        heads = rng.choice((1, 3, 8, 36, 40, 48, 96))
        head_dim = rng.choice((64, 80, 96, 128, 256))
        rot_dim = rng.choice((head_dim, head_dim, 2 * rng.randint(1, head_dim // 2)))
        rows = _log(rng, 1, max(1, min(16384, (30 << 20) // (heads * head_dim))))
        scaling = rng.choice(("none", "linear", "ntk", "yarn"))
        if scaling == "ntk" and rot_dim < 4:
            scaling = "linear"
        return dict(op="rope", rows=rows, heads=heads, head_dim=head_dim, rot_dim=rot_dim,
                    layout=rng.choice(("interleaved", "half")), dtype=rng.choice(("f32", "f16")), scaling=scaling,
                    factor=round(rng.uniform(1.0, 16.0), 3), native_ctx=rng.choice((2048, 4096, 8192)),
                    base=rng.choice((10000.0, 500000.0)), pos=rng.choice((-1, 1)) * _log(rng, 1, 1 << 20),
                    spread=rng.choice(("tree", "run", "same")))
    head_dim = rng.choice((64, 128))
    kv_heads = rng.choice((1, 2, 4, 8, 8, 8, 5))
    kv_dtype = rng.choice(KV_TYPES)
    if op in ("kv_write", "kv_read"):
        rows = _log(rng, 1, 8192)
        ctx = rows + rng.randint(0, 4096)
        slots = rng.choice(("run", "list"))
        return dict(op=op, rows=rows, kv_heads=kv_heads, head_dim=head_dim, kv_dtype=kv_dtype, ctx=ctx, slots=slots,
                    slot=rng.randint(0, ctx - rows) if slots == "run" else 0)
    group = rng.choice((1, 2, 4, 4, 4, 8, 3))
    n = _log(rng, 1, 256)
    most = 64 * 32 * 30784 * 128 // (n * group * kv_heads * head_dim)  # the largest listed case's products
    past = _log(rng, 1, max(1, min(32000, most - n))) - rng.choice((0, 0, 0, 1))
    return dict(op="attn", n=n, heads=group * kv_heads, kv_heads=kv_heads, head_dim=head_dim, kv_dtype=kv_dtype,
                ctx=past + n + rng.randint(0, 300), past=past, mask=rng.choice(("kept", "built")))


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _code_bytes(kv_dtype, head_dim):
    return head_dim if kv_dtype == "q8_0" else head_dim // 2


def _cache(case, g, fill):
    """One layer's cache: k, v (values or codes) and, for the quantized types, their fp16 scales per 32 values.
    fill: random contents (keys with the uneven channels that trained models have), else zeros."""
    kvh, ctx, d, t = case["kv_heads"], case["ctx"], case["head_dim"], case["kv_dtype"]
    if t in ("f32", "f16"):
        dt = torch.float32 if t == "f32" else torch.float16
        if not fill:
            return [torch.zeros(kvh, ctx, d, device="cuda", dtype=dt) for _ in range(2)] + [None, None]
        ch = torch.exp(0.5 * _normal(g, kvh, 1, d))
        return [(_normal(g, kvh, ctx, d) * ch).to(dt), _normal(g, kvh, ctx, d).to(dt), None, None]
    cb = _code_bytes(t, d)
    if not fill:
        return [torch.zeros(kvh, ctx, cb, device="cuda", dtype=torch.uint8) for _ in range(2)] + \
               [torch.zeros(kvh, ctx, d // 32, device="cuda", dtype=torch.float16) for _ in range(2)]
    got = []
    for _ in range(2):
        if t == "q8_0":
            q = (_normal(g, kvh, ctx, cb) * 42).round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
        else:
            q = torch.randint(0, 256, (kvh, ctx, cb), generator=g, device="cuda", dtype=torch.uint8)
        got.append(q)
    for k in range(2):
        s = torch.exp(0.3 * _normal(g, kvh, ctx, d // 32)) * (1 / 42 if t == "q8_0" else 0.2)
        got.append((s if t == "q8_0" else s * torch.sign(_normal(g, kvh, ctx, d // 32) + 1e-9)).to(torch.float16))
    return got


def _slots(case, g):
    """Distinct slots in no order; one in eight rows of a longer list is padding (-1)."""
    if case["slots"] == "run":
        return None
    s = torch.randperm(case["ctx"], generator=g, device="cuda")[: case["rows"]].to(torch.int32)
    if case["rows"] >= 8:
        s[torch.randperm(case["rows"], generator=g, device="cuda")[: case["rows"] // 8]] = -1
    return s


def _parents(n, g):
    """A draft tree: a node's parent is -1 (the last accepted token) or an earlier node, mostly a recent one."""
    back = (torch.rand(n, generator=g, device="cuda") ** 2 * 8).long() + 1
    return (torch.arange(n, device="cuda") - back).clamp_(min=-1).to(torch.int32)


def _ancestors(parent):
    """[n, n] bool: node i sees node j (an ancestor, or itself), and each node's depth."""
    n = parent.numel()
    i = torch.arange(n, device=parent.device)
    see = (i[None, :] == i[:, None]) | (i[None, :] == parent[:, None])
    for _ in range(max(1, (n - 1).bit_length())):  # doubles the generations that are seen
        see = (see.float() @ see.float()) > 0.5
    return see, see.sum(1) - 1


def _pack(see):
    """Bits of [n, n] as int32 words [n, (n + 31) / 32]: bit j % 32 of word j / 32."""
    n = see.shape[0]
    w = (n + 31) // 32
    bits = torch.zeros(n, w * 32, dtype=torch.int64, device=see.device)
    bits[:, :n] = see
    words = (bits.view(n, w, 32) << torch.arange(32, device=see.device)).sum(-1)
    return words.to(torch.int32)  # keeps the low 32 bits


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "rope":
        rows, dt = case["rows"], torch.float32 if case["dtype"] == "f32" else torch.float16
        s["x"] = _normal(g, rows, case["heads"] * case["head_dim"]).to(dt)
        s["out"] = torch.empty_like(s["x"])
        if case["spread"] == "same":
            s["pos"] = torch.full((rows,), case["pos"], dtype=torch.int32, device="cuda")
        elif case["spread"] == "run":
            s["pos"] = None
        else:
            s["pos"] = (case["pos"] + torch.randint(0, 12, (rows,), generator=g, device="cuda")).to(torch.int32)
    elif case["op"] == "attn":
        n, d = case["n"], case["head_dim"]
        # q as it lies in the rows of the fused q | k | v projection
        s["rows"] = _normal(g, n, (case["heads"] + 2 * case["kv_heads"]) * d)
        s["cache"] = _cache(case, g, True)
        s["parent"] = _parents(n, g)
        see, depth = _ancestors(s["parent"])
        s["mask"], s["pos"] = _pack(see), (depth + case["past"]).to(torch.int32)
        s["out"] = torch.empty(n, case["heads"] * d, device="cuda")
        s["ws"] = torch.empty(WORKSPACE, dtype=torch.uint8, device="cuda")
    else:
        w = case["kv_heads"] * case["head_dim"]
        s["slots"] = _slots(case, g)
        s["cache"] = _cache(case, g, case["op"] == "kv_read")
        if case["op"] == "kv_write":
            s["k"], s["v"] = _normal(g, case["rows"], w), _normal(g, case["rows"], w)
        s["k_out"] = torch.zeros(case["rows"], w, device="cuda")
        s["v_out"] = torch.zeros(case["rows"], w, device="cuda")
    return s


# ---------------------------------------------------------------- plain forms

def _inv_freq(case, dtype=torch.float64):
    """Angle per position of each pair, in 64 bits."""
    r, s, base = case["rot_dim"], case["factor"], case["base"]
    if case["scaling"] == "ntk":
        base = base * s ** (r / (r - 2))
    f = base ** (-torch.arange(0, r, 2, device="cuda", dtype=dtype) / r)
    if case["scaling"] == "linear":
        f = f / s
    if case["scaling"] == "yarn":
        turns = case["native_ctx"] * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        f = (1 - keep) * f / s + keep * f
    return f


def _magnitude(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "yarn" else 1.0


def _positions(s):
    c = s["case"]
    return c["pos"] + torch.arange(c["rows"], device="cuda") if s["pos"] is None else s["pos"]


def _rope_plain(s):
    c = s["case"]
    rows, heads, d, r = c["rows"], c["heads"], c["head_dim"], c["rot_dim"]
    angle = _positions(s).double()[:, None] * _inv_freq(c)
    cos = (torch.cos(angle) * _magnitude(c)).float()[:, None, :]
    sin = (torch.sin(angle) * _magnitude(c)).float()[:, None, :]
    x = s["x"].view(rows, heads, d).float()
    out = x.clone()
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if c["layout"] == "interleaved" else (x[..., : r // 2], x[..., r // 2: r])
    ra, rb = a * cos - b * sin, a * sin + b * cos
    if c["layout"] == "interleaved":
        out[..., 0:r:2], out[..., 1:r:2] = ra, rb
    else:
        out[..., : r // 2], out[..., r // 2: r] = ra, rb
    return out.view(rows, heads * d).to(s["x"].dtype)


def _quantize(x, kv_dtype):
    """Codes (bytes) and fp16 scales of [..., d] fp32 values; borders are decided in 64 bits."""
    b = x.double().unflatten(-1, (-1, 32))
    if kv_dtype == "q8_0":
        scale = (b.abs().amax(-1) / 127).float().half()
        d = scale.double()[..., None]
        t = b / torch.where(d == 0, 1.0, d)
        q = torch.sign(t) * torch.floor(t.abs() + 0.5)
        q = torch.where(d == 0, 0.0, q.clamp(-127, 127))
        return q.flatten(-2).to(torch.int8).view(torch.uint8), scale
    m = b.gather(-1, b.abs().argmax(-1, keepdim=True))[..., 0]
    scale = (m / -8).float().half()
    d = scale.double()[..., None]
    n = torch.floor(b / torch.where(d == 0, 1.0, d) + 8.5).clamp(0, 15)
    n = torch.where(d == 0, 8.0, n).flatten(-2).to(torch.uint8)
    return n[..., 0::2] | n[..., 1::2] << 4, scale


def _values(codes, scales, kv_dtype):
    """fp32 values of cache rows [..., d]."""
    if kv_dtype in ("f32", "f16"):
        return codes.float()
    if kv_dtype == "q8_0":
        q = codes.view(torch.int8).float()
    else:
        q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float() - 8
    return (q.unflatten(-1, (-1, 32)) * scales.float()[..., None]).flatten(-2)


def _rows_and_slots(s):
    c = s["case"]
    if s["slots"] is None:
        return slice(None), torch.arange(c["slot"], c["slot"] + c["rows"], device="cuda")
    rows = torch.nonzero(s["slots"] >= 0)[:, 0]
    return rows, s["slots"][rows].long()


def _kv_plain(s):
    c = s["case"]
    t, kvh, d = c["kv_dtype"], c["kv_heads"], c["head_dim"]
    rows, slots = _rows_and_slots(s)
    outs = []
    for i, name in enumerate(("k", "v")):
        data, scales = s["cache"][i], s["cache"][2 + i]
        if c["op"] == "kv_write":
            x = s[name].view(-1, kvh, d)[rows].transpose(0, 1)
            if t in ("f32", "f16"):
                data[:, slots] = x.to(data.dtype)
            else:
                data[:, slots], scales[:, slots] = _quantize(x, t)
        got = _values(data[:, slots], None if scales is None else scales[:, slots], t)
        out = torch.zeros_like(s[name + "_out"])
        out[rows] = got.transpose(0, 1).flatten(1)
        outs.append(out)
    return outs


def _attn_plain(s):
    c = s["case"]
    n, h, kvh, d, past, t = c["n"], c["heads"], c["kv_heads"], c["head_dim"], c["past"], c["kv_dtype"]
    outs = []
    if c["mask"] == "built":
        see, depth = _ancestors(s["parent"])
        outs = [_pack(see), (depth + past).to(torch.int32)]
    else:
        j = torch.arange(n, device="cuda")
        see = (s["mask"][:, j // 32] >> (j % 32)) & 1 == 1
    k, v = (_values(s["cache"][i][:, : past + n], None if s["cache"][2 + i] is None else s["cache"][2 + i][:, : past + n], t)
            for i in (0, 1))
    q = s["rows"][:, : h * d].reshape(n, kvh, h // kvh, d).permute(1, 2, 0, 3).reshape(kvh, -1, d)
    score = (q @ k.transpose(1, 2)) / math.sqrt(d)
    score = score.view(kvh, h // kvh, n, past + n)
    score[..., past:].masked_fill_(~see, -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    p = (p / p.sum(-1, keepdim=True)).view(kvh, -1, past + n)
    out = (p @ v).view(kvh, h // kvh, n, d).permute(2, 0, 1, 3).reshape(n, h * d)
    return [out] + outs


# ---------------------------------------------------------------- one pass

def _run_own(s):
    import gguf_quantized_transformer_gb300 as af
    c = s["case"]
    if c["op"] == "rope":
        if "cfg" not in s:
            s["cfg"] = af.rope_config(c["head_dim"], c["rot_dim"], c["layout"], c["base"], c["scaling"], c["factor"],
                                      c["native_ctx"], magnitude=_magnitude(c))
        w = c["heads"] * c["head_dim"]
        af.af_rope(s["cfg"], s["x"], w, s["out"], w, af.AF_F32 if c["dtype"] == "f32" else af.AF_F16, c["rows"],
                   c["heads"], s["pos"], c["pos"])
        return [s["out"]]
    t = af.KVTYPE[c["kv_dtype"]]
    k, v, ks, vs = s["cache"]
    if c["op"] == "attn":
        n, h, kvh, d = c["n"], c["heads"], c["kv_heads"], c["head_dim"]
        if c["mask"] == "built":
            af.af_tree_mask(s["parent"], n, c["past"], s["mask"], s["pos"])
        af.af_attention_tree(s["rows"], (h + 2 * kvh) * d, k, ks, v, vs, t, h, kvh, d, c["ctx"], c["past"], n, s["mask"],
                             s["ws"], WORKSPACE, s["out"], h * d)
        return [s["out"]] + ([s["mask"], s["pos"]] if c["mask"] == "built" else [])
    w = c["kv_heads"] * c["head_dim"]
    if c["op"] == "kv_write":
        af.af_kv_write(s["k"], s["v"], w, c["rows"], s["slots"], c["slot"], k, ks, v, vs, t, c["kv_heads"],
                       c["head_dim"], c["ctx"])
    af.af_kv_read(k, ks, v, vs, t, c["kv_heads"], c["head_dim"], c["ctx"], c["rows"], s["slots"], c["slot"], s["k_out"],
                  s["v_out"], w)
    return [s["k_out"], s["v_out"]]


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "rope":
        return [_rope_plain(state)]
    return _attn_plain(state) if op == "attn" else _kv_plain(state)


# ---------------------------------------------------------------- what a pass cannot do without

def _row_bytes(case):
    """Bytes of one slot of one kv head, K and V."""
    d = case["head_dim"]
    per = {"f32": 4 * d, "f16": 2 * d, "q8_0": d + d // 16, "q4_0": d // 2 + d // 16}[case["kv_dtype"]]
    return 2 * per


def work(case):
    if case["op"] == "rope":
        n = case["rows"] * case["heads"] * case["head_dim"]
        rot = case["rows"] * case["heads"] * case["rot_dim"]
        return {"bytes": 2 * n * (4 if case["dtype"] == "f32" else 2) + 4 * case["rows"], "flops": 3 * rot}
    kvh, d = case["kv_heads"], case["head_dim"]
    if case["op"] == "attn":
        n, h, past = case["n"], case["heads"], case["past"]
        return {"bytes": 2 * 4 * n * h * d + (past + n) * kvh * _row_bytes(case) + n * ((n + 31) // 32) * MASK_BYTES,
                "flops": 4 * n * h * d * (past + 1)}
    cells = case["rows"] * kvh
    fp32 = 2 * 4 * cells * d
    if case["op"] == "kv_write":  # rows in, cache rows out, rows back
        return {"bytes": 2 * fp32 + cells * _row_bytes(case), "flops": 8 * cells * d}
    return {"bytes": fp32 + cells * _row_bytes(case), "flops": 2 * cells * d}


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_rope(s):
    c = s["case"]
    d, r = c["head_dim"], c["rot_dim"]
    pos = _positions(s).double()
    x = s["x"].double().view(c["rows"], c["heads"], d).clone()
    y = x.clone()
    mag = 1.0
    for i in range(r // 2):
        f = math.pow(c["base"], -2.0 * i / r)
        if c["scaling"] == "linear":
            f /= c["factor"]
        elif c["scaling"] == "ntk":
            f = math.pow(c["base"] * math.pow(c["factor"], r / (r - 2.0)), -2.0 * i / r)
        elif c["scaling"] == "yarn":
            wave = 2 * math.pi / f
            g = min(1.0, max(0.0, (c["native_ctx"] / wave - 1.0) / 31.0))
            f = f * (g + (1 - g) / c["factor"])
            mag = 1.0 + 0.1 * math.log(c["factor"])
        a, b = (2 * i, 2 * i + 1) if c["layout"] == "interleaved" else (i, i + r // 2)
        z = torch.polar(torch.full_like(pos, mag), pos * f)[:, None] * torch.complex(x[..., a], x[..., b])
        y[..., a], y[..., b] = z.real, z.imag
    return [y.view(c["rows"], -1)]


def _exact_cells(data, scales, kv_dtype):
    """float64 values of cache rows, head by head elements in order."""
    if kv_dtype in ("f32", "f16"):
        return data.double()
    u = data.to(torch.int64)
    if kv_dtype == "q8_0":
        q = u - 256 * (u > 127)
    else:
        q = torch.empty(*u.shape[:-1], 2 * u.shape[-1], dtype=torch.int64, device=u.device)
        q[..., 0::2], q[..., 1::2] = u % 16 - 8, u // 16 - 8
    return q.double() * scales.double().repeat_interleave(32, -1)


def _exact_written(x, kv_dtype):
    """What a cache of this type holds of [..., d] fp32 values."""
    if kv_dtype == "f32":
        return x.double()
    if kv_dtype == "f16":
        return x.half().double()
    y = x.double().reshape(*x.shape[:-1], -1, 32)
    if kv_dtype == "q8_0":
        d = (y.abs().max(-1, keepdim=True).values / 127.0).float().half().double()
        lo, hi, off = -127, 127, 0.0
    else:
        big, small = y.max(-1, keepdim=True).values, y.min(-1, keepdim=True).values
        d = (torch.where(big >= -small, big, small) / -8.0).float().half().double()
        lo, hi, off = -8, 7, 0.5
    t = y / d
    q = torch.floor(t + 0.5) if off else torch.where(t >= 0, torch.floor(t + 0.5), torch.ceil(t - 0.5))
    q = torch.where(d == 0, torch.zeros_like(q), q.clamp(lo, hi))
    return (q * d).reshape(x.shape)


def _exact_kv(s):
    c = s["case"]
    kvh, d, rows = c["kv_heads"], c["head_dim"], c["rows"]
    slots = torch.arange(rows, device="cuda") + c["slot"] if s["slots"] is None else s["slots"].long()
    live = slots >= 0
    outs = []
    for i, name in enumerate(("k", "v")):
        if c["op"] == "kv_write":
            y = _exact_written(s[name].view(rows, kvh, d), c["kv_dtype"])
        else:
            at = slots.clamp(min=0)
            sc = None if s["cache"][2 + i] is None else s["cache"][2 + i][:, at]
            y = _exact_cells(s["cache"][i][:, at], sc, c["kv_dtype"]).permute(1, 0, 2)
        outs.append((y * live[:, None, None]).reshape(rows, kvh * d))
    return outs


def _exact_attn(s):
    c = s["case"]
    n, h, kvh, d, past = c["n"], c["heads"], c["kv_heads"], c["head_dim"], c["past"]
    parent = s["parent"].tolist()
    see = torch.zeros(n, n, dtype=torch.bool)
    for i, p in enumerate(parent):
        if p >= 0:
            see[i] = see[p]
        see[i, i] = True
    seen = torch.cat((torch.ones(n, past, dtype=torch.bool), see), 1).cuda()
    out = torch.empty(n, h, d, dtype=torch.float64, device="cuda")
    for g in range(kvh):
        k, v = (_exact_cells(s["cache"][i][g, : past + n],
                             None if s["cache"][2 + i] is None else s["cache"][2 + i][g, : past + n], c["kv_dtype"])
                for i in (0, 1))
        for j in range(g * (h // kvh), (g + 1) * (h // kvh)):
            z = s["rows"][:, j * d:(j + 1) * d].double() @ k.T * d ** -0.5
            out[:, j] = torch.softmax(torch.where(seen, z, -math.inf), -1) @ v
    # the mask words and positions are whole numbers, compared as they are
    return [out.reshape(n, h * d)] + ([None, None] if c["mask"] == "built" else [])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s)
    return _exact_attn(s) if case["op"] == "attn" else _exact_kv(s)
