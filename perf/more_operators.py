"""The operators of a serving step for many requests over one paged KV cache, as measurable cases.

A paged cache is the cache that rows are written to (kv_write), with n_pages * page_size slots: a request's tokens lie in
the pages that its row of the block table names.  A step maps the new tokens of all requests to slots and takes their
pages (pages), and in every layer adds each request's low-rank adapter to the shared projections (lora) and attends
from each new token to its own request's tokens (attn).

``own`` selects the library's kernels; otherwise the operators are computed in their plain form with elementary torch
operations.  Shapes are those of the synthetic models (synth/configs.py).
"""
import math

import numpy as np
import torch

own = False

KV_TYPES = ("f32", "f16", "q8_0", "q4_0")
GOLDEN = 0.6180339887498949  # lengths follow its multiples modulo 1: evenly spread, in no order, the same for every seed


def listed():
    return [
        # one decode step of a serving loop: every request gets a token, a few end and give back their pages
        dict(name="pages step 256", op="pages", n=256, page=16, lo=1, hi=8000, width=513, kind="step", short=0),
        # prompts of the long-context model join: tokens of 24 requests, and one each for 100 that run
        dict(name="pages prompts 24+100", op="pages", n=124, page=64, lo=1, hi=30720, width=512, kind="prompts", short=0),
        # the smallest call: one token of the tiny decoder
        dict(name="attn 1 tiny f32", op="attn", n=1, heads=8, kv_heads=4, head_dim=64, kv_dtype="f32", page=16, lo=31, hi=31,
             rows="all"),
        # 16 requests of the 1B shape, short conversations
        dict(name="attn 16 1b f16", op="attn", n=16, heads=32, kv_heads=8, head_dim=64, kv_dtype="f16", page=16, lo=20,
             hi=2000, rows="all"),
        # 64 requests of the 8B shape, all lengths up to its context
        dict(name="attn 64 8b f16", op="attn", n=64, heads=32, kv_heads=8, head_dim=128, kv_dtype="f16", page=64, lo=1, hi=8192,
             rows="all"),
        # a batch padded to a fixed number of rows over a Q8_0 cache, pages of an odd size
        dict(name="attn 96 8b q8_0", op="attn", n=96, heads=32, kv_heads=8, head_dim=128, kv_dtype="q8_0", page=24, lo=100,
             hi=8000, rows="listed"),
        # one request over a long Q4_0 context: its cache is split over the whole GPU
        dict(name="attn 1 8b q4_0 long", op="attn", n=1, heads=32, kv_heads=8, head_dim=128, kv_dtype="q4_0", page=16, lo=30720,
             hi=30720, rows="all"),
        # the largest: eight long contexts over an fp32 cache
        dict(name="attn 8 8b f32 long", op="attn", n=8, heads=32, kv_heads=8, head_dim=128, kv_dtype="f32", page=128, lo=16384,
             hi=30720, rows="all"),
        # one request's token beside the O projection of the 8B shape
        dict(name="lora 1 r16 4096x4096", op="lora", n=1, used=1, adapters=4, rank=16, K=4096, N=4096, dtype="f16", ranks="full",
             order="mixed", bare=0, plan="kept"),
        # a decode batch beside the fused q | k | v projection: most rows have an adapter of their own, some have none
        dict(name="lora 64 of 40 r16 4096x6144", op="lora", n=64, used=40, adapters=48, rank=16, K=4096, N=6144, dtype="f16",
             ranks="full", order="mixed", bare=9, plan="built"),
        # the down projection, fp32 adapters of several ranks
        dict(name="lora 40 of 12 r64 14336x4096 f32", op="lora", n=40, used=12, adapters=16, rank=64, K=14336, N=4096, dtype="f32",
             ranks="mixed", order="mixed", bare=0, plan="kept"),
        # prompts of five requests beside the gate | up projection
        dict(name="lora 2048 of 5 r32 4096x28672", op="lora", n=2048, used=5, adapters=8, rank=32, K=4096, N=28672, dtype="f16",
             ranks="full", order="grouped", bare=0, plan="kept"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("pages", "attn", "attn", "attn", "lora", "lora"))
    if op == "pages":
        page = rng.choice((1, 8, 16, 16, 24, 32, 64, 128))
        hi = _log(rng, 16, 30720)
        n = _log(rng, 1, max(1, min(1024, 400000 // hi)))
        return dict(op=op, n=n, page=page, lo=1, hi=hi, width=(hi + 600 + page - 1) // page, kind=rng.choice(("step", "prompts", "mixed")),
                    short=rng.choice((0, 0, 1)))
    if op == "attn":
        head_dim = rng.choice((64, 128))
        kv_heads = rng.choice((1, 2, 4, 8, 8, 8, 5))
        kv_dtype = rng.choice(KV_TYPES)
        n = _log(rng, 1, 256)
        most = 8 * 30720 * 8 * 128 // (n * kv_heads * head_dim)  # values of the largest listed case's padded cache
        hi = _log(rng, 1, max(1, min(32000, most)))
        return dict(op=op, n=n, heads=kv_heads * rng.choice((1, 2, 4, 4, 4, 8, 3, 5)), kv_heads=kv_heads, head_dim=head_dim,
                    kv_dtype=kv_dtype, page=rng.choice((1, 8, 16, 16, 24, 32, 64, 128)), lo=_log(rng, 1, hi), hi=hi,
                    rows=rng.choice(("all", "listed")))
    K = 32 * rng.choice((16, 64, 128, 448, rng.randint(4, 448)))
    N = rng.choice((2048, 4096, 6144, 28672, rng.randint(64, 16384)))
    n = _log(rng, 1, max(1, min(2048, 2048 * 28672 // max(K, N))))
    adapters = _log(rng, 1, 64)
    rank = 8 * rng.choice((1, 2, 2, 4, 4, 8, 16, rng.randint(1, 16)))
    while adapters > 1 and adapters * rank * (K + N) > 1 << 28:  # a GB of adapters at most
        adapters //= 2
    return dict(op=op, n=n, used=rng.randint(1, min(n, adapters)), adapters=adapters, rank=rank, K=K, N=N,
                dtype=rng.choice(("f16", "f16", "f32")), ranks=rng.choice(("full", "mixed")), order=rng.choice(("mixed", "grouped")),
                bare=rng.choice((0, 0, 3, 9)), plan=rng.choice(("kept", "built")))


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _perm(g, n):
    return torch.randperm(n, generator=g, device="cuda")


def _spread(n, lo, hi):
    """n whole numbers of lo..hi, evenly spread, the same for every seed."""
    return lo + np.floor((hi - lo + 1) * np.modf((np.arange(n) + 1) * GOLDEN)[0]).astype(np.int64)


def _up(a, b):
    return -(-a // b)


def _requests(case):
    """Cached and new tokens of each request; -1 new tokens: it has ended."""
    n, lo, hi = case["n"], case["lo"], case["hi"]
    ln, new = _spread(n, lo, hi), np.ones(n, np.int64)
    i = np.arange(n)
    if case["kind"] != "prompts":
        new[i % 16 == 7] = -1
    if case["kind"] == "mixed":
        at = i % 8 == 3
        new[at] = np.minimum(ln[at], 512)
    elif case["kind"] == "prompts":
        at = i % 5 == 0
        ln, new = np.where(at, 0, ln), np.where(at, ln, 1)
    return ln, new


def _rows_of(case):
    """Rows of the padded batch."""
    return int(_up(int(np.maximum(_requests(case)[1], 0).sum()) + 1, 8) * 8)


def _lengths(case):
    """Tokens that each row sees; 0: a row of padding."""
    ln = _spread(case["n"], case["lo"], case["hi"])
    if case["rows"] == "listed":
        ln[np.arange(case["n"]) % 8 == 5] = 0
    return ln


def _cache(case, g, slots):
    """One layer's cache: k, v (values or codes) and, for the quantized types, their fp16 scales per 32 values; keys with
    the uneven channels that trained models have."""
    kvh, d, t = case["kv_heads"], case["head_dim"], case["kv_dtype"]
    if t in ("f32", "f16"):
        dt = torch.float32 if t == "f32" else torch.float16
        ch = torch.exp(0.5 * _normal(g, kvh, 1, d))
        return [_normal(g, kvh, slots, d).mul_(ch).to(dt), _normal(g, kvh, slots, d).to(dt), None, None]
    got = []
    for _ in range(2):
        if t == "q8_0":
            q = _normal(g, kvh, slots, d).mul_(42).round_().clamp_(-127, 127).to(torch.int8).view(torch.uint8)
        else:
            q = torch.randint(0, 256, (kvh, slots, d // 2), generator=g, device="cuda", dtype=torch.uint8)
        got.append(q)
    for _ in range(2):
        s = torch.exp(0.3 * _normal(g, kvh, slots, d // 32)) * (1 / 42 if t == "q8_0" else 0.2)
        got.append((s if t == "q8_0" else s * torch.sign(_normal(g, kvh, slots, d // 32) + 1e-9)).to(torch.float16))
    return got


def _pages_state(case, g):
    n, page, width = case["n"], case["page"], case["width"]
    cached, added = _requests(case)
    order = _perm(g, n)
    ln, new = (torch.from_numpy(a).cuda()[order].to(torch.int32) for a in (cached, added))
    have = _up(ln.long(), page)
    held = int(_up(cached, page).sum())
    wanted = int((_up(cached + np.maximum(added, 0), page) - _up(cached, page)).sum())
    n_pages = held + (wanted // 2 if case["short"] else wanted + 64) + 1
    pages = _perm(g, n_pages).to(torch.int32)
    at = torch.arange(width, device="cuda")
    index = (torch.cumsum(have, 0) - have)[:, None] + at
    table = torch.where(at < have[:, None], pages[index.clamp(max=n_pages - 1)], -1).to(torch.int32)
    count = n_pages - held
    head = int(torch.randint(0, n_pages, (1,), generator=g, device="cuda"))
    free = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda")
    free[(head + torch.arange(count, device="cuda")) % n_pages] = pages[held:]
    rows = _rows_of(case)
    new_i32 = lambda *shape: torch.zeros(*shape, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"len": ln, "new": new, "n_pages": n_pages, "rows": rows, "table": table, "free": free,
            "pool": torch.tensor([head, count, 0, 0], dtype=torch.int32, device="cuda"), "len_out": new_i32(n),
            "pool_out": new_i32(4), "start": new_i32(n + 1), "slots": new_i32(rows), "pos": new_i32(rows), "seq": new_i32(rows),
            "ws": torch.empty(64 * n + 1024, dtype=torch.uint8, device="cuda")}


def _attn_state(case, g):
    n, page, h, kvh, d = case["n"], case["page"], case["heads"], case["kv_heads"], case["head_dim"]
    ln = torch.from_numpy(_lengths(case)).cuda()[_perm(g, n)]
    have = _up(ln, page)
    width = int(_up(case["hi"], page)) + 1
    held = int(_up(_lengths(case), page).sum())
    n_pages = held + 3
    pages = _perm(g, n_pages).to(torch.int32)
    at = torch.arange(width, device="cuda")
    index = (torch.cumsum(have, 0) - have)[:, None] + at
    table = torch.where(at < have[:, None], pages[index.clamp(max=n_pages - 1)], -1).to(torch.int32)
    seq = None
    if case["rows"] == "listed":  # rows in another order than the table's, padding among them
        order = _perm(g, n)
        where = torch.empty_like(order)
        where[order] = torch.arange(n, device="cuda")
        table, seq = table[order].contiguous(), torch.where(ln > 0, where, -1).to(torch.int32)
    # q as it lies in the rows of the fused q | k | v projection
    return {"q": _normal(g, n, (h + 2 * kvh) * d), "cache": _cache(case, g, n_pages * page), "table": table, "seq": seq,
            "pos": (ln - 1).to(torch.int32), "n_pages": n_pages, "width": width, "out": torch.empty(n, h * d, device="cuda"),
            "ws": torch.empty(16 << 20, dtype=torch.uint8, device="cuda")}


def _ids(case):
    """The adapter of each row, counted from 0 in order of first use; -1: none."""
    ids = np.minimum(_spread(case["n"], 0, case["used"] - 1), case["used"] - 1)
    ids[: case["used"]] = np.arange(case["used"])
    if case["order"] == "grouped":
        ids = np.sort(ids)
    if case["bare"]:
        ids[np.arange(case["n"]) % case["bare"] == 2] = -1
    return ids


def _ranks(case):
    """The rank of each adapter."""
    r = case["rank"]
    return np.maximum(1, r - (np.arange(case["adapters"]) % 4) * (r // 4)) if case["ranks"] == "mixed" else np.full(case["adapters"], r)


def _lora_state(case, g):
    n, m, r, K, N = case["n"], case["adapters"], case["rank"], case["K"], case["N"]
    dt = torch.float16 if case["dtype"] == "f16" else torch.float32
    ids = torch.from_numpy(_ids(case)).cuda()
    if case["order"] == "mixed":
        ids = ids[_perm(g, n)]
    s = {"ids": ids.to(torch.int32), "rank": torch.from_numpy(_ranks(case)).cuda().to(torch.int32) if case["ranks"] == "mixed" else None,
         "x": _normal(g, n, K) * torch.exp(0.5 * _normal(g, K)), "base": _normal(g, n, N),
         "a": (_normal(g, m, r, K) * K ** -0.5).to(dt), "b": (_normal(g, m, N, r) * r ** -0.5).to(dt),
         "scale": torch.exp(0.5 * _normal(g, m)), "out": torch.empty(n, N, device="cuda")}
    if own:
        import gguf_quantized_transformer_gb300 as af
        s["plan"] = torch.empty(af.af_lora_plan_bytes(n, m), dtype=torch.uint8, device="cuda")
        s["ws"] = torch.empty(max(256, af.af_lora_workspace(n, m, r, K, N)), dtype=torch.uint8, device="cuda")
        if case["plan"] == "kept":  # made once a step for all of its projections
            af.af_lora_plan(s["ids"], n, m, s["plan"], s["plan"].numel())
    return s


def prepare(case, seed):
    g = _gen(seed)
    make = {"pages": _pages_state, "attn": _attn_state, "lora": _lora_state}[case["op"]]
    return {"case": case, **make(case, g)}


# ---------------------------------------------------------------- plain forms

def _pages_plain(s):
    c = s["case"]
    P, width, n_pages, rows = c["page"], c["width"], s["n_pages"], s["rows"]
    ln, new, table, free = s["len"].long(), s["new"].long(), s["table"], s["free"]
    head, count = s["pool"][0].long(), s["pool"][1].long()
    have, ends, grow = _up(ln, P), new < 0, new.clamp(min=0)
    upto = torch.cumsum(grow, 0)
    start = upto - grow
    fits = ~ends & (upto <= rows) & (ln + grow <= width * P)
    need = torch.where(fits, _up(ln + grow, P) - have, 0)
    taken = torch.cumsum(need, 0)
    served = fits & ((need == 0) | (taken <= count))
    back = torch.where(ends, have, 0)
    returned = torch.cumsum(back, 0)
    # rows
    r = torch.arange(rows, device="cuda")
    i = torch.searchsorted(upto, r, right=True)
    live = i < c["n"]
    i = i.clamp(max=c["n"] - 1)
    live &= served[i]
    pos = ln[i] + r - start[i]
    at = (pos // P).clamp(max=width - 1)
    fresh = at >= have[i]
    page = torch.where(fresh, free[(head + taken[i] - need[i] + at - have[i]) % n_pages], table[i, at]).long()
    slots = torch.where(live, page * P + pos % P, -1).to(torch.int32)
    # pages taken and returned
    first = live & fresh & (pos % P == 0)
    table[i[first], at[first]] = page[first].to(torch.int32)
    who = torch.repeat_interleave(torch.arange(c["n"], device="cuda"), back)
    nth = torch.arange(who.numel(), device="cuda") - (returned - back)[who]
    free[(head + count + (returned - back)[who] + nth) % n_pages] = table[who, nth]
    used = torch.where(served & (need > 0), taken, 0).amax()
    pool = torch.stack(((head + used) % n_pages, count - used + returned[-1], (~ends & ~served).sum(), upto[-1]))
    len_out = torch.where(ends, 0, torch.where(served, ln + grow, ln))
    return [slots, torch.where(live, pos, -1).to(torch.int32), torch.where(live, i, -1).to(torch.int32),
            torch.cat((start, upto[-1:])).to(torch.int32), len_out.to(torch.int32), pool.to(torch.int32), table, free]


def _values(codes, scales, kv_dtype):
    """fp32 values of cache rows [..., d]."""
    if kv_dtype in ("f32", "f16"):
        return codes.float()
    if kv_dtype == "q8_0":
        q = codes.view(torch.int8).float()
    else:
        q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float() - 8
    return (q.unflatten(-1, (-1, 32)) * scales.float()[..., None]).flatten(-2)


def _attn_plain(s):
    c = s["case"]
    n, h, kvh, d, P, t, most = c["n"], c["heads"], c["kv_heads"], c["head_dim"], c["page"], c["kv_dtype"], c["hi"]
    at = torch.arange(most, device="cuda")
    table = s["table"] if s["seq"] is None else s["table"][s["seq"].clamp(min=0).long()]
    slot = (table[:, at // P].long() * P + at % P).clamp(min=0)
    k, v = (_values(s["cache"][i][:, slot], None if s["cache"][2 + i] is None else s["cache"][2 + i][:, slot], t) for i in (0, 1))
    q = s["q"][:, : h * d].reshape(n, kvh, h // kvh, d).transpose(0, 1)
    score = (q @ k.transpose(2, 3)) / math.sqrt(d)
    score = torch.where(at <= s["pos"][:, None, None], score, -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    out = (p / p.sum(-1, keepdim=True)) @ v
    out = torch.where(s["pos"][:, None, None] >= 0, out, 0.0)
    return [out.transpose(0, 1).reshape(n, h * d)]


def _lora_plain(s):
    c = s["case"]
    n, m, r = c["n"], c["adapters"], c["rank"]
    ids, col = s["ids"].long(), torch.arange(m * r, device="cuda")
    rank = torch.full((m,), r, device="cuda") if s["rank"] is None else s["rank"].long()
    mine = (col // r == ids[:, None]) & (col % r < rank.repeat_interleave(r))
    hidden = s["x"] @ s["a"].float().view(m * r, -1).T
    hidden = torch.where(mine, hidden * s["scale"].repeat_interleave(r), 0.0)
    return [s["base"] + hidden @ s["b"].float().transpose(1, 2).reshape(m * r, -1)]


# ---------------------------------------------------------------- one pass

def _run_own(s):
    import gguf_quantized_transformer_gb300 as af
    c = s["case"]
    if c["op"] == "pages":
        af.af_kv_pages(s["len"], s["new"], c["n"], c["page"], s["n_pages"], s["pool"], s["free"], s["table"], c["width"],
                       s["len_out"], s["pool_out"], s["start"], s["slots"], s["pos"], s["seq"], s["rows"], s["ws"], s["ws"].numel())
        return [s["slots"], s["pos"], s["seq"], s["start"], s["len_out"], s["pool_out"], s["table"], s["free"]]
    if c["op"] == "attn":
        h, kvh, d = c["heads"], c["kv_heads"], c["head_dim"]
        k, v, ks, vs = s["cache"]
        af.af_attention_paged(s["q"], (h + 2 * kvh) * d, k, ks, v, vs, af.KVTYPE[c["kv_dtype"]], h, kvh, d, c["page"], s["n_pages"],
                              s["table"], s["width"], c["n"], s["seq"], s["pos"], c["n"], s["ws"], s["ws"].numel(), s["out"], h * d)
        return [s["out"]]
    n, m, K, N = c["n"], c["adapters"], c["K"], c["N"]
    if c["plan"] == "built":
        af.af_lora_plan(s["ids"], n, m, s["plan"], s["plan"].numel())
    af.af_lora(s["x"], K, n, s["plan"], s["a"], s["b"], af.AF_F16 if c["dtype"] == "f16" else af.AF_F32, s["scale"], s["rank"], m,
               c["rank"], K, N, s["base"], N, s["out"], N, s["ws"], s["ws"].numel())
    return [s["out"]]


def run(state):
    if own:
        return _run_own(state)
    return {"pages": _pages_plain, "attn": _attn_plain, "lora": _lora_plain}[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def _row_bytes(case):
    """Bytes of one slot of one kv head, K and V."""
    d = case["head_dim"]
    per = {"f32": 4 * d, "f16": 2 * d, "q8_0": d + d // 16, "q4_0": d // 2 + d // 16}[case["kv_dtype"]]
    return 2 * per


def work(case):
    if case["op"] == "pages":
        ln, new = _requests(case)
        P = case["page"]
        moved = int((_up(ln + np.maximum(new, 0), P) - _up(ln, P)).sum() + _up(ln[new < 0], P).sum())
        return {"bytes": 16 * case["n"] + 12 * _rows_of(case) + 8 * moved, "flops": 0}
    if case["op"] == "attn":
        ln = _lengths(case)
        rows, total, h, kvh, d = int((ln > 0).sum()), int(ln.sum()), case["heads"], case["kv_heads"], case["head_dim"]
        return {"bytes": 4 * (rows + case["n"]) * h * d + total * kvh * _row_bytes(case) + 4 * int(_up(ln, case["page"]).sum()),
                "flops": 4 * total * h * d}
    ids, K, N = _ids(case), case["K"], case["N"]
    r = _ranks(case)[np.where(ids >= 0, ids, 0)] * (ids >= 0)
    size = 2 if case["dtype"] == "f16" else 4
    weights = int(_ranks(case)[np.unique(ids[ids >= 0])].sum()) * (K + N) * size
    return {"bytes": 4 * int((ids >= 0).sum()) * K + 8 * case["n"] * N + weights, "flops": 2 * int(r.sum()) * (K + N)}


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_cells(data, scales, kv_dtype):
    """float64 values of cache rows, elements in order."""
    if kv_dtype in ("f32", "f16"):
        return data.double()
    u = data.to(torch.int64)
    if kv_dtype == "q8_0":
        q = u - 256 * (u > 127)
    else:
        q = torch.empty(*u.shape[:-1], 2 * u.shape[-1], dtype=torch.int64, device=u.device)
        q[..., 0::2], q[..., 1::2] = u % 16 - 8, u // 16 - 8
    return q.double() * scales.double().repeat_interleave(32, -1)


def _exact_attn(s):
    c = s["case"]
    n, h, kvh, d, P = c["n"], c["heads"], c["kv_heads"], c["head_dim"], c["page"]
    out = torch.zeros(n, h, d, dtype=torch.float64, device="cuda")
    for r in range(n):
        upto = int(s["pos"][r]) + 1
        who = r if s["seq"] is None else int(s["seq"][r])
        if upto == 0:
            continue
        pages = s["table"][who, : (upto - 1) // P + 1].long()
        slots = (pages[:, None] * P + torch.arange(P, device="cuda")).flatten()[:upto]
        k, v = (_exact_cells(s["cache"][i][:, slots], None if s["cache"][2 + i] is None else s["cache"][2 + i][:, slots], c["kv_dtype"])
                for i in (0, 1))
        z = torch.einsum("gxd,gld->gxl", s["q"][r, : h * d].double().view(kvh, h // kvh, d), k) * d ** -0.5
        out[r] = torch.einsum("gxl,gld->gxd", torch.softmax(z, -1), v).reshape(h, d)
    return [out.reshape(n, h * d)]


def _exact_lora(s):
    c = s["case"]
    y = s["base"].double()
    for a in torch.unique(s["ids"]).tolist():
        if a < 0:
            continue
        r = c["rank"] if s["rank"] is None else int(s["rank"][a])
        rows = torch.nonzero(s["ids"] == a)[:, 0]
        hidden = torch.einsum("nk,rk->nr", s["x"][rows].double(), s["a"][a, :r].double())
        y[rows] += float(s["scale"][a]) * torch.einsum("nr,mr->nm", hidden, s["b"][a, :, :r].double())
    return [y]


def exact(case, seed):
    if case["op"] == "pages":  # whole numbers, compared as they are
        return None
    s = prepare(case, seed)
    return _exact_attn(s) if case["op"] == "attn" else _exact_lora(s)
