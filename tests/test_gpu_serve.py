"""The operators of a serving step over a paged cache against plain implementations in 64 bits: pages and slots, attention of
single tokens over pages, low-rank adapters, and a run of them together."""
import numpy as np
import pytest

from test_gpu_draft import held, new_cache, read, write

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

KV = ["f32", "f16", "q8_0", "q4_0"]


@pytest.fixture(scope="module")
def af():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gguf_quantized_transformer_gb300 as af
    af.build()
    af.lib()
    return af


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def i32(a):
    return _dev(np.asarray(a, np.int32))


# ---------------------------------------------------------------- pages and slots

def pages_ref(ln, new, P, n_pages, width, pool, free, table, max_rows):
    """One step, request by request."""
    free, table, ln = free.copy(), table.copy(), [int(v) for v in ln]
    head, count = int(pool[0]), int(pool[1])
    head = head if 0 <= head < n_pages else 0
    count = min(max(count, 0), n_pages)
    slots, pos, seq, start = [], [], [], [0]
    rows = taken = wanted = back = returned = refused = 0
    before, out = table.copy(), list(ln)
    for i, x in enumerate(int(v) for v in new):
        sound = 0 <= ln[i] <= width * P
        have = -(-ln[i] // P) if sound else 0
        grow = max(x, 0)
        first, rows = rows, rows + grow
        start.append(min(rows, 2 ** 31 - 1))
        ok = False
        if x < 0:
            back += have
            ok = sound and (have == 0 or count + back <= n_pages)
            if ok:
                out[i] = 0
                for k in range(have):
                    free[(head + count + back - have + k) % n_pages] = before[i, k]
                returned = max(returned, back if have else 0)
        elif sound and rows <= max_rows and ln[i] + grow <= width * P:
            need = -(-(ln[i] + grow) // P) - have
            wanted += need
            if need == 0 or wanted <= count:
                ok = True
                for k in range(need):
                    table[i, have + k] = free[(head + wanted - need + k) % n_pages]
                if need:
                    taken = wanted
                out[i] = ln[i] + grow
        refused += not ok
        for t in range(min(grow, max(0, max_rows - first))):
            p = ln[i] + t
            page = int(table[i, p // P]) if ok else -1
            slots.append(page * P + p % P if 0 <= page < n_pages else -1)
            pos.append(p if ok else -1)
            seq.append(i if ok else -1)
    pad = max_rows - len(slots)
    pool = [(head + taken) % n_pages, count - taken + returned, refused, min(rows, 2 ** 31 - 1)]
    return [np.array(v, np.int32) for v in (slots + [-1] * pad, pos + [-1] * pad, seq + [-1] * pad, start, out, pool, table, free)]


def random_pool(rng, lens, P, width, spare):
    """Tables, ring and pool for requests of these lengths."""
    have = [max(0, min(-(-int(x) // P), width)) for x in lens]
    n_pages = sum(have) + spare
    pages = rng.permutation(n_pages).astype(np.int32)
    table = np.full((len(lens), width), -7, np.int32)
    at = 0
    for i, k in enumerate(have):
        table[i, :k] = pages[at:at + k]
        at += k
    head, free = int(rng.integers(0, n_pages)), np.full(n_pages, -9, np.int32)
    for k in range(n_pages - at):
        free[(head + k) % n_pages] = pages[at + k]
    return n_pages, table, free, np.array([head, n_pages - at, 5, 5], np.int32)


def run_pages(af, ln, new, P, n_pages, width, pool, free, table, max_rows, in_place=False, stream=None):
    n = len(ln)
    d = [i32(v) for v in (ln, new, pool, free, table)]
    ln_out, pool_out = (d[0], d[2]) if in_place else (i32(np.full(n, 77)), i32(np.full(4, 77)))
    start, (slots, pos, seq) = i32(np.full(n + 1, 77)), (i32(np.full(max_rows + 1, 77)) for _ in range(3))
    need = af.af_kv_pages_workspace(n)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    af.af_kv_pages(d[0], d[1], n, P, n_pages, d[2], d[3], d[4], width, ln_out, pool_out, start, slots, pos, seq, max_rows, ws, need,
                   stream)
    got = [t.cpu().numpy() for t in (slots, pos, seq, start, ln_out, pool_out, d[4], d[3])]
    for k in range(3):
        assert got[k][max_rows] == 77  # nothing behind the rows is written
        got[k] = got[k][:max_rows]
    return got


NAMES = ["slots", "pos", "seq", "start", "len", "pool", "table", "free"]


def same(got, want):
    for name, a, b in zip(NAMES, got, want):
        assert np.array_equal(a, b), (name, np.flatnonzero(a.ravel() != b.ravel())[:5], a.ravel()[:8], b.ravel()[:8])


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n,P,longest,most_new,pad", [(1, 16, 0, 1, 0), (1, 1, 5, 1, 3), (7, 16, 60, 1, 1), (33, 24, 300, 40, 9),
                                                      (256, 16, 2000, 1, 8), (1024, 64, 500, 3, 0), (1025, 16, 100, 2, 5),
                                                      (3000, 8, 90, 20, 11), (40, 32, 900, 700, 100), (5, 128, 3000, 9000, 1)])
def test_kv_pages(af, n, P, longest, most_new, pad, in_place):
    rng = np.random.default_rng(n + P)
    ln = rng.integers(0, longest + 1, n)
    ln[::3] -= ln[::3] % P  # whole pages
    new = rng.integers(0, most_new + 1, n)
    new[rng.random(n) < 0.15] = -1
    if n > 4:
        new[2], new[n - 1] = 0, -2 ** 31
    width = (longest + most_new) // P + 2
    wanted = int((-(-(ln + np.maximum(new, 0)) // P) + ln // P).sum())
    n_pages, table, free, pool = random_pool(rng, ln, P, width, wanted + 3)
    rows = int(np.maximum(new, 0).sum()) + pad
    args = (ln, new, P, n_pages, width, pool, free, table, rows)
    want = pages_ref(*args)
    assert want[5][2] == 0
    same(run_pages(af, *args, in_place=in_place), want)


@pytest.mark.parametrize("n,rows_cut", [(40, 0), (40, 33), (1500, 0), (1500, 4000), (3, 10 ** 6)])
def test_kv_pages_refuses_requests(af, n, rows_cut):
    """Too few pages, rows or table entries, lengths that are none, a ring that is full: the request stays as it is."""
    rng = np.random.default_rng(n)
    P, width = 8, 6
    ln = rng.integers(0, width * P + 1, n)
    new = rng.integers(0, 20, n)
    ln[1], ln[2] = -3, width * P + 1
    new[rng.random(n) < 0.2] = -1
    if n > 10:
        ln[5], new[5] = 2 ** 31 - 1, 2 ** 31 - 1
        new[n - 3] = 2 ** 31 - 1
    n_pages, table, free, pool = random_pool(rng, np.clip(ln, 0, width * P), P, width, n // 3 + 1)
    rows = max(0, min(int(np.minimum(np.maximum(new, 0), 50).sum()), 20000) - rows_cut)
    for case in (pool, np.array([pool[0], n_pages, 0, 0], np.int32), np.array([-4, -1, 0, 0], np.int32),
                 np.array([2 ** 31 - 1, 2 ** 31 - 1, 0, 0], np.int32)):
        want = pages_ref(ln, new, P, n_pages, width, case, free, table, rows)
        assert want[5][2] > 0
        same(run_pages(af, ln, new, P, n_pages, width, case, free, table, rows), want)


def test_kv_pages_bad_page_numbers_lead_nowhere(af):
    """Entries of the table and the ring that name no page: their rows' slots are -1."""
    P, width, n_pages = 4, 4, 10
    table = np.array([[3, -1, 99, 0], [2 ** 31 - 1, 5, 5, 5]], np.int32)
    free = np.array([10, -5, 7, 1, 1, 1, 1, 1, 1, 1], np.int32)
    args = (np.array([7, 1]), np.array([5, 6]), P, n_pages, width, np.array([0, 10, 0, 0]), free, table, 12)
    want = pages_ref(*args)
    got = run_pages(af, *args)
    same(got, want)
    assert (got[0] == -1).sum() >= 5 and got[0].max() < n_pages * P


@pytest.mark.parametrize("shift", [0, 1])
def test_kv_pages_of_many_requests_and_unaligned_rows(af, shift):
    """The most requests a call takes, no rows at all, and row arrays that begin at any int."""
    rng = np.random.default_rng(13)
    for n, P, rows in ((65536, 16, 70001), (2049, 8, 3000), (9, 4, 0), (700, 16, 701)):
        ln = rng.integers(0, 40, n)
        new = np.where(rng.random(n) < 0.1, -1, 1) if rows else np.zeros(n, int)
        n_pages, table, free, pool = random_pool(rng, ln, P, 12, n)
        want = pages_ref(ln, new, P, n_pages, 12, pool, free, table, rows)
        d = [i32(v) for v in (ln, new, pool, free, table)]
        start, outs = i32(np.zeros(n + 1)), [i32(np.full(rows + 9, 77)) for _ in range(3)]
        ws = torch.full((af.af_kv_pages_workspace(n),), 0xFF, dtype=torch.uint8, device="cuda")
        af.af_kv_pages(d[0], d[1], n, P, n_pages, d[2], d[3], d[4], 12, d[0], d[2], start, *[t[shift:] for t in outs], rows, ws, ws.numel())
        got = [t.cpu().numpy() for t in outs]
        assert all((g[:shift] == 77).all() and (g[shift + rows:] == 77).all() for g in got)
        same([g[shift:shift + rows] for g in got] + [t.cpu().numpy() for t in (start, d[0], d[2], d[4], d[3])], want)


def test_kv_pages_many_steps(af):
    """A loop that serves requests: pages are never lost, shared or outside the pool; captured once and replayed."""
    rng = np.random.default_rng(3)
    n, P, width, n_pages, rows = 48, 16, 10, 250, 300
    ln, pool, free = i32(np.zeros(n)), i32([13, n_pages, 0, 0]), i32((np.arange(n_pages) - 13) % n_pages)
    table = i32(np.full((n, width), -1))
    new, start, (slots, pos, seq) = i32(np.zeros(n)), i32(np.zeros(n + 1)), (i32(np.zeros(rows)) for _ in range(3))
    need = af.af_kv_pages_workspace(n)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def call():
        af.af_kv_pages(ln, new, n, P, n_pages, pool, free, table, width, ln, pool, start, slots, pos, seq, rows, ws, need)
    host = [np.zeros(n, np.int32), free.cpu().numpy(), table.cpu().numpy(), pool.cpu().numpy()]
    call()  # loads the kernel; no request has new tokens
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for step in range(60):
        x = np.where(host[0] == 0, rng.integers(0, 60, n) * (rng.random(n) < 0.3), 1)
        x[(host[0] > 0) & (rng.random(n) < 0.06)] = -1
        new.copy_(i32(x))
        graph.replay()
        want = pages_ref(host[0], x, P, n_pages, width, host[3], host[1], host[2], rows)
        same([t.cpu().numpy() for t in (slots, pos, seq, start, ln, pool, table, free)], want)
        host = [want[4], want[7], want[6], want[5]]
        used = np.concatenate([host[2][i, : -(-int(host[0][i]) // P)] for i in range(n)])
        ring = host[1][(host[3][0] + np.arange(host[3][1])) % n_pages]
        assert sorted(np.concatenate([used, ring]).tolist()) == list(range(n_pages))


# ---------------------------------------------------------------- attention over pages

def attn_tol(q, k, v):
    """Scores in fp32 or from parts that keep 22 bits: |ds| <= 2^-20 sum |q||k| / sqrt(D); p then moves by ds relative, the
    average of v by at most twice that times max |v|, and the parts of p and v, the exponential and the sums add 2^-19
    max |v|."""
    D = q.shape[-1]
    qa, ka = np.abs(q).max(0).max(0), np.abs(k).max(0).max(0)
    return float(np.abs(v).max() * (2 * 2.0 ** -20 * (qa * ka).sum() / np.sqrt(D) + 2.0 ** -19))


def attn_ref(q, k, v, slots):
    """q [n, H, D], k, v [KVH, slots, D] float64, slots: the slots that each row sees."""
    n, H, D = q.shape
    G = H // k.shape[0]
    out = np.zeros((n, H, D))
    for i in range(n):
        if not len(slots[i]):
            continue
        for g in range(k.shape[0]):
            s = q[i, g * G:(g + 1) * G] @ k[g, slots[i]].T / np.sqrt(D)
            p = np.exp(s - s.max(-1, keepdims=True))
            out[i, g * G:(g + 1) * G] = p @ v[g, slots[i]] / p.sum(-1, keepdims=True)
    return out


def attend(af, t, cache, q, kvh, P, n_pages, table, pos, seq=None, pad=0, stream=None, ws=None, out=None):
    n, H, d = q.shape
    qd = torch.full((n, H * d + pad), float("nan"), device="cuda")
    qd[:, :H * d] = _dev(q.reshape(n, H * d).astype(np.float32))
    out = torch.full((n, H * d + pad), 9.0, device="cuda") if out is None else out
    need = af.af_attention_paged_workspace(H, kvh, d)
    if ws is None:
        ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")  # any contents: NaN patterns
    table, pos, seq = i32(table), i32(pos), None if seq is None else i32(seq)
    af.af_attention_paged(qd, H * d + pad, *cache, af.KVTYPE[t], H, kvh, d, P, n_pages, table, table.shape[1], table.shape[0], seq,
                          pos, n, ws, need, out, H * d + pad, stream)
    return out


class Paged:
    """A paged cache with requests of these lengths: random rows in the slots that hold tokens, NaN patterns in all others."""

    def __init__(self, af, t, rng, kvh, d, P, lens, spare=2, spread=1.0, extra=1):
        self.t, self.kvh, self.d, self.P = t, kvh, d, P
        width = max(1, max(-(-int(x) // P) for x in lens)) + extra
        self.n_pages, self.table, _, _ = random_pool(rng, lens, P, width, spare)
        m = self.n_pages * P
        self.slots = [(self.table[i, np.arange(x) // P] * P + np.arange(x) % P).astype(np.int64) for i, x in enumerate(lens)]
        used = np.concatenate(self.slots).astype(np.int32)
        k = (rng.standard_normal((len(used), kvh * d)) * spread).astype(np.float32)
        v = rng.standard_normal((len(used), kvh * d)).astype(np.float32)
        self.cache = new_cache(t, kvh, m, d, 0xFF)
        if len(used):
            write(af, t, self.cache, _dev(k), _dev(v), kvh, d, m, _dev(used))
        self.k, self.v = np.zeros((kvh, m, d)), np.zeros((kvh, m, d))
        self.k[:, used] = held(k.reshape(-1, kvh, d), t).transpose(1, 0, 2)
        self.v[:, used] = held(v.reshape(-1, kvh, d), t).transpose(1, 0, 2)


ATTN = [  # heads, kv heads, head_dim, page size, lengths
    (8, 4, 64, 16, [31]),
    (4, 4, 128, 16, [1]),
    (32, 8, 128, 16, [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100]),
    (32, 8, 64, 64, [700, 3, 1500, 64]),
    (8, 1, 128, 24, [50, 0, 200, 25, 24]),
    (6, 2, 64, 1, [40, 7, 90]),
    (5, 5, 128, 7, [13, 14, 15, 300]),
    (10, 2, 64, 33, [129, 64]),
    (64, 8, 128, 128, [2000, 1000]),
    (16, 1, 64, 16, [333, 90]),
    (12, 1, 128, 16, [333, 90]),
    (64, 1, 64, 8, [77]),
]


@pytest.mark.parametrize("t", KV)
@pytest.mark.parametrize("H,KVH,D,P,lens", ATTN)
def test_attention_paged(af, t, H, KVH, D, P, lens):
    rng = np.random.default_rng(H * D + P)
    c = Paged(af, t, rng, KVH, D, P, lens)
    q = rng.standard_normal((len(lens), H, D)).astype(np.float32)
    got = attend(af, t, c.cache, q, KVH, P, c.n_pages, c.table, np.array(lens) - 1, pad=8).cpu().numpy()
    assert np.all(got[:, H * D:] == 9.0)
    ref = attn_ref(q.astype(np.float64), c.k, c.v, c.slots)
    err, tol = np.abs(got[:, :H * D].reshape(ref.shape) - ref).max(), attn_tol(q, c.k, c.v)
    print(f"err {err:.2e} tol {tol:.2e} rel {np.linalg.norm(got[:, :H * D].ravel() - ref.ravel()) / np.linalg.norm(ref):.2e}")
    assert err <= tol
    assert not got[[i for i, x in enumerate(lens) if x == 0], :H * D].any()


@pytest.mark.parametrize("t", KV)
@pytest.mark.parametrize("H,D", [(8, 64), (16, 128)])
def test_attention_paged_rows_name_requests(af, t, H, D):
    """Rows in any order, padding, several positions of one request, requests and positions that are none."""
    rng = np.random.default_rng(2)
    P, kvh, lens = 16, 2, [90, 5, 0, 200, 33]
    c = Paged(af, t, rng, kvh, D, P, lens)
    seq = [3, 3, 0, -1, 4, 1, 3, 5, 2, 0, 2 ** 31 - 1, -2 ** 31, 4]
    pos = [199, 120, 89, 10, 0, 4, 199, 3, -1, -1, 5, 5, 32]
    q = rng.standard_normal((len(seq), H, D)).astype(np.float32)
    got = attend(af, t, c.cache, q, kvh, P, c.n_pages, c.table, pos, seq).cpu().numpy().reshape(q.shape)
    slots = [c.slots[s][:p + 1] if 0 <= s < 5 and p >= 0 else [] for s, p in zip(seq, pos)]
    assert np.abs(got - attn_ref(q.astype(np.float64), c.k, c.v, slots)).max() <= attn_tol(q, c.k, c.v)
    assert np.array_equal(got[0] == got[6], q[0] == q[6])  # (other queries, so other results)
    assert not got[[i for i, s in enumerate(slots) if not len(s)]].any()


@pytest.mark.parametrize("t", KV)
def test_attention_paged_hides_bad_pages_and_long_positions(af, t):
    rng = np.random.default_rng(4)
    P, kvh, H, D, lens = 16, 2, 8, 128, [200, 100, 64, 130]
    c = Paged(af, t, rng, kvh, D, P, lens, extra=0)
    table = c.table.copy()
    table[0, [0, 5, 12]] = -1, c.n_pages, 2 ** 31 - 1
    table[1, 6] = -2 ** 31
    table[2] = -1
    table[3, 8:] = -1  # 8 whole pages of its own; the position lies far behind the table
    gone = [{0, 5, 12}, {6}, set(range(4)), {8}]
    slots = [[s for k, s in enumerate(c.slots[i]) if k // P not in gone[i]] for i in range(4)]
    pos = np.array([199, 99, 63, 2 ** 31 - 1])
    q = rng.standard_normal((4, H, D)).astype(np.float32)
    got = attend(af, t, c.cache, q, kvh, P, c.n_pages, table, pos).cpu().numpy().reshape(q.shape)
    assert np.abs(got - attn_ref(q.astype(np.float64), c.k, c.v, slots)).max() <= attn_tol(q, c.k, c.v)
    assert not got[2].any()


@pytest.mark.parametrize("t", KV)
@pytest.mark.parametrize("what", [np.nan, np.inf, -np.inf, 3e38])
def test_attention_paged_values_of_others_reach_no_row(af, t, what):
    """A request with non-finite or huge values beside others in the same pages' neighbourhood."""
    rng = np.random.default_rng(5)
    P, kvh, H, D, lens = 8, 2, 8, 64, [40, 37, 50]
    c = Paged(af, t, rng, kvh, D, P, lens)
    q = rng.standard_normal((3, H, D)).astype(np.float32)
    clean = attend(af, t, c.cache, q, kvh, P, c.n_pages, c.table, np.array(lens) - 1).cpu().numpy()
    bad = torch.full((3, kvh * D), float(what), device="cuda")
    at = c.slots[1][[0, 20, 36]].astype(np.int32)
    write(af, t, c.cache, bad, bad, kvh, D, c.n_pages * P, _dev(at))
    got = attend(af, t, c.cache, q, kvh, P, c.n_pages, c.table, np.array(lens) - 1).cpu().numpy()
    assert np.array_equal(got[[0, 2]], clean[[0, 2]])
    if not (t == "f32" and np.isfinite(what)):
        assert not np.isfinite(got[1]).any() or np.isfinite(what)
    # a row that sees the tokens before the last bad one is not touched by it
    pos = np.array(lens) - 1
    pos[1] = 35
    c2 = Paged(af, t, np.random.default_rng(5), kvh, D, P, lens)
    want = attend(af, t, c2.cache, q, kvh, P, c2.n_pages, c2.table, pos).cpu().numpy()
    write(af, t, c2.cache, bad[:1], bad[:1], kvh, D, c2.n_pages * P, _dev(at[2:]))
    assert np.array_equal(attend(af, t, c2.cache, q, kvh, P, c2.n_pages, c2.table, pos).cpu().numpy(), want)


@pytest.mark.parametrize("t,qv,kv", [("f32", 0.5, -np.inf), ("f16", 0.5, -np.inf), ("f32", 2.0 ** 68, -2.0 ** 68)])
def test_attention_paged_row_of_minus_infinities(af, t, qv, kv):
    """Scores that are all -infinity have no softmax: NaN, not the zeros of a row that sees nothing.  One finite score among
    them is what the formula gives, or NaN where the row sees infinities."""
    P, kvh, H, D, m = 16, 1, 4, 64, 1000
    cache = new_cache(t, kvh, 1024, D, 0)
    k = torch.full((m, D), float(kv), device="cuda")
    v = torch.randn(m, D, device="cuda")
    write(af, t, cache, k, v, kvh, D, 1024, slot0=0)
    q = np.full((2, H, D), qv, np.float32)
    table = np.tile(np.arange(64), (2, 1))
    got = attend(af, t, cache, q, kvh, P, 64, table, [999, 10]).cpu().numpy()
    assert np.isnan(got).all()
    write(af, t, cache, torch.zeros(1, D, device="cuda"), v[600:601], kvh, D, 1024, slot0=600)
    got = attend(af, t, cache, q, kvh, P, 64, table, [999, 10]).cpu().numpy().reshape(2, H, D)
    want = held(v[600].cpu().numpy(), t)
    assert np.isnan(got[1]).all()
    assert np.abs(got[0] - want).max() <= 2.0 ** -19 * np.abs(want).max() or (np.isinf(kv) and np.isnan(got[0]).all())


LONG = [  # heads, kv heads, head_dim, page size, lengths: items cut over many CTAs, many short ones, both
    (32, 8, 128, 16, [20011]),
    (8, 1, 128, 64, [9000]),
    (4, 1, 64, 16, [1, 30000, 5, 40]),
    (64, 8, 64, 24, [5000, 1, 7, 2500]),
    (32, 8, 128, 16, list(range(1, 400, 3))),
    (8, 4, 64, 16, [17] * 1000),
    (8, 8, 128, 32, [300] * 60 + [7000]),
]


def attn_ref_gpu(q, c, slots):
    n, H, D = q.shape
    G = H // c.kvh
    k, v = _dev(c.k), _dev(c.v)
    out = torch.zeros(n, H, D, dtype=torch.float64, device="cuda")
    for i in range(n):
        if len(slots[i]):
            at = _dev(np.asarray(slots[i]))
            z = torch.einsum("gxd,gld->gxl", _dev(q[i].astype(np.float64)).view(c.kvh, G, D), k[:, at]) * D ** -0.5
            out[i] = torch.einsum("gxl,gld->gxd", torch.softmax(z, -1), v[:, at]).reshape(H, D)
    return out.cpu().numpy()


@pytest.mark.parametrize("t", KV)
@pytest.mark.parametrize("H,KVH,D,P,lens", LONG)
def test_attention_paged_long_and_many(af, t, H, KVH, D, P, lens):
    rng = np.random.default_rng(H + P)
    c = Paged(af, t, rng, KVH, D, P, lens)
    q = rng.standard_normal((len(lens), H, D)).astype(np.float32)
    got = attend(af, t, c.cache, q, KVH, P, c.n_pages, c.table, np.array(lens) - 1).cpu().numpy().reshape(q.shape)
    ref = attn_ref_gpu(q, c, c.slots)
    err, tol = np.abs(got - ref).max(), attn_tol(q, c.k, c.v)
    rel = max(np.linalg.norm(a - b) / np.linalg.norm(b) for a, b in zip(got, ref))
    print(f"err {err:.2e} tol {tol:.2e} rel {rel:.2e}")
    assert err <= tol


@pytest.mark.parametrize("t", ["f32", "q4_0"])
@pytest.mark.parametrize("n,width", [(2048, 4), (64, 600000), (1, 1 << 26)])
def test_attention_paged_most_rows_and_widest_tables(af, t, n, width):
    """The most rows of a call, of a few requests, and tables so wide that stages are counted in 64 bits."""
    rng = np.random.default_rng(14)
    kvh, H, D, P, lens = 1, 64, 64, 16, [40, 64, 7]
    c = Paged(af, t, rng, kvh, D, P, lens, extra=0)
    reqs = min(3, max(1, (1 << 27) // width))
    table = torch.full((reqs, width), -1, dtype=torch.int32, device="cuda")
    table[:, :c.table.shape[1]] = i32(c.table[:reqs])
    seq = rng.integers(0, reqs, n)
    pos = np.array([rng.integers(-1, lens[s]) for s in seq])
    q = rng.standard_normal((n, H, D)).astype(np.float32)
    qd, out = _dev(q.reshape(n, -1)), torch.full((n, H * D), 9.0, device="cuda")
    ws = torch.full((af.af_attention_paged_workspace(H, kvh, D),), 0xFF, dtype=torch.uint8, device="cuda")
    af.af_attention_paged(qd, H * D, *c.cache, af.KVTYPE[t], H, kvh, D, P, c.n_pages, table, width, reqs, i32(seq), i32(pos), n, ws,
                          ws.numel(), out, H * D)
    ref = attn_ref_gpu(q, c, [c.slots[s][:p + 1] for s, p in zip(seq, pos)])
    assert np.abs(out.cpu().numpy().reshape(ref.shape) - ref).max() <= attn_tol(q, c.k, c.v)


@pytest.mark.parametrize("t,D,slots", [("f32", 128, 1 << 21), ("f16", 64, 1 << 24), ("q8_0", 128, 1 << 24), ("q4_0", 64, 1 << 26)])
def test_attention_paged_far_into_a_large_cache(af, t, D, slots):
    """Pages whose bytes lie past 32 bits."""
    rng = np.random.default_rng(15)
    kvh, H, P, m = 5 if t == "f32" else 4, 20 if t == "f32" else 16, 16, 100
    size = {"f32": 4 * D, "f16": 2 * D, "q8_0": D, "q4_0": D // 2}[t]
    assert kvh * slots * size > 1 << 32
    if t in ("f32", "f16"):
        cache = [x for _ in range(2) for x in (torch.empty(kvh, slots, D, dtype=torch.float32 if t == "f32" else torch.float16,
                                                           device="cuda"), None)]
    else:
        cache = [x for _ in range(2) for x in (torch.empty(kvh, slots, size, dtype=torch.uint8, device="cuda"),
                                               torch.empty(kvh, slots, D // 32, dtype=torch.float16, device="cuda"))]
    n_pages = slots // P
    pages = np.array([[n_pages - 1, 0, n_pages - 3, n_pages // 2, n_pages - 2, 1, n_pages - 9]])
    at = (pages[0, np.arange(m) // P] * P + np.arange(m) % P).astype(np.int32)
    k, v = (rng.standard_normal((m, kvh * D)).astype(np.float32) for _ in range(2))
    write(af, t, cache, _dev(k), _dev(v), kvh, D, slots, _dev(at))
    q = rng.standard_normal((1, H, D)).astype(np.float32)
    got = attend(af, t, cache, q, kvh, P, n_pages, pages, [m - 1]).cpu().numpy().reshape(1, H, D)
    kh, vh = (held(x.reshape(m, kvh, D), t).transpose(1, 0, 2) for x in (k, v))
    ref = attn_ref(q.astype(np.float64), kh, vh, [np.arange(m)])
    assert np.abs(got - ref).max() <= attn_tol(q, kh, vh)


@pytest.mark.parametrize("t", KV)
def test_attention_paged_queries_that_are_not_finite(af, t):
    """A row's query with a NaN, an infinity or fp32's extremes does nothing to the other rows and heads."""
    rng = np.random.default_rng(16)
    P, kvh, H, D, lens = 16, 2, 8, 64, [300, 40, 500, 33]
    c = Paged(af, t, rng, kvh, D, P, lens)
    q = rng.standard_normal((4, H, D)).astype(np.float32)
    pos = np.array(lens) - 1
    clean = attend(af, t, c.cache, q, kvh, P, c.n_pages, c.table, pos).cpu().numpy().reshape(q.shape)
    bad = q.copy()
    bad[0, 3, 5], bad[2, 0, 0], bad[3, 7] = np.nan, np.inf, 0
    bad[1, 2] *= np.float32(1e-41)
    got = attend(af, t, c.cache, bad, kvh, P, c.n_pages, c.table, pos).cpu().numpy().reshape(q.shape)
    same_q = (bad == q).all(-1)
    assert np.array_equal(got[same_q], clean[same_q])
    assert not np.isfinite(got[0, 3]).any() and not np.isfinite(got[2, 0]).any()
    for r, h in ((1, 2), (3, 7)):  # scores of zero: the mean of the values
        want = c.v[h // 4][c.slots[r]].mean(0)
        assert np.abs(got[r, h] - want).max() <= 2.0 ** -19 * np.abs(c.v).max()


@pytest.mark.parametrize("t", KV)
@pytest.mark.parametrize("D,m", [(128, 30000), (64, 8000)])
def test_attention_paged_long_sums(af, t, D, m):
    """Values with a mean and equal weights: sums that lose bits always towards zero would show in the norm.  Parts, sums and
    roundings of v move the mean by 2^-21 each: 2^-19 holds them four times over."""
    rng = np.random.default_rng(8)
    kvh, H, P = 1, 4, 64
    n_pages = -(-m // P)
    cache = new_cache(t, kvh, n_pages * P, D)
    k = torch.zeros(m, D, device="cuda")
    v = 1.0 + 0.25 * torch.randn(m, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    write(af, t, cache, k, v, kvh, D, n_pages * P, slot0=0)
    _, vh = read(af, t, cache, m, kvh, D, n_pages * P)
    q = rng.standard_normal((1, H, D)).astype(np.float32)
    got = attend(af, t, cache, q, kvh, P, n_pages, np.arange(n_pages)[None], [m - 1]).cpu().numpy().reshape(H, D)
    ref = vh.astype(np.float64).mean(0)
    err = np.linalg.norm(got - ref) / np.linalg.norm(np.tile(ref, (H, 1)))
    print(f"rel {err:.2e}")
    assert err <= 2.0 ** -19


@pytest.mark.parametrize("t", KV)
@pytest.mark.parametrize("scale", [1e-6, 1e-3, 30.0, 6e4])
def test_attention_paged_scale_of_values(af, t, scale):
    """Values of any size, and slots whose sizes are far apart."""
    if t == "f16" and scale == 1e-6:
        pytest.skip("below fp16's normal numbers")
    if t in ("q8_0", "q4_0") and scale == 1e-6:
        pytest.skip("below the scales' normal numbers")
    rng = np.random.default_rng(9)
    kvh, H, D, P, m = 2, 8, 128, 16, 700
    cache = new_cache(t, kvh, 704, D)
    k = rng.standard_normal((m, kvh * D)).astype(np.float32)
    v = (rng.standard_normal((m, kvh * D)) * scale / 8).astype(np.float32)
    v[::5] *= 1e-2
    write(af, t, cache, _dev(k), _dev(v), kvh, D, 704, slot0=0)
    kh, vh = (x.astype(np.float64).reshape(m, kvh, D).transpose(1, 0, 2) for x in read(af, t, cache, m, kvh, D, 704))
    q = rng.standard_normal((1, H, D)).astype(np.float32)
    got = attend(af, t, cache, q, kvh, P, 44, np.arange(44)[None], [m - 1]).cpu().numpy().reshape(1, H, D)
    ref = attn_ref(q.astype(np.float64), kh, vh, [np.arange(m)])
    assert np.abs(got - ref).max() <= attn_tol(q, kh, vh)


@pytest.mark.parametrize("t", KV)
@pytest.mark.parametrize("H,spread,qs", [(8, 8.0, 4.0), (16, 30.0, 0.01), (8, 1e-3, 1e4)])
def test_attention_paged_wide_scores(af, t, H, spread, qs):
    rng = np.random.default_rng(10)
    c = Paged(af, t, rng, 2, 64, 16, [900, 50, 1], spread=spread)
    q = (rng.standard_normal((3, H, 64)) * qs).astype(np.float32)
    got = attend(af, t, c.cache, q, 2, 16, c.n_pages, c.table, [899, 49, 0]).cpu().numpy().reshape(q.shape)
    assert np.abs(got - attn_ref(q.astype(np.float64), c.k, c.v, c.slots)).max() <= attn_tol(q, c.k, c.v)


@pytest.mark.parametrize("t", KV)
def test_attention_paged_repeats_captures_and_streams(af, t):
    """The same bits in every call; captured, with new lengths between replays; two calls on two streams with scratch of
    their own, and one workspace for two graphs in order."""
    rng = np.random.default_rng(11)
    P, kvh, H, D, lens = 16, 2, 8, 128, [3000, 17, 900, 250]
    c = Paged(af, t, rng, kvh, D, P, lens)
    q = rng.standard_normal((4, H, D)).astype(np.float32)
    first = attend(af, t, c.cache, q, kvh, P, c.n_pages, c.table, np.array(lens) - 1)
    for _ in range(3):
        assert torch.equal(attend(af, t, c.cache, q, kvh, P, c.n_pages, c.table, np.array(lens) - 1), first)
    qd, table, pos = _dev(q.reshape(4, -1)), i32(c.table), i32(np.array(lens) - 1)
    need = af.af_attention_paged_workspace(H, kvh, D)
    ws = [torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.zeros(4, H * D, device="cuda") for _ in range(2)]

    def call(out, w, stream=None):
        af.af_attention_paged(qd, H * D, *c.cache, af.KVTYPE[t], H, kvh, D, P, c.n_pages, table, table.shape[1], 4, None, pos, 4, w,
                              need, out, H * D, stream)
    torch.cuda.synchronize()
    graphs = []
    for out in outs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(out, ws[0])
        graphs.append(graph)
    for lengths in (lens, [2999, 16, 1, 0], [1, 1, 1, 1]):
        pos.copy_(i32(np.array(lengths) - 1))
        want = attend(af, t, c.cache, q, kvh, P, c.n_pages, c.table, np.array(lengths) - 1)
        for graph, out in zip(graphs, outs):
            out.fill_(5.0)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    pos.copy_(i32(np.array(lens) - 1))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for k in range(2):
            call(outs[k], ws[k], streams[k])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], first) and torch.equal(outs[1], first)


@pytest.mark.parametrize("t", KV)
def test_attention_paged_is_decode_attention(af, t):
    """A cache in pages gives what the same cache gives as one run of slots."""
    rng = np.random.default_rng(12)
    kvh, H, D, P, m = 4, 16, 128, 16, 333
    c = Paged(af, t, rng, kvh, D, P, [m])
    q = rng.standard_normal((1, H, D)).astype(np.float32)
    got = attend(af, t, c.cache, q, kvh, P, c.n_pages, c.table, [m - 1])
    flat = new_cache(t, kvh, m, D)
    k, v = read(af, t, c.cache, m, kvh, D, c.n_pages * P, _dev(c.slots[0].astype(np.int32)))
    write(af, t, flat, _dev(k), _dev(v), kvh, D, m)
    out, mask = torch.empty(1, H * D, device="cuda"), i32([[1]])
    need = af.af_attention_tree_workspace(af.KVTYPE[t], H, kvh, D, m - 1, 1)
    ws = torch.empty(max(256, need), dtype=torch.uint8, device="cuda")
    af.af_attention_tree(_dev(q.reshape(1, -1)), H * D, *flat, af.KVTYPE[t], H, kvh, D, m, m - 1, 1, mask, ws, need, out, H * D)
    assert (got - out).abs().max().item() <= 2 * attn_tol(q, c.k, c.v)


# ---------------------------------------------------------------- adapters

def lora_ref(x, ids, a, b, scale, ranks, base):
    y = base.double().clone()
    m = a.shape[0]
    size = base.double().abs().clone()
    for i in range(m):
        rows = torch.nonzero(ids == i)[:, 0]
        r = a.shape[1] if ranks is None else min(max(int(ranks[i]), 0), a.shape[1])
        s = 1.0 if scale is None else float(scale[i])
        if len(rows) and r:
            h = x[rows].double() @ a[i, :r].double().T
            y[rows] += s * (h @ b[i, :, :r].double().T)
            size[rows] += abs(s) * ((x[rows].double().abs() @ a[i, :r].double().abs().T) @ b[i, :, :r].double().abs().T)
    # parts keep 2^-22 of a factor and products of lo parts are left out, in both products; sums add half a step each
    return y, size * 2.0 ** -19


def lora_call(af, x, ids, a, b, scale, ranks, base, y, N, in_place=False, stream=None, plan=None, ws=None):
    n, K = x.shape
    m, r = a.shape[:2]
    if plan is None:
        plan = torch.full((af.af_lora_plan_bytes(n, m),), 0xFF, dtype=torch.uint8, device="cuda")
        af.af_lora_plan(ids, n, m, plan, plan.numel(), stream)
    need = af.af_lora_workspace(n, m, r, K, N)
    if ws is None:
        ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    af.af_lora(x, x.stride(0), n, plan, a, b, af.AF_F16 if a.dtype == torch.float16 else af.AF_F32, scale, ranks, m, r, K, N, base,
               0 if base is None else base.stride(0), y, y.stride(0), ws, need, stream)


LORA = [  # rows, adapters, rank, K, N, share of rows without an adapter, ranks
    (1, 1, 8, 32, 1, 0, "full"),
    (1, 4, 16, 4096, 4096, 0, "full"),
    (5, 3, 24, 96, 77, 0.4, "mixed"),
    (33, 2, 8, 512, 130, 0.1, "full"),
    (64, 40, 16, 2048, 2048, 0.1, "full"),
    (100, 7, 64, 1408, 512, 0, "mixed"),
    (300, 5, 128, 256, 200, 0.2, "mixed"),
    (257, 300, 32, 512, 258, 0.3, "mixed"),
    (64, 2, 40, 14336, 96, 0, "full"),
    (1000, 1, 72, 160, 1030, 0, "full"),
]


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("n,m,r,K,N,bare,ranks", LORA)
@pytest.mark.parametrize("pad", [0, 1])
def test_lora(af, n, m, r, K, N, bare, ranks, dtype, pad):
    g = torch.Generator(device="cuda").manual_seed(n + r)
    def normal(*s):
        return torch.randn(*s, generator=g, device="cuda")
    xs = torch.full((n, K + 4 * pad), float("nan"), device="cuda")
    x = xs[:, :K]
    x.copy_(normal(n, K) * torch.exp(0.5 * normal(K)))
    a, b = (normal(m, r, K) * K ** -0.5).to(dtype), normal(m, N, r).to(dtype)
    ids = torch.randint(0, m, (n,), generator=g, device="cuda", dtype=torch.int32)
    out_of = torch.tensor([-1, m, 2 ** 31 - 1, -2 ** 31], device="cuda", dtype=torch.int64)
    none = torch.rand(n, generator=g, device="cuda") < bare
    ids = torch.where(none, out_of[torch.arange(n, device="cuda") % 4], ids.long()).to(torch.int32)
    rk = None
    if ranks == "mixed":
        rk = torch.randint(-1, r + 3, (m,), generator=g, device="cuda", dtype=torch.int32)
        for i in range(m):  # what lies behind a rank is not looked at
            a[i, max(0, int(rk[i])):] = float("nan")
            b[i, :, max(0, int(rk[i])):] = float("inf")
    scale = normal(m) if m > 1 else None
    base = torch.full((n, N + pad), 3.0, device="cuda")[:, :N]
    base.copy_(normal(n, N))
    ref, tol = lora_ref(x, ids, a, b, scale, rk, base)
    y = torch.full((n, N + 2 * pad), 9.0, device="cuda")
    lora_call(af, x, ids, a, b, scale, rk, base, y, N)
    assert ((y[:, :N].double() - ref).abs() <= tol).all(), ((y[:, :N].double() - ref).abs() / tol).max()
    assert torch.equal(y[none, :N], base[none])  # rows without an adapter are the base's, and nothing behind N is written
    assert (y[:, N:] == 9.0).all()
    first = y[:, :N].clone()
    lora_call(af, x, ids, a, b, scale, rk, base, base, N)  # in place
    assert torch.equal(base, first)
    # without a base
    ref0, tol0 = lora_ref(x, ids, a, b, scale, rk, torch.zeros(n, N, device="cuda"))
    lora_call(af, x, ids, a, b, scale, rk, None, y, N)
    assert ((y[:, :N].double() - ref0).abs() <= tol0).all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_lora_sizes_of_values(af, dtype):
    """x of any size, non-finite rows beside others, weights that are not finite in other adapters."""
    n, m, r, K, N = 40, 5, 16, 512, 300
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(n, K, generator=g, device="cuda") * torch.exp(torch.arange(n, device="cuda")[:, None] - 20.0)
    a = (torch.randn(m, r, K, generator=g, device="cuda") * K ** -0.5).to(dtype)
    b = torch.randn(m, N, r, generator=g, device="cuda").to(dtype)
    ids = (torch.arange(n, device="cuda") % m).to(torch.int32)
    base = torch.randn(n, N, generator=g, device="cuda")
    ref, tol = lora_ref(x, ids, a, b, None, None, base)
    y = torch.empty_like(base)
    lora_call(af, x, ids, a, b, None, None, base, y, N)
    assert ((y.double() - ref).abs() <= tol).all()
    clean = y.clone()
    x[7, 100], x[22, 3] = float("nan"), float("inf")  # adapter 2
    a[4, 3, 17] = float("inf")
    lora_call(af, x, ids, a, b, None, None, base, y, N)
    hit = torch.zeros(n, dtype=torch.bool, device="cuda")
    hit[[7, 22]] = True
    hit |= ids == 4
    assert torch.equal(y[~hit], clean[~hit]) and not torch.isfinite(y[hit]).any()


@pytest.mark.parametrize("n,r,K,N", [(3, 16, 4096, 512), (40, 8, 256, 4100), (300, 64, 96, 1030)])
def test_lora_chain_of_calls(af, n, r, K, N):
    """Calls behind one another, each on what the last one wrote (its base, its x, the plan in the same buffer): as with a
    synchronisation between them, since a call reads ahead only what is older than its first kernel."""
    g = torch.Generator(device="cuda").manual_seed(n)
    def normal(*s):
        return torch.randn(*s, generator=g, device="cuda")
    m, calls = 5, 8
    a, b = [(normal(m, r, K) * K ** -0.5).half() for _ in range(calls)], [(normal(m, N, r) * r ** -0.5).half() for _ in range(calls)]
    back = [(normal(m, K, r) * r ** -0.5).half() for _ in range(calls)]
    ids = [torch.randint(-1, m, (n,), generator=g, device="cuda", dtype=torch.int32) for _ in range(calls)]
    x0, y0 = normal(n, K), normal(n, N)
    ldn = -(-N // 4) * 4
    plan = torch.empty(af.af_lora_plan_bytes(n, m), dtype=torch.uint8, device="cuda")
    ws = torch.empty(max(af.af_lora_workspace(n, m, r, K, N), af.af_lora_workspace(n, m, r, K, K)), dtype=torch.uint8, device="cuda")

    def run(wait):
        x, y = x0.clone(), torch.zeros(n, ldn, device="cuda")
        y[:, :N] = y0
        torch.cuda.synchronize()
        for i in range(calls):
            for call in (lambda: af.af_lora_plan(ids[i], n, m, plan, plan.numel()),
                         lambda: af.af_lora(x, K, n, plan, a[i], b[i], af.AF_F16, None, None, m, r, K, N, y, ldn, y, ldn, ws, ws.numel()),
                         lambda: af.af_lora(x, K, n, plan, a[i], back[i], af.AF_F16, None, None, m, r, K, K, x, K, x, K, ws, ws.numel())):
                call()
                if wait:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        return x, y

    want = run(True)
    assert all(torch.isfinite(t).all() for t in want) and not torch.equal(want[0], x0)
    for _ in range(5):
        got = run(False)
        assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("ctx", [1024, 6000])
def test_decode_attention_sees_keys_that_an_adapter_wrote_just_before(af, ctx):
    """Rows of one kv head are slots of an fp32 cache, in which the decode attention reads ahead."""
    H, KVH, D, K, r = 32, 8, 128, 64, 16
    g = torch.Generator(device="cuda").manual_seed(ctx)
    def normal(*s):
        return torch.randn(*s, generator=g, device="cuda")
    x, q = [normal(ctx, K) * 2.0 ** i for i in (0, 1)], normal(H * D)
    a, b = (normal(1, r, K) / 8).half(), [(normal(1, D, r) / 4).half() for _ in range(KVH)]
    k, v = torch.zeros(KVH, ctx, D, device="cuda"), normal(KVH, ctx, D)
    plan = torch.empty(af.af_lora_plan_bytes(ctx, 1), dtype=torch.uint8, device="cuda")
    ws = torch.empty(af.af_lora_workspace(ctx, 1, r, K, D), dtype=torch.uint8, device="cuda")
    af.af_lora_plan(torch.zeros(ctx, dtype=torch.int32, device="cuda"), ctx, 1, plan, plan.numel())
    heads = [k[h] for h in range(KVH)]

    def step(i, out):
        for h in range(KVH):
            af.af_lora(x[i], K, ctx, plan, a, b[h], af.AF_F16, None, None, 1, r, K, D, None, 0, heads[h], D, ws, ws.numel())
        af.af_attention_decode_static(q, k, v, af.AF_F32, H, KVH, D, ctx, ctx - 1, out)

    want = [torch.zeros(H * D, device="cuda") for _ in range(2)]
    for i in (0, 1):
        torch.cuda.synchronize()
        step(i, want[i])
    outs = [torch.zeros(H * D, device="cuda") for _ in range(20)]
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        step(i % 2, out)
    torch.cuda.synchronize()
    assert not torch.equal(want[0], want[1])
    assert all(torch.equal(y, want[i % 2]) for i, y in enumerate(outs))


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_lora_values_far_apart(af, dtype):
    """One value of x, of A or of A x that is far larger than its neighbours costs them no bits that the sums would keep: the others
    are down to 2^-30 of it, and only they meet weights that are not zero."""
    n, m, r, K, N = 3, 1, 16, 64, 40
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(n, K, generator=g, device="cuda")
    a = torch.randn(m, r, K, generator=g, device="cuda")
    b = torch.randn(m, N, r, generator=g, device="cuda")
    x[:, ::32] *= 2.0 ** 15
    a[:, :, ::32] = 0
    a[:, 3] *= 2.0 ** 10  # a rank of h far above the others, which B does not use
    b[:, :, 3] = 0
    a, b = a.to(dtype), b.to(dtype)
    y = torch.empty(n, N, device="cuda")
    ids = torch.zeros(n, dtype=torch.int32, device="cuda")
    lora_call(af, x, ids, a, b, None, None, None, y, N)
    ref, tol = lora_ref(x, ids, a, b, None, None, torch.zeros(n, N, device="cuda"))
    assert ((y.double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("n,m", [(1, 1), (5000, 1), (5000, 4096), (65536, 3), (4097, 900), (1023, 4)])
def test_lora_plan_holds_every_row_once(af, n, m):
    """The plan through what it does: A = the row's own 1, so that y is the adapter's number, at every row."""
    g = torch.Generator(device="cuda").manual_seed(n)
    ids = torch.randint(-1, m, (n,), generator=g, device="cuda", dtype=torch.int32)
    r, K, N = 8, 32, 4
    a = torch.zeros(m, r, K, dtype=torch.float16, device="cuda")
    a[:, 0, 0] = 1
    b = torch.zeros(m, N, r, dtype=torch.float16, device="cuda")
    b[:, :, 0] = 1
    scale = torch.arange(1, m + 1, device="cuda", dtype=torch.float32)
    x = torch.zeros(n, K, device="cuda")
    x[:, 0] = torch.arange(1, n + 1, device="cuda") % 1024
    y = torch.empty(n, N, device="cuda")
    lora_call(af, x, ids, a, b, scale, None, None, y, N)
    assert torch.equal(y, (x[:, :1] * (ids[:, None] + 1)).expand(n, N))


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_lora_repeats_captures_and_streams(af, dtype):
    n, m, r, K, N = 70, 9, 16, 1024, 512
    g = torch.Generator(device="cuda").manual_seed(7)
    x, base = torch.randn(n, K, generator=g, device="cuda"), torch.randn(n, N, generator=g, device="cuda")
    a = torch.randn(m, r, K, generator=g, device="cuda").to(dtype)
    b = torch.randn(m, N, r, generator=g, device="cuda").to(dtype)
    ids = torch.randint(-1, m, (n,), generator=g, device="cuda", dtype=torch.int32)
    plans = [torch.empty(af.af_lora_plan_bytes(n, m), dtype=torch.uint8, device="cuda") for _ in range(2)]
    need = af.af_lora_workspace(n, m, r, K, N)
    ws = [torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2)]
    ys = [torch.empty(n, N, device="cuda") for _ in range(2)]

    def step(k, stream=None):
        af.af_lora_plan(ids, n, m, plans[k], plans[k].numel(), stream)
        lora_call(af, x, ids, a, b, None, None, base, ys[k], N, stream=stream, plan=plans[k], ws=ws[k])
    step(0)
    first = ys[0].clone()
    for _ in range(3):
        step(0)
        assert torch.equal(ys[0], first)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(0)
    for shift in (0, 1, 5):
        new = torch.where(ids >= 0, (ids + shift) % m, ids)
        old = ids.clone()
        ids.copy_(new)
        step(1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ys[0], ys[1])
        ids.copy_(old)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for k in range(2):
            step(k, streams[k])
    torch.cuda.synchronize()
    assert torch.equal(ys[0], first) and torch.equal(ys[1], first)


# ---------------------------------------------------------------- a step of a serving loop

@pytest.mark.parametrize("t", KV)
def test_serving_steps(af, t):
    """Prompts join, run and end: each step maps its tokens to slots, projects them with adapters of their requests, rotates,
    writes and attends, in one captured graph; every row against the definition on what the cache holds."""
    import synth
    E, H, kvh, D, P, n, rows, r, m = 256, 4, 2, 64, 8, 6, 40, 8, 3
    width, n_pages = 12, 40
    w = (H + 2 * kvh) * D
    blocks = _dev(synth.matrix("q8_0", 5, synth.TID_TEST_BASE + 60, w, E))
    qw = af.af_qweight_create(af.AF_Q8_0, blocks, w, E)
    g = torch.Generator(device="cuda").manual_seed(8)
    a = (torch.randn(m, r, E, generator=g, device="cuda") * E ** -0.5).half()
    b = torch.randn(m, w, r, generator=g, device="cuda").half()
    scale = torch.tensor([0.5, -1.0, 2.0], device="cuda")
    cache = new_cache(t, kvh, n_pages * P, D, 0xFF)
    ln, pool, free, table = i32(np.zeros(n)), i32([0, n_pages, 0, 0]), i32(np.arange(n_pages)), i32(np.full((n, width), -1))
    new, start, (slots, pos, seq) = i32(np.zeros(n)), i32(np.zeros(n + 1)), (i32(np.zeros(rows)) for _ in range(3))
    adapter_of, ids = i32([0, 1, 2, 0, -1, 1]), i32(np.zeros(rows))
    x, y, rot = torch.zeros(rows, E, device="cuda"), torch.empty(rows, w, device="cuda"), torch.empty(rows, w, device="cuda")
    out = torch.empty(rows, H * D, device="cuda")
    pws = torch.empty(af.af_kv_pages_workspace(n), dtype=torch.uint8, device="cuda")
    plan = torch.empty(af.af_lora_plan_bytes(rows, m), dtype=torch.uint8, device="cuda")
    lws = torch.empty(af.af_lora_workspace(rows, m, r, E, w), dtype=torch.uint8, device="cuda")
    aws = torch.empty(af.af_attention_paged_workspace(H, kvh, D), dtype=torch.uint8, device="cuda")
    cfg = af.rope_config(D, D, "half", 10000.0)

    def step():
        af.af_kv_pages(ln, new, n, P, n_pages, pool, free, table, width, ln, pool, start, slots, pos, seq, rows, pws, pws.numel())
        ids.copy_(torch.where(seq >= 0, adapter_of[seq.clamp(min=0).long()], -1))
        af.af_lora_plan(ids, rows, m, plan, plan.numel())
        af.af_qgemm(qw, x, rows, y)
        af.af_lora(x, E, rows, plan, a, b, af.AF_F16, scale, None, m, r, E, w, y, w, y, w, lws, lws.numel())
        af.af_rope(cfg, y, w, rot, w, af.AF_F32, rows, H + kvh, pos)
        af.af_kv_write(rot[:, H * D:], y[:, (H + kvh) * D:], w, rows, slots, 0, *cache, af.KVTYPE[t], kvh, D, n_pages * P)
        af.af_attention_paged(rot, w, *cache, af.KVTYPE[t], H, kvh, D, P, n_pages, table, width, n, seq, pos, rows, aws, aws.numel(),
                              out, H * D)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    rng = np.random.default_rng(9)
    seen, length = 0, np.zeros(n, int)
    for s in range(14):
        add = np.where(length == 0, rng.integers(0, 12, n), 1)
        add[(length > 15) & (rng.random(n) < 0.4)] = -1
        new.copy_(i32(add))
        x.copy_(torch.randn(rows, E, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        length = np.where(add < 0, 0, length + add)
        assert np.array_equal(ln.cpu().numpy(), length)
        total = int(np.maximum(add, 0).sum())
        base = torch.empty(rows, w, device="cuda")
        af.af_qgemm(qw, x, rows, base)
        ref, tol = lora_ref(x, ids, a, b, scale, None, base)
        assert ((y.double() - ref).abs() <= tol).all()
        kh, vh = (z.astype(np.float64).reshape(-1, kvh, D).transpose(1, 0, 2)
                  for z in read(af, t, cache, n_pages * P, kvh, D, n_pages * P))
        tb, sq, ps = table.cpu().numpy(), seq.cpu().numpy(), pos.cpu().numpy()
        assert (sq[:total] >= 0).all() and (sq[total:] == -1).all()
        where = [tb[i, np.arange(p + 1) // P] * P + np.arange(p + 1) % P if i >= 0 else [] for i, p in zip(sq, ps)]
        q = rot[:, :H * D].cpu().numpy().reshape(rows, H, D)
        used = np.unique(np.concatenate([np.asarray(v, int) for v in where]))
        got = out.cpu().numpy().reshape(rows, H, D)
        live = np.zeros_like(kh), np.zeros_like(vh)
        live[0][:, used], live[1][:, used] = kh[:, used], vh[:, used]
        assert np.abs(got - attn_ref(q.astype(np.float64), *live, where)).max() <= attn_tol(q, *live)
        seen += total
    assert seen > 100
    af.af_qweight_destroy(qw)
