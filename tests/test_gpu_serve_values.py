"""The operators of a serving step at values and in orders where a mistake would be small or rare."""
import numpy as np
import pytest

from test_gpu_draft import new_cache, write
from test_gpu_serve import ATTN, KV, LONG, Paged, af, attend, attn_ref_gpu, i32, lora_call, lora_ref  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


# ---------------------------------------------------------------- adapters: factors far from one

@pytest.mark.parametrize("xs,a_s,bs", [(1e-30, 1e33, 1.0), (1e33, 1e-30, 1.0), (1e-36, 1e36, 1.0), (1e-30, 1.0, 1e33),
                                       (1e30, 1.0, 1e-30), (1e-20, 1e-15, 1e36), (1.0, 1.0, 1.0)])
@pytest.mark.parametrize("n,m,r,K,N", [(1, 1, 16, 96, 128), (9, 1, 24, 512, 77), (40, 3, 64, 256, 260), (70, 2, 8, 64, 64)])
def test_lora_factors_far_from_one(af, xs, a_s, bs, n, m, r, K, N):
    """fp32 weights and rows whose sizes are far apart while their products are not: as with neither of them scaled."""
    g = torch.Generator(device="cuda").manual_seed(n + r)
    def normal(*s):
        return torch.randn(*s, generator=g, device="cuda")
    x, a, b = normal(n, K) * xs, normal(m, r, K) * a_s, normal(m, N, r) * bs
    ids = torch.randint(0, m, (n,), generator=g, device="cuda", dtype=torch.int32)
    y = torch.empty(n, N, device="cuda")
    lora_call(af, x, ids, a, b, None, None, None, y, N)
    ref, tol = lora_ref(x, ids, a, b, None, None, torch.zeros(n, N, device="cuda"))
    assert torch.isfinite(y).all()
    assert ((y.double() - ref).abs() <= tol).all(), ((y.double() - ref).abs() / tol).max()


def test_lora_large_factors_that_do_not_meet(af):
    """The largest of x meet zeros of A and the other way round: what is left is the small sums."""
    n, m, r, K, N = 20, 1, 16, 64, 48
    g = torch.Generator(device="cuda").manual_seed(2)
    x, a = torch.zeros(n, K, device="cuda"), torch.zeros(m, r, K, device="cuda")
    x[:, ::4], a[:, :, 1::4] = 1e38, 1e38
    x[:, 2::4] = torch.randn(n, K // 4, generator=g, device="cuda") * 1e30
    a[:, :, 2::4] = torch.randn(m, r, K // 4, generator=g, device="cuda") * 1e-30
    b = torch.randn(m, N, r, generator=g, device="cuda")
    y = torch.empty(n, N, device="cuda")
    lora_call(af, x, torch.zeros(n, dtype=torch.int32, device="cuda"), a, b, None, None, None, y, N)
    assert torch.isfinite(y).all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("what", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("n,m,r,K,N", [(3, 2, 8, 64, 40), (50, 4, 64, 512, 300)])
def test_lora_values_that_are_not_finite(af, dtype, what, n, m, r, K, N):
    """They reach the rows and columns that the formula takes them to, and no others."""
    g = torch.Generator(device="cuda").manual_seed(3)
    def normal(*s):
        return torch.randn(*s, generator=g, device="cuda")
    x, a, b, base = normal(n, K), normal(m, r, K).to(dtype), normal(m, N, r).to(dtype), normal(n, N)
    ids = (torch.arange(n, device="cuda") % m).to(torch.int32)
    clean = torch.empty(n, N, device="cuda")
    lora_call(af, x, ids, a, b, None, None, base, clean, N)
    hit = torch.zeros(n, N, dtype=torch.bool, device="cuda")
    for kind in ("x", "a", "b"):
        xs, as_, bs, want = x.clone(), a.clone(), b.clone(), hit.clone()
        if kind == "x":
            xs[n // 2, K // 3] = float(what)
            want[n // 2] = True
        elif kind == "a":
            as_[1, r - 1, K - 1] = float(what)
            want[ids == 1] = True
        else:
            bs[1, N // 2, 3] = float(what)
            want[ids == 1, N // 2] = True
        y = torch.empty(n, N, device="cuda")
        lora_call(af, xs, ids, as_, bs, None, None, base, y, N)
        assert torch.equal(~torch.isfinite(y), want)
        assert torch.equal(y[~want], clean[~want])


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("n,m,N", [(40, 6, 260), (7, 300, 33)])
def test_lora_with_a_plan_of_other_sizes(af, dtype, n, m, N):
    """Rows of NaN, whether the plan was made for more or fewer rows or adapters or never; the next call with its own plan is right."""
    K, r = 64, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    def normal(*s):
        return torch.randn(*s, generator=g, device="cuda")
    x, a, b, base = normal(n, K), normal(m, r, K).to(dtype), normal(m, N, r).to(dtype), normal(n, N)
    ids = torch.randint(0, 1 << 30, (5000,), generator=g, device="cuda", dtype=torch.int32)
    plan = torch.zeros(max(af.af_lora_plan_bytes(*s) for s in ((n, m), (5000, 4096))), dtype=torch.uint8, device="cuda")
    right = torch.randint(-1, m, (n,), generator=g, device="cuda", dtype=torch.int32)
    ref, tol = lora_ref(x, right, a, b, None, None, base)
    for other in (0, 0xFF, (n + 1, m), (n - 1, m), (n, m + 1), (n, m - 1), (5000, m), (n, 4096), (5000, 4096), (1, 1)):
        if isinstance(other, int):
            plan.fill_(other)
        else:
            af.af_lora_plan(ids % other[1], *other, plan, plan.numel())
        y = torch.full((n, N + 3), 9.0, device="cuda")
        lora_call(af, x, None, a, b, None, None, base, y, N, plan=plan)
        assert torch.isnan(y[:, :N]).all() and (y[:, N:] == 9.0).all()
        y[:, :N] = base
        lora_call(af, x, None, a, b, None, None, y, y, N, plan=plan)
        assert torch.isnan(y[:, :N]).all() and (y[:, N:] == 9.0).all()
        af.af_lora_plan(right, n, m, plan, plan.numel())
        lora_call(af, x, None, a, b, None, None, base, y, N, plan=plan)
        assert ((y[:, :N].double() - ref).abs() <= tol).all()


# ---------------------------------------------------------------- attention: precision

@pytest.mark.parametrize("t", KV)
@pytest.mark.parametrize("H,KVH,D,P,lens", ATTN + LONG)
def test_attention_paged_precision_of_rows(af, t, H, KVH, D, P, lens):
    """Each row's error against its own norm, with queries, keys and values of unit size: a slot left out or counted twice at a cut,
    or a low part that is lost, shows in rows of any length.  q's parts and p's leave 2^-21 of a value each, the exponential
    2^-22, and scores, up to 8 in powers of two, are rounded by 2^-22 a few times.  These errors differ from slot to slot, so a
    weighted mean of independent values moves by as much of its norm as they do themselves: 2^-19 holds all of them at their
    largest.  (Half the bits of q lost: 2^-12; a slot of 20011 left out: 6e-3 of the row.)"""
    rng = np.random.default_rng(H * D + P + 1)
    c = Paged(af, t, rng, KVH, D, P, lens)
    q = rng.standard_normal((len(lens), H, D)).astype(np.float32)
    got = attend(af, t, c.cache, q, KVH, P, c.n_pages, c.table, np.array(lens) - 1).cpu().numpy().reshape(len(lens), -1)
    ref = attn_ref_gpu(q, c, c.slots).reshape(len(lens), -1)
    size = np.linalg.norm(ref, axis=1)
    err = np.linalg.norm(got - ref, axis=1)
    print(f"largest {(err[size > 0] / size[size > 0]).max():.2e}")
    assert (err <= 2.0 ** -19 * size).all()


def score_bound(t, q, k, v, slots):
    """Per value of the result: scores off by at most d_j = 2^-20 sum |q| max |k_j| / sqrt(D) change the weights by factors of
    exp(+-d_j), which moves the mean by at most sum p_j (exp(d_j) - 1) |v_j - out| / sum p_j exp(-d_j); parts of p and v and the
    sums leave 2^-19 of the weighted mean of |v|.  For fp16 and the codes p, times a value's scale, is held in fp16 parts whose
    smallest step is 2^-24, while the row's largest is at least 2^9 (p = 2^10 at the reference, which is at most the largest; the
    slot's largest scale, to a factor of 2): half a step is 2^-34 of the largest p |v|, of each slot.  (It is all that is left
    of a dim in which the slots that count hold zeros.)"""
    n, H, D = q.shape
    G = H // k.shape[0]
    out, tol = np.zeros((n, H, D)), np.zeros((n, H, D))
    for i in range(n):
        for h in range(H):
            kk, vv = k[h // G, slots[i]], v[h // G, slots[i]]
            s = kk @ q[i, h] / np.sqrt(D)
            d = 2.0 ** -20 * np.abs(q[i, h]).sum() * np.abs(kk).max(1) / np.sqrt(D)
            p = np.exp(s - s.max())
            p /= p.sum()
            out[i, h] = p @ vv
            tol[i, h] = (p * np.expm1(d)) @ np.abs(vv - out[i, h]) / (p @ np.exp(-d)) + 2.0 ** -19 * (p @ np.abs(vv))
            if t != "f32":
                tol[i, h] += len(p) * 2.0 ** -34 * (p * np.abs(vv).max(1)).max()
    return out, tol


@pytest.mark.parametrize("t", KV)
@pytest.mark.parametrize("H,D,spread,qs", [(8, 64, 8.0, 4.0), (16, 64, 30.0, 0.01), (8, 64, 1e-3, 1e4), (4, 128, 3.0, 1.0), (16, 128, 1.0, 8.0)])
def test_attention_paged_precision_of_wide_scores(af, t, H, D, spread, qs):
    """Scores far apart, each value against what its own row's scores allow."""
    rng = np.random.default_rng(17)
    lens = [900, 50, 1, 3000, 333]
    c = Paged(af, t, rng, 2, D, 16, lens, spread=spread)
    q = (rng.standard_normal((5, H, D)) * qs).astype(np.float32)
    got = attend(af, t, c.cache, q, 2, 16, c.n_pages, c.table, np.array(lens) - 1).cpu().numpy().reshape(q.shape)
    ref, tol = score_bound(t, q.astype(np.float64), c.k, c.v, c.slots)
    print(f"largest {(np.abs(got - ref)[tol > 0] / tol[tol > 0]).max():.2f} of the bound")
    assert (np.abs(got - ref) <= tol).all()


# ---------------------------------------------------------------- attention: values that are not finite where work is cut

@pytest.mark.parametrize("what", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("lo,hi,at", [(0, 10000, 5000), (9000, 19900, 9900), (64, 128, 100), (19984, 20000, 19990), (3000, 3400, 3100)])
@pytest.mark.parametrize("G", [4, 8])
def test_attention_paged_values_behind_scores_of_minus_infinity(af, what, lo, hi, at, G):
    """Slots lo..hi have scores of -infinity (fp32 products out of range), one of them a value that is not finite: its weight of
    zero times it is NaN wherever the work on the row is cut; the other dims are finite."""
    kvh, D, P, m, dim = 1, 64, 16, 20000, 5
    cache = new_cache("f32", kvh, m, D, 0)
    k, v = torch.zeros(m, D, device="cuda"), torch.randn(m, D, device="cuda")
    k[lo:hi] = -2.0 ** 68
    v[at, dim] = float(what)
    write(af, "f32", cache, k, v, kvh, D, m, slot0=0)
    q = np.full((3, G, D), 2.0 ** 68, np.float32)
    q[1] = 1.0  # finite scores, but so large that the slots' weights are 0 too
    pos = [m - 1, m - 1, lo + 3 if lo else 3]
    table = np.tile(np.arange(m // P), (3, 1))
    got = attend(af, "f32", cache, q, kvh, P, m // P, table, pos).cpu().numpy().reshape(3, G, D)
    assert np.isnan(got[:2, :, dim]).all()
    keep = np.r_[0:lo, hi:m]
    others = np.arange(D) != dim
    want = v[keep].double().mean(0).cpu().numpy()
    assert np.abs(got[:2, :, others] - want[others]).max() <= 2.0 ** -19 * float(v[torch.isfinite(v)].abs().max())
    # a row that does not see the value is as it was: finite where some of its scores are, NaN where all are -infinity
    assert np.isnan(got[2]).all() if lo == 0 else np.isfinite(got[2]).all()


# ---------------------------------------------------------------- calls that write a cache just before the decode attention

class Chain:
    """One kv head's fp32 cache of `ctx` slots, whose keys are written by adapters just before the decode attention, which reads
    ahead: two sets of keys in turn, each with the result that a synchronisation in between gives."""
    D, K, r, H = 128, 64, 16, 4

    def __init__(self, af, ctx, seed):
        self.af, self.ctx = af, ctx
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.normal = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.q, self.k, self.v = self.normal(self.H * self.D), torch.zeros(1, ctx, self.D, device="cuda"), self.normal(1, ctx, self.D)
        self.a = (self.normal(1, self.r, self.K) / 8).half()

    def adapters(self, n, N):
        """What af_lora needs for n rows of N: two inputs and the rest."""
        af = self.af
        plan = torch.empty(af.af_lora_plan_bytes(n, 1), dtype=torch.uint8, device="cuda")
        ws = torch.empty(af.af_lora_workspace(n, 1, self.r, self.K, N), dtype=torch.uint8, device="cuda")
        af.af_lora_plan(torch.zeros(n, dtype=torch.int32, device="cuda"), n, 1, plan, plan.numel())
        x = [self.normal(n, self.K) * 2.0 ** i for i in (0, 1)]
        b = (self.normal(1, N, self.r) / 4).half()
        return lambda i, y, ldy: af.af_lora(x[i], self.K, n, plan, self.a, b, af.AF_F16, None, None, 1, self.r, self.K, N, None, 0, y, ldy,
                                            ws, ws.numel())

    def attend(self, out):
        self.af.af_attention_decode_static(self.q, self.k, self.v, self.af.AF_F32, self.H, 1, self.D, self.ctx, self.ctx - 1, out)

    def check(self, step):
        """step(i) writes keys i; the attention directly behind it has to see them."""
        want = [torch.zeros(self.H * self.D, device="cuda") for _ in range(2)]
        for i in (0, 1):
            step(i)
            torch.cuda.synchronize()
            self.attend(want[i])
            torch.cuda.synchronize()
        outs = [torch.zeros(self.H * self.D, device="cuda") for _ in range(30)]
        torch.cuda.synchronize()
        for i, out in enumerate(outs):
            step(i % 2)
            self.attend(out)
        torch.cuda.synchronize()
        assert not torch.equal(want[0], want[1])
        assert all(torch.equal(y, want[i % 2]) for i, y in enumerate(outs))


@pytest.mark.parametrize("ctx", [640, 6000])
@pytest.mark.parametrize("between", ["nothing", "plan", "pages"])
def test_decode_attention_sees_an_adapters_keys_behind_other_calls(af, ctx, between):
    """A call in between that lets the next kernel start before its own wait, and touches nothing of the cache."""
    c = Chain(af, ctx, 3)
    keys = c.adapters(ctx, c.D)
    plan = torch.empty(af.af_lora_plan_bytes(64, 4), dtype=torch.uint8, device="cuda")
    ids = torch.zeros(64, dtype=torch.int32, device="cuda")
    zeros = [torch.zeros(k, dtype=torch.int32, device="cuda") for k in (4, 4, 4, 64, 4 * 8, 4, 4, 5, 16, 16, 16)]
    ws = torch.empty(af.af_kv_pages_workspace(4), dtype=torch.uint8, device="cuda")
    ln, new, pool, free, table, ln_out, pool_out, start, slots, pos, seq = zeros

    def step(i):
        keys(i, c.k, c.D)
        if between == "plan":
            af.af_lora_plan(ids, 64, 4, plan, plan.numel())
        elif between == "pages":
            af.af_kv_pages(ln, new, 4, 16, 64, pool, free, table, 8, ln_out, pool_out, start, slots, pos, seq, 16, ws, ws.numel())
    c.check(step)


def test_decode_attention_sees_an_adapters_keys_at_any_stride(af):
    """Rows of an adapter call that are every fourth slot, eight neighbouring slots each, or one row of all slots."""
    c = Chain(af, 6000, 4)
    fourth, eight, one = c.adapters(1500, c.D), c.adapters(750, 8 * c.D), c.adapters(1, 6000 * c.D)
    rows = [c.k[0, i:] for i in range(4)]

    def every_fourth(i):
        for y in rows:
            fourth(i, y, 4 * c.D)
    c.check(every_fourth)
    c.check(lambda i: eight(i, c.k, 8 * c.D))
    c.check(lambda i: one(i, c.k, 6000 * c.D + 4))


@pytest.mark.parametrize("lens", ["short", "long"])
def test_decode_attention_sees_keys_that_the_paged_attention_wrote(af, lens):
    """The paged attention's rows, of eight heads, as eight neighbouring slots each."""
    H, D, P, n = 8, 128, 16, 200
    rng = np.random.default_rng(5)
    lens = rng.integers(1, 40, n) if lens == "short" else rng.integers(1, 400, n)
    lens[::9] = 0  # rows of zeros
    p = Paged(af, "f16", rng, 2, D, P, lens)
    c = Chain(af, n * H, 6)
    q, table, pos = [c.normal(n, H * D) * (i + 1) for i in (0, 1)], i32(p.table), i32(lens - 1)
    ws = torch.empty(af.af_attention_paged_workspace(H, 2, D), dtype=torch.uint8, device="cuda")
    c.check(lambda i: af.af_attention_paged(q[i], H * D, *p.cache, af.KVTYPE["f16"], H, 2, D, P, p.n_pages, table, table.shape[1], n, None,
                                            pos, n, ws, ws.numel(), c.k, H * D))
