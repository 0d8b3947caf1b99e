"""The drafted-tree operators against plain implementations in 64 bits: rotary positions, cache rows of every type,
the mask of a tree and attention over it, and a run of them together."""
import decimal

import numpy as np
import pytest

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


# ---------------------------------------------------------------- rotary positions

def turns(rot, base, scaling, factor, native, low=1, high=32):
    """Turns per position of each pair as exact fractions (50 digits): (numerator, 10^40)."""
    D = decimal.Decimal
    decimal.getcontext().prec = 60
    pi = D("3.14159265358979323846264338327950288419716939937510582097494")
    b, s = D(float(np.float32(base))), D(float(np.float32(factor)))
    if scaling == "ntk":
        b *= (s.ln() * rot / (rot - 2)).exp()
    out = []
    for i in range(rot // 2):
        f = (b.ln() * (-2 * i) / rot).exp()
        if scaling == "linear":
            f /= s
        if scaling == "yarn":
            w = min(D(1), max(D(0), (native * f / (2 * pi) - low) / (high - low)))
            f = f * w + f / s * (1 - w)
        out.append(int(f / (2 * pi) * 10 ** 40))
    return out


def rope_ref(x, pos, rot, layout, tn, mag):
    """x [n, h, D] float64, pos python ints."""
    one = 10 ** 40
    y = x.copy()
    for r, p in enumerate(pos):
        for i, t in enumerate(tn):
            a, b = (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + rot // 2)
            th = 2 * np.pi * (((p * t) % one) / one)
            c, s = mag * np.cos(th), mag * np.sin(th)
            y[r, :, a] = x[r, :, a] * c - x[r, :, b] * s
            y[r, :, b] = x[r, :, a] * s + x[r, :, b] * c
    return y


ROPE_CASES = [  # n, heads, D, rot, layout, scaling, positions
    (1, 8, 64, 64, "interleaved", "none", [0]),
    (3, 40, 128, 128, "interleaved", "none", [4096, 4097, 4097]),
    (5, 3, 128, 96, "half", "yarn", [-512, 0, 1, 30720, 131071]),
    (4, 2, 80, 32, "half", "linear", [7, 8, 9, 10]),
    (4, 2, 80, 20, "half", "ntk", [1 << 20, -(1 << 20), 2 ** 31 - 1, -2 ** 31]),
    (7, 1, 96, 94, "interleaved", "yarn", list(range(100, 107))),
    (2, 5, 256, 256, "half", "none", [12345, 54321]),
    (2, 1, 6, 2, "interleaved", "linear", [3, 1000003]),
]


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("n,heads,D,rot,layout,scaling,pos", ROPE_CASES)
@pytest.mark.parametrize("pad", [0, 3])
def test_rope(af, n, heads, D, rot, layout, scaling, pos, dtype, pad):
    rng = np.random.default_rng(n * D + rot)
    ld = heads * D + pad
    x = rng.standard_normal((n, ld)).astype(np.float32 if dtype == "f32" else np.float16)
    mag = 1.25 if scaling == "yarn" else 1.0
    cfg = af.rope_config(D, rot, layout, 500000.0, scaling, 4.5, 8192, magnitude=mag)
    xd, pd = _dev(x), _dev(np.array(pos, np.int64).astype(np.int32))
    y = torch.full((n, ld), 7.0, dtype=xd.dtype, device="cuda")
    af.af_rope(cfg, xd, ld, y, ld, af.AF_F32 if dtype == "f32" else af.AF_F16, n, heads, pd)
    got = y.cpu().numpy().astype(np.float64)
    xr = x[:, :heads * D].astype(np.float64).reshape(n, heads, D)
    ref = rope_ref(xr, pos, rot, layout, turns(rot, 500000.0, scaling, 4.5, 8192), mag)
    # sin and cos: the argument's rounding (2^-24 of at most pi / 4) and at most two steps of the function's value,
    # under 2^-22 together, the angle's |pos| 2^-53 turns, and three roundings of products and their sum
    size = np.abs(xr).max(-1, keepdims=True) * mag
    tol = 2 * size * (2.0 ** -22 + 2.0 ** -22 + 2 * np.pi * np.abs(np.array(pos, float))[:, None, None] * 2.0 ** -53)
    if dtype == "f16":
        tol = tol + np.abs(ref) * 2.0 ** -11 + 2.0 ** -25
    g = got[:, :heads * D].reshape(n, heads, D)
    assert np.all(np.abs(g - ref) <= tol), np.max(np.abs(g - ref) / tol)
    assert np.array_equal(g[..., rot:], xr[..., rot:])   # the rest of the head is copied
    assert np.all(got[:, heads * D:] == 7.0)             # and nothing behind the heads is written
    # in place, and without positions in memory
    af.af_rope(cfg, xd, ld, xd, ld, af.AF_F32 if dtype == "f32" else af.AF_F16, n, heads, pd)
    assert torch.equal(xd[:, :heads * D], y[:, :heads * D])


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_rope_counted_positions_and_inverse(af, dtype):
    n, heads, D = 700, 8, 128
    x = torch.randn(n, heads * D, device="cuda").to(torch.float32 if dtype == "f32" else torch.float16)
    t = af.AF_F32 if dtype == "f32" else af.AF_F16
    cfg = af.rope_config(D, D, "half", 10000.0)
    y, z = torch.empty_like(x), torch.empty_like(x)
    pos = torch.arange(50, 50 + n, dtype=torch.int32, device="cuda")
    af.af_rope(cfg, x, heads * D, y, heads * D, t, n, heads, None, 50)
    af.af_rope(cfg, x, heads * D, z, heads * D, t, n, heads, pos)
    assert torch.equal(y, z)
    af.af_rope(cfg, y, heads * D, z, heads * D, t, n, heads, -pos)
    # two rotations, each off by at most 2^-20 of the pair's size (and a half-step of fp16)
    tol = 4 * x.abs().max().item() * (2.0 ** -20 + (2.0 ** -11 if dtype == "f16" else 0))
    assert (z.float() - x.float()).abs().max().item() <= tol


@pytest.mark.parametrize("scaling,factor,base", [("none", 1.0, 1234567.9), ("linear", 7.3, 10000.0), ("ntk", 3.7, 10000.0)])
def test_rope_parameters_keep_their_precision(af, scaling, factor, base):
    """Base and factor are taken in 64 bits: in 32, a factor of 7.3 would turn the first pair by 4e-4 at position 100,000."""
    d, pos = 64, [100003, 1 << 20, -777777]
    one, D = 10 ** 40, decimal.Decimal
    decimal.getcontext().prec = 60
    two_pi = 2 * D("3.14159265358979323846264338327950288419716939937510582097494")
    b, s = D(base), D(factor)
    if scaling == "ntk":
        b *= (s.ln() * d / (d - 2)).exp()
    f = [(b.ln() * (-2 * i) / d).exp() / (s if scaling == "linear" else 1) for i in range(d // 2)]
    x = np.random.default_rng(4).standard_normal((len(pos), 1, d)).astype(np.float32)
    cfg = af.rope_config(d, d, "half", base, scaling, factor, 8192)
    y = torch.empty(len(pos), d, device="cuda")
    af.af_rope(cfg, _dev(x), d, y, d, af.AF_F32, len(pos), 1, _dev(np.array(pos, np.int32)))
    ref = rope_ref(x.astype(np.float64), pos, d, "half", [int(v / two_pi * one) for v in f], 1.0)
    # as test_rope's: sines, products and their sum, and the angle's 2^-53 of a turn a position
    tol = 2 * np.abs(x).max() * (2.0 ** -21 + 2 * np.pi * max(map(abs, pos)) * 2.0 ** -53)
    assert np.abs(y.cpu().numpy().reshape(ref.shape) - ref).max() <= tol


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_rope_many_rows(af, layout, dtype):
    """Blocks that walk many rows each, with the positions of every row its own."""
    n, heads, D, rot = 6001, 5, 128, 96
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(n, heads, D, generator=g, device="cuda").to(torch.float32 if dtype == "f32" else torch.float16)
    pos = torch.randint(-(1 << 17), 1 << 17, (n,), generator=g, device="cuda", dtype=torch.int32)
    y = torch.empty_like(x)
    af.af_rope(af.rope_config(D, rot, layout, 500000.0), x, heads * D, y, heads * D, af.AF_F32 if dtype == "f32" else af.AF_F16, n,
               heads, pos)
    f = 500000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    th = (pos.double()[:, None] * f)[:, None]
    a, b = ([slice(0, rot, 2), slice(1, rot, 2)] if layout == "interleaved" else [slice(0, rot // 2), slice(rot // 2, rot)])
    ref = x.double()
    ref[..., a], ref[..., b] = (x[..., a].double() * th.cos() - x[..., b].double() * th.sin(),
                                x[..., a].double() * th.sin() + x[..., b].double() * th.cos())
    # as test_rope's (2^-21, the angle's 2^-53 of a turn a position), and the reference's own angle, 2^-53 of it
    tol = 2 * x.abs().max().item() * (2.0 ** -21 + (2 * np.pi + 2) * 2.0 ** (17 - 53))
    if dtype == "f16":
        tol = tol + ref.abs() * 2.0 ** -11 + 2.0 ** -25
    assert ((y.double() - ref).abs() <= tol).all()


def test_rope_equals_the_models_rotation(af):
    """AF_ROPE_INTERLEAVED with linear scaling is the rotation the model's QKV epilogue applies."""
    import oracle
    D, base, scale = 128, 500000.0, 4.0
    x = np.random.default_rng(3).standard_normal((1, D)).astype(np.float32)
    for p in (0, 1, 4095, 30720):
        cfg = af.rope_config(D, D, "interleaved", base, "linear", scale)
        y = torch.empty(1, D, device="cuda")
        af.af_rope(cfg, _dev(x), D, y, D, af.AF_F32, 1, 1, None, p)
        th = np.array([p / scale / base ** (2 * i / D) for i in range(D // 2)])
        a, b = x[0, 0::2].astype(np.float64), x[0, 1::2].astype(np.float64)
        ref = np.empty(D)
        ref[0::2], ref[1::2] = a * np.cos(th) - b * np.sin(th), a * np.sin(th) + b * np.cos(th)
        assert np.max(np.abs(y.cpu().numpy()[0] - ref)) <= 2 * np.abs(x).max() * 2.0 ** -20
    assert oracle is not None


# ---------------------------------------------------------------- cache rows

def quantize(x, t):
    """Codes (integers) and fp16 scales of float32 blocks [..., 32], decided in float64."""
    b = x.astype(np.float64)
    if t == "q8_0":
        d = (np.abs(b).max(-1) / 127).astype(np.float32).astype(np.float16)
        with np.errstate(divide="ignore", invalid="ignore"):
            r = b / d.astype(np.float64)[..., None]
        q = np.sign(r) * np.floor(np.abs(r) + 0.5)
        q = np.clip(q, -127, 127)
    else:
        m = np.take_along_axis(b, np.abs(b).argmax(-1)[..., None], -1)[..., 0]
        d = (m / -8).astype(np.float32).astype(np.float16)
        with np.errstate(divide="ignore", invalid="ignore"):
            q = np.clip(np.floor(b / d.astype(np.float64)[..., None] + 8.5), 0, 15) - 8
    return np.where(d[..., None] == 0, 0, q), d


def held(x, t):
    """What a cache of type t holds of float32 rows [..., D], as float64."""
    if t == "f32":
        return x.astype(np.float64)
    if t == "f16":
        return x.astype(np.float16).astype(np.float64)
    q, d = quantize(x.reshape(*x.shape[:-1], -1, 32), t)
    return (q * d.astype(np.float64)[..., None]).reshape(x.shape)


def new_cache(t, kvh, ctx, d, fill=0):
    """k, k_scales, v, v_scales filled with a byte value."""
    def plane(*shape, dtype):
        nbytes = int(np.prod(shape)) * np.dtype(dtype).itemsize
        return torch.full((nbytes,), fill, dtype=torch.uint8, device="cuda").view(
            {"f": torch.float32, "e": torch.float16, "B": torch.uint8}[np.dtype(dtype).char]).view(*shape)
    if t in ("f32", "f16"):
        dt = np.float32 if t == "f32" else np.float16
        return [plane(kvh, ctx, d, dtype=dt), None, plane(kvh, ctx, d, dtype=dt), None]
    cb = d if t == "q8_0" else d // 2
    return [x for _ in range(2) for x in (plane(kvh, ctx, cb, dtype=np.uint8), plane(kvh, ctx, d // 32, dtype=np.float16))]


def write(af, t, cache, k, v, kvh, d, ctx, slots=None, slot0=0, stream=None):
    n, ld = k.shape
    af.af_kv_write(k, v, ld, n, slots, slot0, *cache, af.KVTYPE[t], kvh, d, ctx, stream)


def read(af, t, cache, n, kvh, d, ctx, slots=None, slot0=0, fill=0.0):
    k = torch.full((n, kvh * d), fill, device="cuda")
    v = torch.full((n, kvh * d), fill, device="cuda")
    af.af_kv_read(*cache, af.KVTYPE[t], kvh, d, ctx, n, slots, slot0, k, v, kvh * d)
    return k.cpu().numpy(), v.cpu().numpy()


def hard_rows(rng, n, w):
    """Rows with ordinary values, and blocks that sit on the quantizers' borders."""
    x = rng.standard_normal((n, w)).astype(np.float32)
    b = x.reshape(-1, 32)
    for i in range(0, len(b), 7):
        if i % 3 == 0:
            b[i] = 0
        elif i % 3 == 1:  # exact halves of a scale that is a power of two, and their neighbours in fp32
            h = (rng.integers(-8, 8, 32) + 0.5).astype(np.float32) / 64
            b[i] = np.nextafter(h, rng.choice([-9, 9], 32).astype(np.float32))
            b[i, ::3] = h[::3]
            b[i, 5] = -8 / 64
        else:  # ties of the largest magnitude with both signs, tiny and huge scales
            b[i] *= rng.choice([1e-6, 1e-3, 1e3])
            b[i, 3], b[i, 17] = -np.abs(b[i]).max() - 1e-6, np.abs(b[i]).max() + 1e-6
            b[i, 17] = -b[i, 3]
    return x


@pytest.mark.parametrize("t", KV)
@pytest.mark.parametrize("n,kvh,d,listed", [(1, 1, 32, False), (1, 4, 64, True), (16, 8, 128, True), (37, 5, 96, False),
                                            (300, 8, 128, False), (257, 3, 64, True), (9, 2, 256, True)])
def test_kv_rows_bit_exact(af, t, n, kvh, d, listed):
    rng = np.random.default_rng(n + d)
    ctx, w = n + 21, kvh * d
    k, v = hard_rows(rng, n, w), hard_rows(rng, n, w)
    kd = torch.full((n, w + 4), float("nan"), device="cuda")  # rows of a wider buffer
    vd = torch.full((n, w + 4), float("nan"), device="cuda")
    kd[:, :w], vd[:, :w] = _dev(k), _dev(v)
    cache = new_cache(t, kvh, ctx, d, 0x2A)
    before = [None if c is None else c.clone() for c in cache]
    if listed:
        slots = rng.permutation(ctx)[:n].astype(np.int32)
        if n > 4:
            slots[1], slots[n // 2] = -1, ctx
        live = np.flatnonzero((slots >= 0) & (slots < ctx))
        write(af, t, cache, kd, vd, kvh, d, ctx, _dev(slots))
        gk, gv = read(af, t, cache, n, kvh, d, ctx, _dev(slots), fill=5.0)
        assert np.all(gk[np.setdiff1d(np.arange(n), live)] == 5.0)
    else:
        slots = np.arange(n, dtype=np.int32) + 13
        live = np.arange(n)
        write(af, t, cache, kd, vd, kvh, d, ctx, slot0=13)
        gk, gv = read(af, t, cache, n, kvh, d, ctx, slot0=13)
    assert np.array_equal(gk[live].astype(np.float64).reshape(-1, kvh, d), held(k.reshape(n, kvh, d), t)[live])
    assert np.array_equal(gv[live].astype(np.float64).reshape(-1, kvh, d), held(v.reshape(n, kvh, d), t)[live])
    other = np.setdiff1d(np.arange(ctx), slots[live])  # every other slot is as it was
    for a, b in zip(cache, before):
        if a is not None:
            assert torch.equal(a[:, other].view(torch.uint8), b[:, other].view(torch.uint8))


@pytest.mark.parametrize("t", ["q8_0", "q4_0"])
def test_kv_codes_are_the_models_store_format(af, t):
    """Code bytes and scales as af_model_kv_store's: Q8_0 int8 in element order, Q4_0 nibble pairs of n = q + 8."""
    rng = np.random.default_rng(5)
    k = rng.standard_normal((2, 64)).astype(np.float32)
    cache = new_cache(t, 1, 4, 64)
    write(af, t, cache, _dev(k), _dev(k), 1, 64, 4, slot0=1)
    q, d = quantize(k.reshape(2, 2, 32), t)
    codes = cache[0].cpu().numpy()[0, 1:3]
    got = codes.view(np.int8).astype(int) if t == "q8_0" else np.stack((codes & 15, codes >> 4), -1).reshape(2, 64).astype(int) - 8
    assert np.array_equal(got, q.reshape(2, 64))
    assert np.array_equal(cache[1].cpu().numpy()[0, 1:3], d)


@pytest.mark.parametrize("t", KV)
def test_kv_same_slot_twice_last_row_wins(af, t):
    rng = np.random.default_rng(6)
    n, kvh, d, ctx = 700, 2, 64, 50
    k = rng.standard_normal((n, kvh * d)).astype(np.float32)
    slots = rng.integers(-1, ctx, n).astype(np.int32)
    cache = new_cache(t, kvh, ctx, d)
    write(af, t, cache, _dev(k), _dev(-k), kvh, d, ctx, _dev(slots))
    gk, gv = read(af, t, cache, ctx, kvh, d, ctx)
    for s in range(ctx):
        rows = np.flatnonzero(slots == s)
        if len(rows):
            assert np.array_equal(gk[s].astype(np.float64), held(k[rows[-1]].reshape(kvh, d), t).reshape(-1)), s
            assert np.array_equal(gv[s].astype(np.float64), held(-k[rows[-1]].reshape(kvh, d), t).reshape(-1)), s


@pytest.mark.parametrize("n", [4000, 9001, 33333])
def test_kv_many_listed_rows_last_row_wins(af, n):
    """Lists so long that blocks search for several rows at once."""
    kvh, d, ctx = 1, 32, 3001
    rng = np.random.default_rng(n)
    k = rng.standard_normal((n, kvh * d)).astype(np.float32)
    slots = rng.integers(-2, ctx + 2, n).astype(np.int32)
    slots[-1] = slots[0] = 7
    cache = new_cache("f32", kvh, ctx, d)
    write(af, "f32", cache, _dev(k), _dev(-k), kvh, d, ctx, _dev(slots))
    want = np.zeros((ctx, kvh * d), np.float32)
    for r, s in enumerate(slots):
        if 0 <= s < ctx:
            want[s] = k[r]
    gk, gv = read(af, "f32", cache, ctx, kvh, d, ctx)
    assert np.array_equal(gk, want) and np.array_equal(gv, -want)


@pytest.mark.parametrize("t", ["q8_0", "q4_0"])
def test_kv_non_finite_blocks_read_back_as_nan(af, t):
    k = np.random.default_rng(7).standard_normal((1, 128)).astype(np.float32)
    v = k.copy()
    k[0, 3], k[0, 40], k[0, 70] = np.nan, np.inf, -np.inf
    v[0, 100] = 3e38  # the scale overflows fp16
    cache = new_cache(t, 1, 2, 128)
    write(af, t, cache, _dev(k), _dev(v), 1, 128, 2)
    gk, gv = read(af, t, cache, 1, 1, 128, 2)
    assert np.all(np.isnan(gk[0, :96])) and np.array_equal(gk[0, 96:].astype(np.float64), held(k[0, 96:], t))
    assert np.all(np.isnan(gv[0, 96:])) and np.array_equal(gv[0, :96].astype(np.float64), held(v[0, :96], t))


@pytest.mark.parametrize("t", KV)
def test_kv_read_then_write_moves_slots(af, t):
    rng = np.random.default_rng(8)
    kvh, d, ctx, n = 8, 128, 64, 40
    k, v = rng.standard_normal((n, kvh * d)).astype(np.float32), rng.standard_normal((n, kvh * d)).astype(np.float32)
    cache = new_cache(t, kvh, ctx, d)
    write(af, t, cache, _dev(k), _dev(v), kvh, d, ctx)
    path = np.array([3, 4, 9, 17, 39], np.int32)
    before = [None if c is None else c[:, path.astype(np.int64)].clone() for c in cache]
    gk, gv = read(af, t, cache, 5, kvh, d, ctx, _dev(path))
    write(af, t, cache, _dev(gk), _dev(gv), kvh, d, ctx, slot0=50)
    for a, b in zip(cache, before):
        if a is not None:
            assert torch.equal(a[:, 50:55].contiguous().view(torch.uint8), b.view(torch.uint8))


# ---------------------------------------------------------------- trees

def closure(parent):
    n = len(parent)
    see, depth = np.zeros((n, n), bool), np.zeros(n, int)
    for i, p in enumerate(parent):
        if 0 <= p < i:
            see[i], depth[i] = see[p], depth[p] + 1
        see[i, i] = True
    return see, depth


def pack(see):
    n = see.shape[0]
    w = (n + 31) // 32
    bits = np.zeros((n, w * 32), np.uint64)
    bits[:, :n] = see
    words = (bits.reshape(n, w, 32) << np.arange(32, dtype=np.uint64)).sum(-1)
    return words.astype(np.uint32).view(np.int32)


def random_parents(rng, n):
    return np.array([max(-1, i - 1 - int(rng.random() ** 2 * 8)) for i in range(n)], np.int32)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 64, 100, 1000, 1024])
@pytest.mark.parametrize("kind", ["random", "chain", "star", "wild"])
def test_tree_mask(af, n, kind):
    rng = np.random.default_rng(n)
    parent = {"random": random_parents(rng, n), "chain": np.arange(n) - 1, "star": np.full(n, -1),
              "wild": rng.integers(-5, n + 5, n)}[kind].astype(np.int32)
    see, depth = closure(parent)
    mask = torch.full((n + 1, (n + 31) // 32), 0x55, dtype=torch.int32, device="cuda")
    pos = torch.full((n + 1,), -7, dtype=torch.int32, device="cuda")
    af.af_tree_mask(_dev(parent), n, 1000, mask, pos)
    assert np.array_equal(mask[:n].cpu().numpy(), pack(see))
    assert np.array_equal(pos[:n].cpu().numpy(), 1000 + depth)
    assert int(pos[n]) == -7 and bool((mask[n] == 0x55).all())
    again = torch.empty_like(mask)
    af.af_tree_mask(_dev(parent), n, 0, again)  # without positions
    assert torch.equal(again[:n], mask[:n])


def attn_ref(q, k, v, see, past):
    """q [n, H, D], k, v [KVH, past + n, D] float64, see [n, n]: row by row over what the row sees."""
    n, H, D = q.shape
    G = H // k.shape[0]
    out = np.zeros((n, H, D))
    for i in range(n):
        at = np.concatenate([np.arange(past), past + np.flatnonzero(see[i])])
        if not len(at):
            continue
        for g in range(k.shape[0]):
            s = q[i, g * G:(g + 1) * G] @ k[g, at].T / np.sqrt(D)
            p = np.exp(s - s.max(-1, keepdims=True))
            out[i, g * G:(g + 1) * G] = p @ v[g, at] / p.sum(-1, keepdims=True)
    return out


def attn_tol(q, k, v):
    """Scores in fp32 or from parts that keep 22 bits: |ds| <= 2^-20 sum |q||k| / sqrt(D) (the parts' 2^-21 and the sum's
    roundings); p then moves by ds relative, the average of v by at most twice that times max |v|, and the parts of
    p and v, the exponential and the sums add 2^-19 max |v|."""
    D = q.shape[-1]
    qa, ka = np.abs(q).max(0).max(0), np.abs(k).max(0).max(0)
    return float(np.abs(v).max() * (2 * 2.0 ** -20 * (qa * ka).sum() / np.sqrt(D) + 2.0 ** -19))


def attend(af, t, cache, q, H, kvh, d, ctx, past, see, pad=0, stream=None, ws=None, out=None):
    n = q.shape[0]
    qd = torch.full((n, H * d + pad), float("nan"), device="cuda")
    qd[:, :H * d] = _dev(q.reshape(n, H * d).astype(np.float32))
    out = torch.full((n, H * d + pad), 9.0, device="cuda") if out is None else out
    need = af.af_attention_tree_workspace(af.KVTYPE[t], H, kvh, d, past, n)
    if ws is None:
        ws = torch.full((max(need, 256),), 0xFF, dtype=torch.uint8, device="cuda")  # any contents: NaN patterns
    af.af_attention_tree(qd, H * d + pad, *cache, af.KVTYPE[t], H, kvh, d, ctx, past, n, _dev(pack(see)), ws, need, out,
                         H * d + pad, stream)
    return out


def filled(af, t, rng, kvh, d, ctx, m, spread=1.0):
    """A cache whose first m slots hold random rows (written by af_kv_write), the rest 0xFF bytes (NaN)."""
    k = (rng.standard_normal((m, kvh * d)) * spread).astype(np.float32)
    v = rng.standard_normal((m, kvh * d)).astype(np.float32)
    cache = new_cache(t, kvh, ctx, d, 0xFF)
    write(af, t, cache, _dev(k), _dev(v), kvh, d, ctx)
    return cache, held(k.reshape(m, kvh, d), t).transpose(1, 0, 2), held(v.reshape(m, kvh, d), t).transpose(1, 0, 2)


ATTN = [  # H, KVH, D, past, n
    (8, 4, 64, 0, 1), (8, 4, 64, 31, 1), (1, 1, 64, 1, 1), (32, 8, 128, 300, 16), (32, 8, 64, 1024, 17),
    (12, 4, 128, 77, 5), (5, 1, 64, 129, 33), (64, 1, 128, 500, 3), (32, 8, 128, 4097, 64), (8, 8, 128, 0, 100),
    (32, 4, 64, 640, 100), (8, 8, 128, 257, 200), (3, 1, 128, 3000, 40), (24, 8, 64, 2111, 300), (64, 1, 64, 320, 2),
    (32, 4, 64, 15, 31), (16, 2, 128, 255, 128), (7, 7, 64, 63, 9), (2, 2, 128, 3, 700), (4, 1, 64, 1, 1024),
]


@pytest.mark.parametrize("t", KV)
@pytest.mark.parametrize("H,KVH,D,past,n", ATTN)
def test_attention_tree(af, t, H, KVH, D, past, n):
    rng = np.random.default_rng(past * 7 + n)
    ctx = past + n + (n % 3) * 5
    cache, k, v = filled(af, t, rng, KVH, D, ctx, past + n)
    q = rng.standard_normal((n, H, D)).astype(np.float32)
    see, _ = closure(random_parents(rng, n))
    out = attend(af, t, cache, q, H, KVH, D, ctx, past, see, pad=4)
    got = out.cpu().numpy().astype(np.float64)
    assert np.all(got[:, H * D:] == 9.0)
    ref = attn_ref(q.astype(np.float64), k, v, see, past)
    err, tol = np.abs(got[:, :H * D].reshape(n, H, D) - ref).max(), attn_tol(q, k, v)
    print(f"err {err:.2e} tol {tol:.2e} rel {np.linalg.norm(got[:, :H * D].ravel() - ref.ravel()) / np.linalg.norm(ref):.2e}")
    assert err <= tol


@pytest.mark.parametrize("t", KV)
@pytest.mark.parametrize("past,n", [(0, 40), (70, 40), (33, 300)])
def test_attention_tree_masks(af, t, past, n):
    """Rows that see nothing, everything, one slot, later slots (any mask goes, not only a tree's)."""
    H, KVH, D = 8, 2, 128
    rng = np.random.default_rng(n)
    cache, k, v = filled(af, t, rng, KVH, D, past + n, past + n)
    q = rng.standard_normal((n, H, D)).astype(np.float32)
    see = rng.random((n, n)) < 0.3
    see[0], see[1], see[2] = False, True, False
    see[2, n - 1] = True
    see[5:25] = False
    got = attend(af, t, cache, q, H, KVH, D, past + n, past, see).cpu().numpy().astype(np.float64).reshape(n, H, D)
    ref = attn_ref(q.astype(np.float64), k, v, see, past)
    assert np.abs(got - ref).max() <= attn_tol(q, k, v)
    if past == 0:
        assert np.all(got[5:25] == 0.0) and np.all(got[0] == 0.0)


@pytest.mark.parametrize("t", KV)
@pytest.mark.parametrize("what", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("past,n", [(50, 20), (0, 130)])
def test_attention_tree_hidden_slots_reach_no_row(af, t, what, past, n):
    """A slot that holds NaN or infinities changes the rows that see it and no other."""
    H, KVH, D = 8, 2, 64
    rng = np.random.default_rng(11)
    cache, k, v = filled(af, t, rng, KVH, D, past + n, past + n)
    q = rng.standard_normal((n, H, D)).astype(np.float32)
    see, _ = closure(random_parents(rng, n))
    see[:, 3] = False
    see[7, 3] = True
    clean = attend(af, t, cache, q, H, KVH, D, past + n, past, see).cpu().numpy()
    bad = torch.full((1, KVH * D), float(what), device="cuda")
    write(af, t, cache, bad, bad, KVH, D, past + n, slot0=past + 3)
    got = attend(af, t, cache, q, H, KVH, D, past + n, past, see).cpu().numpy()
    rest = np.arange(n) != 7
    assert np.abs(got[rest] - clean[rest]).max() <= attn_tol(q.astype(np.float64), k, v)  # (False for a NaN)
    assert not np.array_equal(got[7], clean[7])


@pytest.mark.parametrize("t,what", [("f32", "k"), ("f16", "k"), ("f32", "v"), ("f16", "v"), ("q8_0", "v"), ("q4_0", "v")])
@pytest.mark.parametrize("n", [3, 24, 70])
def test_attention_tree_infinities_in_the_past(af, t, what, n):
    """An infinite key, value or value's scale among the slots that every row sees: a result is what the definition gives
    or not finite, never a finite number that left slots out."""
    H, KVH, D, past = 8, 2, 128, 300
    rng = np.random.default_rng(19)
    cache, k, v = filled(af, t, rng, KVH, D, past + n, past + n)
    q = rng.standard_normal((n, H, D)).astype(np.float32)
    see, _ = closure(random_parents(rng, n))
    tol = attn_tol(q, k, v)
    ki, ksi, vi, vsi = cache
    x, scales = (ki, ksi) if what == "k" else (vi, vsi)
    if t in ("f32", "f16"):
        x.view(torch.float32 if t == "f32" else torch.float16).view(KVH, past + n, D)[:, 37, 40] = float("inf")
    else:
        scales.view(torch.float16).view(KVH, past + n, D // 32)[:, 37, 1] = float("inf")
    got = attend(af, t, cache, q, H, KVH, D, past + n, past, see).cpu().numpy().astype(np.float64).reshape(n, H, D)
    if what == "k":
        k = k.copy()
        k[:, 37, 40] = np.inf
    else:
        assert not np.isfinite(got[:, :, 40]).any()
    with np.errstate(invalid="ignore"):
        ref = attn_ref(q.astype(np.float64), k, v, see, past)
    assert not np.isfinite(got[~np.isfinite(ref)]).any()
    fine = np.isfinite(got)
    assert np.abs(got - ref)[fine].max(initial=0) <= tol


@pytest.mark.parametrize("t", KV)
def test_attention_tree_wide_scores_and_small_values(af, t):
    """Scores far apart (one slot takes nearly all the weight), and values whose sizes differ by blocks and slots."""
    H, KVH, D, past, n = 8, 2, 128, 700, 24
    rng = np.random.default_rng(12)
    m = past + n
    k = (rng.standard_normal((m, KVH * D)) * 6).astype(np.float32)
    v = (rng.standard_normal((m, KVH * D)) * np.exp(rng.uniform(-6, 3, (m, 1)))).astype(np.float32)
    cache = new_cache(t, KVH, m, D)
    write(af, t, cache, _dev(k), _dev(v), KVH, D, m)
    q = (rng.standard_normal((n, H, D)) * 4).astype(np.float32)
    see, _ = closure(random_parents(rng, n))
    got = attend(af, t, cache, q, H, KVH, D, m, past, see).cpu().numpy().astype(np.float64).reshape(n, H, D)
    kh, vh = held(k.reshape(m, KVH, D), t).transpose(1, 0, 2), held(v.reshape(m, KVH, D), t).transpose(1, 0, 2)
    assert np.abs(got - attn_ref(q.astype(np.float64), kh, vh, see, past)).max() <= attn_tol(q, kh, vh)


@pytest.mark.parametrize("t,scale", [("f32", 1e-4), ("f32", 3e4), ("f16", 1e-4), ("f16", 1e4), ("q8_0", 1e-3), ("q8_0", 1e4),
                                     ("q4_0", 1e-3), ("q4_0", 1e4)])
@pytest.mark.parametrize("past,n", [(200, 3), (200, 70), (900, 70)])
def test_attention_tree_scale_of_values(af, t, scale, past, n):
    """The result scales with the values: nothing under- or overflows on the way, at small row counts or large."""
    H, KVH, D = 8, 2, 64
    rng = np.random.default_rng(13)
    m = past + n
    k = rng.standard_normal((m, KVH * D)).astype(np.float32)
    v = (rng.standard_normal((m, KVH * D)) * scale).astype(np.float32)
    cache = new_cache(t, KVH, m, D)
    write(af, t, cache, _dev(k), _dev(v), KVH, D, m)
    q = rng.standard_normal((n, H, D)).astype(np.float32)
    see, _ = closure(random_parents(rng, n))
    got = attend(af, t, cache, q, H, KVH, D, m, past, see).cpu().numpy().astype(np.float64).reshape(n, H, D)
    kh, vh = held(k.reshape(m, KVH, D), t).transpose(1, 0, 2), held(v.reshape(m, KVH, D), t).transpose(1, 0, 2)
    assert np.abs(got - attn_ref(q.astype(np.float64), kh, vh, see, past)).max() <= attn_tol(q, kh, vh)


@pytest.mark.parametrize("t", ["f32", "f16"])
def test_attention_tree_of_one_node_is_decode_attention(af, t):
    H, KVH, D, past = 32, 8, 128, 1000
    rng = np.random.default_rng(14)
    cache, k, v = filled(af, t, rng, KVH, D, past + 1, past + 1)
    q = rng.standard_normal((1, H, D)).astype(np.float32)
    got = attend(af, t, cache, q, H, KVH, D, past + 1, past, np.ones((1, 1), bool)).cpu().numpy()
    dec = torch.empty(H * D, device="cuda")
    af.af_attention_decode(_dev(q.reshape(-1)), cache[0], cache[2], af.KVTYPE[t], H, KVH, D, past + 1, past, dec)
    assert np.abs(got.reshape(-1) - dec.cpu().numpy()).max() <= 2 * 1e-3 * np.abs(got).max()  # both within 1e-3 normwise


@pytest.mark.parametrize("t", KV)
@pytest.mark.parametrize("past,n", [(2000, 8), (900, 96)])
def test_attention_tree_repeats_captures_and_streams(af, t, past, n):
    """The same bits from call to call, from a replayed graph over new inputs, and from two streams at once."""
    H, KVH, D = 32, 8, 128
    rng = np.random.default_rng(15)
    ctx = past + n
    cache, k, v = filled(af, t, rng, KVH, D, ctx, ctx)
    qs = [rng.standard_normal((n, H * D)).astype(np.float32) for _ in range(2)]
    see, _ = closure(random_parents(rng, n))
    want = [attend(af, t, cache, q, H, KVH, D, ctx, past, see) for q in qs]
    assert torch.equal(want[0], attend(af, t, cache, qs[0], H, KVH, D, ctx, past, see))
    need = max(256, af.af_attention_tree_workspace(af.KVTYPE[t], H, KVH, D, past, n))
    q, out, mask = _dev(qs[0]), torch.zeros(n, H * D, device="cuda"), _dev(pack(see))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        af.af_attention_tree(q, H * D, *cache, af.KVTYPE[t], H, KVH, D, ctx, past, n, mask, ws, need, out, H * D)
    for i in (1, 0, 1):
        q.copy_(_dev(qs[i]))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])
    streams = [torch.cuda.Stream() for _ in range(2)]
    bufs = [(_dev(qs[i]), torch.empty(need, dtype=torch.uint8, device="cuda"), torch.zeros(n, H * D, device="cuda"))
            for i in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (qd, w, o) in zip(streams, bufs):
            af.af_attention_tree(qd, H * D, *cache, af.KVTYPE[t], H, KVH, D, ctx, past, n, mask, w, need, o, H * D, s)
    torch.cuda.synchronize()
    assert torch.equal(bufs[0][2], want[0]) and torch.equal(bufs[1][2], want[1])


@pytest.mark.parametrize("t", KV)
@pytest.mark.parametrize("past,n", [(2000, 8), (900, 96)])
@pytest.mark.parametrize("nstreams", [1, 2])
def test_attention_tree_calls_in_a_row(af, t, past, n, nstreams):
    """Calls that follow one another without a pause (a call's blocks start while the one before it ends) give the bits of
    a call by itself."""
    H, KVH, D = 32, 8, 128
    rng = np.random.default_rng(17)
    ctx = past + n
    cache, k, v = filled(af, t, rng, KVH, D, ctx, ctx)
    q = rng.standard_normal((n, H * D)).astype(np.float32)
    see, _ = closure(random_parents(rng, n))
    want = attend(af, t, cache, q, H, KVH, D, ctx, past, see)
    need = max(256, af.af_attention_tree_workspace(af.KVTYPE[t], H, KVH, D, past, n))
    qd, mask = _dev(q), _dev(pack(see))
    streams = [torch.cuda.Stream() for _ in range(nstreams)]
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in streams]
    outs = [[torch.zeros(n, H * D, device="cuda") for _ in range(20)] for _ in streams]
    torch.cuda.synchronize()
    for i in range(20):
        for s, w, o in zip(streams, ws, outs):
            af.af_attention_tree(qd, H * D, *cache, af.KVTYPE[t], H, KVH, D, ctx, past, n, mask, w, need, o[i], H * D, s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for o in outs for x in o)


@pytest.mark.parametrize("t", KV)
@pytest.mark.parametrize("past,n", [(500, 8), (60, 64)])
def test_attention_tree_sees_rows_written_just_before(af, t, past, n):
    """Writes and attention in turn, without a pause between them: each attention sees the rows written before it, and no
    older ones that an SM still holds."""
    H, KVH, D = 32, 8, 128
    rng = np.random.default_rng(20)
    ctx = past + n + 3
    cache, _, _ = filled(af, t, rng, KVH, D, ctx, past + n)
    rows = [_dev((rng.standard_normal((n, KVH * D)) * 4.0 ** i).astype(np.float32)) for i in range(3)]
    q = _dev(rng.standard_normal((n, H * D)).astype(np.float32))
    see, _ = closure(random_parents(rng, n))
    mask = _dev(pack(see))
    need = max(256, af.af_attention_tree_workspace(af.KVTYPE[t], H, KVH, D, past, n))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def step(i, out):
        write(af, t, cache, rows[i], rows[i], KVH, D, ctx, slot0=past)
        af.af_attention_tree(q, H * D, *cache, af.KVTYPE[t], H, KVH, D, ctx, past, n, mask, ws, need, out, H * D)

    want = [torch.zeros(n, H * D, device="cuda") for _ in rows]
    for i, out in enumerate(want):
        torch.cuda.synchronize()
        step(i, out)
    outs = [torch.zeros(n, H * D, device="cuda") for _ in range(30)]
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        step(i % 3, out)
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[i % 3]) for i, x in enumerate(outs))


@pytest.mark.parametrize("t", ["f32", "f16"])
@pytest.mark.parametrize("ctx", [1024, 6000])
@pytest.mark.parametrize("how", ["write", "rope"])
def test_decode_attention_sees_a_cache_changed_just_before(af, t, ctx, how):
    """The decode attention reads ahead in the cache, so the kernel before it must not let it start early."""
    H, KVH, D, pos = 32, 8, 128, ctx - 1
    rng = np.random.default_rng(21)
    cache, _, _ = filled(af, t, rng, KVH, D, ctx, ctx)
    rows = [_dev((rng.standard_normal((ctx, KVH * D)) * 2.0 ** i).astype(np.float32)) for i in range(2)]
    q = _dev(rng.standard_normal(H * D).astype(np.float32))
    cfg = af.rope_config(D, D, "half", 10000.0)
    keys = [cache[0].clone(), cache[0].flip(1).contiguous()]

    def step(i, out):
        if how == "write":
            write(af, t, cache, rows[i], rows[i], KVH, D, ctx)
        else:
            af.af_rope(cfg, keys[i], D, cache[0], D, af.AF_F32 if t == "f32" else af.AF_F16, KVH * ctx, 1, None, 0)
        af.af_attention_decode_static(q, cache[0], cache[2], af.KVTYPE[t], H, KVH, D, ctx, pos, out)

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
    assert all(torch.equal(x, want[i % 2]) for i, x in enumerate(outs))


@pytest.mark.parametrize("t", KV)
@pytest.mark.parametrize("ctx", [1024, 6000])
def test_decode_attention_sees_slots_read_back_just_before(af, t, ctx):
    """A kv head's slots, read back by one call a head, are an fp32 cache for the decode attention behind them."""
    H, KVH, D, pos = 32, 8, 128, ctx - 1
    rng = np.random.default_rng(22)
    src = [filled(af, t, rng, KVH, D, ctx, ctx)[0] for _ in range(2)]
    heads = [[[None if x is None else x[h] for x in c] for h in range(KVH)] for c in src]
    k, v = (torch.zeros(KVH, ctx, D, device="cuda") for _ in range(2))
    kd, vd = [k[h] for h in range(KVH)], [v[h] for h in range(KVH)]
    q = _dev(rng.standard_normal(H * D).astype(np.float32))

    def step(i, out):
        for h in range(KVH):
            af.af_kv_read(*heads[i][h], af.KVTYPE[t], 1, D, ctx, ctx, None, 0, kd[h], vd[h], D)
        af.af_attention_decode_static(q, k, v, af.AF_F32, H, KVH, D, ctx, pos, out)

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
    assert all(torch.equal(x, want[i % 2]) for i, x in enumerate(outs))


@pytest.mark.parametrize("t", KV)
def test_attention_tree_long_sums(af, t):
    """Over 125 tiles in one block the error does not grow with their number: the tensor cores cut their sums by up to
    2^-23 at each of the 12 products of a tile, over 2 tiles at most; with the two-part operands, the exponential and the
    row sum (2^-21 together, and as much for the joining of the sums) 24 * 2^-23 + 2^-20 of the result's norm."""
    H, KVH, D, past, n = 8, 8, 128, 15500, 1000
    rng = np.random.default_rng(18)
    cache, k, v = filled(af, t, rng, KVH, D, past + n, past + n)
    q = rng.standard_normal((n, H, D)).astype(np.float32)
    see, _ = closure(random_parents(rng, n))
    got = attend(af, t, cache, q, H, KVH, D, past + n, past, see).double().cpu().view(n, H, D)
    seen = torch.cat((torch.ones(n, past, dtype=torch.bool), torch.from_numpy(see)), 1).cuda()
    err = norm = 0.0
    for h in range(H):
        z = torch.from_numpy(q[:, h].astype(np.float64)).cuda() @ torch.from_numpy(k[h].astype(np.float64)).cuda().T * D ** -0.5
        z = torch.softmax(torch.where(seen, z, -torch.inf), -1) @ torch.from_numpy(v[h].astype(np.float64)).cuda()
        err += float((got[:, h].cuda() - z).square().sum())
        norm += float(z.square().sum())
    print(f"err {(err / norm) ** 0.5:.2e}")
    assert (err / norm) ** 0.5 <= 24 * 2.0 ** -23 + 2.0 ** -20


def on_gpu(af, t, k, v, kvh, d):
    """A cache of k, v [m, kvh, d] (device, fp32) and what it holds, float64 [kvh, m, d] on the device."""
    m = k.shape[0]
    cache = new_cache(t, kvh, m, d)
    write(af, t, cache, k.reshape(m, kvh * d), v.reshape(m, kvh * d), kvh, d, m)
    back = [torch.empty(m, kvh * d, device="cuda") for _ in range(2)]
    af.af_kv_read(*cache, af.KVTYPE[t], kvh, d, m, m, None, 0, *back, kvh * d)
    return cache, *(x.view(m, kvh, d).transpose(0, 1).double() for x in back)


def attn_ref_gpu(q, k, v, see, past):
    """attn_ref on the device: q [n, H, D] float32 array, k and v [KVH, m, D] float64 on the device -> [n, H, D]."""
    n, H, D = q.shape
    G = H // k.shape[0]
    seen = torch.cat((torch.ones(n, past, dtype=torch.bool), torch.from_numpy(see)), 1).cuda()
    out = torch.empty(n, H, D, dtype=torch.float64, device="cuda")
    for h in range(H):
        z = torch.from_numpy(q[:, h].astype(np.float64)).cuda() @ k[h // G].T * D ** -0.5
        out[:, h] = torch.softmax(torch.where(seen, z, -torch.inf), -1) @ v[h // G]
    return out


LARGE = [("f32", 1e3), ("f32", 1e4), ("f32", 1e6), ("f32", 1e30), ("f32", float(np.finfo(np.float32).max)),
         ("f16", 65504.0), ("q8_0", 1e3), ("q8_0", 1e6), ("q8_0", 127 * 65504.0), ("q4_0", 1e3), ("q4_0", 8 * 65504.0)]


@pytest.mark.parametrize("t,size", LARGE)
@pytest.mark.parametrize("what", ["k", "v", "kv"])
@pytest.mark.parametrize("D,past,n", [(64, 50, 20), (128, 50, 24), (128, 0, 130), (64, 300, 130)])
def test_attention_tree_large_hidden_slots_reach_no_row(af, t, size, what, D, past, n):
    """A slot that holds large finite numbers (an unwritten one of a padded tree, a mask's lowest value) costs the rows that
    do not see it nothing, in slots next to it and in later ones.  In the result's norm: the parts of q, k, p and v move
    scores and products by 2^-21 each, sums, exponential and join by as much: 2^-18 holds them four times over."""
    H, KVH, j = 8, 2, 1
    rng = np.random.default_rng(23)
    m = past + n
    k, v = (rng.standard_normal((m, KVH, D)).astype(np.float32) for _ in range(2))
    q = rng.standard_normal((n, H, D)).astype(np.float32)
    see, _ = closure(random_parents(rng, n))
    see[:, j] = False
    see[j, j] = True
    tol = attn_tol(q, k.transpose(1, 0, 2), v.transpose(1, 0, 2))
    big = (rng.choice([-1.0, 1.0], (KVH, D)) * rng.uniform(0.5, 1, (KVH, D)) * size).astype(np.float32)
    big[:, ::32] = np.float32(size)  # the largest magnitude of each block
    if t == "q4_0":
        big[:, ::32] = -np.float32(size)
    if "k" in what:
        k[past + j] = big
    if "v" in what:
        v[past + j] = big
    cache, kh, vh = on_gpu(af, t, _dev(k), _dev(v), KVH, D)
    assert torch.isfinite(kh).all() and torch.isfinite(vh).all()
    got = attend(af, t, cache, q, H, KVH, D, m, past, see).double().view(n, H, D)
    ref = attn_ref_gpu(q, kh, vh, see, past)
    rest = [i for i in range(n) if i != j]
    err = (got - ref)[rest].abs().max().item()
    assert err <= tol, (err, tol)
    norm = ((got - ref)[rest].norm() / ref[rest].norm()).item()
    print(f"norm {norm:.2e}")
    assert norm <= 2.0 ** -18


@pytest.mark.parametrize("t,size", LARGE)
@pytest.mark.parametrize("what", ["k", "v", "kv"])
@pytest.mark.parametrize("D,past,n", [(64, 50, 2), (128, 50, 3), (64, 40, 7)])
def test_attention_tree_large_hidden_slots_of_few_rows(af, t, size, what, D, past, n):
    test_attention_tree_large_hidden_slots_reach_no_row(af, t, size, what, D, past, n)


@pytest.mark.parametrize("t,size", [("f32", 1e3), ("f32", 1e6), ("f32", 1e30), ("f16", 6e4), ("q8_0", 1e3), ("q8_0", 1e6),
                                    ("q4_0", 1e3), ("q4_0", 1e5)])
@pytest.mark.parametrize("at", [5, 290, 611])
@pytest.mark.parametrize("n", [1, 3, 8, 24, 70])
def test_attention_tree_large_slot_of_no_weight(af, t, size, at, n):
    """A slot that every row sees, with a key far from all queries (its weight is below 2^-150) and large values: the other
    slots' scores and values keep their precision."""
    H, KVH, D, past = 8, 2, 128, 700
    rng = np.random.default_rng(24)
    m = past + n
    k, v = (rng.standard_normal((m, KVH, D)).astype(np.float32) for _ in range(2))
    q = (rng.standard_normal((n, H, D)) + 0.5).astype(np.float32)
    see, _ = closure(random_parents(rng, n))
    tol = attn_tol(q, k.transpose(1, 0, 2), v.transpose(1, 0, 2))
    k[at], v[at] = -200.0, size * rng.choice([-1.0, 1.0], (KVH, D))
    cache, kh, vh = on_gpu(af, t, _dev(k), _dev(v), KVH, D)
    got = attend(af, t, cache, q, H, KVH, D, m, past, see).double().view(n, H, D)
    z = torch.einsum("nhd,hd->nh", torch.from_numpy(q).cuda().double(), kh[:, at].repeat_interleave(H // KVH, 0)) * D ** -0.5
    far = z < -150 - 20  # (the others' scores are above -20)
    assert far.float().mean() > 0.9
    err = ((got - attn_ref_gpu(q, kh, vh, see, past)).abs().amax(-1) * far).max().item()
    assert err <= tol, (err, tol)


SMALL = [  # H, KVH, D, past, n: few rows over many slots
    (32, 32, 128, 8200, 1), (32, 32, 64, 8200, 8), (32, 32, 128, 8200, 12), (32, 32, 64, 8200, 16), (32, 32, 128, 8200, 24),
    (32, 32, 64, 8200, 32), (32, 8, 128, 40000, 2), (32, 8, 128, 40000, 8), (4, 1, 128, 60000, 1), (16, 1, 64, 60000, 2),
]


@pytest.mark.parametrize("t", KV)
@pytest.mark.parametrize("H,KVH,D,past,n", SMALL)
def test_attention_tree_few_rows_over_many_slots(af, t, H, KVH, D, past, n):
    """Long walks of the small-row kernel: its rings go round, maxima and scales of values move on the way, the result is a
    join of many parts.  Scores drift and values grow along the cache."""
    g = torch.Generator(device="cuda").manual_seed(past + n)
    m = past + n
    along = torch.linspace(-1, 1, m, device="cuda")[:, None, None]
    q = torch.randn(n, H, D, generator=g, device="cuda") + 0.3
    k = torch.randn(m, KVH, D, generator=g, device="cuda") + 3 * along
    v = torch.randn(m, KVH, D, generator=g, device="cuda") * torch.exp(3 * along)
    cache, kh, vh = on_gpu(af, t, k, v, KVH, D)
    see = np.tril(np.ones((n, n), bool))
    q = q.cpu().numpy()
    splits = af.af_attention_tree_workspace(af.KVTYPE[t], H, KVH, D, past, n) // (n * H * (D + 2) * 4)
    if KVH == 1:
        assert splits > 32
    else:  # at most 384 slots a round of a block's warps
        assert 1 < splits and m / splits > 5 * 384
    got = attend(af, t, cache, q, H, KVH, D, m, past, see).double().view(n, H, D)
    tol = attn_tol(q, kh.cpu().numpy(), vh.cpu().numpy())
    err = (got - attn_ref_gpu(q, kh, vh, see, past)).abs().max().item()
    print(f"err {err:.2e} tol {tol:.2e}")
    assert err <= tol, (err, tol)


@pytest.mark.parametrize("t", KV)
@pytest.mark.parametrize("D,n", [(128, 1), (128, 8), (128, 16), (64, 8), (64, 16), (128, 32)])
def test_attention_tree_few_rows_long_sums(af, t, D, n):
    """Values of one sign over some 80 stages a warp: the tensor cores cut their sums (by up to 2^-23 at each product, always
    towards zero), so a sum of all of them would be off by 3e-5.  A stage's sum starts from zero: at most 12 products,
    12 * 2^-23, and 2^-20 for the parts, the exponential, the row sum and the joining of the sums, of the result's norm."""
    H = KVH = 32
    past = 30000
    g = torch.Generator(device="cuda").manual_seed(n)
    m = past + n
    k = torch.randn(m, KVH, D, generator=g, device="cuda")
    v = torch.rand(m, KVH, D, generator=g, device="cuda") + 0.5
    q = torch.randn(n, H, D, generator=g, device="cuda").cpu().numpy()
    cache, kh, vh = on_gpu(af, t, k, v, KVH, D)
    see = np.tril(np.ones((n, n), bool))
    got = attend(af, t, cache, q, H, KVH, D, m, past, see).double().view(n, H, D)
    ref = attn_ref_gpu(q, kh, vh, see, past)
    err = ((got - ref).norm() / ref.norm()).item()
    print(f"err {err:.2e} mean {((got - ref) / ref).mean().item():.2e}")
    assert err <= 12 * 2.0 ** -23 + 2.0 ** -20


@pytest.mark.parametrize("t", KV)
@pytest.mark.parametrize("H,KVH,D,past,n", [(8, 8, 128, 1000, 1), (32, 8, 128, 6000, 3), (8, 2, 128, 6000, 3), (32, 8, 64, 6000, 3),
                                            (32, 8, 128, 1000, 8), (8, 2, 128, 6000, 40), (8, 8, 64, 3454, 14)])
def test_attention_tree_scores_are_not_cut_over_the_whole_head(af, t, H, KVH, D, past, n):
    """Scores summed 32 dims at a time: 12 products, each cut by half of 2^-23 of the sum so far on average, and that grows
    evenly, so together by 6.5 * 2^-24 of the block's score, which moves the slot's weight by as much; and 2^-21 of the
    result's norm for all else (parts, exponential and row sum are off by 2^-22 at random).  tcgen05 sums the small lo
    products first, then 8 over the head."""
    m = past + n
    g = torch.Generator(device="cuda").manual_seed(past)
    q = torch.randn(n, H, D, generator=g, device="cuda")
    k = torch.randn(m, KVH, D, generator=g, device="cuda") * torch.exp(0.5 * torch.randn(1, KVH, D, generator=g, device="cuda"))
    v = torch.randn(m, KVH, D, generator=g, device="cuda")
    cache, kh, vh = on_gpu(af, t, k, v, KVH, D)
    see = np.tril(np.ones((n, n), bool))
    got = attend(af, t, cache, q.cpu().numpy(), H, KVH, D, m, past, see).double().view(n, H, D)
    ref = attn_ref_gpu(q.cpu().numpy(), kh, vh, see, past)
    blocks = torch.einsum("nhbd,hmbd->nhmb", q.double().view(n, H, -1, 32),
                          kh.repeat_interleave(H // KVH, 0).view(H, m, -1, 32)).abs().sum(-1).mean().item() * D ** -0.5
    err = ((got - ref).norm() / ref.norm()).item()
    print(f"err {err:.2e} bound {6.5 * 2.0 ** -24 * blocks + 2.0 ** -21:.2e}")
    assert err <= 6.5 * 2.0 ** -24 * blocks + 2.0 ** -21


@pytest.mark.parametrize("t", KV)
@pytest.mark.parametrize("D,n", [(128, 1), (128, 16), (64, 32), (128, 70)])
@pytest.mark.parametrize("run", [16, 384])
def test_attention_tree_sizes_of_values_that_take_turns(af, t, D, n, run):
    """Values of one sign whose size changes 64-fold every few slots: the powers of two that follow them lose nothing.  The
    bound of the long sums (tcgen05: 24 products over two tiles)."""
    H = KVH = 32
    past = 12000
    m = past + n
    g = torch.Generator(device="cuda").manual_seed(n)
    turn = (torch.arange(m, device="cuda") // run % 2 * 6 - 3).float().exp2()[:, None, None]
    k = torch.randn(m, KVH, D, generator=g, device="cuda")
    v = (torch.rand(m, KVH, D, generator=g, device="cuda") + 0.5) * turn
    q = torch.randn(n, H, D, generator=g, device="cuda").cpu().numpy()
    cache, kh, vh = on_gpu(af, t, k, v, KVH, D)
    see = np.tril(np.ones((n, n), bool))
    got = attend(af, t, cache, q, H, KVH, D, m, past, see).double().view(n, H, D)
    ref = attn_ref_gpu(q, kh, vh, see, past)
    err = ((got - ref).norm() / ref.norm()).item()
    print(f"err {err:.2e}")
    assert err <= 24 * 2.0 ** -23 + 2.0 ** -20


@pytest.mark.parametrize("t", KV)
@pytest.mark.parametrize("H,KVH,D,n", [(1, 1, 64, 33), (4, 1, 128, 9), (40, 1, 64, 1), (64, 1, 128, 40)])
def test_attention_tree_of_a_cache_smaller_than_a_tile(af, t, H, KVH, D, n):
    rng = np.random.default_rng(27)
    cache, k, v = filled(af, t, rng, KVH, D, n, n)
    q = rng.standard_normal((n, H, D)).astype(np.float32)
    see, _ = closure(random_parents(rng, n))
    got = attend(af, t, cache, q, H, KVH, D, n, 0, see).cpu().numpy().reshape(n, H, D)
    assert np.abs(got - attn_ref(q.astype(np.float64), k, v, see, 0)).max() <= attn_tol(q, k, v)


@pytest.mark.parametrize("t,qv,kv", [("f32", 0.5, -np.inf), ("f16", 0.5, -np.inf), ("f32", 2.0 ** 68, -2.0 ** 68)])
@pytest.mark.parametrize("past,n", [(0, 2), (40, 3), (600, 3), (0, 70), (600, 70)])
def test_attention_tree_rows_that_see_only_minus_infinity(af, t, qv, kv, past, n):
    """Scores that are all -infinity (or below fp32's range) have no softmax: such a row is not the zeros of a row that sees
    nothing."""
    H, KVH, D = 8, 2, 64
    m = past + n
    q = np.full((n, H, D), qv, np.float32)
    k = torch.full((m, KVH, D), kv, device="cuda")
    see = np.eye(n, dtype=bool)
    if past == 0:
        see[0] = False
    cache = new_cache(t, KVH, m, D)
    write(af, t, cache, k.view(m, -1), torch.ones(m, KVH * D, device="cuda"), KVH, D, m)
    got = attend(af, t, cache, q, H, KVH, D, m, past, see)
    blind = 1 if past == 0 else 0
    assert got[blind:].isnan().all()
    assert (got[:blind] == 0).all()


def test_attention_tree_workspace_has_a_bound(af):
    """Smaller calls may need more scratch than larger ones, but none more than 512 * SMs * (head_dim + 2) bytes."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    shapes = [(1, 1, 64), (8, 4, 64), (32, 8, 128), (64, 1, 128), (40, 5, 128), (32, 32, 64), (96, 96, 128), (128, 2, 64),
              (300, 150, 64)]
    for t in KV:
        for H, KVH, D in shapes:
            need = [af.af_attention_tree_workspace(af.KVTYPE[t], H, KVH, D, past, n)
                    for past in (0, 100, 700, 1500, 1600, 4096, 9000, 30000, 1 << 20) for n in range(1, 1025)]
            assert max(need) <= 512 * sms * (D + 2), (t, H, KVH, D)
            assert max(need) > 0 or KVH > sms // 2  # (one split a head fills the SMs)
    H, KVH, D, past = 32, 8, 128, 4096
    ws = torch.empty(512 * sms * (D + 2), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(25)
    cache, k, v = filled(af, "f16", rng, KVH, D, past + 40, past + 40)
    for n in (1, 8, 32, 33, 40):  # 32 nodes need more than 33
        q = rng.standard_normal((n, H, D)).astype(np.float32)
        see = np.tril(np.ones((n, n), bool))
        out = torch.empty(n, H * D, device="cuda")
        af.af_attention_tree(_dev(q.reshape(n, H * D)), H * D, *cache, af.AF_F16, H, KVH, D, past + 40, past, n, _dev(pack(see)),
                             ws, ws.numel(), out, H * D)
        ref = attn_ref(q.astype(np.float64), k[:, :past + n], v[:, :past + n], see, past)
        assert np.abs(out.cpu().numpy().reshape(n, H, D) - ref).max() <= attn_tol(q, k, v)


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("t", KV)
@pytest.mark.parametrize("n", [5, 40])
def test_draft_step_in_one_graph(af, t, n):
    """Mask, rotation, write, attention and read of a drafted tree, captured together and replayed over other inputs, give
    the bits of the calls one by one."""
    H, KVH, D, past, ctx = 32, 8, 128, 700, 800
    rng = np.random.default_rng(26)
    start, _, _ = filled(af, t, rng, KVH, D, ctx, past)
    w = (H + 2 * KVH) * D
    inputs = [(_dev(rng.standard_normal((n, w)).astype(np.float32)), _dev(random_parents(rng, n).astype(np.int32))) for _ in range(3)]
    cfg = af.rope_config(D, D, "half", 500000.0)
    need = max(256, af.af_attention_tree_workspace(af.KVTYPE[t], H, KVH, D, past, n))
    cache = [None if x is None else x.clone() for x in start]
    rows, parent = inputs[0][0].clone(), inputs[0][1].clone()
    rot, pos = torch.zeros(n, w, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    mask = torch.zeros(n, (n + 31) // 32, dtype=torch.int32, device="cuda")
    ws, out = torch.empty(need, dtype=torch.uint8, device="cuda"), torch.zeros(n, H * D, device="cuda")
    kr, vr = torch.zeros(n, KVH * D, device="cuda"), torch.zeros(n, KVH * D, device="cuda")

    def step(pause):
        for call in (lambda: af.af_tree_mask(parent, n, past, mask, pos),
                     lambda: af.af_rope(cfg, rows, w, rot, w, af.AF_F32, n, H + KVH, pos),
                     lambda: af.af_kv_write(rot[:, H * D:], rows[:, (H + KVH) * D:], w, n, None, past, *cache, af.KVTYPE[t], KVH, D, ctx),
                     lambda: af.af_attention_tree(rot, w, *cache, af.KVTYPE[t], H, KVH, D, ctx, past, n, mask, ws, need, out, H * D),
                     lambda: af.af_kv_read(*cache, af.KVTYPE[t], KVH, D, ctx, n, None, past, kr, vr, KVH * D)):
            call()
            if pause:
                torch.cuda.synchronize()

    def put(i):
        rows.copy_(inputs[i][0])
        parent.copy_(inputs[i][1])
        for x in (rot, pos, mask, out, kr, vr):
            x.zero_()

    want = []
    for i in range(3):
        put(i)
        step(True)
        want.append([x.clone() for x in (rot[:, :(H + KVH) * D], pos, mask, out, kr, vr)])
    assert not torch.equal(want[0][3], want[1][3])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(False)
    for i in (2, 0, 1, 1, 2):
        put(i)
        graph.replay()
        torch.cuda.synchronize()
        got = [rot[:, :(H + KVH) * D], pos, mask, out, kr, vr]
        assert all(torch.equal(x, y) for x, y in zip(got, want[i]))


@pytest.mark.parametrize("t", KV)
def test_draft_verify_and_move(af, t):
    """A drafted tree through rotary positions, cache write, mask and attention equals, node by node, the definition
    on the node's own path; the accepted branch, moved with a read and a write, serves the next call."""
    H, KVH, D, past, n, ctx = 16, 4, 128, 90, 23, 160
    rng = np.random.default_rng(16)
    parent = random_parents(rng, n)
    see, depth = closure(parent)
    cache, k0, v0 = filled(af, t, rng, KVH, D, ctx, past)
    fused = rng.standard_normal((n, (H + 2 * KVH) * D)).astype(np.float32)
    w = fused.shape[1]
    rows, rot = _dev(fused), torch.empty(n, w, device="cuda")
    mask = torch.empty(n, 1, dtype=torch.int32, device="cuda")
    pos = torch.empty(n, dtype=torch.int32, device="cuda")
    cfg = af.rope_config(D, D, "interleaved", 500000.0)
    af.af_tree_mask(_dev(parent), n, past, mask, pos)
    af.af_rope(cfg, rows, w, rot, w, af.AF_F32, n, H + KVH, pos)          # q and k heads in one call
    kd, vd = rot[:, H * D:], rows[:, (H + KVH) * D:]
    af.af_kv_write(kd, vd, w, n, None, past, *cache, af.KVTYPE[t], KVH, D, ctx)
    need = af.af_attention_tree_workspace(af.KVTYPE[t], H, KVH, D, past, n)
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    out = torch.empty(n, H * D, device="cuda")
    af.af_attention_tree(rot, w, *cache, af.KVTYPE[t], H, KVH, D, ctx, past, n, mask, ws, need, out, H * D)
    r = rot.cpu().numpy()
    th = rope_ref(fused[:, :(H + KVH) * D].astype(np.float64).reshape(n, H + KVH, D), [past + int(x) for x in depth], D,
                  "interleaved", turns(D, 500000.0, "none", 1, 1), 1.0)
    assert np.abs(r[:, :(H + KVH) * D].reshape(n, H + KVH, D) - th).max() <= 2 * np.abs(fused).max() * 2.0 ** -20
    q = r[:, :H * D].reshape(n, H, D).astype(np.float64)
    kn = held(r[:, H * D:(H + KVH) * D].reshape(n, KVH, D), t).transpose(1, 0, 2)
    vn = held(fused[:, (H + KVH) * D:].reshape(n, KVH, D), t).transpose(1, 0, 2)
    k, v = np.concatenate([k0, kn], 1), np.concatenate([v0, vn], 1)
    assert np.abs(out.cpu().numpy().reshape(n, H, D) - attn_ref(q, k, v, see, past)).max() <= attn_tol(q, k, v)
    # the accepted branch: the path to the last node, moved to the slots after the past
    path = np.flatnonzero(see[n - 1])
    m = len(path)
    slots = _dev((past + path).astype(np.int32))
    kr, vr = torch.empty(m, KVH * D, device="cuda"), torch.empty(m, KVH * D, device="cuda")
    af.af_kv_read(*cache, af.KVTYPE[t], KVH, D, ctx, m, slots, 0, kr, vr, KVH * D)
    af.af_kv_write(kr, vr, KVH * D, m, None, past, *cache, af.KVTYPE[t], KVH, D, ctx)
    got = attend(af, t, cache, q[n - 1:], H, KVH, D, ctx, past + m - 1, np.ones((1, 1), bool))
    # the same slots in another order of summation
    assert np.abs(got.cpu().numpy().reshape(H, D) - out[n - 1].cpu().numpy().reshape(H, D)).max() <= 2 * attn_tol(q, k, v)
