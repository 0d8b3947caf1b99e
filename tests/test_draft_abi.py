"""Refusals of the drafted-tree operators (af_rope, af_kv_write, af_kv_read, af_tree_mask, af_attention_tree): every
check runs on the host before anything is launched, so no GPU is needed.  Pointers are dummies, never dereferenced."""
import ctypes

import pytest

P = 4096  # an aligned address nothing reads


def _af():
    import gguf_quantized_transformer_gb300 as af
    af.build()
    return af


def _rope(L, af, cfg=None, x=P, y=P, ldx=1024, ldy=1024, dtype=0, n=4, heads=8, pos=P, pos0=0, **kw):
    base = dict(head_dim=128, rot_dim=128, layout="interleaved", base=10000.0)
    base.update(kw)
    c = cfg or af.rope_config(**base)
    return L.af_rope(ctypes.byref(c), x, ldx, y, ldy, dtype, n, heads, pos, pos0, None)


def test_rope_refusals():
    af = _af()
    L = af.lib()
    E, R, N = af.AF_EINVAL, af.AF_ERANGE, af.AF_ENOTIMPL
    assert L.af_rope(None, P, 1024, P, 1024, 0, 4, 8, P, 0, None) == E
    assert _rope(L, af, x=None) == E and _rope(L, af, y=None) == E
    assert _rope(L, af, head_dim=127) == E and _rope(L, af, head_dim=258, rot_dim=2) == N
    assert _rope(L, af, rot_dim=0) == E and _rope(L, af, rot_dim=130) == E and _rope(L, af, rot_dim=63) == E
    assert _rope(L, af, base=1.0) == E and _rope(L, af, base=float("nan")) == E and _rope(L, af, base=float("inf")) == E
    assert _rope(L, af, scaling="linear", factor=0.0) == E and _rope(L, af, scaling="linear", factor=float("inf")) == E
    assert _rope(L, af, scaling="ntk", rot_dim=2, factor=2.0) == E
    assert _rope(L, af, scaling="yarn", factor=2.0, native_ctx=0) == E
    assert _rope(L, af, scaling="yarn", factor=2.0, native_ctx=64, turns_low=32.0, turns_high=32.0) == E
    assert _rope(L, af, magnitude=-1.0) == E and _rope(L, af, magnitude=float("nan")) == E
    c = af.rope_config(128, 128)
    c.layout = 2
    assert _rope(L, af, cfg=c) == E
    c = af.rope_config(128, 128)
    c.scaling = 4
    assert _rope(L, af, cfg=c) == E
    assert _rope(L, af, dtype=2) == E and _rope(L, af, heads=0) == E and _rope(L, af, n=-1) == R
    assert _rope(L, af, ldx=1023) == E and _rope(L, af, ldy=1000) == E
    assert _rope(L, af, x=P + 2) == E and _rope(L, af, pos=P + 1) == E and _rope(L, af, dtype=1, y=P + 1) == E
    assert _rope(L, af, ldy=2048) == E  # in place with another stride
    assert _rope(L, af, pos=None, pos0=2 ** 31 - 4, n=5) == R
    assert _rope(L, af, n=0) == af.AF_OK


def _rows(L, af, write, k=P, v=P, ld=1024, n=4, slots=None, slot0=0, kc=P, ks=None, vc=P, vs=None, t=0, kvh=8, d=128,
          ctx=64):
    if write:
        return L.af_kv_write(k, v, ld, n, slots, slot0, kc, ks, vc, vs, t, kvh, d, ctx, None)
    return L.af_kv_read(kc, ks, vc, vs, t, kvh, d, ctx, n, slots, slot0, k, v, ld, None)


@pytest.mark.parametrize("write", [True, False])
def test_kv_rows_refusals(write):
    af = _af()
    L = af.lib()
    E, R, N = af.AF_EINVAL, af.AF_ERANGE, af.AF_ENOTIMPL
    def call(**kw):
        return _rows(L, af, write, **kw)
    assert call(k=None) == E and call(v=None) == E and call(kc=None) == E and call(vc=None) == E
    assert call(t=7) == E and call(t=-1) == E
    assert call(t=af.AF_KV_Q8_0) == E and call(t=af.AF_KV_Q8_0, ks=P) == E and call(t=0, ks=P, vs=P) == E
    assert call(kvh=0) == E and call(d=0) == E and call(ctx=0) == E
    assert call(d=48) == N and call(d=288, ld=4096) == N and call(kvh=1 << 14, ld=1 << 30) == N
    assert call(ld=1023) == E and call(ld=1026) == E and call(ld=1020) == E
    assert call(k=P + 4) == E and call(vc=P + 8) == E and call(t=af.AF_KV_Q4_0, ks=P + 2, vs=P) == E
    assert call(slots=P + 2) == E
    assert call(n=-1) == R and call(n=65) == R and call(slot0=-1) == R and call(slot0=61) == R
    assert call(slot0=2 ** 31 - 1) == R
    assert call(n=0) == af.AF_OK and call(n=0, slots=P) == af.AF_OK


def test_tree_refusals():
    af = _af()
    L = af.lib()
    E, R, N = af.AF_EINVAL, af.AF_ERANGE, af.AF_ENOTIMPL
    assert L.af_tree_mask(None, 4, 0, P, P, None) == E and L.af_tree_mask(P, 4, 0, None, P, None) == E
    assert L.af_tree_mask(P, 0, 0, P, P, None) == R and L.af_tree_mask(P, 1025, 0, P, P, None) == R
    assert L.af_tree_mask(P, 4, -1, P, P, None) == R and L.af_tree_mask(P, 4, 2 ** 31 - 1, P, P, None) == R
    assert L.af_tree_mask(P + 2, 4, 0, P, P, None) == E

    def call(q=P, ldq=4096, kc=P, ks=None, vc=P, vs=None, t=1, h=32, kvh=8, d=128, ctx=64, past=10, n=4, mask=P, ws=P,
             wsb=1 << 40, out=P, ldo=4096):
        return L.af_attention_tree(q, ldq, kc, ks, vc, vs, t, h, kvh, d, ctx, past, n, mask, ws, wsb, out, ldo, None)
    assert call(q=None) == E and call(mask=None) == E and call(out=None) == E and call(kc=None) == E
    assert call(t=5) == E and call(t=2) == E and call(t=2, ks=P) == E and call(t=1, ks=P, vs=P) == E
    assert call(h=0) == E and call(kvh=0) == E and call(h=30) == E and call(d=-1) == E
    assert call(d=96) == N and call(d=256) == N and call(h=520, kvh=8, ldq=1 << 20, ldo=1 << 20) == N
    assert call(n=0) == R and call(n=1025) == R and call(past=-1) == R and call(past=61) == R
    assert call(past=2 ** 31 - 1) == R
    assert call(q=P + 4) == E and call(out=P + 8) == E and call(mask=P + 1) == E and call(vc=P + 4) == E
    assert call(ldq=4095) == E and call(ldq=4098) == E and call(ldo=4092) == E
    ws = af.af_attention_tree_workspace(af.AF_F16, 32, 8, 128, 4096, 64)
    if ws:
        assert call(ctx=8192, past=4096, n=64, wsb=ws - 1) == E and "workspace" in af.af_last_error()
        assert call(ctx=8192, past=4096, n=64, ws=None) == E and call(ctx=8192, past=4096, n=64, ws=P + 16) == E
    assert af.af_attention_tree_workspace(af.AF_F16, 32, 8, 96, 4096, 64) == 0


def test_workspace_covers_the_documented_range():
    af = _af()
    for t in (af.AF_F32, af.AF_F16, af.AF_KV_Q8_0, af.AF_KV_Q4_0):
        for h, kvh, d in ((1, 1, 64), (8, 4, 64), (32, 8, 128), (64, 1, 128), (40, 5, 128)):
            for past in (0, 1, 31, 4096, 30720, 1 << 20):
                for n in (1, 4, 64, 1024):
                    assert 0 <= af.af_attention_tree_workspace(t, h, kvh, d, past, n) <= 256 << 20


def test_tree_pasts_at_the_end_of_the_integers():
    """Slots are counted in 32 bits, tiles past the last one among them: a past that leaves no room for a tile is refused."""
    af = _af()
    L = af.lib()
    big = 2 ** 31 - 1
    for t in (af.AF_F32, af.AF_F16):
        for n in (1, 40, 1024):
            for past in (big - n, big - 1024, big - 2047):
                assert L.af_attention_tree(P, 64, P, None, P, None, t, 1, 1, 64, big, past, n, P, None, 0, P, 64,
                                           None) == af.AF_ERANGE
                assert af.af_attention_tree_workspace(t, 1, 1, 64, past, n) == 0
    assert af.af_attention_tree_workspace(af.AF_F32, 1, 1, 64, big - 2048, 1024) <= 256 << 20


# The binding's calls, whose arguments go over as one packed record: every argument with a value that only it can be refused
# for, so that a member that lies elsewhere in the record than in the call is seen.  (stream is passed on unread.)
GOOD = {
    "af_rope": dict(cfg=None, x=P, ldx=1024, y=2 * P, ldy=1024, dtype=0, n=4, n_heads=8, pos=None, pos0=0),
    "af_kv_write": dict(k=P, v=P, ld=1024, n=4, slots=None, slot0=0, kc=P, ks=P, vc=P, vs=P, t=2, kvh=8, d=128, ctx=64),
    "af_kv_read": dict(kc=P, ks=P, vc=P, vs=P, t=2, kvh=8, d=128, ctx=64, n=4, slots=None, slot0=0, k=P, v=P, ld=1024),
    "af_tree_mask": dict(parent=P, n=4, pos0=0, mask=P, pos=None),
    "af_attention_tree": dict(q=P, ldq=4096, kc=P, ks=P, vc=P, vs=P, t=2, h=32, kvh=8, d=128, ctx=64, past=10, n=4, mask=P,
                              ws=P, wsb=1 << 40, out=P, ldo=4096),
}
BAD = {
    "af_rope": dict(x=P + 1, ldx=1000, y=P + 3, ldy=1001, dtype=3, n=-7, n_heads=-5, pos=P + 2, pos0=2 ** 31 - 2),
    "af_kv_write": dict(k=P + 4, v=None, ld=1022, n=77, slots=P + 1, slot0=-9, kc=None, ks=None, vc=P + 8, vs=P + 2, t=9, kvh=0,
                        d=96 * 3, ctx=-2),
    "af_kv_read": dict(kc=None, ks=None, vc=P + 8, vs=P + 2, t=9, kvh=0, d=96 * 3, ctx=-2, n=77, slots=P + 1, slot0=-9, k=P + 4,
                       v=None, ld=1022),
    "af_tree_mask": dict(parent=None, n=1031, pos0=-11, mask=P + 1, pos=P + 2),
    "af_attention_tree": dict(q=P + 4, ldq=4095, kc=None, ks=None, vc=P + 8, vs=P + 2, t=9, h=31, kvh=-1, d=96, ctx=13, past=-3,
                              n=1029, mask=P + 1, out=P + 8, ldo=4094),
}


@pytest.mark.parametrize("name", list(GOOD))
def test_packed_calls_refuse_what_the_calls_refuse(name):
    af = _af()
    cfg = af.rope_config(128, 128)
    for arg, bad in BAD[name].items():
        args = {**GOOD[name], arg: bad}
        if "cfg" in args:
            args["cfg"] = cfg
        with pytest.raises(Exception) as refused:
            getattr(af, name)(*args.values(), stream=0)
        packed = af.af_last_error()
        args = [ctypes.byref(cfg) if a is cfg else a for a in args.values()]
        rc = getattr(af.lib(), name)(*args, None)
        assert rc not in (af.AF_OK, af.AF_ECUDA), arg
        assert packed == af.af_last_error() and af.STATUS_NAMES[rc] in str(refused.value), arg


def test_packed_call_refuses_what_is_no_call():
    L = _af().lib()
    assert L.af_packed_call(5, b"\0" * 256) == 1 and L.af_packed_call(-1, b"\0" * 256) == 1 and L.af_packed_call(0, None) == 1
