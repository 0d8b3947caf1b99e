"""Refusals of the serving operators (af_kv_pages, af_attention_paged, af_lora_plan, af_lora): every check runs on the host
before anything is launched, so no GPU is needed.  Pointers are dummies, never dereferenced."""
import pytest

P = 4096  # an aligned address nothing reads
BIG = 1 << 40


def _af():
    import gguf_quantized_transformer_gb300 as af
    af.build()
    return af


GOOD = {
    "af_kv_pages": dict(ln=P, new=P, n_seqs=4, page=16, n_pages=64, pool=P, free=P, table=P, width=8, len_out=P, pool_out=P,
                        start=P, slots=P, pos=P, seq=P, max_rows=8, ws=P, wsb=BIG),
    "af_attention_paged": dict(q=P, ldq=4096, kc=P, ks=P, vc=P, vs=P, t=2, h=32, kvh=8, d=128, page=16, n_pages=64, table=P,
                               width=8, n_seqs=4, seq=None, pos=P, n=4, ws=P, wsb=BIG, out=P, ldo=4096),
    "af_lora_plan": dict(ids=P, n=4, adapters=3, plan=P, bytes=BIG),
    "af_lora": dict(x=P, ldx=512, n=4, plan=P, a=P, b=P, dtype=1, scale=P, ranks=P, adapters=3, rank=16, K=512, N=96, base=P,
                    ldb=96, y=2 * P, ldy=96, ws=P, wsb=BIG),
}
E, R, N = 1, 2, 6  # AF_EINVAL, AF_ERANGE, AF_ENOTIMPL
BAD = {
    "af_kv_pages": [(k, v, E) for k in ("ln", "new", "pool", "free", "table", "len_out", "pool_out", "start", "slots", "pos", "seq")
                    for v in (None, P + 2)] +
                   [("n_seqs", 0, R), ("n_seqs", 65537, R), ("page", 0, E), ("page", 2 ** 26, R), ("n_pages", -1, E),
                    ("n_pages", 2 ** 27, R), ("width", 0, E), ("width", 2 ** 27, R), ("max_rows", -1, R), ("ws", None, E),
                    ("ws", P + 8, E), ("wsb", 79, E)],
    "af_attention_paged": [("q", None, E), ("q", P + 8, E), ("ldq", 4095, E), ("ldq", 4098, E), ("kc", None, E), ("kc", P + 4, E),
                           ("ks", None, E), ("vc", None, E), ("vs", P + 2, E), ("t", 9, E), ("t", 0, E), ("h", 31, E), ("h", 0, E),
                           ("h", 8 * 65, N), ("kvh", 0, E), ("d", 96, N), ("d", -64, E), ("page", 0, E), ("page", 2 ** 26, R),
                           ("n_pages", 0, E), ("n_pages", 2 ** 24, N), ("table", None, E), ("table", P + 1, E), ("width", 0, E),
                           ("width", 2 ** 27, R), ("n_seqs", 0, R), ("n_seqs", 3, R), ("n_seqs", 65537, R), ("seq", P + 2, E),
                           ("pos", None, E), ("pos", P + 3, E), ("n", 0, R), ("n", 5, R), ("n", 2049, R), ("ws", None, E),
                           ("ws", P + 16, E), ("out", None, E), ("out", P + 4, E), ("ldo", 4092, E), ("ldo", 4097, E)],
    "af_lora_plan": [("ids", None, E), ("ids", P + 1, E), ("n", 0, R), ("n", 65537, R), ("adapters", 0, R), ("adapters", 4097, R),
                     ("plan", None, E), ("plan", P + 4, E), ("bytes", 15, E)],
    "af_lora": [("x", None, E), ("x", P + 4, E), ("ldx", 508, E), ("ldx", 514, E), ("n", 0, R), ("n", 65537, R), ("plan", None, E),
                ("plan", P + 8, E), ("a", None, E), ("a", P + 2, E), ("b", None, E), ("b", P + 8, E), ("dtype", 2, E),
                ("scale", P + 1, E), ("ranks", P + 2, E), ("adapters", 0, R), ("adapters", 4097, R), ("rank", 0, E), ("rank", 12, N),
                ("rank", 136, N), ("K", 0, E), ("K", 2 ** 24 + 32, N), ("N", 2 ** 24 + 1, N), ("K", 500, N), ("N", 0, E), ("N", 97, E), ("base", P + 2, E), ("ldb", 95, E),
                ("y", None, E), ("y", P + 1, E), ("ldy", 95, E), ("ws", None, E), ("ws", P + 16, E), ("wsb", 100, E)],
}


@pytest.mark.parametrize("name", list(GOOD))
def test_refusals_by_call_and_by_record(name):
    """Every argument with values that only it can be refused for, through the header's call and through the binding's packed
    record, which must say the same: a member that lies elsewhere in the record than in the call is seen."""
    af = _af()
    for arg, bad, want in BAD[name]:
        args = {**GOOD[name], arg: bad}
        with pytest.raises(af.AfError) as refused:
            getattr(af, name)(*args.values(), stream=0)
        packed = af.af_last_error()
        rc = getattr(af.lib(), name)(*args.values(), None)
        assert rc == want and refused.value.code == want and packed == af.af_last_error(), (arg, bad, packed)


def test_attention_paged_cache_types():
    af = _af()
    def call(**kw):
        return af.lib().af_attention_paged(*{**GOOD["af_attention_paged"], **kw}.values(), None)
    assert call(t=af.AF_KV_Q4_0, ks=None) == E and call(t=af.AF_F16, ks=P, vs=None) == E and call(t=-1) == E
    need = af.af_attention_paged_workspace(32, 8, 128)
    if need:
        assert call(wsb=need - 1) == E and "workspace" in af.af_last_error()


def test_lora_in_place_needs_one_stride():
    af = _af()
    args = {**GOOD["af_lora"], "base": P, "y": P, "ldb": 100}
    assert af.lib().af_lora(*args.values(), None) == E and "in place" in af.af_last_error()


def test_sizes_of_scratch():
    af = _af()
    assert af.af_kv_pages_workspace(0) == 0 and af.af_kv_pages_workspace(65537) == 0
    assert 16 * 256 <= af.af_kv_pages_workspace(256) <= 64 * 256
    assert af.af_attention_paged_workspace(32, 8, 96) == 0 and af.af_attention_paged_workspace(30, 8, 128) == 0
    assert af.af_lora_plan_bytes(0, 1) == 0 and af.af_lora_plan_bytes(1, 0) == 0
    for n in (1, 31, 32, 33, 2048, 65536):
        for m in (1, 7, 4096):
            assert 4 * n <= af.af_lora_plan_bytes(n, m) <= 4 * n + 16 * (n // 32 + min(n, m + 1) + 2)
    assert af.af_lora_workspace(4, 3, 12, 512, 96) == 0 and af.af_lora_workspace(4, 3, 16, 500, 96) == 0
