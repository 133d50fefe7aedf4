"""Host-side validation of the attention block's calls: every refusal comes
before any CUDA launch, so no GPU is needed."""
import ctypes

import pytest

import q4_weight_matmul_gb300 as q4k

OK, INVALID, ALIGN, UNSUPPORTED = 0, 1, 2, 3
P = ctypes.c_void_p(0x100000)
ODD16, ODD4 = ctypes.c_void_p(0x100008), ctypes.c_void_p(0x100002)


@pytest.fixture(scope="module")
def lib():
    q4k.build()
    return q4k.lib()


def cache(**kw):
    d = dict(k=P, v=P, num_pages=10, page_size=16, kv_heads=2, head_dim=128, type=0)
    d.update(kw)
    return ctypes.byref(q4k.KvCache(*(d[n] for n, _ in q4k.KvCache._fields_)))


BAD_CACHE = [(dict(page_size=8), INVALID), (dict(page_size=48), INVALID), (dict(page_size=512), INVALID),
             (dict(kv_heads=0), INVALID), (dict(kv_heads=3), INVALID), (dict(num_pages=-1), INVALID),
             (dict(num_pages=2 ** 27), INVALID), (dict(type=2), INVALID), (dict(type=7), INVALID),
             (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=256), UNSUPPORTED)]


def rope(lib, c=None, **kw):
    d = dict(q=P, k=P, v=P, tokens=3, heads=4, cache=c or cache(), qw=P, kw=P, eps=1e-6, cs=P, max_pos=64, rot=128,
             inter=0, pos=P, slot=P, out=P)
    d.update(kw)
    return lib.q4k_qk_norm_rope(*d.values(), None)


def test_qk_norm_rope_refusals(lib):
    for bad, status in BAD_CACHE:
        assert rope(lib, cache(**bad)) == status, bad
    for bad, status in [(dict(tokens=-1), INVALID), (dict(heads=0), INVALID), (dict(heads=3), INVALID),
                        (dict(rot=12), INVALID), (dict(rot=136), INVALID), (dict(rot=-8), INVALID),
                        (dict(max_pos=-1), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=-1.0), INVALID),
                        (dict(qw=None), INVALID), (dict(kw=None), INVALID), (dict(q=None), INVALID),
                        (dict(cs=None), INVALID), (dict(pos=None), INVALID), (dict(slot=None), INVALID),
                        (dict(out=None), INVALID), (dict(q=ODD16), ALIGN), (dict(qw=ODD16), ALIGN),
                        (dict(out=ODD16), ALIGN), (dict(pos=ODD4), ALIGN), (dict(slot=ODD4), ALIGN),
                        (dict(cache=cache(k=ODD16)), ALIGN), (dict(cache=cache(v=None)), INVALID),
                        (dict(cache=None), INVALID), (dict(tokens=0, q=None, slot=None), OK)]:
        assert rope(lib, **bad) == status, bad


def attn(lib, **kw):
    d = dict(q=P, tokens=3, heads=4, cache=cache(), table=P, max_pages=4, cu=P, kv=P, n_req=2, max_q=2, scale=0.1,
             window=0, out=P, out_type=2, ws=P, ws_bytes=1 << 40)
    d.update(kw)
    return lib.q4k_paged_attn(*d.values(), None)


def test_paged_attn_refusals(lib):
    for bad, status in BAD_CACHE:
        if bad != dict(type=2):                   # with out_type 2 that reads as a type that is not the cache's
            assert attn(lib, cache=cache(**bad)) == status, bad
    for bad, status in [(dict(tokens=-1), INVALID), (dict(heads=5), INVALID), (dict(n_req=-1), INVALID),
                        (dict(n_req=0), INVALID), (dict(max_q=0), INVALID), (dict(max_q=-1), INVALID),
                        (dict(max_pages=-1), INVALID), (dict(max_pages=2 ** 27), INVALID), (dict(window=-1), INVALID),
                        (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID),
                        (dict(out_type=1), INVALID), (dict(out_type=3), INVALID), (dict(q=None), INVALID),
                        (dict(table=None), INVALID), (dict(cu=None), INVALID), (dict(kv=None), INVALID),
                        (dict(out=None), INVALID), (dict(ws=None), INVALID), (dict(ws_bytes=8), INVALID),
                        (dict(q=ODD16), ALIGN), (dict(out=ODD16), ALIGN), (dict(ws=ODD16), ALIGN),
                        (dict(table=ODD4), ALIGN), (dict(cu=ODD4), ALIGN), (dict(kv=ODD4), ALIGN),
                        (dict(tokens=2 ** 22, heads=2048, max_q=2 ** 22), UNSUPPORTED),
                        (dict(tokens=0, q=None, out=None, ws=None), OK)]:
        assert attn(lib, **bad) == status, bad
    ws = lib.q4k_paged_attn_workspace_bytes
    assert ws(cache(), 4, 3, 2, 2, 4, 2) > 0
    assert ws(cache(), 4, 0, 2, 2, 4, 2) == 0 and ws(cache(page_size=8), 4, 3, 2, 2, 4, 2) == 0
    assert ws(cache(), 5, 3, 2, 2, 4, 2) == 0 and ws(cache(), 4, 3, 2, 2, 4, 1) == 0


def lora(lib, mats=None, **kw):
    m = dict(a=P, b=P, base=P, y=P, rows=100)
    rows = [dict(m, **c) for c in (mats if mats is not None else [{}])]
    arr = (q4k.LoraMat * max(1, len(rows)))(*(q4k.LoraMat(*r.values()) for r in rows))
    d = dict(n=len(rows), mats=arr, n_adapters=3, rank=16, type=0, cols=512, x=P, tokens=5, order=P, start=P, ad=P,
             n_seg=2, scale=P, ws=P, ws_bytes=1 << 40)
    d.update(kw)
    return lib.q4k_lora_add(*d.values(), None)


def test_lora_add_refusals(lib):
    for bad, status in [(dict(n=-1), INVALID), (dict(n=5), UNSUPPORTED), (dict(mats=None), INVALID),
                        (dict(n_adapters=-1), INVALID), (dict(rank=0), INVALID), (dict(rank=12), INVALID),
                        (dict(rank=136), INVALID), (dict(type=2), INVALID), (dict(cols=300), INVALID),
                        (dict(cols=0), INVALID), (dict(tokens=-1), INVALID), (dict(n_seg=0), INVALID),
                        (dict(n_seg=-1), INVALID), (dict(x=None), INVALID), (dict(order=None), INVALID),
                        (dict(start=None), INVALID), (dict(ad=None), INVALID), (dict(scale=None), INVALID),
                        (dict(ws=None), INVALID), (dict(ws_bytes=8), INVALID), (dict(x=ODD16), ALIGN),
                        (dict(order=ODD4), ALIGN), (dict(start=ODD4), ALIGN), (dict(ad=ODD4), ALIGN),
                        (dict(ws=ODD16), ALIGN), (dict(tokens=0, x=None), OK)]:
        if bad == dict(mats=None):
            assert lib.q4k_lora_add(1, None, 3, 16, 0, 512, P, 5, P, P, P, 2, P, P, 1 << 40, None) == status
        else:
            assert lora(lib, **bad) == status, bad
    for bad, status in [(dict(a=None), INVALID), (dict(b=None), INVALID), (dict(y=None), INVALID),
                        (dict(rows=-1), INVALID), (dict(a=ODD16), ALIGN), (dict(b=ODD16), ALIGN),
                        (dict(base=ODD16), ALIGN), (dict(y=ODD16), ALIGN)]:
        assert lora(lib, mats=[{}, bad]) == status, bad
    assert lora(lib, mats=[dict(rows=0, y=None)]) == OK and lora(lib, mats=[]) == OK
    assert lib.q4k_lora_workspace_bytes(1, 16, 5) > 0 and lib.q4k_lora_workspace_bytes(1, 12, 5) == 0
    need = [lib.q4k_lora_workspace_bytes(2, 16, t) for t in range(1, 6000)]
    assert need == sorted(need)                              # serves fewer tokens as well
    assert lib.q4k_lora_workspace_bytes(0, 16, 5) == 0 and lib.q4k_lora_workspace_bytes(5, 16, 5) == 0


def test_segments_helper():
    order, start, ad = (t.tolist() for t in q4k.q4k_lora_segments([2, -1, 0, 2, -7, 0], device="cpu"))
    assert order == [1, 4, 2, 5, 0, 3] and start == [0, 2, 4, 6] and ad == [-1, 0, 2]
    order, start, ad = (t.tolist() for t in q4k.q4k_lora_segments([], device="cpu"))
    assert order == [] and start == [0] and ad == []
