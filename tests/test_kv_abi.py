"""The KV cache calls refuse bad arguments on the host, before any device
work (no GPU needed): statuses of the C ABI, and the binding's checks."""
import ctypes

import pytest

rw4 = pytest.importorskip("rotated_w4a4_amd", reason="librw4.so not built")
torch = pytest.importorskip("torch")
from rotated_w4a4_amd import kv as rkv  # noqa: E402

lib = rw4.lib
OK, ARG, SHAPE, UNSUP, HIP, NOMEM = range(6)
P = 0x10000  # 16-byte aligned, never dereferenced: every case fails validation first


def _call(fn, names, base, **change):
    args = dict(base)
    assert set(change) <= set(names)
    args.update(change)
    return fn(*[args[n] for n in names])


def _cache(**change):
    f = dict(k_codes=P, k_scales=P, v_codes=P, v_scales=P, pages=4, page_size=16, heads=2, head_dim=128,
             code_page=2048, code_head=1024, code_slot=64, scale_page=32, scale_head=16, scale_slot=1)
    f.update(change)
    return rkv._CacheStruct(**f)


BAD_CACHES = [
    (dict(head_dim=96), SHAPE), (dict(head_dim=512), SHAPE), (dict(page_size=8), SHAPE), (dict(page_size=48), SHAPE),
    (dict(page_size=1 << 21), SHAPE), (dict(pages=0), SHAPE), (dict(pages=1 << 31), SHAPE), (dict(heads=0), SHAPE),
    (dict(heads=1025), SHAPE), (dict(pages=1 << 30, page_size=64), SHAPE), (dict(k_codes=None), ARG),
    (dict(v_scales=None), ARG), (dict(k_codes=P + 8), ARG), (dict(v_scales=P + 2), ARG), (dict(code_slot=56), ARG),
    (dict(code_page=-2048), ARG), (dict(scale_head=-1), ARG), (dict(code_page=1 << 40), ARG),
    (dict(code_slot=32), ARG),  # rows of 64 bytes overlap
    (dict(scale_slot=0), ARG), (dict(code_head=64), ARG), (dict(scale_page=16), ARG),
]

SLOTS = "ctx new B page table width free cap state state_out kv cu served slots pos tokens stream".split()
SLOTS_OK = dict(ctx=P, new=P, B=2, page=16, table=P, width=4, free=P, cap=8, state=P, state_out=P, kv=P, cu=P,
                served=P, slots=P, pos=P, tokens=4, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(B=-1), SHAPE), (dict(B=4097), SHAPE), (dict(page=0), SHAPE), (dict(page=24), SHAPE), (dict(page=1 << 21), SHAPE),
    (dict(width=-1), SHAPE), (dict(width=1 << 31), SHAPE), (dict(cap=0), SHAPE), (dict(cap=1 << 31), SHAPE),
    (dict(tokens=-1), SHAPE), (dict(tokens=1 << 31), SHAPE), (dict(ctx=None), ARG), (dict(new=None), ARG),
    (dict(table=None), ARG), (dict(free=None), ARG), (dict(state=None), ARG), (dict(state_out=None), ARG),
    (dict(kv=None), ARG), (dict(cu=None), ARG), (dict(served=None), ARG), (dict(slots=None), ARG), (dict(pos=None), ARG)])
def test_slots_refusals(change, want):
    assert _call(lib.rw4_kv_slots, SLOTS, SLOTS_OK, **change) == want


ROWS = ("q qt qh k kt kh dt T heads kv_heads D wq wk eps cs max_pos rot inter pos rotate qo qot qoh ko kot koh odt "
        "stream").split()
ROWS_OK = dict(q=P, qt=1024, qh=128, k=P, kt=1024, kh=128, dt=1, T=3, heads=4, kv_heads=2, D=128, wq=P, wk=P, eps=1e-6,
               cs=P, max_pos=100, rot=128, inter=0, pos=P, rotate=0, qo=P, qot=512, qoh=128, ko=P, kot=256, koh=128,
               odt=1, stream=None)
ROW_CHANGES = [
    (dict(dt=2), ARG), (dict(odt=7), ARG), (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE), (dict(eps=-1.0), ARG),
    (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG), (dict(heads=1025), SHAPE),
    (dict(rot=8), SHAPE), (dict(rot=40), SHAPE), (dict(rot=144), SHAPE), (dict(max_pos=0), SHAPE), (dict(pos=None), ARG),
    (dict(cs=P + 4), ARG), (dict(q=P + 2), ARG), (dict(qt=1028), ARG), (dict(qh=-128), ARG), (dict(qt=1 << 40), ARG),
    (dict(k=None), ARG), (dict(kh=4), ARG), (dict(qo=None), ARG), (dict(qot=500), ARG), (dict(qoh=64), ARG),
    (dict(wq=P + 4), ARG), (dict(wk=P + 8), ARG), (dict(dt=0, qh=130), ARG),
]


@pytest.mark.parametrize("change,want", ROW_CHANGES + [
    (dict(D=96), SHAPE), (dict(heads=0), SHAPE), (dict(kv_heads=-1), SHAPE), (dict(kv_heads=1025), SHAPE),
    (dict(q=None), ARG), (dict(ko=None), ARG), (dict(kot=128), ARG), (dict(T=0, q=None, k=None, qo=None, ko=None), OK)])
def test_norm_rope_refusals(change, want):
    assert _call(lib.rw4_qk_norm_rope, ROWS, ROWS_OK, **change) == want


APPEND = ("cache k kt kh v vt vh slots q qt qh heads dt T wq wk eps cs max_pos rot inter pos rotate qo qot qoh odt "
          "stream").split()


def _append_ok(cache):
    return {**{n: ROWS_OK[n] for n in APPEND if n in ROWS_OK}, "cache": ctypes.addressof(cache), "v": P, "vt": 1024,
            "vh": 128, "slots": P}


@pytest.mark.parametrize("change,want", ROW_CHANGES + [
    (dict(heads=0), SHAPE), (dict(v=None), ARG), (dict(vt=3), ARG), (dict(slots=None), ARG), (dict(cache=None), ARG),
    (dict(T=0, q=None, k=None, v=None, slots=None, qo=None), OK)])
def test_append_refusals(change, want):
    c = _cache()
    assert _call(lib.rw4_kv_append, APPEND, _append_ok(c), **change) == want


@pytest.mark.parametrize("change,want", BAD_CACHES)
def test_bad_caches_are_refused(change, want):
    c = _cache(**change)
    assert _call(lib.rw4_kv_append, APPEND, _append_ok(c)) == want
    assert _call(lib.rw4_kv_attention, ATT, _att_ok(c)) == want


ATT = ("cache q qdt qt qh T heads table width kv cu B most scale causal window unrotate out odt ot oh lse ws wbytes "
       "stream").split()


def _att_ok(cache):
    return dict(cache=ctypes.addressof(cache), q=P, qdt=1, qt=512, qh=128, T=3, heads=4, table=P, width=4, kv=P, cu=P,
                B=2, most=3, scale=0.1, causal=1, window=0, unrotate=1, out=P, odt=1, ot=512, oh=128, lse=P, ws=P,
                wbytes=1 << 40, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(cache=None), ARG), (dict(qdt=3), ARG), (dict(odt=-1), ARG), (dict(scale=float("nan")), ARG),
    (dict(scale=float("inf")), ARG), (dict(T=-1), SHAPE), (dict(heads=3), SHAPE), (dict(heads=1), SHAPE),
    (dict(heads=130), SHAPE), (dict(B=-1), SHAPE), (dict(B=65536), SHAPE), (dict(width=-1), SHAPE),
    (dict(width=1 << 31), SHAPE), (dict(most=-1), SHAPE), (dict(window=-1), SHAPE), (dict(window=5, causal=0), UNSUP),
    (dict(q=None), ARG), (dict(q=P + 4), ARG), (dict(qt=510), ARG), (dict(out=None), ARG), (dict(oh=64), ARG),
    (dict(ot=256), ARG), (dict(table=None), ARG), (dict(kv=None), ARG), (dict(cu=None), ARG), (dict(ws=None), ARG),
    (dict(ws=P + 8), ARG), (dict(wbytes=8), ARG), (dict(T=0, q=None, out=None, ws=None), OK),
    (dict(B=0, q=None, out=None, ws=None), OK)])
def test_attention_refusals(change, want):
    c = _cache()
    assert _call(lib.rw4_kv_attention, ATT, _att_ok(c), **change) == want


def test_workspace_sizes():
    ws = lib.rw4_kv_attention_workspace_bytes
    assert ws(1, 1, 32, 8, 128) > 0
    assert ws(-1, 1, 32, 8, 128) == 0 and ws(1, 1, 30, 8, 128) == 0 and ws(1, 1, 32, 8, 100) == 0
    assert ws(1, 65536, 32, 8, 128) == 0 and ws(1, 1, 8, 0, 128) == 0


def test_binding_refuses_host_tensors():
    i32 = torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(2, 2, 128)
    codes, scales = torch.zeros(2, 2, 16, 64, dtype=torch.uint8), torch.zeros(2, 2, 16)
    with pytest.raises(ValueError, match="GPU"):
        rw4.KVCache(codes, codes, scales, scales)
    with pytest.raises(ValueError, match="GPU"):
        rw4.kv_slots(i32, i32, i32.view(2, 1), i32, i32, 16, 4)
    with pytest.raises(ValueError, match="GPU"):
        rw4.qk_norm_rope(q, q)


def test_rope_table_values():
    t = rw4.rope_table(3, 4, base=100.0, device="cpu").double()
    a = torch.tensor([[0.0, 0.0], [1.0, 0.1], [2.0, 0.2]], dtype=torch.float64)
    assert (t - torch.cat([a.cos(), a.sin()], 1)).abs().max() <= 2.0 ** -24
