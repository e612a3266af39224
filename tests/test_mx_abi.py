"""The MXFP4 calls refuse bad arguments on the host, before any device work (no
GPU needed): statuses of the C ABI, and the binding's checks."""
import ctypes

import pytest

rw4 = pytest.importorskip("rotated_w4a4_amd", reason="librw4.so not built")
torch = pytest.importorskip("torch")

lib = rw4.lib
OK, ARG, SHAPE, UNSUP = range(4)
P = 0x10000  # 16-byte aligned, never dereferenced: every case fails validation first


def _call(fn, names, base, **change):
    args = dict(base)
    assert set(change) <= set(names)
    args.update(change)
    return fn(*[args[n] for n in names])


ACT = "t x dt M K ldx q s stream".split()
ACT_OK = dict(t=None, x=P, dt=1, M=3, K=256, ldx=256, q=P, s=P, stream=None)
SIZES = [(dict(K=0), SHAPE), (dict(K=-128), SHAPE), (dict(K=100), SHAPE), (dict(K=192), SHAPE), (dict(K=1 << 24), SHAPE),
         (dict(q=None), ARG), (dict(s=None), ARG), (dict(q=P + 8), ARG), (dict(s=P + 4), ARG), (dict(dt=2), ARG),
         (dict(dt=-1), ARG)]


@pytest.mark.parametrize("change,want", SIZES + [
    (dict(M=-1), SHAPE), (dict(M=(1 << 28) + 1), SHAPE), (dict(x=None), ARG), (dict(x=P + 2), ARG), (dict(ldx=255), ARG),
    (dict(ldx=260), ARG), (dict(ldx=1 << 40), ARG), (dict(dt=0, ldx=258), ARG), (dict(M=0, x=None, q=None, s=None), OK)])
def test_quantize_refusals(change, want):
    assert _call(lib.rw4_mx_quantize_act, ACT, ACT_OK, **change) == want


PACK = "t w dt N K sk sn q s stream".split()
PACK_OK = dict(t=None, w=P, dt=0, N=3, K=256, sk=3, sn=1, q=P, s=P, stream=None)


@pytest.mark.parametrize("change,want", SIZES + [
    (dict(N=-1), SHAPE), (dict(N=1 << 32), SHAPE), (dict(w=None), ARG), (dict(w=P + 2), ARG), (dict(dt=1, w=P + 1), ARG),
    (dict(sk=0), ARG), (dict(sn=0), ARG), (dict(sk=-1), ARG), (dict(sn=1 << 40), ARG), (dict(sk=1 << 40), ARG),
    (dict(N=0, w=None), OK)])
def test_pack_refusals(change, want):
    assert _call(lib.rw4_mx_pack_weight, PACK, PACK_OK, **change) == want


DEQ = "q s M K out dt ldo stream".split()
DEQ_OK = dict(q=P, s=P, M=3, K=256, out=P, dt=1, ldo=256, stream=None)


@pytest.mark.parametrize("change,want", SIZES + [
    (dict(M=-1), SHAPE), (dict(out=None), ARG), (dict(out=P + 8), ARG), (dict(ldo=255), ARG), (dict(ldo=260), ARG),
    (dict(ldo=1 << 40), ARG), (dict(M=0, q=None), OK)])
def test_dequantize_refusals(change, want):
    assert _call(lib.rw4_mx_dequantize, DEQ, DEQ_OK, **change) == want


GEMM = "qa sa qw sw M N K y dt ldy stream".split()
GEMM_OK = dict(qa=P, sa=P, qw=P, sw=P, M=3, N=5, K=256, y=P, dt=1, ldy=5, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(M=-1), SHAPE), (dict(N=-1), SHAPE), (dict(M=1 << 32), SHAPE), (dict(N=1 << 32), SHAPE), (dict(K=0), SHAPE),
    (dict(K=64), SHAPE), (dict(K=1 << 24), SHAPE), (dict(qa=None), ARG), (dict(sa=None), ARG), (dict(qw=None), ARG),
    (dict(sw=None), ARG), (dict(y=None), ARG), (dict(qa=P + 8), ARG), (dict(sa=P + 4), ARG), (dict(qw=P + 1), ARG),
    (dict(sw=P + 8), ARG), (dict(y=P + 2), ARG), (dict(ldy=4), ARG), (dict(ldy=1 << 40), ARG), (dict(dt=7), ARG),
    (dict(M=0, qa=None, y=None), OK), (dict(N=0, ldy=0, qw=None), OK)])
def test_gemm_refusals(change, want):
    assert _call(lib.rw4_mx_gemm, GEMM, GEMM_OK, **change) == want


def _transform(K, block):
    h = ctypes.c_void_p()
    assert lib.rw4_transform_hadamard(K, block, None, ctypes.byref(h)) == OK
    return h


@pytest.mark.parametrize("K,block,want_k,want", [(1024, 128, 1024, ARG), (1024, 128, 512, SHAPE), (1024, 512, 1024, ARG),
                                                 (1024, 1024, 1024, UNSUP), (4096, 4096, 4096, UNSUP)])
def test_transforms(K, block, want_k, want):
    # ARG: the transform passed, the null input did not
    t = _transform(K, block)
    try:
        assert lib.rw4_mx_quantize_act(t, None, 1, 3, want_k, want_k, P, P, None) == want
        assert lib.rw4_mx_pack_weight(t, None, 1, 3, want_k, 1, want_k, P, P, None) == want
    finally:
        lib.rw4_transform_destroy(t)


def test_binding_wants_gpu_tensors():
    x = torch.zeros(2, 128)
    q, s = torch.zeros(2, 64, dtype=torch.uint8), torch.zeros(1, 2, 4, dtype=torch.uint8)
    for call in (lambda: rw4.mx_quantize_act(None, x), lambda: rw4.mx_pack_weight(None, x),
                 lambda: rw4.mx_dequantize(q, s), lambda: rw4.mx_gemm(q, s, q, s)):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_scale_rows():
    s = torch.arange(24, dtype=torch.uint8).reshape(3, 8)
    o = rw4.mx_scale_rows(s)
    assert o.shape == (2, 3, 4) and o.is_contiguous()
    assert all(o[b // 4, r, b % 4] == s[r, b] for r in range(3) for b in range(8))
    with pytest.raises(ValueError):
        rw4.mx_scale_rows(s[:, :6])
    with pytest.raises(ValueError):
        rw4.mx_scale_rows(s.int())
