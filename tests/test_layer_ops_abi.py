"""Argument checks and host-side helpers of lora_rmsnorm, lora_w4_project and
lora_rope_append, without a GPU: every call here is refused, or has nothing to
do, before any CUDA call."""
import ctypes
import math

import pytest
import torch

from scatter_gemm_b200 import lora
from scatter_gemm_b200.build import build

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = 0x10000  # a fake address, aligned; never read


@pytest.fixture(scope="module")
def L():
    build()
    return lora.lib()


def norm(lib, **kw):
    a = dict(x=P, ld_x=64, res=P, ld_res=64, ro=P, ld_ro=64, w=P, w0=0.0, eps=1e-6, out=P,
             ld_out=64, q=P, ld_q=64, sc=P, tok=4, H=64, dt=0)
    a.update(kw)
    return lib.lora_rmsnorm(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=2), UNSUPPORTED), (dict(dt=7), UNSUPPORTED), (dict(tok=-1), INVALID),
    (dict(H=0), INVALID), (dict(ld_x=63), INVALID), (dict(ld_res=63), INVALID),
    (dict(ld_ro=10), INVALID), (dict(ld_out=63), INVALID), (dict(ld_q=63), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID), (dict(out=None, q=None, sc=None), INVALID),
    (dict(res=None), INVALID), (dict(ro=None), INVALID), (dict(sc=None), INVALID),
    (dict(q=None), INVALID), (dict(x=None), INVALID), (dict(w=None), INVALID),
    (dict(x=P + 1), INVALID), (dict(ro=P + 1), INVALID), (dict(out=P + 1), INVALID),
    (dict(sc=P + 2), INVALID), (dict(w=P + 1), INVALID),
    (dict(H=65537, ld_x=65537, ld_res=65537, ld_ro=65537, ld_out=65537, ld_q=65537), UNSUPPORTED),
    (dict(tok=1 << 30), UNSUPPORTED), (dict(tok=0), OK), (dict(tok=0, x=None, w=None), OK),
])
def test_norm_argument_checks(L, kw, want):
    assert norm(L, **kw) == want


def w4(lib, **kw):
    a = dict(x=P, ld_x=128, sx=None, W=P, ld_w=64, s=P, z=P, ld_s=16, out=P, ld_out=16, tok=4,
             K=128, N=16, group=128, xdt=0, dt=0, ws=None, wsb=0)
    a.update(kw)
    return lib.lora_w4_project(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=2), UNSUPPORTED), (dict(xdt=1), UNSUPPORTED), (dict(xdt=3), UNSUPPORTED),
    (dict(group=16), UNSUPPORTED), (dict(group=256), UNSUPPORTED), (dict(group=0), UNSUPPORTED),
    (dict(tok=-1), INVALID), (dict(K=0), INVALID), (dict(N=-1), INVALID), (dict(ld_x=127), INVALID),
    (dict(ld_out=15), INVALID), (dict(ld_s=15), INVALID), (dict(ld_w=48), INVALID),
    (dict(K=129, ld_x=129), INVALID),                       # 129 values need 80 bytes a row
    (dict(sx=P), INVALID), (dict(xdt=2), INVALID),          # a scale goes with e4m3 alone
    (dict(xdt=2, sx=P + 2), INVALID), (dict(x=None), INVALID), (dict(W=None), INVALID),
    (dict(s=None), INVALID), (dict(out=None), INVALID), (dict(x=P + 1), INVALID),
    (dict(s=P + 1), INVALID), (dict(out=P + 1), INVALID),
    (dict(W=P + 8), UNSUPPORTED), (dict(ld_w=72), UNSUPPORTED),
    (dict(wsb=64), INVALID), (dict(ws=P + 8, wsb=64), INVALID),
    (dict(tok=1 << 30), UNSUPPORTED), (dict(N=(1 << 28) + 1, ld_out=1 << 29, ld_s=1 << 29), UNSUPPORTED),
    (dict(tok=0), OK), (dict(N=0), OK), (dict(tok=0, x=None), OK),
])
def test_w4_argument_checks(L, kw, want):
    assert w4(L, **kw) == want


def rope(lib, off=(0, 256, 384, 512), ks=(1024, 128, 64), vs=(1024, 128, 64), amap=None, **kw):
    a = dict(qkv=P, ld=512, off=None if off is None else (ctypes.c_int32 * 4)(*off), D=64, R=64,
             pos=P, ld_pos=8, axes=1, amap=None if amap is None else bytes(amap), cs=P, max_pos=10,
             inter=0, qw=None, kw=None, w0=0.0, eps=1e-6, q=P, ld_q=256, kc=P,
             ks=None if ks is None else (ctypes.c_int64 * 3)(*ks), vc=P,
             vs=None if vs is None else (ctypes.c_int64 * 3)(*vs), pages=4, page=8, cdt=0, ksc=1.0,
             vsc=1.0, slots=P, ib=8, tok=3, dt=0)
    a.update(kw)
    return lib.lora_rope_append(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=2), UNSUPPORTED), (dict(cdt=1), UNSUPPORTED), (dict(cdt=5), UNSUPPORTED),
    (dict(ib=2), UNSUPPORTED), (dict(off=None), INVALID), (dict(ks=None), INVALID),
    (dict(vs=None), INVALID), (dict(tok=-1), INVALID), (dict(D=0), INVALID), (dict(R=66), INVALID),
    (dict(R=63), INVALID), (dict(R=-2), INVALID), (dict(axes=0), INVALID), (dict(axes=5), UNSUPPORTED),
    (dict(pages=-1), INVALID), (dict(page=0), INVALID), (dict(eps=-1.0), INVALID),
    (dict(D=514, off=(0, 514, 514, 514), ld=600, ld_q=600), UNSUPPORTED),
    (dict(off=(-1, 256, 384, 512)), INVALID), (dict(off=(0, 256, 128, 512)), INVALID),
    (dict(off=(0, 256, 384, 513)), INVALID), (dict(off=(0, 250, 378, 506)), INVALID),
    (dict(off=(0, 256, 384, 448)), INVALID),          # more heads of k than of v
    (dict(ld=511), INVALID), (dict(ld_q=255), INVALID), (dict(qw=P), INVALID), (dict(kw=P), INVALID),
    (dict(ksc=0.0), INVALID), (dict(vsc=-1.0), INVALID), (dict(ksc=math.nan), INVALID),
    (dict(max_pos=0), INVALID), (dict(axes=2), INVALID), (dict(axes=2, amap=[0] * 32, ld_pos=2), INVALID),
    (dict(axes=2, amap=[2] * 32), INVALID), (dict(ks=(-1, 1, 1)), INVALID),
    (dict(qkv=None), INVALID), (dict(slots=None), INVALID), (dict(q=None), INVALID),
    (dict(kc=None), INVALID), (dict(pos=None), INVALID), (dict(cs=None), INVALID),
    (dict(qkv=P + 1), INVALID), (dict(slots=P + 4), INVALID), (dict(pos=P + 4), INVALID),
    (dict(kc=P + 1), INVALID), (dict(cs=P + 2), INVALID), (dict(tok=1 << 30), UNSUPPORTED),
    (dict(tok=0), OK), (dict(off=(0, 0, 0, 0), ld_q=0), OK),
])
def test_rope_argument_checks(L, kw, want):
    assert rope(L, **kw) == want


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def test_norm_binding_refusals(L):
    x, w = bf16(4, 32), bf16(32)
    q, s = torch.zeros(4, 32).to(torch.float8_e4m3fn), torch.zeros(4)
    for bad, err in ((dict(x=x[0]), ValueError), (dict(x=x.float()), TypeError),
                     (dict(weight=bf16(31)), ValueError), (dict(weight=w.half()), TypeError),
                     (dict(out=bf16(3, 32)), ValueError), (dict(out=bf16(4, 31)), ValueError),
                     (dict(out=bf16(32, 4).T), ValueError), (dict(out=None), ValueError),
                     (dict(out=bf16(1, 32).expand(4, 32)), ValueError),
                     (dict(residual=x.half()), TypeError), (dict(residual_out=x), ValueError),
                     (dict(out_q=q), ValueError), (dict(out_scale=s), ValueError),
                     (dict(out_q=x, out_scale=s), TypeError),
                     (dict(out_q=q, out_scale=s[:3]), ValueError),
                     (dict(), ValueError)):  # the last: CPU tensors
        a = dict(x=x, weight=w, out=bf16(4, 32))
        a.update(bad)
        with pytest.raises(err):
            lora.lora_rmsnorm(**a)
    assert lora.lora_rmsnorm(x[:0], w, bf16(0, 32)).shape == (0, 32)


def test_w4_binding_refusals(L):
    x, out = bf16(4, 64), bf16(4, 8)
    w, s = torch.zeros(8, 32, dtype=torch.uint8), bf16(1, 8)
    x8, sx = torch.zeros(4, 64).to(torch.float8_e4m3fn), torch.zeros(4)
    for bad, err in ((dict(x=x.half()), TypeError), (dict(x=x[0]), ValueError),
                     (dict(w_packed=w.to(torch.int8)), TypeError),
                     (dict(w_packed=w[:, :16]), ValueError), (dict(w_packed=w[:7]), ValueError),
                     (dict(w_scales=bf16(2, 8)), ValueError), (dict(w_scales=s.float()), TypeError),
                     (dict(w_zeros=torch.zeros(1, 7, dtype=torch.uint8)), ValueError),
                     (dict(w_zeros=torch.zeros(1, 16, dtype=torch.uint8)[:, ::2]), ValueError),
                     (dict(group_size=48), ValueError), (dict(out=out.float()), TypeError),
                     (dict(out=bf16(4, 7)), ValueError), (dict(x=x[:, :0]), ValueError),
                     (dict(x_scale=sx), ValueError), (dict(x=x8), ValueError),
                     (dict(x=x8, x_scale=sx[:2]), ValueError), (dict(x=x8, x_scale=sx.double()), TypeError),
                     (dict(), ValueError)):
        a = dict(x=x, w_packed=w, w_scales=s, out=out, group_size=128)
        a.update(bad)
        with pytest.raises(err):
            lora.lora_w4_project(**a)
    assert lora.lora_w4_project(x[:0], w, s, out[:0], group_size=128).shape == (0, 8)


def test_rope_binding_refusals(L):
    D, off = 16, [0, 64, 96, 128]
    a0 = dict(qkv=bf16(3, 128), slice_offsets=off, head_dim=D, positions=torch.zeros(3, dtype=torch.int64),
              cos_sin=torch.zeros(5, D), k_cache=bf16(2, 4, 2, D), v_cache=bf16(2, 4, 2, D),
              slots=torch.zeros(3, dtype=torch.int64))
    i64 = torch.int64
    for bad, err in ((dict(qkv=bf16(3, 128).float()), TypeError), (dict(qkv=bf16(3, 127)), ValueError),
                     (dict(slice_offsets=[0, 64, 96]), ValueError), (dict(slice_offsets=[0, 64, 95, 126]), ValueError),
                     (dict(head_dim=24), ValueError), (dict(positions=torch.zeros(3)), TypeError),
                     (dict(positions=torch.zeros(3, dtype=torch.int32)), TypeError),
                     (dict(positions=torch.zeros(2, dtype=i64)), ValueError),
                     (dict(positions=torch.zeros(2, 3, dtype=i64)), ValueError),
                     (dict(positions=torch.zeros(5, 3, dtype=i64), axis_map=[0] * 8), ValueError),
                     (dict(positions=torch.zeros(2, 3, dtype=i64), axis_map=[0] * 7), ValueError),
                     (dict(positions=torch.zeros(2, 3, dtype=i64), axis_map=[2] * 8), ValueError),
                     (dict(axis_map=[0] * 8), ValueError), (dict(cos_sin=torch.zeros(5, 18)), ValueError),
                     (dict(cos_sin=torch.zeros(5, 15)), ValueError), (dict(cos_sin=torch.zeros(0, D)), ValueError),
                     (dict(cos_sin=torch.zeros(5, D).double()), ValueError),
                     (dict(k_cache=bf16(2, 4, 3, D)), ValueError), (dict(k_cache=bf16(3, 4, 2, D)), ValueError),
                     (dict(k_cache=bf16(2, 4, 2, D).half()), ValueError),
                     (dict(k_cache=bf16(2, 4, 2, D).float(), v_cache=bf16(2, 4, 2, D).float()), TypeError),
                     (dict(k_cache=bf16(2, 4, 2, 2 * D)[..., ::2]), ValueError),
                     (dict(slots=torch.zeros(4, dtype=i64)), ValueError), (dict(slots=torch.zeros(3)), TypeError),
                     (dict(q_out=bf16(3, 63)), ValueError), (dict(q_weight=bf16(D)), ValueError),
                     (dict(q_weight=bf16(D), k_weight=bf16(D + 1)), ValueError),
                     (dict(), ValueError)):
        with pytest.raises(err):
            lora.lora_rope_append(**{**a0, **bad})


def test_w4_pack_round_trip_and_refusals():
    g = torch.Generator().manual_seed(1)
    for N, K in ((1, 1), (3, 31), (5, 32), (2, 33), (7, 1000)):
        q = torch.randint(0, 16, (N, K), generator=g)
        p = lora.w4_pack(q)
        assert p.shape == (N, -(-K // 32) * 16) and p.dtype == torch.uint8
        assert torch.equal(lora.w4_unpack(p, K).long(), q)
    # value i of a word stands at bit (0, 16, 4, 20, 8, 24, 12, 28)[i]
    word = lora.w4_pack(torch.arange(8)[None]).view(torch.int32)[0, 0].item() & 0xFFFFFFFF
    assert [(word >> s) & 15 for s in (0, 16, 4, 20, 8, 24, 12, 28)] == list(range(8))
    for bad in (torch.full((2, 2), 16), torch.full((2, 2), -1), torch.zeros(4, dtype=torch.int64),
                torch.zeros(2, 2), torch.zeros(2, 2, dtype=torch.bool)):
        with pytest.raises(ValueError):
            lora.w4_pack(bad)
    with pytest.raises(ValueError):
        lora.w4_unpack(torch.zeros(2, 16, dtype=torch.uint8), 33)
    with pytest.raises(ValueError):
        lora.w4_unpack(torch.zeros(2, 15, dtype=torch.uint8), 3)


@pytest.mark.parametrize("zeros", [False, True])
def test_w4_quantize(zeros):
    g = torch.Generator().manual_seed(2)
    W = (torch.randn(9, 200, generator=g) * 0.1 + (0.2 if zeros else 0.0)).to(torch.bfloat16)
    W[3, 64:128] = 0
    p, s, z = lora.w4_quantize(W, 64, zeros=zeros)
    assert s.shape == (4, 9) and (z is None) == (not zeros)
    of = torch.arange(200) // 64
    zp = 8.0 if z is None else z.double()[of].T
    back = (lora.w4_unpack(p, 200).double() - zp) * s.double()[of].T
    # half a step, a step where the zero point is rounded too; the stored scale
    # may be 2^-8 small over up to 15 steps
    step = s.double()[of].T
    assert ((back - W.double()).abs() <= step * (1.0 if zeros else 0.5) + step * 15 * 2.0 ** -8).all()
    assert (back[3, 64:128] == 0).all()
    with pytest.raises(ValueError):
        lora.w4_quantize(W, 48)
    with pytest.raises(TypeError):
        lora.w4_quantize(W.float())


def test_w4_workspace_size(L):
    assert lora.w4_workspace_size(10, 7, torch.bfloat16) == 160
    assert lora.w4_workspace_size(3, 33, torch.float8_e4m3fn) == 3 * 48
    assert lora.w4_workspace_size(0, 33, torch.float16) == 0
    assert L.lora_w4_workspace_size(-1, 3, 0) == 0


def test_rope_axis_map():
    assert lora.rope_axis_map([2, 1, 3]) == [0, 0, 1, 2, 2, 2]
    assert lora.rope_axis_map([3, 2, 2], interleaved=True) == [0, 1, 2, 0, 1, 2, 0]
    assert lora.rope_axis_map([4]) == [0] * 4
    for bad in ([], [1] * 5, [2, -1]):
        with pytest.raises(ValueError):
            lora.rope_axis_map(bad)


def test_packed_calls_give_what_the_calls_give(L):
    assert L.lora_rmsnorm_packed(None) == L.lora_w4_project_packed(None) == INVALID
    assert L.lora_rope_append_packed(None) == INVALID
    n = lambda **k: L.lora_rmsnorm_packed(lora._WORDS["lora_rmsnorm"](*{**dict(
        x=P, ld_x=64, res=P, ld_res=64, ro=P, ld_ro=64, w=P, w0=0.0, eps=1e-6, out=P, ld_out=64,
        q=P, ld_q=64, sc=P, tok=0, H=64, dt=0, st=0), **k}.values()))
    for kw, want in ((dict(), OK), (dict(dt=2), UNSUPPORTED), (dict(eps=-1.0), INVALID),
                     (dict(res=0), INVALID), (dict(sc=0), INVALID), (dict(ld_q=63), INVALID),
                     (dict(tok=1 << 40), INVALID)):
        assert n(**kw) == want, kw
    w = lambda **k: L.lora_w4_project_packed(lora._WORDS["lora_w4_project"](*{**dict(
        x=P, ld_x=128, sx=0, W=P, ld_w=64, s=P, z=P, ld_s=16, out=P, ld_out=16, tok=0, K=128, N=16,
        group=128, xdt=0, dt=0, ws=0, wsb=0, st=0), **k}.values()))
    for kw, want in ((dict(), OK), (dict(xdt=2), INVALID), (dict(group=16), UNSUPPORTED),
                     (dict(ld_out=15), INVALID), (dict(tok=3, W=P + 8), UNSUPPORTED)):
        assert w(**kw) == want, kw
    r = lambda tail=b"", **k: L.lora_rope_append_packed(lora._WORDS["lora_rope_append"](*{**dict(
        qkv=P, ld=512, o0=0, o1=256, o2=384, o3=512, D=64, R=64, pos=P, ld_pos=8, axes=1, amap=0,
        cs=P, max_pos=10, inter=0, qw=0, kw=0, w0=0.0, eps=1e-6, q=P, ld_q=256, kc=P, k0=1024,
        k1=128, k2=64, vc=P, v0=1024, v1=128, v2=64, pages=4, page=8, cdt=0, ksc=1.0, vsc=1.0,
        slots=P, ib=8, tok=0, dt=0, st=0), **k}.values()) + tail)
    for tail, kw, want in ((b"", dict(), OK), (b"", dict(o3=500), INVALID), (b"", dict(k1=-1), INVALID),
                           (b"", dict(v2=-1), INVALID), (b"", dict(axes=2), INVALID),
                           (bytes([0, 1] * 16), dict(axes=2, amap=1), OK),
                           (bytes([0, 2] * 16), dict(axes=2, amap=1), INVALID),
                           (b"", dict(vsc=0.0), INVALID), (b"", dict(page=0), INVALID),
                           (b"", dict(cdt=1), UNSUPPORTED), (b"", dict(ib=2), UNSUPPORTED)):
        assert r(tail, **kw) == want, kw
