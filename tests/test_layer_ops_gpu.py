"""lora_rmsnorm, lora_w4_project and lora_rope_append against their formulas in
64 bits.  Tolerances: half a step of the stored type, plus the fp32 error of
the sums behind it, bounded in each reference below."""
import pytest
import torch

from scatter_gemm_b200 import lora

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3 = torch.float8_e4m3fn
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # eps / 2, relative
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}         # half a subnormal step
SENT = 72.0  # exact in every type, e4m3 included


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def strided(t, pad=0, lead=0):
    """t's values in rows `pad` elements longer than they need be, the first
    `lead` elements into an allocation."""
    rows, cols = t.shape
    flat = torch.full((lead + rows * (cols + pad),), SENT, device="cuda").to(t.dtype)
    v = flat[lead:].view(rows, cols + pad)[:, :cols]
    v.copy_(t)
    return v


def new(tok, n, dtype, pad=0, lead=0):
    return strided(torch.full((tok, n), SENT, device="cuda").to(dtype), pad, lead)


def padding_intact(v):
    """Everything around the strided tensor's rows still holds the sentinel."""
    base = v._base if v._base is not None else v
    n = base.numel()
    flat = base.view(-1).float()
    inside = torch.zeros(n, dtype=torch.bool, device="cuda")
    rows = torch.arange(v.shape[0], device="cuda")[:, None] * v.stride(0) + v.storage_offset()
    inside[(rows + torch.arange(v.shape[1], device="cuda")).flatten()] = True
    return bool((flat[~inside] == SENT).all())


def within(got, ref, tol, what):
    got, bad = got.double(), None
    assert got.shape == ref.shape, what
    nan = ref.isnan()
    assert torch.equal(got.isnan(), nan), f"{what}: NaNs differ"
    err = (got - ref).abs()
    bad = ~nan & (err > tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst "
                           f"{float((err - tol)[bad].max()):.3g} over")


# ----------------------------------------------------------------------------
# RMS norm
# ----------------------------------------------------------------------------

def check_norm(x, w, res=None, eps=1e-6, w0=0.0, mode="both", pad=0, lead=0, in_place=False,
               qpad=0):
    tok, H = x.shape
    dt = x.dtype
    xs = strided(x, pad, lead)
    rs = None if res is None else strided(res, pad, lead)
    ro = None if res is None or in_place else new(tok, H, dt, pad, lead)
    out = new(tok, H, dt, pad, lead) if mode != "8bit" else None
    q = new(tok, H, E4M3, qpad) if mode != "rounded" else None
    sc = torch.full((tok,), SENT, device="cuda") if q is not None else None
    r = lora.lora_rmsnorm(xs, w, out, residual=rs, residual_out=ro, eps=eps, weight_offset=w0,
                          out_q=q, out_scale=sc)
    torch.cuda.synchronize()
    assert r is (out if out is not None else q)
    h = x
    if res is not None:
        h = (x.float() + res.float()).to(dt)
        stream = rs if in_place else ro
        assert torch.equal(stream, h) or bool(h.isnan().any())
        assert padding_intact(stream)
    hd = h.double()
    v = hd * torch.rsqrt(hd.pow(2).mean(1, keepdim=True) + eps) * (w.double() + w0)
    # a sum of squares whose chains are under 128 long, halved by the root, a
    # root good to 2 steps and three products: under 2^-17
    rel = 2.0 ** -17
    if out is not None:
        within(out, v, v.abs() * (HALF[dt] + rel) + TINY[dt], "out")
        assert padding_intact(out)
    if q is not None:
        top = v.abs().amax(1) / 448
        within(sc, top, top * 2 * rel, "scale")
        # half a step of e4m3: 2^-4 of the value, 2^-10 among its subnormals
        tol = v.abs() * (2.0 ** -4 + 4 * rel) + 2.0 ** -10 * sc.double()[:, None]
        within(q.double() * sc.double()[:, None], v, tol, "q")
        assert padding_intact(q)
    return out, q, sc


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("tok,H", [(1, 1), (1, 4096), (3, 7), (5, 8), (2, 65), (300, 64), (17, 520),
                                   (200, 3583), (149, 5120), (33, 8192), (2, 16384), (1, 65536),
                                   (160, 40000), (2, 65531)])
def test_norm_sizes(dtype, tok, H):
    g = gen(tok * 131 + H)
    x, res = (rand(g, tok, H, dtype=DT[dtype], std=s) for s in (1.0, 3.0))
    w = (1 + rand(g, H, std=0.2)).to(DT[dtype])
    check_norm(x, w, res)


@pytest.mark.parametrize("mode", ["rounded", "8bit", "both"])
@pytest.mark.parametrize("with_res", [False, True])
@pytest.mark.parametrize("pad,lead,qpad", [(0, 0, 0), (8, 8, 8), (3, 0, 5), (0, 1, 0), (8, 4, 1)])
def test_norm_strides_and_outputs(mode, with_res, pad, lead, qpad):
    g = gen(5)
    x, res = rand(g, 37, 264, dtype=torch.bfloat16), rand(g, 37, 264, dtype=torch.bfloat16)
    w = rand(g, 264, dtype=torch.bfloat16)
    check_norm(x, w, res if with_res else None, mode=mode, pad=pad, lead=lead, qpad=qpad, w0=1.0)


def test_norm_rows_of_different_alignment():
    # each tensor starts at another element of its 16-byte block
    g = gen(6)
    x, res = (rand(g, 9, 171, dtype=torch.float16) for _ in range(2))
    w = rand(g, 171, dtype=torch.float16)
    a, b, c, d = strided(x, 5, 1), strided(res, 2, 3), new(9, 171, x.dtype, 1, 2), new(9, 171, x.dtype, 4, 6)
    lora.lora_rmsnorm(a, w, c, residual=b, residual_out=d)
    h = (x.float() + res.float()).half()
    assert torch.equal(d, h)
    hd = h.double()
    v = hd * torch.rsqrt(hd.pow(2).mean(1, keepdim=True) + 1e-6) * w.double()
    within(c, v, v.abs() * (2.0 ** -11 + 2.0 ** -17) + 2.0 ** -25, "out")
    assert all(padding_intact(t) for t in (a, b, c, d))


@pytest.mark.parametrize("H", [256, 771])
def test_norm_in_place(H):
    g = gen(7)
    x, res = rand(g, 50, H, dtype=torch.bfloat16), rand(g, 50, H, dtype=torch.bfloat16)
    w = rand(g, H, dtype=torch.bfloat16)
    check_norm(x, w, res, in_place=True)
    want = torch.empty_like(x)
    lora.lora_rmsnorm(x, w, want, residual=res.clone())
    x2, r2 = x.clone(), res.clone()
    lora.lora_rmsnorm(x2, w, x2, residual=r2)
    assert torch.equal(x2, want) and torch.equal(r2, (x.float() + res.float()).bfloat16())


def test_norm_rows_of_zeros_and_non_finite_values():
    g = gen(8)
    x = rand(g, 8, 320, dtype=torch.bfloat16)
    x[1] = 0
    x[3, 17] = float("nan")
    x[5, 300] = float("inf")
    x[6] = x[6] * 1e-30
    w = rand(g, 320, dtype=torch.bfloat16)
    out, q = new(8, 320, x.dtype), new(8, 320, E4M3)
    sc = torch.empty(8, device="cuda")
    lora.lora_rmsnorm(x, w, out, out_q=q, out_scale=sc, eps=0.0)
    # a row of zeros over a zero eps is 0 * inf
    assert out[1].isnan().all() and sc[1].isnan()
    lora.lora_rmsnorm(x, w, out, out_q=q, out_scale=sc)
    assert (out[1] == 0).all() and (q[1].float() == 0).all() and sc[1] == 0
    assert out[3].isnan().all() and sc[3].isnan() and q[3].float().isnan().all()
    assert out[5, 300].isnan() and sc[5].isnan()
    rest = [0, 2, 4, 7]
    check_norm(x[rest].contiguous(), w)
    ref = torch.empty(4, 320, dtype=x.dtype, device="cuda")
    lora.lora_rmsnorm(x[rest].contiguous(), w, ref)
    assert torch.equal(out[rest], ref)  # a bad row does not touch its neighbours


# ----------------------------------------------------------------------------
# 4-bit projection
# ----------------------------------------------------------------------------

def w4_inputs(seed, tok, K, N, dtype, group, zeros, x8, pad=0, lead=0, wpad=0):
    g = gen(seed)
    dt = DT[dtype]
    G = -(-K // group)
    q = torch.randint(0, 16, (N, K), generator=g, device="cuda")
    packed = lora.w4_pack(q)
    if wpad:
        wide = torch.full((N, packed.shape[1] + wpad), 0xAB, dtype=torch.uint8, device="cuda")
        wide[:, :packed.shape[1]] = packed
        packed = wide[:, :packed.shape[1]]
    s = (0.01 * torch.exp(rand(g, G, N, std=0.5))).to(dt)
    z = torch.randint(0, 16, (G, N), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    x = rand(g, tok, K)
    sx = None
    if x8:
        sx = (x.abs().amax(1) / 448).clamp(min=1e-9)
        x = (x / sx[:, None]).clamp(-448, 448).to(E4M3)
    else:
        x = x.to(dt)
    return strided(x, pad, lead), sx, q, packed, s, z


def check_w4(seed, tok, K, N, dtype="bf16", group=128, zeros=False, x8=False, pad=0, lead=0,
             wpad=0, opad=0, olead=0):
    x, sx, q, packed, s, z = w4_inputs(seed, tok, K, N, dtype, group, zeros, x8, pad, lead, wpad)
    dt = DT[dtype]
    out = new(tok, N, dt, opad, olead)
    lora.lora_w4_project(x, packed, s, out, group_size=group, w_zeros=z, x_scale=sx)
    torch.cuda.synchronize()
    assert lora.device_error() == 0
    of = torch.arange(K, device="cuda") // group
    zero = 8.0 if z is None else z.double()[of].T
    W = (q.double() - zero) * s.double()[of].T
    f = 1.0 if sx is None else sx.double()[:, None]
    ref = (x.double() @ W.T) * f
    mag = (x.double().abs() @ W.abs().T) * f
    # sums in steps of 16 products within a group, then over the groups and at
    # most 32 parts of K; a step of a tensor-core sum may cut off 2^-22
    depth = min(K, group) / 16 + -(-K // group) + 40
    within(out, ref, ref.abs() * HALF[dt] + mag * depth * 2.0 ** -22 + TINY[dt], "out")
    assert padding_intact(out)
    return x, sx, packed, s, z, out


@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("tok", [1, 2, 3, 5, 8, 9, 16, 17, 32, 33, 50, 64, 65, 128, 129, 200, 300])
def test_w4_token_counts(tok, dtype, x8):
    check_w4(tok, tok, 512, 384, dtype, x8=x8)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("tok", [1, 7, 24, 100, 257])
def test_w4_groups(tok, group, zeros):
    check_w4(tok + group, tok, 1024, 200, "fp16", group, zeros)
    check_w4(tok + group + 1, tok, 1024, 200, "bf16", group, zeros, x8=True)


@pytest.mark.parametrize("tok", [1, 4, 13, 40, 130])
@pytest.mark.parametrize("K,N", [(1, 1), (5, 3), (31, 17), (33, 128), (127, 129), (129, 15),
                                 (500, 1031), (3583, 65), (4100, 8), (64, 5000)])
def test_w4_odd_sizes(tok, K, N):
    check_w4(tok + K, tok, K, N, "bf16", 64, True)
    check_w4(tok + K + 1, tok, K, N, "fp16", 128, False, x8=True)


@pytest.mark.parametrize("tok", [1, 6, 20, 140])
@pytest.mark.parametrize("pad,lead,wpad,opad,olead", [(8, 8, 16, 8, 8), (1, 0, 32, 3, 1),
                                                      (0, 1, 0, 0, 5), (16, 0, 16, 1, 0)])
@pytest.mark.parametrize("x8", [False, True])
def test_w4_strides(tok, pad, lead, wpad, opad, olead, x8):
    check_w4(3, tok, 576, 312, "bf16", 32, True, x8, pad, lead, wpad, opad, olead)


@pytest.mark.parametrize("tok", [1, 8, 50, 200])
def test_w4_qkv_shape_and_determinism(tok):
    x, sx, packed, s, z, out = check_w4(4, tok, 4096, 6144)
    again = torch.empty_like(out)
    for _ in range(3):
        lora.lora_w4_project(x, packed, s, again, group_size=128)
        assert torch.equal(again, out)


@pytest.mark.parametrize("tok", [1, 12, 30, 150])
@pytest.mark.parametrize("x8", [False, True])
def test_w4_non_finite_values_stay_in_their_rows(tok, x8):
    x, sx, q, packed, s, z = w4_inputs(9, tok, 256, 160, "bf16", 64, True, x8)
    want = torch.empty(tok, 160, dtype=torch.bfloat16, device="cuda")
    lora.lora_w4_project(x, packed, s, want, group_size=64, w_zeros=z, x_scale=sx)
    s[1, 40] = float("nan")
    if tok > 1:
        x[tok // 2, 33] = float("nan")
    got = torch.empty_like(want)
    lora.lora_w4_project(x, packed, s, got, group_size=64, w_zeros=z, x_scale=sx)
    bad = torch.zeros_like(want, dtype=torch.bool)
    bad[:, 40] = True
    if tok > 1:
        bad[tok // 2] = True
    assert got[bad].isnan().all()
    assert torch.equal(got[~bad], want[~bad])


def test_w4_quantized_weight_is_near_the_weight():
    g = gen(12)
    W = rand(g, 96, 300, dtype=torch.bfloat16, std=0.05)
    W[5] = 0
    eye = torch.eye(300, dtype=torch.bfloat16, device="cuda")
    for zeros in (False, True):
        packed, s, z = lora.w4_quantize(W, 64, zeros=zeros)
        out = torch.empty(300, 96, dtype=torch.bfloat16, device="cuda")
        lora.lora_w4_project(eye, packed, s, out, group_size=64, w_zeros=z)
        step = s.double()[torch.arange(300, device="cuda") // 64]
        # half a 4-bit step; the stored scale may be 2^-8 small over up to 15
        # steps, and a zero point is rounded too
        tol = step * (1.0 if zeros else 0.5) + step * 15 * 2.0 ** -8 + W.double().T.abs() * 2.0 ** -8
        within(out, W.double().T, tol, f"zeros={zeros}")


# ----------------------------------------------------------------------------
# rotate and append
# ----------------------------------------------------------------------------

def rope_ref(qkv, off, D, pos, cs, R, amap, inter, qw, kw, eps, w0):
    tok = qkv.shape[0]
    x = qkv.double()
    q, k, v = (x[:, off[i]:off[i + 1]].reshape(tok, -1, D) for i in range(3))
    outs, mags = [], []
    for t, w in ((q, qw), (k, kw)):
        if w is not None:
            t = t * torch.rsqrt(t.pow(2).mean(2, keepdim=True) + eps) * (w.double() + w0)
        y, mag = t.clone(), t.abs().clone()
        for i in range(R // 2):
            p = (pos if pos.dim() == 1 else pos[amap[i] if amap else 0]).long()
            p = p.clamp(0, cs.shape[0] - 1)
            c, s = cs[p, i].double()[:, None], cs[p, R // 2 + i].double()[:, None]
            a, b = (2 * i, 2 * i + 1) if inter else (i, i + R // 2)
            ta, tb = t[:, :, a], t[:, :, b]
            y[:, :, a], y[:, :, b] = ta * c - tb * s, tb * c + ta * s
            mag[:, :, a] = (ta * c).abs() + (tb * s).abs()
            mag[:, :, b] = (tb * c).abs() + (ta * s).abs()
        outs.append(y)
        mags.append(mag)
    return outs[0], outs[1], v, mags[0], mags[1]


def check_rope(seed, tok, hq, hkv, D, dtype="bf16", R=None, axes=1, amap=None, inter=False,
               norm=False, c8=False, page=16, idx=torch.int64, hnd=False, pad=0, lead=0,
               col_lead=0, in_place=False, w0=0.0, slots=None, cpad=0, clead=0, max_pos=500,
               positions=None):
    g = gen(seed)
    dt = DT[dtype]
    R = D if R is None else R
    off = [col_lead, col_lead + hq * D, col_lead + (hq + hkv) * D, col_lead + (hq + 2 * hkv) * D]
    src = rand(g, tok, off[3], dtype=dt)
    qkv = strided(src, pad, lead)
    cs = rand(g, max_pos, R).clamp(-1, 1)
    if positions is None:
        positions = torch.randint(0, max_pos, (tok,) if axes == 1 and amap is None else (axes, tok),
                                  generator=g, device="cuda")
    positions = positions.to(idx)
    pages = -(-tok // page) + 3
    if slots is None:
        slots = torch.randperm(pages * page, generator=g, device="cuda")[:tok]
        slots[::5] = -1
        if tok > 3:
            slots[3] = pages * page  # behind the cache
    slots = slots.to(idx)
    cdt = E4M3 if c8 else dt

    def cache():
        shape = (pages, hkv, page, D) if hnd else (pages, page, hkv, D)
        flat = torch.full((pages * page * hkv * (D + cpad) + clead,), SENT, device="cuda").to(cdt)
        v = flat[clead:].view(*shape[:3], D + cpad)[..., :D]
        return v.transpose(1, 2) if hnd else v

    kc, vc = cache(), cache()
    before = [c.float().clone() for c in (kc, vc)]
    qw, kw = (rand(g, D, dtype=dt) for _ in range(2)) if norm else (None, None)
    ksc, vsc = (0.02, 0.03) if c8 else (1.0, 1.0)
    q_out = None if in_place else new(tok, hq * D, dt, pad, lead)
    got = lora.lora_rope_append(qkv, off, D, positions, cs, kc, vc, slots, q_out=q_out,
                                axis_map=amap, interleaved=inter, q_weight=qw, k_weight=kw,
                                eps=1e-5, weight_offset=w0, k_scale=ksc, v_scale=vsc)
    torch.cuda.synchronize()
    q, k, v, mq, mk = rope_ref(src, off, D, positions, cs, R, amap, inter, qw, kw, 1e-5, w0)
    # two products and a sum: 2^-22 of their magnitudes; the head's norm 2^-17
    rel = 2.0 ** -17 if norm else 2.0 ** -22
    within(got.reshape(tok, hq, D), q, q.abs() * HALF[dt] + mq * rel + TINY[dt], "q")
    if not in_place:
        assert torch.equal(qkv, src) and padding_intact(q_out)
    else:
        assert torch.equal(qkv[:, off[1]:], src[:, off[1]:])
        assert torch.equal(qkv[:, :off[0]], src[:, :off[0]])
    assert padding_intact(qkv)
    live = (slots >= 0) & (slots < pages * page)
    at = slots[live].long()
    for c, b, val, mag, sc, what in ((kc, before[0], k, mk, ksc, "k"),
                                     (vc, before[1], v, v.abs(), vsc, "v")):
        flat = c.float().reshape(pages * page, hkv, D)
        want = val[live] / sc
        if c8:
            want = want.clamp(-448, 448)
            tol = want.abs() * 2.0 ** -4 + 2.0 ** -10 + mag[live] / sc * 2 * rel
        else:
            tol = want.abs() * (HALF[dt] + 2.0 ** -22) + mag[live] * rel + TINY[dt]
        within(flat[at], want, tol, what)
        rest = torch.ones(pages * page, dtype=torch.bool, device="cuda")
        rest[at] = False
        assert torch.equal(flat[rest], b.reshape(pages * page, hkv, D)[rest]), f"{what}: other slots"
        root = c._base if c._base is not None else c
        if cpad:
            assert (root.view(-1)[clead:].view(-1, D + cpad)[:, D:].float() == SENT).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,R", [(2, 2), (64, 64), (128, 128), (80, 80), (80, 40), (96, 48), (96, 96),
                                 (192, 64), (256, 256), (512, 512), (128, 0), (70, 6), (33, 32), (512, 32)])
def test_rope_head_sizes(dtype, inter, D, R):
    check_rope(D + R, 23, 4, 2, D, dtype, R, inter=inter)
    check_rope(D + R + 1, 9, 3, 3, D, dtype, R, inter=inter, norm=True, w0=1.0, c8=True)


@pytest.mark.parametrize("tok,hq,hkv", [(1, 32, 8), (1, 1, 1), (3, 5, 1), (64, 7, 7), (700, 8, 1), (2000, 2, 1)])
def test_rope_batches(tok, hq, hkv):
    check_rope(tok, tok, hq, hkv, 128, page=7)
    check_rope(tok, tok, hq, hkv, 128, page=1, idx=torch.int32, c8=True, norm=True)


@pytest.mark.parametrize("sections,mixed", [([8, 12, 12], False), ([11, 11, 10], True), ([32], False),
                                            ([16, 16], False), ([8, 8, 8, 8], True), ([0, 32], False)])
@pytest.mark.parametrize("inter", [False, True])
def test_rope_axes(sections, mixed, inter):
    amap = lora.rope_axis_map(sections, interleaved=mixed)
    check_rope(11, 41, 6, 2, 80, R=64, axes=len(sections), amap=amap, inter=inter)


@pytest.mark.parametrize("kw", [dict(hnd=True), dict(pad=8, lead=8), dict(pad=3, lead=1),
                                dict(cpad=8), dict(cpad=8, clead=8), dict(cpad=3, clead=1),
                                dict(in_place=True), dict(in_place=True, pad=8, norm=True),
                                dict(col_lead=16), dict(col_lead=5), dict(hnd=True, cpad=16, c8=True),
                                dict(cpad=3, clead=1, c8=True), dict(idx=torch.int32)])
@pytest.mark.parametrize("D", [128, 48])
def test_rope_layouts(kw, D):
    check_rope(21, 37, 6, 2, D, **kw)


def test_rope_positions_outside_the_table_are_clamped():
    pos = torch.tensor([-1, 0, 499, 500, 1 << 40, -(1 << 40)], device="cuda")
    check_rope(31, 6, 2, 1, 64, positions=pos)


def test_rope_no_live_slot_and_infinite_values():
    check_rope(32, 8, 2, 1, 64, slots=torch.full((8,), -1, device="cuda"))
    g = gen(33)
    qkv = rand(g, 4, 4 * 64, dtype=torch.bfloat16)
    qkv[1, 130] = float("inf")   # k
    qkv[2, 200] = float("nan")   # v
    cs = rand(g, 10, 64)
    pos = torch.arange(4, device="cuda")
    kc, vc = (torch.zeros(1, 4, 1, 64, device="cuda").to(E4M3) for _ in range(2))
    out = lora.lora_rope_append(qkv, [0, 128, 192, 256], 64, pos, cs, kc, vc, pos,
                                q_out=torch.empty(4, 128, dtype=qkv.dtype, device="cuda"))
    assert out.isfinite().all()
    assert kc.float().abs().eq(448).sum() == 2          # both of the infinite element's pair
    assert vc.float().isnan().sum() == 1


def test_rope_offsets_beyond_32_bits():
    # a cache of over 2^31 elements: page strides reach the far end of it
    D, hkv, page = 128, 8, 64
    pages = (1 << 31) // (page * hkv * D) + 40
    g = gen(34)
    kc = torch.zeros(pages, page, hkv, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    tok = 5
    qkv = rand(g, tok, (2 + 2 * hkv) * D, dtype=torch.bfloat16)
    cs = torch.cat([torch.ones(4, D // 2), torch.zeros(4, D // 2)], 1).cuda()
    slots = torch.tensor([0, pages * page - 1, pages * page - 65, 77, (1 << 31) // (hkv * D) + 1],
                         device="cuda")
    pos = torch.zeros(tok, dtype=torch.int64, device="cuda")
    off = [0, 2 * D, (2 + hkv) * D, (2 + 2 * hkv) * D]
    lora.lora_rope_append(qkv, off, D, pos, cs, kc, vc, slots)
    assert torch.equal(kc.view(-1, hkv, D)[slots], qkv[:, off[1]:off[2]].reshape(tok, hkv, D))
    assert torch.equal(vc.view(-1, hkv, D)[slots], qkv[:, off[2]:off[3]].reshape(tok, hkv, D))
    assert int(torch.count_nonzero(kc.view(-1, hkv * D).any(1))) == tok


# ----------------------------------------------------------------------------
# large K, paths, streams, and the operators one after the other
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("tok", [1, 2, 8])
def test_w4_long_rows(tok):
    # x of 8 tokens does not fit shared memory: the tensor-core kernel takes it
    check_w4(tok, tok, 65536 if tok == 1 else 40000, 48, "bf16", 128)
    check_w4(tok, tok, 131072, 33, "fp16", 128, zeros=True)


def test_w4_long_rows_off_the_16_byte_grid():
    check_w4(5, 20, 30001, 40, "bf16", 64)
    # up to 8 tokens nothing is copied, and these rows fit neither kernel
    x = new(2, 120000, torch.bfloat16, pad=1)
    out = new(2, 16, torch.bfloat16)
    with pytest.raises(lora.LoraError) as e:
        lora.lora_w4_project(x, torch.zeros(16, 60000, dtype=torch.uint8, device="cuda"),
                             torch.zeros(938, 16, dtype=torch.bfloat16, device="cuda"), out,
                             group_size=128)
    assert e.value.status == lora.LORA_ERR_UNSUPPORTED
    assert (out == SENT).all()


def test_w4_paths_and_launches():
    for tok, N, want, launches in ((8, 512, lora.PATH_GENERAL, 1), (9, 19000, lora.PATH_TENSOR, 1),
                                   (9, 512, lora.PATH_TENSOR | lora.PATH_SPLITK, 1),
                                   # 150 tiles on 148 SMs: a wave and two tiles left over
                                   (128, 150 * 128, lora.PATH_TENSOR | lora.PATH_SPLITK, 2)):
        x, sx, q, packed, s, z = w4_inputs(tok, tok, 256, N, "bf16", 128, False, False)
        out = torch.empty(tok, N, dtype=x.dtype, device="cuda")
        lora.reset_launch_count()
        lora.lora_w4_project(x, packed, s, out, group_size=128)
        if torch.cuda.get_device_properties(0).multi_processor_count == 148:
            assert lora.last_path() == want and lora.launch_count() == launches, (tok, N)


@pytest.mark.parametrize("group", [32, 128])
def test_w4_tiles_left_over(group):
    # whole waves of tiles and a few more, rows and tokens ragged
    check_w4(6, 130, 640, 75 * 128 + 5, "bf16", group, True)
    check_w4(7, 200, 384, 80 * 128 - 3, "fp16", group, False, x8=True)


def test_on_another_stream():
    g = gen(40)
    x, res = rand(g, 30, 512, dtype=torch.bfloat16), rand(g, 30, 512, dtype=torch.bfloat16)
    w = rand(g, 512, dtype=torch.bfloat16)
    want = torch.empty_like(x)
    lora.lora_rmsnorm(x, w, want, residual=res.clone())
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got, r2 = torch.empty_like(x), res.clone()
    torch.cuda.synchronize()
    lora.lora_rmsnorm(x, w, got, residual=r2, stream=st)
    st.synchronize()
    assert torch.equal(got, want)
    with torch.cuda.stream(st):  # the current stream is the default
        got2 = torch.empty_like(x)
        lora.lora_rmsnorm(x, w, got2, residual=res.clone())
    st.synchronize()
    assert torch.equal(got2, want)


def test_two_streams_at_once():
    # kernels that take tensor memory and clusters, from two streams, many times
    jobs = []
    for tok, K, N, x8 in ((40, 2048, 1024, False), (130, 1024, 19500, True)):
        x, sx, q, packed, s, z = w4_inputs(tok, tok, K, N, "bf16", 128, False, x8)
        want = torch.empty(tok, N, dtype=torch.bfloat16, device="cuda")
        lora.lora_w4_project(x, packed, s, want, group_size=128, x_scale=sx)
        jobs.append((x, packed, s, sx, want, [torch.empty_like(want) for _ in range(20)],
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    for i in range(20):
        for x, packed, s, sx, want, outs, st in jobs:
            lora.lora_w4_project(x, packed, s, outs[i], group_size=128, x_scale=sx, stream=st)
    torch.cuda.synchronize()
    for x, packed, s, sx, want, outs, st in jobs:
        assert all(torch.equal(o, want) for o in outs)
    assert lora.device_error() == 0


class Step:
    """The attention input of one decoder layer for a batch of adapted requests:
    norm, 4-bit projection of its 8-bit output, LoRA pair on its 16-bit output,
    rotation and append."""

    def __init__(self, seed, tok, hidden=1024, hq=8, hkv=2, D=128, rank=16, adapters=4, big=False):
        g = gen(seed)
        dt = torch.bfloat16
        self.off = [0, hq * D, (hq + hkv) * D, (hq + 2 * hkv) * D]
        N = self.off[3]
        self.D, self.rank = D, rank
        self.x, self.res = rand(g, tok, hidden, dtype=dt), rand(g, tok, hidden, dtype=dt)
        self.w = (1 + rand(g, hidden, std=0.2)).to(dt)
        W = rand(g, N, hidden, dtype=dt, std=hidden ** -0.5)
        self.packed, self.s, self.z = lora.w4_quantize(W, 128, zeros=True)
        self.A = rand(g, adapters, 3 * rank, hidden, dtype=dt, std=0.02)
        self.B = rand(g, adapters, N, rank, dtype=dt, std=0.02)
        cut = sorted(torch.randint(0, tok + 1, (adapters - 1,), generator=g, device="cuda").tolist())
        self.si = torch.tensor([0] + cut + [tok], dtype=torch.int32, device="cuda")
        self.wi = torch.arange(adapters, dtype=torch.int32, device="cuda").flip(0).contiguous()
        self.pm = torch.randperm(tok, generator=g, device="cuda").to(torch.int32)
        self.sc = torch.tensor([2.0, 0.5, 0.0, 1.0], device="cuda")[:adapters].contiguous()
        self.cs = rand(g, 300, D).clamp(-1, 1)
        self.pos = torch.randint(0, 300, (tok,), generator=g, device="cuda")
        self.slots = torch.randperm(4 * 64, generator=g, device="cuda")[:tok]
        self.kc, self.vc = (torch.zeros(4, 64, hkv, D, dtype=dt, device="cuda") for _ in range(2))
        self.qw, self.kw = rand(g, D, dtype=dt), rand(g, D, dtype=dt)
        self.out = torch.empty_like(self.x)
        self.q8 = torch.empty(tok, hidden, dtype=E4M3, device="cuda")
        self.sx = torch.empty(tok, device="cuda")
        self.r = torch.empty(tok, 3 * rank, dtype=dt, device="cuda")
        self.qkv = torch.empty(tok, N, dtype=dt, device="cuda")
        self.q = torch.empty(tok, self.off[1], dtype=dt, device="cuda")

    def run(self):
        lora.lora_rmsnorm(self.x, self.w, self.out, residual=self.res, out_q=self.q8,
                          out_scale=self.sx)
        lora.lora_w4_project(self.q8, self.packed, self.s, self.qkv, group_size=128,
                             w_zeros=self.z, x_scale=self.sx)
        lora.lora_shrink_expand(self.out, self.A, self.B, self.si, self.wi, self.pm, self.off,
                                self.sc, self.r, self.qkv)
        lora.lora_rope_append(self.qkv, self.off, self.D, self.pos, self.cs, self.kc, self.vc,
                              self.slots, q_out=self.q, q_weight=self.qw, k_weight=self.kw)


@pytest.mark.parametrize("tok", [1, 7, 50, 200])
def test_a_layer_of_them(tok):
    s = Step(tok, tok)
    x0, r0 = s.x.clone(), s.res.clone()
    s.run()
    torch.cuda.synchronize()
    h = (x0.float() + r0.float()).bfloat16()
    assert torch.equal(s.res, h) and torch.equal(s.x, x0)
    v = h.double() * torch.rsqrt(h.double().pow(2).mean(1, keepdim=True) + 1e-6) * s.w.double()
    within(s.out, v, v.abs() * (2.0 ** -8 + 2.0 ** -17), "x")
    # from what each operator was given: the projection, then the LoRA term
    of = torch.arange(v.shape[1], device="cuda") // 128
    q = lora.w4_unpack(s.packed, v.shape[1]).double()
    W = (q - s.z.double()[of].T) * s.s.double()[of].T
    x8 = s.q8.double() * s.sx.double()[:, None]
    base = x8 @ W.T
    R = s.rank
    lo = torch.zeros_like(base)
    si = s.si.tolist()
    for g_, a in enumerate(s.wi.tolist()):
        rows = s.pm[si[g_]:si[g_ + 1]].long()
        ra = s.out[rows].double() @ s.A[a].double().T
        for t in range(3):
            c0, c1 = s.off[t], s.off[t + 1]
            lo[rows, c0:c1] = float(s.sc[a]) * ra[:, t * R:(t + 1) * R] @ s.B[a, c0:c1].double().T
    # the projection rounded, the rank activations rounded, their sum rounded
    ref = base + lo
    tol = (base.abs() + ref.abs()) * 2.0 ** -8 + 2e-2 * lo.abs() + 2.0 ** -8
    within(s.qkv, ref, tol, "q/k/v")
    qr, kr, vr, mq, mk = rope_ref(s.qkv, s.off, s.D, s.pos, s.cs, s.D, None, False, s.qw, s.kw, 1e-6, 0.0)
    within(s.q.reshape(qr.shape), qr, qr.abs() * 2.0 ** -8 + mq * 2.0 ** -17, "q")
    at = s.slots
    hkv = s.kc.shape[2]
    within(s.kc.view(-1, hkv, s.D)[at], kr, kr.abs() * 2.0 ** -8 + mk * 2.0 ** -17, "k")
    assert torch.equal(s.vc.view(-1, hkv, s.D)[at].double(), vr)
    # x in 8 bits is near x: half a step of e4m3 in 448 steps' range of a row
    assert (x8 - v).abs().le(v.abs() * 2.0 ** -4 + 2.0 ** -10 * s.sx.double()[:, None] +
                             v.abs() * 2.0 ** -15).all()


@pytest.mark.parametrize("tok", [3, 60])
def test_a_layer_of_them_in_a_graph(tok):
    s, t = Step(70 + tok, tok), Step(80 + tok, tok)
    s.run()  # first calls of each kernel outside of the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    # the other step's inputs in the first one's buffers
    for n in ("x", "res", "w", "packed", "s", "z", "A", "B", "si", "wi", "pm", "sc", "cs", "pos",
              "slots", "qw", "kw"):
        getattr(s, n).copy_(getattr(t, n))
    s.kc.zero_(), s.vc.zero_()
    graph.replay()
    t.run()
    torch.cuda.synchronize()
    for n in ("res", "out", "sx", "qkv", "q", "kc", "vc"):
        assert torch.equal(getattr(s, n), getattr(t, n)), n
    assert torch.equal(s.q8.view(torch.uint8), t.q8.view(torch.uint8))
    assert lora.device_error() == 0


def test_w4_tiles_left_over_in_a_graph():
    # two launches, the second of which starts early, replayed on new inputs
    x, sx, q, packed, s, z = w4_inputs(50, 140, 512, 76 * 128, "bf16", 64, True, False)
    x2 = w4_inputs(51, 140, 512, 76 * 128, "bf16", 64, True, False)[0]
    want = torch.empty(140, 76 * 128, dtype=x.dtype, device="cuda")
    lora.lora_w4_project(x2, packed, s, want, group_size=64, w_zeros=z)
    torch.cuda.synchronize()
    got, after = torch.empty_like(want), torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lora.lora_w4_project(x, packed, s, got, group_size=64, w_zeros=z)
        after.copy_(got)  # what follows sees both launches' tiles
    for _ in range(3):
        got.zero_()
        x.copy_(x2)
        graph.replay()
        assert torch.equal(after, want)


@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("given", ["none", "enough", "short"])
def test_w4_workspace_for_rows_off_the_16_byte_grid(x8, given):
    # 20 tokens whose rows start at any element: copied to aligned rows first,
    # or (too short a workspace) read as they are
    x, sx, q, packed, s, z = w4_inputs(60, 20, 333, 200, "bf16", 64, True, x8, pad=0, lead=3)
    need = lora.w4_workspace_size(20, 333, x.dtype)
    ws = None
    if given != "none":
        guard = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device="cuda")
        ws = guard[:need if given == "enough" else 16]
    out = new(20, 200, torch.bfloat16)
    lora.reset_launch_count()
    lora.lora_w4_project(x, packed, s, out, group_size=64, w_zeros=z, x_scale=sx, workspace=ws)
    assert lora.launch_count() == (1 if given == "short" else 2)
    want = torch.empty_like(out)
    even = torch.zeros(20, 336, device="cuda").to(x.dtype)[:, :333]
    if x8:  # rows of 336 bytes are on the grid too
        assert even.stride(0) % 16 == 0
    even.copy_(x)
    lora.lora_w4_project(even, packed, s, want, group_size=64, w_zeros=z, x_scale=sx)
    if given != "short":
        assert torch.equal(out, want)
        if ws is not None:
            assert (guard[need:] == 0x5A).all()
    else:
        # each within half a step of the exact value, and its sums' error
        tol = want.double().abs() * 2.0 ** -7 + x.double().abs().sum(1)[:, None] * \
            (1.0 if sx is None else sx.double()[:, None]) * 15 * s.double().max() * 60 * 2.0 ** -21
        within(out, want.double(), tol, "out")


def test_w4_scratch_belongs_to_the_calls_stream():
    # the scratch of calls on a side stream must not be handed to the current
    # stream's allocations while those calls run
    x, sx, q, packed, s, z = w4_inputs(61, 200, 4001, 2048, "bf16", 128, False, False)
    want = torch.empty(200, 2048, dtype=x.dtype, device="cuda")
    lora.lora_w4_project(x, packed, s, want, group_size=128)
    torch.cuda.synchronize()
    n = lora.w4_workspace_size(200, 4001, x.dtype)
    for st in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        outs = [torch.empty_like(want) for _ in range(12)]
        torch.cuda.synchronize()
        for o in outs:
            lora.lora_w4_project(x, packed, s, o, group_size=128, stream=st)
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)


def test_norm_offsets_beyond_32_bits():
    tok, H = 66000, 32776  # over 2^31 elements; the first and last rows count
    g = gen(70)
    x = torch.ones(tok, H, dtype=torch.bfloat16, device="cuda")
    rows = [0, 1, tok // 2, tok - 2, tok - 1]
    for r in rows:
        x[r] = rand(g, H, dtype=x.dtype)
    w = rand(g, H, dtype=x.dtype)
    out = torch.zeros_like(x)
    q = torch.zeros(tok, H, dtype=torch.uint8, device="cuda").view(E4M3)
    sc = torch.empty(tok, device="cuda")
    lora.lora_rmsnorm(x, w, out, out_q=q, out_scale=sc)
    few = torch.empty(len(rows), H, dtype=x.dtype, device="cuda")
    fq, fs = torch.empty(len(rows), H, dtype=torch.uint8, device="cuda").view(E4M3), torch.empty(len(rows), device="cuda")
    lora.lora_rmsnorm(x[rows].contiguous(), w, few, out_q=fq, out_scale=fs)
    # the same thread layout for few rows and many is not given: sums may differ
    within(out[rows], few.double(), few.double().abs() * 2.0 ** -7, "out")
    within(sc[rows], fs.double(), fs.double() * 2.0 ** -15, "scale")
    d = fq.double() * fs.double()[:, None]
    within(q[rows].double() * sc[rows].double()[:, None], d, d.abs() * 2.0 ** -3 + 2.0 ** -9 * fs.double()[:, None], "q")


def test_w4_offsets_beyond_32_bits():
    tok, K, N = 66000, 64, 32800
    g = gen(71)
    x = rand(g, tok, K, dtype=torch.bfloat16)
    packed = lora.w4_pack(torch.randint(0, 16, (N, K), generator=g, device="cuda"))
    s = (0.01 * torch.exp(rand(g, 1, N, std=0.3))).to(x.dtype)
    out = torch.zeros(tok, N, dtype=x.dtype, device="cuda")
    lora.lora_w4_project(x, packed, s, out, group_size=64)
    rows = [0, 127, 128, 40000, 65520, tok - 1]
    xf = torch.zeros(40, K, dtype=x.dtype, device="cuda")
    xf[:len(rows)] = x[rows]
    few = torch.empty(40, N, dtype=x.dtype, device="cuda")
    lora.lora_w4_project(xf, packed, s, few, group_size=64)
    assert torch.equal(out[rows], few[:len(rows)])  # one group: one sum, however tiled
