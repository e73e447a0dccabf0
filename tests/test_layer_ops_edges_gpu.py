"""Edges of lora_rmsnorm, lora_w4_project and lora_rope_append, against their
formulas in 64 bits: the values of 8-bit outputs, the range of the element
types, infinities, and the kernel variants that serve prompts.  Tolerances as
in test_layer_ops_gpu.py."""
import os
import subprocess
import sys

import pytest
import torch

from scatter_gemm_b200 import lora
from tests.test_layer_ops_gpu import (DT, E4M3, HALF, SENT, TINY, check_norm, check_rope, check_w4,
                                      gen, new, padding_intact, rand, rope_ref, strided,
                                      w4_inputs, within)

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("tok,H,pad", [(3, 4096, 0), (5, 1003, 1), (2, 40000, 0)])
def test_norm_8bit_values_are_products_with_the_rounded_reciprocal(dtype, tok, H, pad):
    # with x = +-1 and eps = 0 the norm's factor is 1 and v is the weight
    g = gen(90 + H)
    x = (torch.randint(0, 2, (tok, H), generator=g, device="cuda") * 2 - 1).to(DT[dtype])
    w = rand(g, H, dtype=DT[dtype])
    q, sc = new(tok, H, E4M3, pad), torch.empty(tok, device="cuda")
    lora.lora_rmsnorm(strided(x, pad), w, None, eps=0.0, out_q=q, out_scale=sc)
    v = x.float() * w.float()
    assert torch.equal(sc, v.abs().amax(1) / torch.full((tok,), 448.0, device="cuda"))
    want = (v * sc.reciprocal()[:, None]).clamp(-448, 448).to(E4M3)
    assert torch.equal(q.float(), want.float())
    assert padding_intact(q)


@pytest.mark.parametrize("D", [64, 33])
@pytest.mark.parametrize("tok", [7, 1500])
@pytest.mark.parametrize("c8", [False, True])
def test_rope_cache_values_are_products_with_the_rounded_reciprocal(tok, D, c8):
    # a rotation by nothing: k' is k
    hq, hkv = 18, 3
    g = gen(91 + tok)
    off = [0, hq * D, (hq + hkv) * D, (hq + 2 * hkv) * D]
    qkv, R = rand(g, tok, off[3], dtype=torch.bfloat16), D // 2 * 2
    cs = torch.cat([torch.ones(1, R // 2), torch.zeros(1, R // 2)], 1).cuda()
    at = torch.arange(tok, device="cuda")
    dt = E4M3 if c8 else qkv.dtype
    kc, vc = (torch.zeros(tok, 1, hkv, D, device="cuda").to(dt) for _ in range(2))
    lora.lora_rope_append(qkv, off, D, torch.zeros_like(at), cs, kc, vc, at, k_scale=0.03, v_scale=0.02)
    for c, lo, hi, scale in ((kc, off[1], off[2], 0.03), (vc, off[2], off[3], 0.02)):
        want = qkv[:, lo:hi].float() * torch.tensor(scale).reciprocal().cuda()
        want = (want.clamp(-448, 448) if c8 else want).to(dt)
        assert torch.equal(c.float().reshape(tok, -1), want.float())


@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("K,group", [(40, 32), (70, 64), (200, 32), (130, 128), (300, 64)])
@pytest.mark.parametrize("tok", [1, 8, 20, 100])
def test_w4_infinite_scale_of_the_last_group(tok, K, group, x8):
    # the groups that would follow behind K add nothing, whatever that scale
    x, sx, q, packed, s, z = w4_inputs(104, tok, K, 50, "bf16", group, True, x8)
    s[-1, 7], s[-1, 30] = float("inf"), float("-inf")
    out = new(tok, 50, torch.bfloat16)
    lora.lora_w4_project(x, packed, s, out, group_size=group, w_zeros=z, x_scale=sx)
    g0 = (-(-K // group) - 1) * group
    last = x[:, g0:].double() @ (q[:, g0:].double() - z[-1].double()[:, None]).T
    for col, sign in ((7, 1.0), (30, -1.0)):
        want = last[:, col] * sign * float("inf")  # NaN where the group's sum is 0
        assert torch.equal(out[:, col].double().nan_to_num(7.0), want.nan_to_num(7.0))
    out[:, [7, 30]] = 0
    assert out.isfinite().all()


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("tok,lead", [(1, 0), (5, 0), (8, 0), (9, 0), (13, 1), (40, 0)])
def test_w4_range_of_bf16_x(tok, lead, zeros):
    # rows of x from near the smallest to near the largest normal bf16, one of
    # both: a row's result does not depend on how many others there are
    _, _, q, packed, s, z = w4_inputs(91, tok, 520, 70, "bf16", 64, zeros, False)
    g = gen(92)
    x = rand(g, tok, 520)
    mags = [1e-33, 1e35, 1e-20, 1e20, 1.0]
    for t in range(tok):
        x[t] *= mags[(t + tok) % 5]
    x[0, ::2] *= 1e-25 if mags[tok % 5] > 1e-6 else 1e25
    x = strided(x.bfloat16(), 0, lead)
    out = new(tok, 70, x.dtype)
    lora.lora_w4_project(x, packed, s, out, group_size=64, w_zeros=z)
    of = torch.arange(520, device="cuda") // 64
    W = (q.double() - (8.0 if z is None else z.double()[of].T)) * s.double()[of].T
    ref, mag = x.double() @ W.T, x.double().abs() @ W.abs().T
    depth = 64 / 16 + 9 + 40
    # TINY: results near the smallest normal value are rounded among subnormals
    within(out, ref, ref.abs() * 2.0 ** -8 + mag * depth * 2.0 ** -22 + 2.0 ** -133, "out")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("tok,lead", [(1, 0), (6, 0), (9, 0), (14, 3), (30, 0), (100, 0)])
def test_w4_infinities_are_products_of_their_weights(tok, lead, group, dtype):
    # inf * (q - z): an infinity of the weight's sign, NaN where q = z
    x, _, q, packed, s, z = w4_inputs(93, tok, 300, 90, dtype, group, True, False, lead=lead)
    rows = [0] if tok == 1 else [1, tok - 1]
    x[rows[0], 77] = float("inf")
    x[rows[-1], 299] = float("-inf")
    out = new(tok, 90, x.dtype)
    lora.lora_w4_project(x, packed, s, out, group_size=group, w_zeros=z)
    of = torch.arange(300, device="cuda") // group
    d = q.double() - z.double()[of].T
    W = d * s.double()[of].T
    assert (d[:, 77] == 0).any() and (d[:, 77] > 0).any() and (d[:, 77] < 0).any()
    hit = torch.zeros(tok, dtype=torch.bool, device="cuda")
    hit[rows] = True
    want = x.double() @ W.T
    assert torch.equal(out[hit].double().nan_to_num(7.0), want[hit].nan_to_num(7.0))
    rest, mag = want[~hit], x[~hit].double().abs() @ W.abs().T
    within(out[~hit], rest, rest.abs() * HALF[x.dtype] + mag * 60 * 2.0 ** -22 + TINY[x.dtype], "rest")


@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("tok,lead", [(1, 0), (8, 0), (12, 1), (20, 0)])
def test_w4_weights_at_their_zero_point_add_nothing(tok, lead, x8):
    # columns of large x whose weights all equal their zero point, as in a
    # pruned model: what is left is a sum of small products
    _, _, q, _, s, z = w4_inputs(94, tok, 256, 100, "fp16", 64, True, x8)
    of = torch.arange(256, device="cuda") // 64
    big = torch.tensor([5, 70, 77, 130, 255], device="cuda")
    q[:, big] = z.long()[of[big]].T
    g = gen(95)
    x = rand(g, tok, 256, std=0.01)
    x[:, big] = rand(g, tok, 5, std=200.0)
    sx = None
    if x8:
        sx = torch.full((tok,), 2.0, device="cuda")
        x = (x / 2).clamp(-448, 448).to(E4M3)
    else:
        x = x.half()
    x = strided(x, 0, lead)
    out = new(tok, 100, torch.float16)
    lora.lora_w4_project(x, lora.w4_pack(q), s, out, group_size=64, w_zeros=z, x_scale=sx)
    W = (q.double() - z.double()[of].T) * s.double()[of].T
    f = 1.0 if sx is None else sx.double()[:, None]
    ref, mag = (x.double() @ W.T) * f, (x.double().abs() @ W.abs().T) * f
    within(out, ref, ref.abs() * 2.0 ** -11 + mag * 60 * 2.0 ** -22 + 2.0 ** -25, "out")


@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("K", [8191, 16383, 70001])
@pytest.mark.parametrize("tok", [6, 8, 9, 16])
def test_w4_long_rows_off_the_grid_are_copied(tok, K, x8):
    # where shared memory does not hold all tokens' rows at once, the rows are
    # copied to the workspace and W is read once
    check_w4(tok, tok, K, 40, "bf16", 128, False, x8)
    copies = lora.lib().lora_w4_copies_x(tok, K)
    assert bool(lora.last_path() & lora.PATH_TENSOR) == bool(copies)
    assert copies == ((tok, K) not in ((6, 8191), (8, 8191), (9, 8191)))


@pytest.mark.parametrize("tok,most", [(1, 94080), (3, 94080), (9, 85888), (40, 85888)])
def test_w4_long_rows_off_the_grid_without_a_workspace(tok, most):
    # as long as shared memory holds one of them
    for K, want in ((most, lora.LORA_OK), (most + 1, lora.LORA_ERR_UNSUPPORTED)):
        x, _, q, packed, s, z = w4_inputs(tok, tok, K, 20, "bf16", 128, False, False, lead=1)
        out = new(tok, 20, x.dtype)
        got = lora.lib().lora_w4_project(
            x.data_ptr(), x.stride(0), None, packed.data_ptr(), packed.stride(0), s.data_ptr(), None,
            s.stride(0), out.data_ptr(), out.stride(0), tok, K, 20, 128, 0, 0, None, 0,
            torch.cuda.current_stream().cuda_stream)
        assert got == want
        if want:
            assert (out == SENT).all()
            continue
        W = (q.double() - 8) * s.double()[torch.arange(K, device="cuda") // 128].T
        ref, mag = x.double() @ W.T, x.double().abs() @ W.abs().T
        depth = 128 / 16 + -(-K // 128) + 40
        within(out, ref, ref.abs() * 2.0 ** -8 + mag * depth * 2.0 ** -22, "out")


@pytest.mark.parametrize("tok", [1, 2, 16])
def test_w4_longest_rows_off_the_grid_take_a_given_workspace(tok):
    K = 120000
    x, _, q, packed, s, z = w4_inputs(5, tok, K, 20, "fp16", 128, False, False, lead=1)
    out, want = new(tok, 20, x.dtype), new(tok, 20, x.dtype)
    with pytest.raises(lora.LoraError):
        lora.lora_w4_project(x, packed, s, out, group_size=128)
    assert (out == SENT).all()
    ws = torch.empty(lora.w4_workspace_size(tok, K, x.dtype), dtype=torch.uint8, device="cuda")
    lora.lora_w4_project(x, packed, s, out, group_size=128, workspace=ws)
    lora.lora_w4_project(x.clone(), packed, s, want, group_size=128)
    assert torch.equal(out, want)


FIRST_CALLS = r"""
import hashlib, sys, torch
from scatter_gemm_b200 import lora
from tests.test_layer_ops_gpu import w4_inputs
captured = sys.argv[1] == "captured"
got = {}
for tok in eval(sys.argv[2]):
    x, _, _, packed, s, _ = w4_inputs(tok, tok, 2048, 1024, "bf16", 128, False, False)
    out = torch.zeros(tok, 1024, dtype=x.dtype, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    if captured:
        with torch.cuda.graph(graph):
            lora.lora_w4_project(x, packed, s, out, group_size=128)
        graph.replay()
    else:
        lora.lora_w4_project(x, packed, s, out, group_size=128)
    got[tok] = hashlib.sha1(out.view(torch.int16).cpu().numpy().tobytes()).hexdigest()
assert lora.device_error() == 0
print(sorted(got.items()))
"""


def test_w4_results_do_not_depend_on_the_calls_before():
    # nor on whether a kernel's first call is a captured one
    said = set()
    for how, order in (("plain", [4, 12, 40, 60, 300]), ("plain", [300, 60, 40, 12, 4]),
                       ("captured", [40, 300, 4, 12, 60])):
        r = subprocess.run([sys.executable, "-c", FIRST_CALLS, how, str(order)], cwd=ROOT, text=True,
                           capture_output=True, timeout=300)
        assert r.returncode == 0, r.stderr[-2000:]
        said.add(r.stdout)
    assert len(said) == 1


def test_w4_one_groups_zeros_of_any_row_stride():
    x, _, q, packed, s, z = w4_inputs(96, 3, 100, 50, "bf16", 128, True, False)
    want = torch.empty(3, 50, dtype=x.dtype, device="cuda")
    lora.lora_w4_project(x, packed, s, want, group_size=128, w_zeros=z)
    wide = torch.full((2, 70), 0xAB, dtype=torch.uint8, device="cuda")
    wide[:1, :50] = z
    got = torch.empty_like(want)
    lora.lora_w4_project(x, packed, s, got, group_size=128, w_zeros=wide[:1, :50])
    assert torch.equal(got, want)
    # with two groups the strides must agree
    x, _, q, packed, s, z = w4_inputs(97, 3, 200, 50, "bf16", 128, True, False)
    wide = torch.zeros(2, 70, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        lora.lora_w4_project(x, packed, s, got, group_size=128, w_zeros=wide[:, :50])


def test_w4_a_single_row_of_any_stride():
    # the stride of an only row says nothing: 120000 columns are more than
    # shared memory holds, so TMA has to take them
    x, _, q, packed, s, z = w4_inputs(98, 2, 120000, 33, "bf16", 128, False, False, pad=1)
    assert x.stride(0) % 8
    out, want = (torch.empty(1, 33, dtype=x.dtype, device="cuda") for _ in range(2))
    lora.lora_w4_project(x[:1].clone(), packed, s, want, group_size=128)
    lora.lora_w4_project(x[:1], packed, s, out, group_size=128)
    assert torch.equal(out, want)


def test_one_token_of_any_stride():
    # norm and rotation of the first row of a padded batch
    g = gen(99)
    x = strided(rand(g, 2, 520, dtype=torch.bfloat16), 3)[:1]
    w = rand(g, 520, dtype=x.dtype)
    check_norm(x.clone(), w)
    got, want = new(1, 520, x.dtype), new(1, 520, x.dtype)
    lora.lora_rmsnorm(x, w, got)
    lora.lora_rmsnorm(x.clone(), w, want)
    assert torch.equal(got, want)
    check_rope(99, 1, 4, 2, 64, pad=3)


@pytest.mark.parametrize("tok", [1, 12])
def test_w4_one_output_of_any_row_stride(tok):
    x, _, q, packed, s, z = w4_inputs(100, tok, 200, 1, "bf16", 64, True, False)
    wide = torch.full((2, packed.shape[1] + 7), 0xAB, dtype=torch.uint8, device="cuda")[:1, :packed.shape[1]]
    wide.copy_(packed)
    out, want = (torch.empty(tok, 1, dtype=x.dtype, device="cuda") for _ in range(2))
    lora.lora_w4_project(x, packed, s, want, group_size=64, w_zeros=z)
    lora.lora_w4_project(x, wide, s, out, group_size=64, w_zeros=z)
    assert torch.equal(out, want)
    got = lora.lib().lora_w4_project(
        x.data_ptr(), 200, None, wide.data_ptr(), wide.stride(0), s.data_ptr(), z.data_ptr(), 1,
        out.zero_().data_ptr(), 1, tok, 200, 1, 64, 0, 0, None, 0,
        torch.cuda.current_stream().cuda_stream)
    assert got == lora.LORA_OK and torch.equal(out, want)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("mode", ["rounded", "both", "8bit"])
@pytest.mark.parametrize("tok,H,pad", [(1200, 5120, 0), (1300, 8191, 1), (1190, 12000, 3),
                                       (3, 24576, 0), (2, 32768, 0), (3, 30001, 5),
                                       (150, 16400, 0), (2, 65536, 0), (2, 65530, 1)])
def test_norm_of_wide_rows_and_many_rows(tok, H, pad, mode, in_place):
    # four and eight blocks of eight a thread, up to 256, 512 and 1024 threads a row
    g = gen(tok + H)
    x, res = (rand(g, tok, H, dtype=torch.bfloat16, std=s) for s in (1.0, 3.0))
    w = (1 + rand(g, H, std=0.2)).bfloat16()
    check_norm(x, w, res, mode=mode, pad=pad, in_place=in_place)


@pytest.mark.parametrize("tok,H,pad", [(1200, 5120, 0), (1300, 8191, 1), (2, 65536, 0), (2, 40000, 1)])
def test_norm_written_over_x(tok, H, pad):
    g = gen(tok * H)
    x, res = (rand(g, tok, H, dtype=torch.float16) for _ in range(2))
    w = rand(g, H, dtype=torch.float16)
    want, want_r = strided(x, pad), strided(res, pad)
    lora.lora_rmsnorm(strided(x, pad), w, want, residual=want_r)
    a, b = strided(x, pad), strided(res, pad)
    lora.lora_rmsnorm(a, w, a, residual=b)           # out over x, the stream over the residual
    assert torch.equal(a, want) and torch.equal(b, want_r)
    a, out = strided(x, pad), new(tok, H, x.dtype, pad)
    lora.lora_rmsnorm(a, w, out, residual=res, residual_out=a)   # the stream over x
    assert torch.equal(out, want) and torch.equal(a, want_r)


PROMPT_ROPE = [
    dict(tok=1500, hq=18, hkv=2, D=128),                       # a step that holds two heads of four
    dict(tok=1500, hq=18, hkv=2, D=128, norm=True, w0=1.0),
    dict(tok=1501, hq=37, hkv=3, D=64, c8=True, norm=True),
    dict(tok=1499, hq=37, hkv=3, D=64, R=32, inter=True),
    dict(tok=1507, hq=20, hkv=4, D=80, R=40, inter=True, page=7),
    dict(tok=1507, hq=21, hkv=4, D=80, c8=True, idx=torch.int32),
    dict(tok=1502, hq=9, hkv=2, D=256, norm=True),
    dict(tok=1502, hq=9, hkv=2, D=256, c8=True, inter=True, norm=True),
    dict(tok=1503, hq=5, hkv=1, D=512),
    dict(tok=1503, hq=5, hkv=1, D=512, norm=True, c8=True),
    dict(tok=1504, hq=12, hkv=4, D=128, hnd=True, in_place=True),
    dict(tok=1504, hq=12, hkv=4, D=128, norm=True, in_place=True, inter=True),
    dict(tok=8200, hq=5, hkv=1, D=128),
    dict(tok=8200, hq=7, hkv=2, D=64, norm=True, c8=True),
    dict(tok=8200, hq=3, hkv=1, D=96, R=48, inter=True, norm=True),
]


@pytest.mark.parametrize("kw", PROMPT_ROPE)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_rope_prompts(kw, dtype):
    # several steps of heads a warp, two under way, the last ones partly filled
    kw = dict(kw)
    args = [kw.pop(n) for n in ("tok", "hq", "hkv", "D")]
    check_rope(100 + args[0], *args, dtype, **kw)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("sections,mixed", [([24, 20, 20], True), ([16, 24, 24], False), ([32, 32], False)])
def test_rope_prompts_of_several_axes(sections, mixed, norm):
    amap = lora.rope_axis_map(sections, interleaved=mixed)
    check_rope(101, 1600, 14, 4, 128, axes=len(sections), amap=amap, norm=norm)
    check_rope(102, 8195, 3, 1, 128, axes=len(sections), amap=amap, norm=norm, c8=True)


@pytest.mark.parametrize("tok", [5, 1500])
@pytest.mark.parametrize("D", [33, 64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_rope_scaled_cache_of_16_bits(dtype, D, tok):
    dt, hq, hkv = DT[dtype], 9, 3
    g = gen(103)
    off = [0, hq * D, (hq + hkv) * D, (hq + 2 * hkv) * D]
    qkv, R = rand(g, tok, off[3], dtype=dt), D // 2 * 2
    cs = rand(g, 50, R).clamp(-1, 1)
    pos = torch.randint(0, 50, (tok,), generator=g, device="cuda")
    kc, vc = (torch.full((tok, 1, hkv, D), SENT, device="cuda").to(dt) for _ in range(2))
    slots = torch.randperm(tok, generator=g, device="cuda")
    q = torch.empty(tok, hq * D, dtype=dt, device="cuda")
    lora.lora_rope_append(qkv, off, D, pos, cs, kc, vc, slots, q_out=q, k_scale=0.7, v_scale=1.9)
    rq, rk, rv, mq, mk = rope_ref(qkv, off, D, pos, cs, R, None, False, None, None, 1e-6, 0.0)
    within(q.reshape(rq.shape), rq, rq.abs() * HALF[dt] + mq * 2.0 ** -22 + TINY[dt], "q")
    # the scale and its reciprocal in fp32, and two products: 2^-21
    for c, ref, mag, sc in ((kc, rk, mk, 0.7), (vc, rv, rv.abs(), 1.9)):
        ref, mag = ref / sc, mag / sc
        within(c[slots, 0], ref, ref.abs() * HALF[dt] + mag * 2.0 ** -21 + TINY[dt], "cache")


