"""Edges of lora_rmsnorm, lora_w4_project and lora_rope_append, against their
formulas in 64 bits: the values of 8-bit outputs, the range of the element
types, infinities, and the kernel variants that serve prompts.  Tolerances as
in test_layer_ops_gpu.py."""
import pytest
import torch

from scatter_gemm_b200 import lora
from tests.test_layer_ops_gpu import (DT, E4M3, HALF, SENT, TINY, check_norm, check_rope, check_w4,
                                      gen, new, padding_intact, rand, rope_ref, strided,
                                      w4_inputs, within)

pytestmark = pytest.mark.gpu


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


