"""The operators around the adapted projection of a decoder layer, as cases to
time and compare: the RMS norm that makes the projection's input, the base
projection with 4-bit weights that the LoRA expand adds to, and the rotation of
its q/k/v slices with the append to a paged cache.

``run`` computes a case in plain torch (fp32, rounded once at the end) where
``own`` is false, and through ``scatter_gemm_b200.lora`` where it is true.
"""
import math

import torch

own = False

BF16, FP16, E4M3 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
DTYPES = {"bf16": BF16, "fp16": FP16, "e4m3": E4M3}
E4M3_MAX = 448.0
EPS = 1e-6


def _norm_case(name, tok, hidden, dtype, out="rounded", residual=True):
    return {"name": name, "op": "rmsnorm", "tok": tok, "hidden": hidden, "dtype": dtype,
            "out": out, "residual": residual}


def _w4_case(name, tok, K, N, dtype, group, zeros=False, x8=False):
    return {"name": name, "op": "w4_project", "tok": tok, "K": K, "N": N, "dtype": dtype,
            "group": group, "zeros": zeros, "x8": x8}


def _rope_case(name, tok, heads, kv_heads, head_dim, dtype, rotary=None, axes=1,
               interleaved=False, head_norm=False, cache="same", page=16):
    return {"name": name, "op": "rope_append", "tok": tok, "heads": heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "rotary": rotary or head_dim, "dtype": dtype, "axes": axes,
            "interleaved": interleaved, "head_norm": head_norm, "cache": cache, "page": page}


def listed():
    return [
        # one decode step of a single request: the launch and one row's latency
        _norm_case("norm_one_token", 1, 4096, "bf16"),
        # a ragged prompt batch of an odd hidden size, whose rows have no 16-byte alignment
        _norm_case("norm_odd_rows", 777, 3583, "fp16"),
        # a long prompt: the adapters' x and the quantised projection's 8-bit x in one pass
        _norm_case("norm_prompt_8bit", 8192, 5120, "bf16", out="both"),
        # q/k/v projection of one token: the weights are read once for a single row
        _w4_case("w4_one_token", 1, 4096, 6144, "bf16", 128),
        # gate/up projection of a small decode batch, 8-bit x from the norm
        _w4_case("w4_decode_8bit", 8, 4096, 24576, "bf16", 128, x8=True),
        # odd sizes in every direction, zero points, the smallest groups
        _w4_case("w4_odd_sizes", 13, 3583, 6159, "fp16", 32, zeros=True),
        # gate/up projection of a large decode batch
        _w4_case("w4_batch", 128, 4096, 24576, "bf16", 64, zeros=True),
        # q/k/v projection of a prompt chunk, 16-bit x
        _w4_case("w4_prompt", 2048, 5120, 7168, "bf16", 128),
        # one decode step of a single request
        _rope_case("rope_one_token", 1, 32, 8, 128, "bf16"),
        # a decode batch with per-head norms of q and k and an 8-bit cache
        _rope_case("rope_decode_8bit", 256, 32, 8, 128, "bf16", head_norm=True, cache="e4m3"),
        # part of an odd-sized head rotated, neighbouring elements paired
        _rope_case("rope_partial", 1031, 20, 4, 80, "fp16", rotary=40, interleaved=True, page=7),
        # a long prompt with images: time, height and width positions
        _rope_case("rope_prompt_axes", 8192, 40, 8, 128, "bf16", axes=3, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rmsnorm", "w4_project", "rope_append"])
    dtype = rng.choice(["bf16", "fp16"])
    if kind == "rmsnorm":
        hidden = _log(rng, 64, 16384)
        if rng.random() < 0.7:  # most models' rows are 16-byte aligned, some are not
            hidden = max(8, hidden // 8 * 8)
        tok = max(1, min(_log(rng, 1, 16384), 8192 * 5120 // hidden))
        c = _norm_case("", tok, hidden, dtype, out=rng.choice(["rounded", "8bit", "both"]),
                       residual=rng.random() < 0.75)
    elif kind == "w4_project":
        K = _log(rng, 128, 16384)
        step = rng.choice([128, 128, 32, 1])
        K = max(step, K // step * step)
        N = _log(rng, 16, 28672)
        tok = _log(rng, 1, 4096)
        cap = 2048 * 5120 * 7168
        while tok * K * N > cap or K * N > 4096 * 24576:
            if tok > 1 and tok * K * N > cap:
                tok = max(1, tok // 2)
            else:
                N = max(16, N // 2)
        c = _w4_case("", tok, K, N, dtype, rng.choice([32, 64, 128]),
                     zeros=rng.random() < 0.5, x8=rng.random() < 0.4)
    else:
        kv = rng.choice([1, 2, 4, 8, 10])
        heads = kv * rng.choice([1, 4, 5, 7, 8])
        dim = rng.choice([64, 80, 96, 128, 128, 128, 192, 256])
        rot = rng.choice([dim, dim, dim // 2])
        tok = _log(rng, 1, 8192)
        while tok * (heads + 2 * kv) * dim > 8192 * 56 * 128:
            tok //= 2
        c = _rope_case("", tok, heads, kv, dim, dtype, rotary=rot, axes=rng.choice([1, 1, 2, 3]),
                       interleaved=rng.random() < 0.3, head_norm=rng.random() < 0.4,
                       cache=rng.choice(["same", "same", "e4m3"]),
                       page=rng.choice([1, 7, 16, 32, 64]))
    del c["name"]
    return c


def _axis_map(rotary, axes):
    """The position axis of each frequency: `axes` sections of neighbouring frequencies."""
    half = rotary // 2
    edges = [half * a // axes for a in range(axes + 1)]
    return [a for a in range(axes) for _ in range(edges[a], edges[a + 1])]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda").mul_(std)

    def integers(lo, hi, shape, dtype=torch.int64):
        return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=dtype)

    s = {"case": case}
    tok = case["tok"]
    if case["op"] == "rmsnorm":
        H = case["hidden"]
        s["x"] = normal(tok, H).to(dt)
        # a residual stream has a few columns far larger than the others
        col = torch.where(torch.rand(H, generator=g, device="cuda") < 0.01, 20.0, 1.0)
        s["residual"] = (normal(tok, H) * col).to(dt) if case["residual"] else None
        s["weight"] = (1.0 + normal(H, std=0.2)).to(dt)
        s["residual_out"] = torch.empty(tok, H, dtype=dt, device="cuda") if case["residual"] else None
        s["out"] = torch.empty(tok, H, dtype=dt, device="cuda") if case["out"] != "8bit" else None
        if case["out"] != "rounded":
            s["out_q"] = torch.empty(tok, H, dtype=E4M3, device="cuda")
            s["out_scale"] = torch.empty(tok, dtype=torch.float32, device="cuda")
    elif case["op"] == "w4_project":
        K, N, group = case["K"], case["N"], case["group"]
        G = -(-K // group)
        x = normal(tok, K)
        if case["x8"]:  # one scale for each row, as the norm writes them
            s["x_scale"] = x.abs().amax(dim=1) / E4M3_MAX
            s["x"] = (x / s["x_scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3)
        else:
            s["x"], s["x_scale"] = x.to(dt), None
        # packed weights: two 4-bit values a byte, rows padded to 32 values
        s["w"] = integers(0, 256, (N, -(-K // 32) * 16), torch.uint8)
        s["w_scales"] = (0.004 * torch.exp(normal(G, N, std=0.3))).to(dt)
        s["w_zeros"] = integers(5, 11, (G, N), torch.uint8) if case["zeros"] else None
        s["out"] = torch.empty(tok, N, dtype=dt, device="cuda")
    else:
        D, R, hq, hk = case["head_dim"], case["rotary"], case["heads"], case["kv_heads"]
        page, axes = case["page"], case["axes"]
        s["qkv"] = normal(tok, (hq + 2 * hk) * D).to(dt)
        s["offsets"] = [0, hq * D, (hq + hk) * D, (hq + 2 * hk) * D]
        max_pos = 16384
        freq = 1e6 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
        angle = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None] * freq
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], dim=1).float()
        s["positions"] = integers(0, max_pos, (tok,) if axes == 1 else (axes, tok))
        s["axis_map"] = _axis_map(R, axes) if axes > 1 else None
        # a cache in use: the pages of this step's tokens lie anywhere in it
        pages = -(-tok // page) * 2 + 1
        cdt = dt if case["cache"] == "same" else E4M3
        s["k_cache"] = normal(pages, page, hk, D).to(cdt)
        s["v_cache"] = normal(pages, page, hk, D).to(cdt)
        slots = torch.randperm(pages * page, generator=g, device="cuda")[:tok]
        if tok > 4:  # padding of the batch
            slots[-1] = -1
        s["slots"] = slots
        s["scales"] = (1.0, 1.0) if case["cache"] == "same" else (0.03, 0.02)
        s["q_out"] = torch.empty(tok, hq * D, dtype=dt, device="cuda")
        for n in ("q_weight", "k_weight"):
            s[n] = (1.0 + normal(D, std=0.2)).to(dt) if case["head_norm"] else None
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(op, s)
    return {"rmsnorm": _plain_norm, "w4_project": _plain_w4, "rope_append": _plain_rope}[op](s)


def _run_own(op, s):
    from scatter_gemm_b200 import lora
    c = s["case"]
    if op == "rmsnorm":
        lora.lora_rmsnorm(s["x"], s["weight"], s["out"], residual=s["residual"],
                          residual_out=s["residual_out"], eps=EPS, out_q=s.get("out_q"),
                          out_scale=s.get("out_scale"))
        return [s[n] for n in ("residual_out", "out", "out_q", "out_scale") if s.get(n) is not None]
    if op == "w4_project":
        return lora.lora_w4_project(s["x"], s["w"], s["w_scales"], s["out"], group_size=c["group"],
                                    w_zeros=s["w_zeros"], x_scale=s["x_scale"])
    lora.lora_rope_append(s["qkv"], s["offsets"], c["head_dim"], s["positions"], s["cos_sin"],
                          s["k_cache"], s["v_cache"], s["slots"], q_out=s["q_out"],
                          axis_map=s["axis_map"], interleaved=c["interleaved"],
                          q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                          k_scale=s["scales"][0], v_scale=s["scales"][1])
    return [s["q_out"], s["k_cache"], s["v_cache"]]


def _plain_norm(s):
    c = s["case"]
    h = s["x"]
    outs = []
    if s["residual"] is not None:
        h = (h.float() + s["residual"].float()).to(h.dtype)
        outs.append(h)
    h = h.float()
    v = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS) * s["weight"].float()
    if c["out"] != "8bit":
        outs.append(v.to(s["x"].dtype))
    if c["out"] != "rounded":
        scale = v.abs().amax(dim=1) / E4M3_MAX
        outs.append((v / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3))
        outs.append(scale)
    return outs


#: Within four packed bytes (eight values), the place of each value: its byte and its shift.
_BYTE = (0, 2, 0, 2, 1, 3, 1, 3)
_SHIFT = (0, 0, 4, 4, 0, 0, 4, 4)


def _unpack(w, K):
    words = w.view(w.shape[0], -1, 4)
    shift = torch.tensor(_SHIFT, dtype=torch.uint8, device=w.device)
    q = (words[:, :, list(_BYTE)] >> shift) & 15
    return q.reshape(w.shape[0], -1)[:, :K]


def _plain_w4(s):
    c = s["case"]
    K, group = c["K"], c["group"]
    q = _unpack(s["w"], K).float()
    of = torch.arange(K, device=q.device) // group
    zero = 8.0 if s["w_zeros"] is None else s["w_zeros"].float()[of].T
    W = (q - zero) * s["w_scales"].float()[of].T
    out = s["x"].float() @ W.T
    if s["x_scale"] is not None:
        out = out * s["x_scale"][:, None]
    return out.to(s["out"].dtype)


def _plain_rotate(x, cos, sin, R, interleaved):
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., :R // 2], x[..., R // 2:R])
    a2, b2 = a * cos - b * sin, b * cos + a * sin
    if interleaved:
        rot = torch.stack([a2, b2], dim=-1).flatten(-2)
    else:
        rot = torch.cat([a2, b2], dim=-1)
    return torch.cat([rot, x[..., R:]], dim=-1)


def _plain_append(cache, val, slots, scale):
    live = slots >= 0
    val = val[live] / scale
    if cache.dtype == E4M3:
        val = val.clamp(-E4M3_MAX, E4M3_MAX)
    bits = torch.uint8 if cache.dtype == E4M3 else torch.int16
    flat = cache.view(bits).view(-1, *cache.shape[2:])
    flat[slots[live]] = val.to(cache.dtype).view(bits)


def _plain_rope(s):
    c = s["case"]
    D, R, hq, hk, tok = c["head_dim"], c["rotary"], c["heads"], c["kv_heads"], c["tok"]
    half = R // 2
    qkv = s["qkv"].float()
    q, k, v = (t.reshape(tok, -1, D) for t in qkv.split([hq * D, hk * D, hk * D], dim=1))
    if s["q_weight"] is not None:
        q = q * torch.rsqrt((q * q).mean(-1, keepdim=True) + EPS) * s["q_weight"].float()
        k = k * torch.rsqrt((k * k).mean(-1, keepdim=True) + EPS) * s["k_weight"].float()
    freq = torch.arange(half, device=q.device)
    if c["axes"] == 1:
        row = s["positions"][:, None]
    else:
        row = s["positions"][torch.tensor(s["axis_map"], device=q.device)].T
    cos, sin = (s["cos_sin"][row, freq + o][:, None, :] for o in (0, half))
    q = _plain_rotate(q, cos, sin, R, c["interleaved"])
    k = _plain_rotate(k, cos, sin, R, c["interleaved"])
    s["q_out"].copy_(q.reshape(tok, -1))
    _plain_append(s["k_cache"], k, s["slots"], s["scales"][0])
    _plain_append(s["v_cache"], v, s["slots"], s["scales"][1])
    return [s["q_out"], s["k_cache"], s["v_cache"]]


def work(case):
    c = case
    tok = c["tok"]
    if c["op"] == "rmsnorm":
        n = tok * c["hidden"]
        b = 2 * n + (4 * n if c["residual"] else 0) + 2 * c["hidden"]
        b += 2 * n if c["out"] != "8bit" else 0
        b += n + 4 * tok if c["out"] != "rounded" else 0
        return {"bytes": b, "flops": 6 * n}
    if c["op"] == "w4_project":
        K, N = c["K"], c["N"]
        G = -(-K // c["group"])
        b = N * -(-K // 2) + G * N * (3 if c["zeros"] else 2) + 2 * tok * N
        b += tok * (K + 4) if c["x8"] else 2 * tok * K
        return {"bytes": b, "flops": 2 * tok * N * K}
    D, hq, hk = c["head_dim"], c["heads"], c["kv_heads"]
    e = 2 if c["cache"] == "same" else 1
    b = tok * (hq + 2 * hk) * D * 2 + tok * hq * D * 2 + tok * 2 * hk * D * e
    b += tok * (4 * c["rotary"] + 8 * c["axes"] + 8)
    return {"bytes": b, "flops": tok * (hq + hk) * (3 * c["rotary"] + (4 * D if c["head_norm"] else 0))}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rmsnorm":
        return _exact_norm(case, s)
    if case["op"] == "w4_project":
        return _exact_w4(case, s)
    return _exact_rope(case, s)


def _exact_norm(case, s):
    h = s["x"].double()
    res = []
    if case["residual"]:
        res = [h + s["residual"].double()]
        h = res[0].to(s["x"].dtype).double()  # what the stream holds is what is normalised
    rms = (h.pow(2).sum(1) / case["hidden"] + EPS).sqrt()
    v = h / rms[:, None] * s["weight"].double()
    top = v.abs().max(1).values / E4M3_MAX
    if case["out"] != "8bit":
        res.append(v)
    if case["out"] != "rounded":
        res += [v / top[:, None], top]
    return res


def _exact_w4(case, s):
    K, group = case["K"], case["group"]
    words = s["w"].view(torch.int32).to(torch.int64)
    q = torch.empty(case["N"], words.shape[1] * 8, dtype=torch.float64, device=words.device)
    for i in range(8):  # value i of a word: even ones in its low half, odd ones in its high half
        q[:, i::8] = ((words >> (16 * (i % 2) + 4 * (i // 2))) & 15).double()
    out = torch.zeros(case["tok"], case["N"], dtype=torch.float64, device=words.device)
    x = s["x"].double()
    for i in range(-(-K // group)):
        lo, hi = i * group, min(K, (i + 1) * group)
        zero = 8.0 if s["w_zeros"] is None else s["w_zeros"][i].double()[:, None]
        out += (x[:, lo:hi] @ (q[:, lo:hi] - zero).T) * s["w_scales"][i].double()
    if s["x_scale"] is not None:
        out *= s["x_scale"].double()[:, None]
    return out


def _exact_rope(case, s):
    D, R, hq, hk = case["head_dim"], case["rotary"], case["heads"], case["kv_heads"]
    tok, off = case["tok"], s["offsets"]
    qkv = s["qkv"].double()
    parts = [qkv[:, off[i]:off[i + 1]].reshape(tok, n, D) for i, n in enumerate((hq, hk, hk))]
    turned = []
    for x, w in zip(parts, (s["q_weight"], s["k_weight"])):
        if w is not None:
            x = x / (x.pow(2).sum(2, keepdim=True) / D + EPS).sqrt() * w.double()
        y = x.clone()
        for i in range(R // 2):
            pos = s["positions"] if case["axes"] == 1 else s["positions"][s["axis_map"][i]]
            turn = torch.complex(s["cos_sin"][pos, i].double(), s["cos_sin"][pos, R // 2 + i].double())
            a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + R // 2)
            z = torch.complex(x[:, :, a], x[:, :, b]) * turn[:, None]
            y[:, :, a], y[:, :, b] = z.real, z.imag
        turned.append(y)
    live = torch.nonzero(s["slots"] >= 0).flatten()
    caches = []
    for cache, val, scale in zip((s["k_cache"], s["v_cache"]), (turned[1], parts[2]), s["scales"]):
        full = cache.double().reshape(-1, hk, D)
        val = val / scale
        if cache.dtype == E4M3:
            val = val.clamp(-E4M3_MAX, E4M3_MAX)
        full[s["slots"][live]] = val[live]
        caches.append(full.reshape(cache.shape))
    return [turned[0].reshape(tok, hq * D)] + caches
