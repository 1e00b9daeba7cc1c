"""Measured cases of the decode-step operators: appending to an 8-bit paged key/value
cache with the rotary rotation, attention over that cache, and the product with 4-bit
weights and group scales.

The cache holds E4M3 codes [pages, kv_heads, page_size, head_dim] for keys and for
values, with one FP32 scale per page and head ([pages, kv_heads]); a sequence's pages
are the entries of its row of `page_table`. `lens[b]` counts sequence b's tokens with
the call's new ones, the last T of them. `own` selects the framework's kernels; the
plain forms are elementary torch operations in 32 bits.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
MIN_SCALE = 2.0 ** -60        # the smallest page scale that the append writes


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # one user's next token: every launch counts
        dict(name="append_b1_t1", op="append", B=1, T=1, ctx=1000, Hq=32, Hkv=8, D=128, rot=128, P=16,
             interleaved=False, dtype="bf16"),
        # a serving batch's next tokens at ragged lengths, rotation of half the head
        dict(name="append_b48_t1", op="append", B=48, T=1, ctx=700, Hq=32, Hkv=8, D=128, rot=64, P=32,
             interleaved=True, dtype="bf16"),
        # prompts entering the cache: odd length, pages that begin and end inside the chunk
        dict(name="append_b4_t1501", op="append", B=4, T=1501, ctx=1600, Hq=32, Hkv=8, D=128, rot=128, P=64,
             interleaved=False, dtype="f16"),
        # one user's next token over a short context: latency
        dict(name="attn_b1_t1_l1000", op="attn", B=1, T=1, ctx=1000, ragged=False, Hq=32, Hkv=8, D=128, P=16,
             dtype="bf16"),
        # a serving batch of ragged lengths
        dict(name="attn_b32_t1_l8191", op="attn", B=32, T=1, ctx=8191, ragged=True, Hq=32, Hkv=8, D=128, P=64,
             dtype="bf16"),
        # one user far into a long document
        dict(name="attn_b1_t1_l131000", op="attn", B=1, T=1, ctx=131000, ragged=False, Hq=64, Hkv=8, D=128, P=64,
             dtype="bf16"),
        # checking a draft of five tokens, as many key heads as query heads, small heads
        dict(name="attn_b16_t5_l2001", op="attn", B=16, T=5, ctx=2001, ragged=True, Hq=16, Hkv=16, D=64, P=32,
             dtype="f16"),
        # a prompt's later chunk over what the cache already holds
        dict(name="attn_b1_t1024_l8192", op="attn", B=1, T=1024, ctx=8192, ragged=False, Hq=32, Hkv=8, D=128,
             P=64, dtype="bf16"),
        # a square projection for one token
        dict(name="w4_m1_n4096_k4096", op="w4", M=1, N=4096, K=4096, group=128, zeros=False, scales="f32",
             pad=0, dtype="bf16"),
        # fused QKV for a small batch, asymmetric codes
        dict(name="w4_m8_n12288_k4096", op="w4", M=8, N=12288, K=4096, group=64, zeros=True, scales="same",
             pad=0, dtype="f16"),
        # the widest up-projection for one token, the finest groups
        dict(name="w4_m1_n28672_k8192", op="w4", M=1, N=28672, K=8192, group=32, zeros=False, scales="same",
             pad=0, dtype="bf16"),
        # a batch of 32 with padded rows, as in the strided workload
        dict(name="w4_m32_n14336_k5120", op="w4", M=32, N=14336, K=5120, group=128, zeros=True, scales="f32",
             pad=64, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        c = _draw(rng)
        if 3072 in c.values():
            continue
        w = work(c)
        top = [work(x) for x in listed() if x["op"] == c["op"]]
        if w["bytes"] <= max(x["bytes"] for x in top) and w["flops"] <= max(x["flops"] for x in top):
            return c


def _draw(rng):
    op = rng.choice(["append", "attn", "w4"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "w4":
        group = rng.choice([32, 64, 128])
        return dict(op=op, M=rng.choice([1, 1, 2, 3, 4, 7, 8, 12, 16, 24, 32]), N=_log_int(rng, 256, 28672),
                    K=group * max(1, _log_int(rng, 512, 8192) // group), group=group, zeros=rng.random() < 0.5,
                    scales=rng.choice(["f32", "same"]), pad=rng.choice([0, 0, 64]), dtype=dtype)
    D = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8, 16])
    c = dict(op=op, Hkv=hkv, Hq=hkv * rng.choice([1, 2, 4, 7, 8]), D=D, P=rng.choice([16, 32, 64, 128]), dtype=dtype)
    if op == "append":
        T = rng.choice([1, 1, 1, 2, 5, _log_int(rng, 8, 1500)])
        return dict(c, B=_log_int(rng, 1, 48) if T < 8 else rng.choice([1, 2, 4]), T=T,
                    ctx=T + _log_int(rng, 1, 1000), rot=rng.choice([D, D // 2, 48]), interleaved=rng.random() < 0.5)
    T = rng.choice([1, 1, 1, 2, 5, _log_int(rng, 8, 1024)])
    return dict(c, B=_log_int(rng, 1, 32) if T < 8 else 1, T=T, ctx=max(T, _log_int(rng, 100, 131000)),
                ragged=rng.random() < 0.5)


def _lens(case):
    """Tokens per sequence, this call's included: all at ctx, or spread over [ctx/4, ctx]."""
    B, ctx, T = case["B"], case["ctx"], case["T"]
    if case["op"] == "attn" and not case["ragged"]:
        return [ctx] * B
    return [max(T, ctx - (b * (ctx - ctx // 4)) // B) for b in range(B)]


def work(case):
    c = case
    if c["op"] == "w4":
        groups = c["N"] * (c["K"] // c["group"])
        b = c["N"] * c["K"] // 2 + groups * (4 if c["scales"] == "f32" else 2) + (groups if c["zeros"] else 0)
        return {"bytes": b + 2 * c["M"] * (c["K"] + c["N"]), "flops": 2 * c["M"] * c["N"] * c["K"]}
    lens, B, T, D, P = _lens(c), c["B"], c["T"], c["D"], c["P"]
    if c["op"] == "append":
        tok = B * T
        pages = sum(-(-n // P) - (n - T) // P for n in lens)
        return {"bytes": tok * D * (4 * c["Hq"] + 6 * c["Hkv"]) + pages * c["Hkv"] * 16 + tok * c["rot"] * 4
                + pages * 4 + 4 * B,
                "flops": tok * D * (3 * c["Hq"] + 6 * c["Hkv"])}
    pages = sum(-(-n // P) for n in lens)
    pairs = sum(T * (n - T) + T * (T + 1) // 2 for n in lens)
    return {"bytes": 2 * sum(lens) * c["Hkv"] * D + pages * (8 * c["Hkv"] + 4) + 4 * B * T * c["Hq"] * D + 4 * B,
            "flops": 4 * pairs * c["Hq"] * D}


# ------------------------------------------------------------------ inputs --
def _page_scale(amax):
    """The smallest power of two s with amax <= 448 s, not below 2^-60."""
    m, e = torch.frexp(amax)                                  # amax = m 2^e, m in [0.5, 1)
    s = torch.ldexp(torch.ones_like(amax), e - 9 + (m > 0.875).to(e.dtype))
    return torch.where(amax > 0, s, torch.zeros_like(s)).clamp_min(MIN_SCALE)


def _cache(pages, Hkv, P, D, g, dev, outliers):
    x = torch.randn(pages, Hkv, P, D, generator=g, device=dev)
    if outliers:                                              # keys carry a few large channels
        x = x * (1.0 + 4.0 * (torch.rand(1, Hkv, 1, D, generator=g, device=dev) < 0.04).float())
    scale = _page_scale(x.abs().amax((2, 3)))
    return (x / scale[:, :, None, None]).to(E4M3), scale


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 11)
    dt = DTYPES[c["dtype"]]
    s = dict(case=c)
    if c["op"] == "w4":
        M, N, K, grp = c["M"], c["N"], c["K"], c["group"]
        s["A"] = torch.randn(M, K + c["pad"], generator=g, device=dev).to(dt)[:, :K]
        s["W"] = torch.randint(0, 256, (N, K // 2), generator=g, device=dev, dtype=torch.uint8)
        s["scale"] = ((0.5 + torch.rand(N, K // grp, generator=g, device=dev)) * 0.004).to(
            torch.float32 if c["scales"] == "f32" else dt)
        s["zeros"] = (torch.randint(4, 12, (N, K // grp), generator=g, device=dev, dtype=torch.uint8)
                      if c["zeros"] else None)
        s["C"] = torch.zeros(M, N + c["pad"], device=dev, dtype=dt)[:, :N]
        return s
    B, T, D, P, Hkv, Hq = c["B"], c["T"], c["D"], c["P"], c["Hkv"], c["Hq"]
    lens = _lens(c)
    per_seq = -(-max(lens) // P)
    used = [-(-n // P) for n in lens]
    pages = sum(used)
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(B, per_seq, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    s["table"] = table
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["k_codes"], s["k_scale"] = _cache(pages, Hkv, P, D, g, dev, True)
    s["v_codes"], s["v_scale"] = _cache(pages, Hkv, P, D, g, dev, False)
    s["q"] = torch.randn(B * T, Hq, D, generator=g, device=dev).to(dt)
    if c["op"] == "append":
        qkv = torch.randn(B * T, (Hq + 2 * Hkv) * D, generator=g, device=dev).to(dt)   # the fused projection's rows
        s["q"] = qkv[:, :Hq * D].view(B * T, Hq, D)
        s["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].view(B * T, Hkv, D)
        s["v"] = qkv[:, (Hq + Hkv) * D:].view(B * T, Hkv, D)
        inv = 10000.0 ** (-torch.arange(c["rot"] // 2, device=dev, dtype=torch.float64) * 2 / c["rot"])
        ang = torch.arange(c["ctx"] + 1, device=dev, dtype=torch.float64)[:, None] * inv
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
    s["out"] = torch.zeros(B * T, Hq, D, device=dev, dtype=dt)
    if own:
        import fp8_weight_only_gemm_gb300 as w8
        s["cache"] = w8.KVCache(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
        if c["op"] == "attn":
            s["ws"] = torch.empty(w8.kv_attention_workspace_bytes(s["cache"], B, T, Hq), dtype=torch.uint8, device=dev)
    return s


# --------------------------------------------------------------------- run --
def run(s):
    op = s["case"]["op"]
    if op == "append":
        return _append_own(s) if own else _append_plain(s)
    if op == "attn":
        return _attn_own(s) if own else _attn_plain(s)
    return _w4_own(s) if own else _w4_plain(s)


def _append_own(s):
    import fp8_weight_only_gemm_gb300 as w8
    w8.kv_append(s["cache"], s["k"], s["v"], s["table"], s["lens"], s["cos"], s["sin"], q=s["q"], q_out=s["out"],
                 interleaved=s["case"]["interleaved"])
    return s["out"], s["k_codes"], s["k_scale"], s["v_codes"], s["v_scale"]


def _attn_own(s):
    import fp8_weight_only_gemm_gb300 as w8
    return w8.kv_attention(s["cache"], s["q"], s["table"], s["lens"], s["out"], workspace=s["ws"])


def _w4_own(s):
    import fp8_weight_only_gemm_gb300 as w8
    return w8.gemm_w4(s["A"], s["W"], s["scale"], s["C"], zeros=s["zeros"])


def _rotate(x, cos, sin, rot, interleaved):
    """x [N, H, D] in 32 bits; cos, sin [N, 1, rot/2]."""
    r = x[..., :rot]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((r, x[..., rot:]), -1)


def _append_plain(s):
    c = s["case"]
    B, T, P, D, H = c["B"], c["T"], c["P"], c["D"], c["Hkv"]
    dev = s["q"].device
    lens = s["lens"].long()
    first = (lens - T)[:, None]                                # position of each sequence's first new token
    pos = (first + torch.arange(T, device=dev)).reshape(-1)
    cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
    s["out"].copy_(_rotate(s["q"].float(), cos, sin, c["rot"], c["interleaved"]))
    new = {"k": _rotate(s["k"].float(), cos, sin, c["rot"], c["interleaved"]), "v": s["v"].float()}
    # every page that the new tokens touch (the last one again where a sequence touches fewer)
    n = (T + P - 2) // P + 1
    pg = torch.minimum(first // P + torch.arange(n, device=dev), ((lens - 1) // P)[:, None])   # [B, n]
    phys = s["table"].long().gather(1, pg).reshape(-1)
    slot_pos = pg[:, :, None] * P + torch.arange(P, device=dev)                                # [B, n, P]
    t = slot_pos - first[:, :, None]
    is_new = ((t >= 0) & (t < T)).reshape(B * n, 1, P, 1)
    is_old = (t < 0).reshape(B * n, 1, P, 1)
    row = (torch.arange(B, device=dev)[:, None, None] * T + t.clamp(0, T - 1)).reshape(B * n, P)
    for name in ("k", "v"):
        codes, scales = s[name + "_codes"], s[name + "_scale"]
        x = new[name][row].transpose(1, 2)                     # [B n, H, P, D]
        old_codes, old_scale = codes.view(torch.uint8)[phys].view(E4M3).float(), scales[phys]
        scale = _page_scale(torch.where(is_new, x.abs(), 0.0).amax((2, 3)))
        scale = torch.where(is_old.any(2)[:, :, 0], torch.maximum(scale, old_scale), scale)
        e = scale[:, :, None, None]
        y = torch.where(is_new, x / e, torch.where(is_old, old_codes * (old_scale[:, :, None, None] / e), old_codes))
        codes.view(torch.uint8)[phys] = y.to(E4M3).view(torch.uint8)
        scales[phys] = scale
    return s["out"], s["k_codes"], s["k_scale"], s["v_codes"], s["v_scale"]


def _attn_plain(s):
    c = s["case"]
    B, T, P, D, H = c["B"], c["T"], c["P"], c["D"], c["Hkv"]
    dev = s["q"].device
    table = s["table"].long()
    L = table.shape[1] * P

    def pages(codes, scale):                                   # [B, H, L, D]
        x = codes.view(torch.uint8)[table].view(E4M3).float() * scale[table][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(B, H, L, D)

    q = s["q"].float().view(B, T, H, c["Hq"] // H, D).permute(0, 2, 3, 1, 4).reshape(B, H, -1, D)
    x = torch.matmul(q, pages(s["k_codes"], s["k_scale"]).transpose(2, 3)) / math.sqrt(D)
    last = s["lens"].long()[:, None] - T + torch.arange(T, device=dev)                          # [B, T]
    seen = torch.arange(L, device=dev) <= last[:, :, None]                                      # [B, T, L]
    x = x.view(B, H, -1, T, L).masked_fill(~seen[:, None, None], -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    p = (p / p.sum(-1, keepdim=True)).view(B, H, -1, L)
    o = torch.matmul(p, pages(s["v_codes"], s["v_scale"])).view(B, H, -1, T, D)
    s["out"].copy_(o.permute(0, 3, 1, 2, 4).reshape(B * T, c["Hq"], D))
    return s["out"]


def _w4_plain(s):
    N, K = s["W"].shape[0], s["W"].shape[1] * 2
    grp = s["case"]["group"]
    codes = torch.stack((s["W"] & 15, s["W"] >> 4), -1).view(N, K // grp, grp).float()
    zero = 8.0 if s["zeros"] is None else s["zeros"].float()[..., None]
    w = ((codes - zero) * s["scale"].float()[..., None]).view(N, K)
    s["C"].copy_(torch.matmul(s["A"].float(), w.t()))
    return s["C"]


# ------------------------------------------------------------------- exact --
def exact(case, seed):
    """The definition in 64 bits, one sequence (or block of rows) at a time."""
    s = prepare(case, seed)
    if case["op"] == "append":
        return _append_exact(case, s)
    if case["op"] == "attn":
        return _attn_exact(case, s)
    A = s["A"].double()
    blocks = []
    for n0 in range(0, case["N"], 1024):
        W = s["W"][n0:n0 + 1024].int()
        w = torch.empty(W.shape[0], case["K"], dtype=torch.float64, device=A.device)
        w[:, 0::2], w[:, 1::2] = W % 16, W // 16
        w -= 8.0 if s["zeros"] is None else s["zeros"][n0:n0 + 1024].double().repeat_interleave(case["group"], 1)
        w *= s["scale"][n0:n0 + 1024].double().repeat_interleave(case["group"], 1)
        blocks.append(torch.einsum("mk,nk->mn", A, w))
    return torch.cat(blocks, 1)


def _attn_exact(c, s):
    T, P, D, H, G = c["T"], c["P"], c["D"], c["Hkv"], c["Hq"] // c["Hkv"]
    out = torch.zeros(c["B"] * T, c["Hq"], D, dtype=torch.float64, device=s["q"].device)
    for b, n in enumerate(_lens(c)):
        ids = s["table"][b, :-(-n // P)].long()
        pos = torch.arange(n, device=ids.device)
        mask = pos[None, :] > (n - T + torch.arange(T, device=ids.device))[:, None]
        for h in range(H):
            k = s["k_codes"].view(torch.uint8)[ids, h].view(E4M3).double() * s["k_scale"][ids, h].double()[:, None, None]
            v = s["v_codes"].view(torch.uint8)[ids, h].view(E4M3).double() * s["v_scale"][ids, h].double()[:, None, None]
            k, v = k.reshape(-1, D)[:n], v.reshape(-1, D)[:n]
            for i in range(G):
                x = s["q"][b * T:(b + 1) * T, h * G + i].double() @ k.t() * D ** -0.5
                x[mask] = -math.inf
                out[b * T:(b + 1) * T, h * G + i] = torch.softmax(x, -1) @ v
    return out


def _e4m3_round(x):
    """The nearest E4M3 value (ties to the even mantissa) of 64-bit numbers within +-448."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp_min(-6) - 3)
    return torch.round(x / step) * step


def _append_exact(c, s):
    T, P, D, rot = c["T"], c["P"], c["D"], c["rot"]
    dev = s["q"].device
    j = torch.arange(rot // 2, device=dev)
    lo, hi = (2 * j, 2 * j + 1) if c["interleaved"] else (j, j + rot // 2)
    pos = torch.cat([torch.arange(n - T, n, device=dev) for n in _lens(c)])
    cos, sin = s["cos"].double()[pos][:, None], s["sin"].double()[pos][:, None]

    def turn(x):
        y = x.double().clone()
        y[..., lo] = x[..., lo].double() * cos - x[..., hi].double() * sin
        y[..., hi] = x[..., lo].double() * sin + x[..., hi].double() * cos
        return y

    done = []
    for new, codes, scales in ((turn(s["k"]), s["k_codes"], s["k_scale"]), (s["v"].double(), s["v_codes"], s["v_scale"])):
        codes, scales = codes.double(), scales.double()
        for b, n in enumerate(_lens(c)):
            for page in range((n - T) // P, (n - 1) // P + 1):
                id = int(s["table"][b, page])
                a, z = max(page * P, n - T), min((page + 1) * P, n)
                x = new[b * T + a - (n - T):b * T + z - (n - T)].transpose(0, 1)      # [H, new, D]
                amax = x.abs().amax((1, 2))
                scale = torch.exp2(torch.ceil(torch.log2(amax / 448.0))).clamp_min(MIN_SCALE)
                if a > page * P:
                    scale = torch.maximum(scale, scales[id])
                    held = codes[id, :, :a - page * P] * (scales[id] / scale)[:, None, None]
                    codes[id, :, :a - page * P] = _e4m3_round(held)
                codes[id, :, a - page * P:z - page * P] = _e4m3_round(x / scale[:, None, None])
                scales[id] = scale
        done += [codes, scales]
    return (turn(s["q"]), *done)
