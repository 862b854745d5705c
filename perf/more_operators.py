"""FP8 products with a scale for each block of 128, their quantisation, the
norms and rotations of query and key heads, and the quantised paged cache:
cases, plain forms and measurement hooks.

``run`` computes one pass of an operator, in plain torch operations (32 bits
inside, one rounding at the end) or, where ``own`` is set, through the
package's public calls.  ``exact`` computes the same outputs in 64 bits.

Operators
  quantize  bf16 [T,H] to E4M3 codes and fp32 scales of blocks of 128 of a
            row (block_rows 1: activations) or 128 by 128 (weights)
  product   out = A B^T in bf16, of codes and block scales
  experts   out[s] = x[rows[s]] W_e^T for the slots s of every expert e, of
            codes and block scales
  heads     RMSNorm of every query and key head and the rotation by position
            in one pass; keys and values may go straight into the cache
  cache     keys and values written to a paged cache in 8 or 4 bits, and the
            sequences' contexts read back in bf16
"""
import math

import torch

own = False

DEV = "cuda"
# The NVFP4 caches' tensor scale: an amax of 16 maps to the largest code
# times the largest block scale.
G = 168.0
EPS = 1e-6


def listed():
    return [
        # Activations of one decoding step.
        dict(name="quantize_decode", op="quantize", T=16, H=4096, rows=1),
        # A projection's weights, once at load time.
        dict(name="quantize_weights", op="quantize", T=10240, H=5120, rows=128),
        # A projection of one token: reading the weights.
        dict(name="product_one_token", op="product", T=1, N=8192, H=8192),
        # Sizes off every tile; the last block of a row has 16 elements.
        dict(name="product_ragged", op="product", T=1237, N=4100, H=2064),
        # A projection of the prefill workload.
        dict(name="product_prefill", op="product", T=8192, N=8192, H=8192),
        # Second expert product of a decoding batch: a handful of rows for
        # every expert.
        dict(name="experts_decode", op="experts", T=64, K=8, E=64, H=2048, N=7168, gather=False,
             skew=0.5),
        # First expert product of a prefill of 4096 tokens (the MoE combine
        # workload's hidden size and experts per token).
        dict(name="experts_prefill", op="experts", T=4096, K=8, E=64, H=7168, N=4096, gather=True,
             skew=0.5),
        # One decoding step of 16 sequences: heads of the decode workload's
        # hidden size, keys and values into an FP8 cache.
        dict(name="heads_decode", op="heads", T=16, HQ=32, HKV=8, D=128, R=128, axes=1,
             interleaved=False, format="fp8"),
        # A prefill of 8192 tokens: heads of the headline's hidden size.
        dict(name="heads_prefill", op="heads", T=8192, HQ=40, HKV=8, D=128, R=128, axes=1,
             interleaved=False, format="fp8"),
        # Image or video tokens: positions in time, height and width, a part
        # of every head rotated, in pairs of neighbours; keys stay in bf16.
        dict(name="heads_axes", op="heads", T=4099, HQ=16, HKV=16, D=80, R=64, axes=3,
             interleaved=True, format=""),
        # A chunk of a prompt appended to a 4-bit cache and the contexts read
        # back for it.
        dict(name="cache_chunk_nvfp4", op="cache", B=4, L=4000, new=512, HKV=8, D=128, page=16,
             format="nvfp4"),
        # Long contexts of many sequences read back from an 8-bit cache.
        dict(name="cache_read_fp8", op="cache", B=32, L=5120, new=0, HKV=8, D=128, page=64,
             format="fp8"),
    ]


def _log(rng, lo, hi, step=1):
    """A size in lo..hi, even over its logarithm, in multiples of `step`."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return int(min(hi, max(lo, step * round(v / step))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "experts", "experts", "heads", "heads",
                     "cache", "cache"])
    if op == "quantize":
        return dict(op=op, T=_log(rng, 1, 8192), H=_log(rng, 100, 5120), rows=rng.choice([1, 128]))
    if op == "product":
        return dict(op=op, T=_log(rng, 1, 8192), N=_log(rng, 100, 8192), H=_log(rng, 256, 8192, 16))
    if op == "experts":
        E = _log(rng, 2, 64)
        return dict(op=op, T=_log(rng, 1, 4096), K=rng.randint(1, min(8, E)), E=E,
                    H=_log(rng, 256, 7168, 16), N=_log(rng, 100, 4096),
                    gather=rng.random() < 0.5, skew=rng.choice([0.0, 0.5, 1.0]))
    if op == "heads":
        D = rng.choice([64, 80, 96, 128, 192, 256])
        HKV = rng.choice([1, 2, 4, 8])
        return dict(op=op, T=_log(rng, 1, 4096), HQ=HKV * rng.choice([1, 2, 5]), HKV=HKV, D=D,
                    R=rng.choice([D, D // 32 * 16]), axes=rng.choice([1, 1, 2, 3]),
                    interleaved=rng.random() < 0.5, format=rng.choice(["", "fp8"]))
    return dict(op=op, B=_log(rng, 1, 32), L=_log(rng, 1, 4096), new=_log(rng, 1, 256),
                HKV=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 96, 128, 256]),
                page=rng.choice([1, 16, 64]), format=rng.choice(["fp8", "nvfp4"]))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _codes(shape, g):
    """E4M3 codes of normal values whose largest use the type's range."""
    v = torch.randn(shape, device=DEV, generator=g, dtype=torch.bfloat16)
    return v.mul_(100.0).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _scales(shape, size, g):
    return (0.5 + torch.rand(shape, device=DEV, generator=g)) * (size / 100.0)


def _routing(case, g):
    """A routing of T tokens to K of E experts each, some experts favoured
    over others by `skew`: rows (the token of each slot) and offsets (the
    first slot of each expert), the slots sorted by expert, then token."""
    T, K, E = case["T"], case["K"], case["E"]
    liking = case["skew"] * torch.randn(E, device=DEV, generator=g)
    noise = torch.rand(T, E, device=DEV, generator=g)
    experts = (liking - (-(noise + 1e-9).log()).log()).topk(K, dim=1).indices.reshape(-1)
    order = experts.sort(stable=True).indices
    counts = torch.bincount(experts, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = counts.cumsum(0)
    return (order // K).to(torch.int32), offsets, int(counts.max())


def _contexts(B, L):
    """Lengths of B contexts, between L / 2 and L, one of three or more empty:
    a sequence that begins."""
    old = [L // 2 + i * 7919 % (L - L // 2 + 1) for i in range(B)]
    if B > 2:
        old[B // 2] = 0
    return old


def _empty_cache(slots, HKV, D, fmt, page, g):
    """A cache in use: codes and scales of other tokens in every slot."""
    pages = -(-slots // page)

    def half():
        shape = (pages, page, HKV)
        if fmt == "fp8":
            return _codes(shape + (D,), g), _scales(shape, 1.0, g)
        codes = torch.randint(0, 256, shape + (D // 2,), device=DEV, generator=g,
                              dtype=torch.uint8)
        # block scales of 8 to 120
        scales = torch.randint(0x50, 0x70, shape + (D // 16,), device=DEV, generator=g,
                               dtype=torch.uint8)
        return codes, scales
    (kc, ks), (vc, vs) = half(), half()
    return kc, vc, ks, vs


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "quantize":
        T, H = case["T"], case["H"]
        x = torch.randn(T, H, device=DEV, generator=g)
        # outliers as the prefill workload has them, and a run of zeros
        x *= torch.where(torch.rand(T, H, device=DEV, generator=g) < 0.001, 50.0, 1.0)
        x[T // 2, :128] = 0.0
        return dict(case, x=x.to(torch.bfloat16))
    if op == "product":
        T, N, H = case["T"], case["N"], case["H"]
        HB, NB = -(-H // 128), -(-N // 128)
        return dict(case, a=_codes((T, H), g), sa=_scales((T, HB), 1.0, g), b=_codes((N, H), g),
                    sb=_scales((NB, HB), H ** -0.5, g))
    if op == "experts":
        T, K, E, H, N = (case[k] for k in ("T", "K", "E", "H", "N"))
        HB, NB = -(-H // 128), -(-N // 128)
        rows, offsets, most = _routing(case, g)
        n = T if case["gather"] else T * K
        return dict(case, a=_codes((n, H), g), sa=_scales((n, HB), 1.0, g),
                    b=_codes((E, N, H), g), sb=_scales((E, NB, HB), H ** -0.5, g),
                    offsets=offsets, token=rows if case["gather"] else None, most=most)
    if op == "heads":
        T, HQ, HKV, D, R, axes = (case[k] for k in ("T", "HQ", "HKV", "D", "R", "axes"))
        qkv = torch.randn(T, (HQ + 2 * HKV) * D, device=DEV, generator=g).to(torch.bfloat16)
        weigh = lambda: (1.0 + 0.1 * torch.randn(D, device=DEV, generator=g)).to(torch.bfloat16)  # noqa: E731
        half = R // 2
        freqs = (1e6 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)).float()
        # one axis: tokens of a sequence that is far along; more: time,
        # height and width
        first = torch.randint(0, 100000, (1,), device=DEV, generator=g)
        at = torch.arange(T, device=DEV)
        sides = [first + at] if axes == 1 else [first + at // 576, at // 24 % 24, at % 24][:axes]
        part = half // axes
        s = dict(case, qkv=qkv, wq=weigh(), wk=weigh(), freqs=freqs,
                 positions=torch.stack(sides).to(torch.int32).contiguous(),
                 sections=str([half - part * (axes - 1)] + [part] * (axes - 1)))
        if case["format"]:
            slots = torch.randperm(T + T // 4 + 16, device=DEV, generator=g)[:T].to(torch.int32)
            if T > 8:
                slots[T - T // 16 - 1:] = -1                # padding of the batch
            s.update(slots=slots, cache=_empty_cache(T + T // 4 + 16, HKV, D, case["format"], 16, g))
        return s
    if op == "cache":
        B, L, HKV, D, page = (case[k] for k in ("B", "L", "HKV", "D", "page"))
        old = torch.tensor(_contexts(B, L), device=DEV)
        lengths = old + case["new"]
        width = -(-(L + case["new"]) // page)
        table = torch.randperm(B * width, device=DEV, generator=g).view(B, width).to(torch.int32)
        offsets = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
        offsets[1:] = lengths.cumsum(0)
        s = dict(case, table=table, offsets=offsets, total=int(offsets[-1]),
                 cache=_empty_cache(B * width * page, HKV, D, case["format"], page, g))
        if case["new"]:
            pos = old[:, None] + torch.arange(case["new"], device=DEV)
            s["slots"] = (table.long().gather(1, pos // page) * page + pos % page).view(-1).to(
                torch.int32)
            for name in ("k", "v"):
                x = torch.randn(B * case["new"], HKV, D, device=DEV, generator=g)
                s[name] = x.to(torch.bfloat16)
        return s
    raise ValueError(op)


# ------------------------------------------------------------ plain forms
def _to_e4m3(x, amax):
    """Codes and scale of values whose largest magnitude is `amax`."""
    top = amax.new_full((), 448.0)      # on the device: a division, no product with 1 / 448
    scale = torch.where(amax > 0, amax / top, 1.0)
    inv = torch.where(amax > 0, top / amax, 1.0)
    return (x * inv).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale


def _quantize(s):
    T, H, br = s["T"], s["H"], s["rows"]
    TB, HB = -(-T // br), -(-H // 128)
    x = torch.zeros(TB * br, HB * 128, device=s["x"].device)
    x[:T, :H] = s["x"].float()
    x = x.view(TB, br, HB, 128)
    codes, scale = _to_e4m3(x, x.abs().amax(dim=(1, 3), keepdim=True))
    codes = codes.view(torch.uint8).view(TB * br, HB * 128)[:T, :H].contiguous()
    return dict(codes=codes.view(torch.float8_e4m3fn), scales=scale.view(TB, HB))


def _wide(codes, scales, rows):
    """code * scale in 32 bits; `rows` rows share a scale."""
    T, H = codes.shape[-2:]
    s = scales.repeat_interleave(128, dim=-1)[..., :H]
    if rows > 1:
        s = s.repeat_interleave(rows, dim=-2)[..., :T, :]
    return codes.view(torch.float8_e4m3fn).float() * s


def _product(s):
    return torch.matmul(_wide(s["a"], s["sa"], 1), _wide(s["b"], s["sb"], 128).t()).to(
        torch.bfloat16)


def _experts(s):
    a, offsets, E, most = _wide(s["a"], s["sa"], 1), s["offsets"].long(), s["E"], s["most"]
    S = s["T"] * s["K"]
    slot = torch.arange(S, device=a.device)
    e = torch.searchsorted(offsets, slot, right=True) - 1
    at = slot - offsets[e]
    padded = torch.zeros(E, most, s["H"], device=a.device)
    padded[e, at] = a if s["token"] is None else a[s["token"].long()]
    w = _wide(s["b"], s["sb"], 128)
    return torch.bmm(padded, w.transpose(1, 2))[e, at].to(torch.bfloat16)


def _sections(s):
    return [int(v) for v in s["sections"][1:-1].split(",")]


def _split(s):
    q, k, v = s["qkv"].split([s["HQ"] * s["D"], s["HKV"] * s["D"], s["HKV"] * s["D"]], dim=1)
    T, D = s["T"], s["D"]
    return q.view(T, -1, D), k.view(T, -1, D), v.view(T, -1, D)


def _rotated(x, w, cos, sin, R, interleaved):
    x = x.float()
    x = x / (x.square().mean(dim=2, keepdim=True) + EPS).sqrt() * w.float()
    y, rest = x[..., :R], x[..., R:]
    if interleaved:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=3).flatten(2)
    else:
        a, b = y[..., :R // 2], y[..., R // 2:]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=2)
    return torch.cat((y, rest), dim=2)


def _heads(s):
    q, k, v = _split(s)
    axis = torch.repeat_interleave(
        torch.arange(s["axes"], device=q.device),
        torch.tensor(_sections(s), device=q.device))
    # angles of far positions need 64 bits
    angle = (s["positions"].double()[axis].t() * s["freqs"].double()).unsqueeze(1)
    cos, sin = angle.cos().float(), angle.sin().float()
    q = _rotated(q, s["wq"], cos, sin, s["R"], s["interleaved"])
    k = _rotated(k, s["wk"], cos, sin, s["R"], s["interleaved"])
    if not s["format"]:
        return dict(q=q.to(torch.bfloat16), k=k.to(torch.bfloat16))
    kc, vc, ks, vs = s["cache"]
    live = s["slots"] >= 0
    at = s["slots"][live].long()
    for x, codes, scales in ((k, kc, ks), (v.float(), vc, vs)):
        c, scale = _to_e4m3(x, x.abs().amax(dim=2, keepdim=True))
        codes.view(-1, s["HKV"], s["D"])[at] = c.view(torch.uint8)[live]
        scales.view(-1, s["HKV"])[at] = scale[live].squeeze(2)
    return dict(q=q.to(torch.bfloat16), k=kc.view(torch.float8_e4m3fn), ks=ks,
                v=vc.view(torch.float8_e4m3fn), vs=vs)


def _to_nvfp4(x):
    """Packed codes and block scale bytes of values [n, HKV, D]."""
    n, h, d = x.shape
    x = x.float().view(n, h, d // 16, 16)
    six, g = x.new_full((), 6.0), x.new_full((), G)
    scale = (x.abs().amax(dim=3, keepdim=True) / six * g).clamp(max=448.0).to(torch.float8_e4m3fn)
    sv = scale.float()
    x = torch.where(sv > 0, x * (g / sv), 0.0)
    m = x.abs()
    # the code of a magnitude: how many of the borders between codes it is
    # beyond; a tie goes to the even code
    code = (m > 0.25).int() + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) \
        + (m > 5.0)
    code = (code + 8 * torch.signbit(x)).view(n, h, d // 2, 2)
    packed = (code[..., 0] + 16 * code[..., 1]).to(torch.uint8)
    return packed, scale.view(torch.uint8).view(n, h, d // 16)


def _cache(s):
    kc, vc, ks, vs = s["cache"]
    HKV, D, page, fp8 = s["HKV"], s["D"], s["page"], s["format"] == "fp8"
    if s["new"]:
        at = s["slots"].long()
        for x, codes, scales in ((s["k"], kc, ks), (s["v"], vc, vs)):
            if fp8:
                x = x.float()
                c, scale = _to_e4m3(x, x.abs().amax(dim=2, keepdim=True))
                codes.view(-1, HKV, D)[at] = c.view(torch.uint8)
                scales.view(-1, HKV)[at] = scale.squeeze(2)
            else:
                codes.view(-1, HKV, D // 2)[at], scales.view(-1, HKV, D // 16)[at] = _to_nvfp4(x)
    token = torch.arange(s["total"], device=kc.device)
    b = torch.searchsorted(s["offsets"].long(), token, right=True) - 1
    pos = token - s["offsets"].long()[b]
    at = s["table"].long()[b, pos // page] * page + pos % page
    out = []
    for codes, scales in ((kc, ks), (vc, vs)):
        if fp8:
            c = codes.view(-1, HKV, D)[at].view(torch.float8_e4m3fn).float()
            v = c * scales.view(-1, HKV)[at].unsqueeze(2)
        else:
            c = codes.view(-1, HKV, D // 2)[at]
            c = torch.stack((c & 15, c >> 4), dim=3).view(-1, HKV, D // 16, 16).long()
            half = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=c.device)
            f = scales.view(-1, HKV, D // 16)[at].view(torch.float8_e4m3fn).float() / G
            v = (torch.cat((half, -half))[c] * f.unsqueeze(3)).view(-1, HKV, D)
        out.append(v.to(torch.bfloat16))
    return dict(k=out[0], v=out[1])


def run(state):
    s = state
    op = s["op"]
    if own:
        import rank_sum_residual_gb300 as farn
        if op == "quantize":
            codes, scales = farn.fp8_quantize(s["x"], block_rows=s["rows"])
            return dict(codes=codes.view(torch.float8_e4m3fn), scales=scales)
        if op == "product":
            return farn.fp8_matmul(s["a"], s["sa"], s["b"], s["sb"])
        if op == "experts":
            return farn.fp8_grouped_matmul(s["a"], s["sa"], s["b"], s["sb"], s["offsets"],
                                           rows=s["token"])
        if op == "heads":
            q, k, v = _split(s)
            rest = dict(sections=_sections(s), interleaved=s["interleaved"])
            if not s["format"]:
                q, k = farn.qk_norm_rope(q, k, s["wq"], s["wk"], EPS, s["positions"], s["freqs"],
                                         **rest)
                return dict(q=q, k=k)
            q = farn.qk_norm_rope_cache(q, k, v, s["wq"], s["wk"], EPS, s["positions"],
                                        s["freqs"], s["cache"], s["slots"], **rest)
            kc, vc, ks, vs = s["cache"]
            return dict(q=q, k=kc.view(torch.float8_e4m3fn), ks=ks,
                        v=vc.view(torch.float8_e4m3fn), vs=vs)
        scale = None if s["format"] == "fp8" else (G, G)
        if s["new"]:
            farn.kv_write(s["k"], s["v"], s["cache"], s["slots"], tensor_scales=scale)
        k, v = farn.kv_read(s["cache"], s["table"], s["offsets"], s["total"], tensor_scales=scale)
        return dict(k=k, v=v)
    return dict(quantize=_quantize, product=_product, experts=_experts, heads=_heads,
                cache=_cache)[op](s)


def work(case):
    op = case["op"]
    if op == "quantize":
        T, H, br = case["T"], case["H"], case["rows"]
        return dict(bytes=3 * T * H + 4 * -(-T // br) * -(-H // 128), flops=3 * T * H)
    if op == "product":
        T, N, H = case["T"], case["N"], case["H"]
        return dict(bytes=(T + N) * H + 2 * T * N + 4 * (T + -(-N // 128)) * -(-H // 128),
                    flops=2 * T * N * H)
    if op == "experts":
        T, K, E, H, N = (case[k] for k in ("T", "K", "E", "H", "N"))
        # the experts that T draws of K out of E reach, in the mean
        reached = E * (1.0 - (1.0 - K / E) ** T)
        n = T if case["gather"] else T * K
        return dict(bytes=n * H + reached * N * H + 2 * T * K * N + 4 * (E + 1)
                    + 4 * (n + reached * -(-N // 128)) * -(-H // 128)
                    + (4 * T * K if case["gather"] else 0), flops=2 * T * K * N * H)
    if op == "heads":
        T, HQ, HKV, D = (case[k] for k in ("T", "HQ", "HKV", "D"))
        n = T * (HQ + HKV) * D
        if not case["format"]:
            return dict(bytes=4 * n + 4 * T * case["axes"], flops=10 * n)
        return dict(bytes=2 * T * (HQ + 2 * HKV) * D + 2 * T * HQ * D + 2 * T * HKV * (D + 4)
                    + 8 * T, flops=10 * n)
    B, L, HKV, D = (case[k] for k in ("B", "L", "HKV", "D"))
    row = D + 4 if case["format"] == "fp8" else D * 9 / 16
    read = sum(_contexts(B, L)) + B * case["new"]
    return dict(bytes=2 * HKV * (read * (row + 2 * D) + B * case["new"] * (row + 2 * D)),
                flops=2 * HKV * D * read)


# ------------------------------------------------------- 64-bit definition
def _e4m3_value(codes):
    """The value of E4M3 codes, from the format's definition."""
    c = codes.long()
    e, f = (c >> 3) & 15, (c & 7).double() / 8
    v = torch.where(e == 0, f * 2.0 ** -6, (1 + f) * torch.exp2(e.double() - 7))
    return torch.where(c >= 128, -v, v)


def _round(v, low, top, bits):
    """|v| to the nearest value with `bits` fraction bits, exponents from
    `low`, at most `top`; ties to the even one."""
    e = torch.frexp(v).exponent.double() - 1
    step = torch.exp2(e.clamp(min=low) - bits)
    return ((v / step).round() * step).clamp(max=top)


def _f32(v):
    return v.float().double()


def _exact_e4m3(x, amax):
    """The definition rounds both quotients and the product to 32 bits."""
    inv = torch.where(amax > 0, _f32(448.0 / amax), 1.0)
    return _round(_f32(x.abs() * inv), -6, 448.0, 3) * x.sign(), \
        torch.where(amax > 0, _f32(amax / 448.0), 1.0)


def _exact_quantize(s):
    T, H, br = s["T"], s["H"], s["rows"]
    TB, HB = -(-T // br), -(-H // 128)
    codes = torch.empty(T, H, device=DEV, dtype=torch.float64)
    scales = torch.empty(TB, HB, device=DEV, dtype=torch.float64)
    x = s["x"].double()
    for j in range(HB):
        part = x[:, j * 128:(j + 1) * 128]
        most = part.abs().amax(dim=1)
        most = torch.cat((most, most.new_zeros(TB * br - T))).view(TB, br).amax(dim=1)
        codes[:, j * 128:(j + 1) * 128], scale = _exact_e4m3(
            part, most.repeat_interleave(br)[:T, None])
        scales[:, j] = most.new_ones(TB) if TB == 0 else torch.where(most > 0, _f32(most / 448.0),
                                                                     1.0)
    return dict(codes=codes, scales=scales)


def _sum_of_blocks(a, sa, b, sb):
    """Block by block, as the definition has it."""
    out = torch.zeros(a.shape[0], b.shape[0], device=a.device, dtype=torch.float64)
    block = torch.arange(b.shape[0], device=a.device) // 128
    step = 8192 if a.shape[0] * b.shape[0] > 1 << 24 else 128
    for h in range(0, a.shape[1], step):
        n = min(step, a.shape[1] - h)
        at = (h + torch.arange(n, device=a.device)) // 128
        va = _e4m3_value(a[:, h:h + n]) * sa.double()[:, at]
        vb = _e4m3_value(b[:, h:h + n]) * sb.double()[block][:, at]
        out += va @ vb.t()
    return out


def _exact_product(s):
    return _sum_of_blocks(s["a"], s["sa"], s["b"], s["sb"])


def _exact_experts(s):
    offsets = s["offsets"].tolist()
    out = torch.empty(s["T"] * s["K"], s["N"], device=DEV, dtype=torch.float64)
    for e in range(s["E"]):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            at = slice(lo, hi) if s["token"] is None else s["token"][lo:hi].long()
            out[lo:hi] = _sum_of_blocks(s["a"][at], s["sa"][at], s["b"][e], s["sb"][e])
    return out


def _exact_heads(s):
    HQ, HKV, D, R, T = (s[k] for k in ("HQ", "HKV", "D", "R", "T"))
    x = s["qkv"].double().view(T, HQ + 2 * HKV, D)
    axis = [a for a, n in enumerate(_sections(s)) for _ in range(n)]
    turn = torch.polar(torch.ones(T, R // 2, device=DEV, dtype=torch.float64),
                       torch.stack([s["positions"][a].double() * s["freqs"][i].double()
                                    for i, a in enumerate(axis)], dim=1))

    def rotate(y, w):
        rms = torch.sqrt((y * y).sum(dim=2, keepdim=True) / D + EPS)
        y = y / rms * w.double()
        first = torch.arange(R // 2, device=DEV)
        a, b = (2 * first, 2 * first + 1) if s["interleaved"] else (first, first + R // 2)
        z = torch.complex(y[..., a], y[..., b]) * turn[:, None]
        y = y.clone()
        y[..., a], y[..., b] = z.real, z.imag
        return y
    q, k, v = rotate(x[:, :HQ], s["wq"]), rotate(x[:, HQ:HQ + HKV], s["wk"]), x[:, HQ + HKV:]
    if not s["format"]:
        return dict(q=q, k=k)
    out = dict(q=q)
    live = (s["slots"] >= 0).nonzero()[:, 0]
    at = s["slots"][live].long()
    kc, vc, ks, vs = s["cache"]
    for name, y, codes, scales in (("k", k, kc, ks), ("v", v, vc, vs)):
        c, sc = _e4m3_value(codes).view(-1, HKV, D), scales.double().view(-1, HKV)
        amax = y.abs().amax(dim=2, keepdim=True)
        # of values that no smaller type holds: the quotients stay in 64 bits
        c[at] = (_round((y * (448.0 / amax)).abs(), -6, 448.0, 3) * y.sign())[live]
        sc[at] = (amax / 448.0)[live].squeeze(2)
        out[name], out[name + "s"] = c.view(codes.shape), sc.view(scales.shape)
    return out


def _exact_cache(s):
    HKV, D, page = s["HKV"], s["D"], s["page"]
    kc, vc, ks, vs = s["cache"]
    offsets, out = s["offsets"].tolist(), {}
    for name, codes, scales in (("k", kc, ks), ("v", vc, vs)):
        if s["format"] == "fp8":
            value = _e4m3_value(codes) * scales.double().unsqueeze(3)
        else:
            c = torch.empty(codes.shape[:3] + (D,), dtype=torch.int64, device=DEV)
            c[..., 0::2], c[..., 1::2] = (codes % 16).long(), (codes // 16).long()
            e, f = (c >> 1) & 3, (c & 1).double()
            m = torch.where(e == 0, 0.5 * f, torch.exp2(e.double() - 1) * (1 + 0.5 * f))
            value = torch.where(c >= 8, -m, m) * (
                _e4m3_value(scales) / G).repeat_interleave(16, dim=3)
        value = value.view(-1, HKV, D)
        if s["new"]:
            x = s[name].double()
            if s["format"] == "fp8":
                c, scale = _exact_e4m3(x, x.abs().amax(dim=2, keepdim=True))
                new = c * scale
            else:
                y = x.view(-1, HKV, D // 16, 16)
                sc = _round(_f32(_f32(y.abs().amax(dim=3) / 6.0) * G), -6, 448.0, 3)
                inv = torch.where(sc > 0, _f32(G / sc), 0.0)[..., None]
                new = _round(_f32(y.abs() * inv), 0, 6.0, 1) * y.sign() * sc[..., None] / G
            value[s["slots"].long()] = new.view(-1, HKV, D)
        parts = []
        for b, row in enumerate(s["table"].long()):
            n = offsets[b + 1] - offsets[b]
            parts.append(value.view(-1, page, HKV, D)[row].view(-1, HKV, D)[:n])
        out[name] = torch.cat(parts)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return dict(quantize=_exact_quantize, product=_exact_product, experts=_exact_experts,
                heads=_exact_heads, cache=_exact_cache)[case["op"]](s)
