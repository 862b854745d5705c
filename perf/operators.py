"""The MoE router, the products grouped by expert, and the NVFP4 quantisation
and product: cases, plain forms and measurement hooks.

``run`` computes one pass of an operator, in plain torch operations (32 bits
inside, one rounding at the end) or, where ``own`` is set, through the
package's public calls.  ``exact`` computes the same outputs in 64 bits.

Operators
  route     the top-K experts of every token, their softmax gates, and the
            slots of the (token, expert) pairs sorted by expert
  experts   out[s] = x[rows[s]] W_e^T for the slots s of every expert e
  quantize  bf16 [T,H] to NVFP4 codes and block scales, and the values back
  product   out = (A / ga) (B / gb)^T of two NVFP4 tensors, in bf16
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
# The tensor scale of the benchmark's NVFP4 workload: an amax of 16 maps to
# the largest code times the largest block scale.
G = 168.0


def listed():
    return [
        # The router of one decoding step of 16 sequences.
        dict(name="route_decode", op="route", T=16, E=128, K=8, dtype="f32", renorm=True, pad=0),
        # The router of a long prefill whose batch is padded: logits of the
        # padding are masked, so those tokens choose no expert.
        dict(name="route_prefill", op="route", T=16384, E=256, K=8, dtype="bf16", renorm=False,
             pad=1500),
        # First expert product of one token: eight experts' weights are read
        # for one row each.
        dict(name="experts_one_token", op="experts", T=1, K=8, E=64, H=7168, N=2048, gather=True,
             skew=0.0),
        # Second expert product of a decoding batch: a handful of rows for
        # every expert.
        dict(name="experts_decode", op="experts", T=64, K=8, E=64, H=2048, N=7168, gather=False,
             skew=0.5),
        # Few, unevenly loaded experts with sizes off every tile.
        dict(name="experts_ragged", op="experts", T=1003, K=3, E=7, H=2056, N=1100, gather=True,
             skew=1.0),
        # First expert product of a prefill of 4096 tokens (the MoE combine
        # workload's hidden size and experts per token).
        dict(name="experts_prefill", op="experts", T=4096, K=8, E=64, H=7168, N=4096, gather=True,
             skew=0.5),
        # Activations of one decoding step, quantised.
        dict(name="quantize_decode", op="quantize", T=16, H=4096),
        # Activations of the prefill workload, quantised.
        dict(name="quantize_prefill", op="quantize", T=8192, H=8192),
        # A projection of one token: reading the 4-bit weights.
        dict(name="product_one_token", op="product", T=1, N=8192, H=8192),
        # A projection of a decoding batch.
        dict(name="product_decode", op="product", T=128, N=10240, H=5120),
        # Sizes off every tile; H a multiple of 32 only.
        dict(name="product_ragged", op="product", T=1237, N=4100, H=2080),
        # A projection of the prefill workload.
        dict(name="product_prefill", op="product", T=8192, N=8192, H=8192),
    ]


def _log(rng, lo, hi, step=1):
    """A size in lo..hi, even over its logarithm, in multiples of `step`."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return int(min(hi, max(lo, step * round(v / step))))


def draw(rng):
    op = rng.choice(["route", "experts", "experts", "quantize", "product", "product"])
    if op == "route":
        T, E = _log(rng, 1, 16384), _log(rng, 4, 256)
        return dict(op=op, T=T, E=E, K=rng.randint(1, min(8, E)),
                    dtype=rng.choice(["f32", "bf16"]), renorm=rng.random() < 0.5,
                    pad=int(T * rng.choice([0, 0, 0.1, 0.4])))
    if op == "experts":
        E = _log(rng, 2, 64)
        return dict(op=op, T=_log(rng, 1, 4096), K=rng.randint(1, min(8, E)), E=E,
                    H=_log(rng, 256, 7168, 8), N=_log(rng, 100, 4096),
                    gather=rng.random() < 0.5, skew=rng.choice([0.0, 0.5, 1.0]))
    if op == "quantize":
        return dict(op=op, T=_log(rng, 1, 8192), H=_log(rng, 256, 8192, 16))
    return dict(op=op, T=_log(rng, 1, 8192), N=_log(rng, 100, 8192), H=_log(rng, 256, 8192, 32))


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


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


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "route":
        T, E = case["T"], case["E"]
        x = 2.0 * torch.randn(T, E, device=DEV, generator=g)
        if case["pad"]:
            x[T - case["pad"]:] = -math.inf
        return dict(case, logits=x.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32))
    if op == "experts":
        T, K, E, H, N = (case[k] for k in ("T", "K", "E", "H", "N"))
        rows, offsets, most = _routing(case, g)
        n = T if case["gather"] else T * K
        x = torch.randn(n, H, device=DEV, generator=g, dtype=torch.bfloat16)
        w = torch.randn(E, N, H, device=DEV, generator=g, dtype=torch.bfloat16)
        w *= H ** -0.5
        return dict(case, x=x, w=w, offsets=offsets, rows=rows if case["gather"] else None,
                    most=most)
    if op == "quantize":
        T, H = case["T"], case["H"]
        x = torch.randn(T, H, device=DEV, generator=g)
        # outliers as the prefill workload has them, and a block of zeros
        x *= torch.where(torch.rand(T, H, device=DEV, generator=g) < 0.001, 50.0, 1.0)
        x[T // 2, :16] = 0.0
        return dict(case, x=x.to(torch.bfloat16))
    if op == "product":
        T, N, H = case["T"], case["N"], case["H"]

        def tensor(rows):
            codes = torch.randint(0, 256, (rows, H // 2), device=DEV, generator=g,
                                  dtype=torch.uint8)
            # block scales of 8 to 120, and one block in 64 of zeros
            scales = torch.randint(0x50, 0x70, (rows, H // 16), device=DEV, generator=g,
                                   dtype=torch.uint8)
            scales *= torch.randint(0, 64, scales.shape, device=DEV, generator=g,
                                    dtype=torch.uint8) != 0
            return codes, scales
        a, b = tensor(T), tensor(N)
        return dict(case, aq=a[0], ascale=a[1], bq=b[0], bscale=b[1])
    raise ValueError(op)


# ------------------------------------------------------------ plain forms
def _route(s):
    x, K, E = s["logits"].float(), s["K"], s["E"]
    T = x.shape[0]
    top, experts = x.sort(dim=1, descending=True, stable=True)
    first = top[:, :1]
    over = top[:, :K] if s["renorm"] else top
    # an expert masked with -inf weighs nothing, and a token without experts
    # has no gates
    weigh = lambda v: torch.where(v == -math.inf, 0.0, (v - first).exp())  # noqa: E731
    total = weigh(over).sum(dim=1, keepdim=True)
    top, experts = top[:, :K], experts[:, :K]
    gates = torch.where(total > 0, weigh(top) / total, 0.0)
    experts = torch.where(top == -math.inf, -1, experts)
    flat = experts.reshape(-1)
    key, order = torch.where(flat < 0, E, flat).sort(stable=True)
    slot = torch.arange(T * K, device=x.device)
    index = torch.empty_like(flat)
    index[order] = torch.where(key < E, slot, -1)
    rows = torch.where(key < E, order // K, -1)
    offsets = torch.searchsorted(key, torch.arange(E + 1, device=x.device))
    i32 = torch.int32
    return dict(experts=experts.to(i32), gates=gates, index=index.reshape(T, K).to(i32),
                rows=rows.to(i32), offsets=offsets.to(i32))


def _experts(s):
    x, w, offsets, E, most = s["x"], s["w"], s["offsets"].long(), s["E"], s["most"]
    S = s["T"] * s["K"]
    slot = torch.arange(S, device=x.device)
    e = torch.searchsorted(offsets, slot, right=True) - 1
    at = slot - offsets[e]
    padded = torch.zeros(E, most, s["H"], device=x.device)
    padded[e, at] = (x if s["rows"] is None else x[s["rows"].long()]).float()
    return torch.bmm(padded, w.float().transpose(1, 2))[e, at].to(torch.bfloat16)


def _quantize(s):
    T, H = s["x"].shape
    x = s["x"].float().view(T, H // 16, 16)
    amax = x.abs().amax(dim=2, keepdim=True)
    scale = (amax / 6.0 * G).clamp(max=448.0).to(torch.float8_e4m3fn)
    sv = scale.float()
    v = torch.where(sv > 0, x * (G / sv), 0.0)
    m = v.abs()
    half = [(m > 0.25), (m >= 0.75), (m > 1.25), (m >= 1.75)]
    one = [(m > 2.5), (m >= 3.5)]
    mag = 0.5 * (half[0].float() + half[1].float() + half[2].float() + half[3].float()) \
        + one[0].float() + one[1].float() + 2.0 * (m > 5.0).float()
    values = torch.copysign(mag, v) * (sv / G)
    return dict(values=values.view(T, H).to(torch.bfloat16), scales=scale.view(T, H // 16))


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _values(codes, scales):
    table = torch.tensor(_E2M1 + [-v for v in _E2M1], device=codes.device)
    both = torch.stack((codes & 15, codes >> 4), dim=2).long()
    rows, blocks = scales.shape
    v = table[both].view(rows, blocks, 16)
    return (v * scales.view(torch.float8_e4m3fn).float()[:, :, None]).view(rows, blocks * 16)


def _product(s):
    a, b = _values(s["aq"], s["ascale"]), _values(s["bq"], s["bscale"])
    return (torch.matmul(a, b.t()) / (G * G)).to(torch.bfloat16)


def run(state):
    op = state["op"]
    if own:
        import rank_sum_residual_gb300 as farn
        if op == "route":
            experts, gates, index, rows, offsets = farn.moe_route(
                state["logits"], state["K"], renormalize=state["renorm"])
            return dict(experts=experts, gates=gates, index=index, rows=rows, offsets=offsets)
        if op == "experts":
            return farn.grouped_matmul(state["x"], state["w"], state["offsets"],
                                       rows=state["rows"])
        if op == "quantize":
            codes, scales = farn.nvfp4_quantize(state["x"], G)
            return dict(values=farn.nvfp4_dequantize(codes, scales, G),
                        scales=scales.view(torch.float8_e4m3fn))
        return farn.nvfp4_matmul(state["aq"], state["ascale"], G,
                                 state["bq"], state["bscale"], G)
    return dict(route=_route, experts=_experts, quantize=_quantize, product=_product)[op](state)


def work(case):
    op = case["op"]
    if op == "route":
        T, E, K = case["T"], case["E"], case["K"]
        return dict(bytes=T * E * (2 if case["dtype"] == "bf16" else 4) + 4 * 4 * T * K
                    + 4 * (E + 1), flops=4 * T * E)
    if op == "experts":
        T, K, E, H, N = (case[k] for k in ("T", "K", "E", "H", "N"))
        # the experts that T draws of K out of E reach, in the mean
        reached = E * (1.0 - (1.0 - K / E) ** T)
        n = T if case["gather"] else T * K
        return dict(bytes=2 * (n * H + reached * N * H + T * K * N) + 4 * (E + 1)
                    + (4 * T * K if case["gather"] else 0), flops=2 * T * K * N * H)
    if op == "quantize":
        n = case["T"] * case["H"]
        # quantise: 2 bytes in, 9/16 out; back to values: 9/16 in, 2 out
        return dict(bytes=5.125 * n, flops=4 * n)
    T, N, H = case["T"], case["N"], case["H"]
    return dict(bytes=(T + N) * H * 9 / 16 + 2 * T * N, flops=2 * T * N * H)


# ------------------------------------------------------- 64-bit definition
def _exact_route(s):
    x = s["logits"].double().cpu().numpy()
    T, E = x.shape
    K = s["K"]
    order = np.argsort(-x, axis=1, kind="stable")[:, :K]
    top = np.take_along_axis(x, order, axis=1)
    live = np.isfinite(top)
    some = live[:, :1]
    m = np.where(some, top[:, :1], 0.0)
    p = np.where(np.isfinite(x), np.exp(x - m), 0.0)
    chosen = np.take_along_axis(p, order, axis=1)
    total = (chosen if s["renorm"] else p).sum(axis=1, keepdims=True)
    gates = np.divide(chosen, total, out=np.zeros_like(chosen), where=total > 0)
    experts = np.where(live, order, -1)
    index = np.full(T * K, -1)
    rows = np.full(T * K, -1)
    offsets = np.zeros(E + 1, dtype=np.int64)
    flat, at = experts.reshape(-1), 0
    for e in range(E):
        hit = np.flatnonzero(flat == e)
        index[hit] = at + np.arange(hit.size)
        rows[at:at + hit.size] = hit // K
        at += hit.size
        offsets[e + 1] = at
    return dict(experts=experts, gates=gates, index=index.reshape(T, K), rows=rows,
                offsets=offsets)


def _exact_experts(s):
    offsets = s["offsets"].tolist()
    out = torch.empty(s["T"] * s["K"], s["N"], device=s["x"].device, dtype=torch.float64)
    for e in range(s["E"]):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            x = s["x"][lo:hi] if s["rows"] is None else s["x"][s["rows"][lo:hi].long()]
            out[lo:hi] = x.double() @ s["w"][e].double().t()
    return out


def _exact_round(v, low, top, bits):
    """|v| to the nearest value with `bits` fraction bits, exponents from
    `low`, at most `top`; ties to the even one."""
    e = torch.frexp(v).exponent.double() - 1
    step = torch.exp2(e.clamp(min=low) - bits)
    return ((v / step).round() * step).clamp(max=top)


def _exact_quantize(s):
    # The definition rounds amax / 6, its product with the tensor scale, the
    # quotient and the scaled value to 32 bits each.
    f32 = lambda v: v.float().double()  # noqa: E731
    T, H = s["x"].shape
    values = torch.empty(T, H, device=s["x"].device, dtype=torch.float64)
    scales = torch.empty(T, H // 16, device=s["x"].device, dtype=torch.float64)
    x = s["x"].double().reshape(T, H // 16, 16)
    sc = _exact_round(f32(f32(x.abs().amax(dim=2) / 6.0) * G), -6, 448.0, 3)
    inv = torch.where(sc > 0, f32(G / sc), 0.0)[:, :, None]
    q = _exact_round(f32(x.abs() * inv), 0, 6.0, 1) * x.sign()
    scales[:] = sc
    values[:] = (q * sc[:, :, None] / G).reshape(T, H)
    return dict(values=values, scales=scales)


def _exact_product(s):
    def values(codes, scales):
        rows, blocks = scales.shape
        c = torch.empty(rows, blocks * 16, dtype=torch.int64, device=codes.device)
        c[:, 0::2] = (codes % 16).long()
        c[:, 1::2] = (codes // 16).long()
        e, f, neg = (c >> 1) & 3, (c & 1).double(), c >= 8
        v = torch.where(e == 0, 0.5 * f, torch.exp2(e.double() - 1) * (1 + 0.5 * f))
        b = scales.long()
        se, sf = (b >> 3) & 15, (b & 7).double() / 8
        sv = torch.where(se == 0, sf * 2.0 ** -6, (1 + sf) * torch.exp2(se.double() - 7))
        return torch.where(neg, -v, v) * sv.repeat_interleave(16, dim=1)
    return values(s["aq"], s["ascale"]) @ values(s["bq"], s["bscale"]).t() / (G * G)


def exact(case, seed):
    s = prepare(case, seed)
    return dict(route=_exact_route, experts=_exact_experts, quantize=_exact_quantize,
                product=_exact_product)[case["op"]](s)
