"""Cases that time the mixture-of-experts operators against their plain form.

The operators are ``mxfp4_moe_route`` (router scores to experts and weights),
``mxfp4_moe_linear`` (each routed token times its expert's MXFP4 weights) and
``mxfp4_moe_ffn`` (the experts' whole gated network, weighted and summed, with
the residual).  ``run`` computes them with elementary torch operations in 32
bits (the router's choice, where scores lie next to one another, in 64), or,
where ``own`` is true, with the library's kernels.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

BLOCK = 32


# ------------------------------------------------------------------- cases
def listed() -> list[dict]:
    return [
        # one decode step of 16 users: sigmoid scores, a bias for balance, 4 of 8 groups
        dict(name="route step of 16", op="route", T=16, E=256, k=8, score="sigmoid", bias=True, groups=8, keep=4, top=2,
             renorm=True, scale=2.5, half=False, hidden=False),
        # a prompt of 8192 tokens: softmax scores of a bf16 gate, renormalised
        dict(name="route prompt of 8192", op="route", T=8192, E=128, k=8, score="softmax", bias=False, groups=1, keep=1,
             top=1, renorm=True, scale=1.0, half=True, hidden=False),
        # the largest batch of tokens, groups and bias, experts that are switched off
        dict(name="route prompt of 16384", op="route", T=16384, E=256, k=8, score="sigmoid", bias=True, groups=8, keep=4,
             top=2, renorm=True, scale=2.5, half=False, hidden=True),
        # one product of a small step, with biases
        dict(name="linear 37 x 4 of 32", op="linear", T=37, E=32, k=4, K=1024, N=5120, bias=True, pad=False),
        # odd sizes, an ordinary number of tokens
        dict(name="linear 1500 x 2 of 9", op="linear", T=1500, E=9, k=2, K=1510, N=1001, bias=True, pad=True),
        # one user: latency, eight experts' weights
        dict(name="ffn 1 x 8 of 128", op="ffn", T=1, E=128, k=8, K=5120, I=1024, N=5120, act="silu", bias=False,
             res=True, pad=False),
        # a small decode batch
        dict(name="ffn 16 x 8 of 128", op="ffn", T=16, E=128, k=8, K=5120, I=1024, N=5120, act="silu", bias=False,
             res=True, pad=False),
        # the largest decode batch of the linears, its tail padding of a captured graph: nearly all experts' weights
        dict(name="ffn 64 x 8 of 128", op="ffn", T=64, E=128, k=8, K=5120, I=1024, N=5120, act="silu", bias=False,
             res=True, pad=True),
        # odd widths, clamped activation and biases
        dict(name="ffn 300 x 3 of 20", op="ffn", T=300, E=20, k=3, K=1000, I=362, N=1000, act="swiglu", bias=True,
             res=False, pad=False),
        # a chunk of prompts: neither the weights nor the products alone bound it
        dict(name="ffn 1024 x 8 of 64", op="ffn", T=1024, E=64, k=8, K=5120, I=1024, N=5120, act="silu", bias=False,
             res=True, pad=False),
        # one expert: a dense gated network of the linears' widths
        dict(name="ffn 2048 dense", op="ffn", T=2048, E=1, k=1, K=5120, I=14336, N=5120, act="gelu", bias=False,
             res=True, pad=False),
        # a prompt of 8192 tokens (the largest M of the linears' prefill)
        dict(name="ffn 8192 x 8 of 64", op="ffn", T=8192, E=64, k=8, K=5120, I=1024, N=5120, act="silu", bias=False,
             res=True, pad=False),
    ]


def _log_int(rng, lo: int, hi: int) -> int:
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng) -> dict:
    op = rng.choice(("route", "linear", "ffn", "ffn"))
    if op == "route":
        E = rng.choice((8, 16, 60, 64, 96, 128, 160, 256, 384, 512))
        groups = rng.choice((1, 1, 4, 8) if E % 8 == 0 else (1, 4))
        keep = rng.randint(1, groups)
        k = rng.randint(1, min(16, E // groups * keep))
        return dict(op=op, T=_log_int(rng, 1, 16384), E=E, k=k, score=rng.choice(("softmax", "sigmoid")),
                    bias=rng.random() < 0.5, groups=groups, keep=keep, top=rng.choice((1, 2)),
                    renorm=rng.random() < 0.7, scale=rng.choice((1.0, 2.5)), half=rng.random() < 0.5,
                    hidden=rng.random() < 0.3)
    E = _log_int(rng, 1, 128)
    k = rng.randint(1, min(8, E))
    if op == "linear":
        return dict(op=op, T=_log_int(rng, 1, 4096), E=E, k=k, K=2 * _log_int(rng, 32, 2560), N=_log_int(rng, 64, 5120),
                    bias=rng.random() < 0.5, pad=rng.random() < 0.5)
    K = 2 * _log_int(rng, 128, 2560)
    return dict(op=op, T=_log_int(rng, 1, 4096), E=E, k=k, K=K, I=2 * _log_int(rng, 32, 1024),
                N=K, act=rng.choice(("silu", "gelu", "swiglu")), bias=rng.random() < 0.5, res=rng.random() < 0.5,
                pad=rng.random() < 0.3)


# ------------------------------------------------------------------ inputs
def _bf16(g, *shape, scale: float = 1.0):
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(torch.bfloat16)


def _weights(g, E: int, N: int, K: int):
    """FP4 codes [E, N, K / 2] and E8M0 scales [E, N, ceil(K / 32)] whose products with unit rows are near 1."""
    codes = torch.randint(0, 256, (E, N, K // 2), device="cuda", generator=g, dtype=torch.uint8)
    at = 127 - round(math.log2(2.9 * math.sqrt(K)))
    scales = torch.randint(at - 1, at + 2, (E, N, -(-K // BLOCK)), device="cuda", generator=g, dtype=torch.uint8)
    return codes, scales


def _packed(codes, scales):
    """The packed weights a program keeps, one matrix per expert (the layout of include/mxfp4.h)."""
    E, N, half = codes.shape
    P, KT = -(-N // 256), -(-half // 128)
    c = torch.zeros(E, P * 256, KT * 128, dtype=torch.uint8, device=codes.device)
    c[:, :N, :half] = codes
    c = c.view(E, P, 2, 128, KT, 8, 16).permute(0, 1, 4, 2, 3, 5, 6)
    i = torch.arange(128, device=c.device)[:, None]
    c = c[:, :, :, :, i, torch.arange(8, device=c.device) ^ (i % 8)]
    s = torch.full((E, P * 256, KT * 8), 127, dtype=torch.uint8, device=codes.device)
    s[:, :N, : scales.shape[2]] = scales
    s = s.view(E, P, 2, 4, 32, KT, 2, 4).permute(0, 1, 5, 2, 6, 4, 3, 7)
    return torch.cat((c.reshape(E, P, KT, 32768), s.reshape(E, P, KT, 2048)), 3).flatten()


def _liked(E: int) -> torch.Tensor:
    """How much more the router likes one expert than another."""
    return 0.6 * torch.sin(torch.arange(E, dtype=torch.float32) * 2.4)


def _routing(g, T: int, E: int, k: int, pad: bool):
    x = torch.randn(T, E, device="cuda", generator=g) + _liked(E).cuda()
    top, ids = x.topk(k, dim=1)
    ids = ids.to(torch.int32)
    if pad:
        ids[T - T // 8:] = -1                           # padding tokens of a captured batch
    return ids, torch.softmax(top, 1)


def prepare(case: dict, seed: int) -> dict:
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 29)
    dev, T, E, k = "cuda", case["T"], case["E"], case["k"]
    if case["op"] == "route":
        x = 1.5 * torch.randn(T, E, device=dev, generator=g) + _liked(E).to(dev)
        if case["hidden"]:                              # every eleventh expert is switched off, and all for token 0
            x[:, ::11] = -math.inf
            x[0] = -math.inf
        return dict(case, logits=x.to(torch.bfloat16) if case["half"] else x,
                    balance=0.05 * torch.randn(E, device=dev, generator=g) if case["bias"] else None,
                    weights=torch.empty(T, k, device=dev), ids=torch.empty(T, k, dtype=torch.int32, device=dev))
    K, N = case["K"], case["N"]
    x = _bf16(g, T, K)
    ids, w = _routing(g, T, E, k, case["pad"])
    if case["op"] == "linear":
        codes, scales = _weights(g, E, N, K)
        return dict(case, x=x, ids=ids, codes=codes, scales=scales, packed=_packed(codes, scales),
                    b=_bf16(g, E, N, scale=0.2) if case["bias"] else None,
                    out=torch.empty(T, k, N, dtype=torch.bfloat16, device=dev))
    I = case["I"]
    c1, s1 = _weights(g, E, 2 * I, K)                   # row 2 i: gate i, row 2 i + 1: up i
    c2, s2 = _weights(g, E, N, I)
    return dict(case, x=x, ids=ids, weights=w, c1=c1, s1=s1, c2=c2, s2=s2, p1=_packed(c1, s1), p2=_packed(c2, s2),
                b1=_bf16(g, E, 2 * I, scale=0.2) if case["bias"] else None,
                b2=_bf16(g, E, N, scale=0.2) if case["bias"] else None,
                residual=_bf16(g, T, N) if case["res"] else None,
                out=torch.empty(T, N, dtype=torch.bfloat16, device=dev))


# -------------------------------------------------------------- plain forms
def _route_plain(st: dict):
    T, E, k, G = st["T"], st["E"], st["k"], st["groups"]
    x = st["logits"].double()                           # the choice falls between near values: 64 bits
    x = torch.where(x.isnan(), -math.inf, x)
    if st["score"] == "softmax":
        m = x.amax(1, keepdim=True)
        p = torch.where(x == m, 1.0, torch.exp(x - m)) * (x > -math.inf)
        s = p / p.sum(1, keepdim=True).clamp(min=1.0)
    else:
        s = 1 / (1 + torch.exp(-x))
    c = x if st["balance"] is None else torch.where(x > -math.inf, s + st["balance"].double(), -math.inf)
    if G > 1:
        v = s if st["balance"] is None and st["top"] == 2 else c
        v = torch.where(x > -math.inf, v, -math.inf).view(T, G, E // G)
        best = v.sort(dim=2, descending=True)[0][..., : st["top"]]
        score = torch.where(best > -math.inf, best, 0.0).sum(2)
        score = torch.where(best[..., 0] > -math.inf, score, -math.inf)
        kept = score.sort(dim=1, descending=True, stable=True)[1][:, : st["keep"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, kept, True)
        c = torch.where(keep.repeat_interleave(E // G, 1), c, -math.inf)
    c, at = c.sort(dim=1, descending=True, stable=True)
    at, found = at[:, :k], c[:, :k] > -math.inf
    w = torch.where(found, s.gather(1, at), 0.0)
    if st["renorm"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    return (st["scale"] * w).float(), torch.where(found, at, -1).to(torch.int32)


def _values(codes):
    """The values of packed E2M1 codes: [.., n] bytes to [.., 2 n] fp32."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    grid = torch.cat((grid, -grid))
    both = torch.stack((grid.repeat(16), grid.repeat_interleave(16)), 1)
    return both[codes.int()].flatten(-2)


def _matrix(codes, scales):
    """The weights that codes and scales stand for, fp32."""
    w = _values(codes)
    return w.mul_(torch.exp2(scales.float() - 127).repeat_interleave(BLOCK, -1)[..., : w.shape[-1]])


def _rounded(x):
    """x in MXFP4 per 1x32, as the values that it stands for."""
    n = x.shape[-1]
    b = torch.nn.functional.pad(x, (0, -n % BLOCK)).unflatten(-1, (-1, BLOCK))
    e = torch.frexp(b.abs().amax(-1, keepdim=True))[1].clamp(min=-124) - 3
    a = torch.ldexp(b, -e)
    step = torch.where(a.abs() < 2, 0.5, torch.where(a.abs() < 4, 1.0, 2.0))
    q = (torch.round(a / step) * step).clamp(-6, 6)
    return torch.ldexp(q, e).flatten(-2)[..., :n]


def _products(x, ids, codes, scales, bias):
    """x [P, K] fp32 times the transposed weights of each row's expert, plus its bias; zeros where there is none."""
    P, E = x.shape[0], codes.shape[0]
    live = ids >= 0
    e = torch.where(live, ids, E).long()
    if P <= E:                                          # few rows: their experts' weights row by row
        some = e.clamp(max=E - 1)
        y = torch.matmul(_matrix(codes[some], scales[some]), x[:, :, None])[..., 0]
    else:                                               # the rows of each expert side by side, one batched product
        order = torch.argsort(e, stable=True)
        count = torch.bincount(e, minlength=E + 1)
        slot = torch.empty_like(order)
        slot[order] = torch.arange(P, device=x.device) - (count.cumsum(0) - count)[e[order]]
        most = int(count[:E].max())
        at = torch.where(live, e * most + slot, E * most)           # (a last row takes what has no expert)
        rows = torch.zeros(E * most + 1, x.shape[1], device=x.device)
        rows[at] = x
        y = torch.matmul(rows[:-1].view(E, most, -1), _matrix(codes, scales).transpose(1, 2)).flatten(0, 1)
        y = y[at.clamp(max=E * most - 1)]
    if bias is not None:
        y = y + bias.float()[e.clamp(max=E - 1)]
    return torch.where(live[:, None], y, 0.0)


def _gated(z, act: str):
    gate, up = z[..., 0::2], z[..., 1::2]
    if act == "silu":
        return gate / (1 + torch.exp(-gate)) * up
    if act == "gelu":
        return 0.5 * gate * (1 + torch.tanh(math.sqrt(2 / math.pi) * (gate + 0.044715 * gate ** 3))) * up
    gate, up = gate.clamp(max=7.0), up.clamp(-7.0, 7.0)
    return gate / (1 + torch.exp(-1.702 * gate)) * (up + 1)


def _linear_plain(st: dict):
    T, k = st["T"], st["k"]
    x = _rounded(st["x"].float()).repeat_interleave(k, 0)
    y = _products(x, st["ids"].flatten(), st["codes"], st["scales"], st["b"])
    return y.to(torch.bfloat16).view(T, k, -1)


def _ffn_plain(st: dict):
    T, k = st["T"], st["k"]
    ids = st["ids"].flatten()
    x = _rounded(st["x"].float()).repeat_interleave(k, 0)
    h = _rounded(_gated(_products(x, ids, st["c1"], st["s1"], st["b1"]), st["act"]))
    y = _products(h, ids, st["c2"], st["s2"], st["b2"])
    y = (y.view(T, k, -1) * st["weights"][..., None]).sum(1)
    return (y if st["residual"] is None else y + st["residual"].float()).to(torch.bfloat16)


# ----------------------------------------------------------------- kernels
def _scratch(st: dict, n: int):
    """The caller's workspace, kept as for the GEMMs."""
    if "workspace" not in st:
        st["workspace"] = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    return st["workspace"]


def _route_own(st: dict):
    from mxfp4_quantized_gemm_gb300 import capi
    x, T, E = st["logits"], st["T"], st["E"]
    capi.mxfp4_moe_route(x, capi.DTYPE_BF16 if st["half"] else capi.DTYPE_F32, x.stride(0), st["balance"], T, E, st["k"],
                         capi.MOE_SOFTMAX if st["score"] == "softmax" else capi.MOE_SIGMOID, st["groups"], st["keep"],
                         st["top"], st["renorm"], st["scale"], st["weights"], st["ids"])
    return st["weights"], st["ids"]


def _linear_own(st: dict):
    from mxfp4_quantized_gemm_gb300 import capi
    T, k, E, N, K = st["T"], st["k"], st["E"], st["N"], st["K"]
    ws = _scratch(st, capi.mxfp4_moe_linear_workspace_bytes(T, k, E, N, K))
    capi.mxfp4_moe_linear(st["x"], st["x"].stride(0), st["ids"], st["packed"], st["b"], st["out"], N, T, k, E, N, K, ws,
                          ws.numel())
    return st["out"]


def _ffn_own(st: dict):
    from mxfp4_quantized_gemm_gb300 import capi
    T, k, E, K, I, N = st["T"], st["k"], st["E"], st["K"], st["I"], st["N"]
    act = {"silu": capi.MOE_SILU, "gelu": capi.MOE_GELU_TANH, "swiglu": capi.MOE_SWIGLU_CLAMP}[st["act"]]
    ws = _scratch(st, capi.mxfp4_moe_ffn_workspace_bytes(T, k, E, K, I, N))
    capi.mxfp4_moe_ffn(st["x"], st["x"].stride(0), st["ids"], st["weights"], st["p1"], st["b1"], st["p2"], st["b2"],
                       st["residual"], N, st["out"], N, T, k, E, K, I, N, act, 1.702, 7.0, ws, ws.numel())
    return st["out"]


def run(state: dict):
    forms = {"route": (_route_plain, _route_own), "linear": (_linear_plain, _linear_own),
             "ffn": (_ffn_plain, _ffn_own)}[state["op"]]
    return forms[1 if own else 0](state)


# -------------------------------------------------------------------- work
def _active(T: int, E: int, k: int) -> float:
    """Experts that T tokens reach, on average, where the router likes some more than others."""
    if T * k >= 16 * E:
        return float(E)
    g = np.random.default_rng(0)
    n = max(1, 2048 // T)
    x = g.standard_normal((n, T, E)) + _liked(E).numpy()
    at = np.argpartition(-x, k - 1, axis=2)[..., :k].reshape(n, -1)
    return float(np.mean([len(np.unique(r)) for r in at]))


def _weight_bytes(N: int, K: int) -> int:
    return N * K // 2 + N * -(-K // BLOCK)


def work(case: dict) -> dict:
    T, E, k = case["T"], case["E"], case["k"]
    if case["op"] == "route":
        return {"bytes": T * E * (2 if case["half"] else 4) + T * k * 8 + (4 * E if case["bias"] else 0),
                "flops": T * E * (5 + k)}
    live = T - T // 8 if case["pad"] else T
    K, N = case["K"], case["N"]
    some = _active(live, E, k)
    if case["op"] == "linear":
        return {"bytes": some * (_weight_bytes(N, K) + (2 * N if case["bias"] else 0)) + T * (2 * K + 4 * k + 2 * k * N),
                "flops": 2 * live * k * N * K}
    I = case["I"]
    return {"bytes": some * (_weight_bytes(2 * I, K) + _weight_bytes(N, I) + (4 * I + 2 * N if case["bias"] else 0))
            + T * (2 * K + 8 * k + (4 if case["res"] else 2) * N),
            "flops": 2 * live * k * (2 * I * K + I * N)}


# ------------------------------------------------------------ 64-bit values
def _exact_rounded(x):
    """MXFP4 of x [rows, n] in 64 bits, by the distances to the values that there are."""
    rows, n = x.shape
    b = torch.zeros(rows, -(-n // BLOCK) * BLOCK, dtype=torch.float64, device=x.device)
    b[:, :n] = x
    b = b.view(rows, -1, BLOCK)
    most = b.abs().amax(2, keepdim=True)
    low = torch.floor(torch.log2(torch.where(most > 0, most, 1.0)))
    low = low + (torch.exp2(low + 1) <= most).double() - (torch.exp2(low) > most).double()
    unit = torch.exp2(torch.where(most > 0, low, -126.0).clamp(min=-125.0) - 2)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    a = (b / unit).abs().contiguous()
    up, down = torch.bucketize(a, mid, right=True), torch.bucketize(a, mid)
    code = torch.where((up != down) & (up % 2 == 1), down, up)          # halfway: the even code
    return (torch.sign(b) * grid[code] * unit).view(rows, -1)[:, :n]


def _exact_matrix(codes, scales, K: int):
    """One expert's weights in 64 bits."""
    v = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=codes.device)
    w = torch.empty(codes.shape[0], K, dtype=torch.float64, device=codes.device)
    for half, nib in ((0, codes & 15), (1, codes >> 4)):
        w[:, half::2] = v[(nib & 7).long()] * (1 - 2 * (nib >> 3).double())
    for b in range(scales.shape[1]):
        w[:, b * BLOCK:(b + 1) * BLOCK] *= torch.exp2(scales[:, b:b + 1].double() - 127)
    return w


def _exact_route(st: dict):
    x = st["logits"].double()
    T, E, k, G = st["T"], st["E"], st["k"], st["groups"]
    on = x > -math.inf
    s = torch.where(on, torch.softmax(torch.where(on.any(1, keepdim=True), x, 0.0), 1)
                    if st["score"] == "softmax" else torch.sigmoid(x), 0.0)
    c = s if st["balance"] is None else s + st["balance"].double()
    c = torch.where(on, c, -math.inf)
    if G > 1:
        v = torch.topk(c.view(T, G, -1), min(st["top"], E // G), 2)[0]
        score = torch.where(v[..., 0] == -math.inf, -math.inf, torch.where(v == -math.inf, 0.0, v).sum(2))
        last = score.sort(dim=1, descending=True)[0][:, st["keep"] - 1, None]
        c = c.view(T, G, -1).masked_fill((score < last)[..., None], -math.inf).view(T, E)
    top, at = torch.topk(c, k, 1)
    w = torch.where(top > -math.inf, s.gather(1, at), 0.0)
    if st["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    return st["scale"] * w, None


def exact(case: dict, seed: int):
    """The operators' definitions, expert by expert, in 64 bits."""
    st = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(st)
    T, k, K, N = case["T"], case["k"], case["K"], case["N"]
    ids = st["ids"].long()
    x = _exact_rounded(st["x"].double())
    y = torch.zeros(T, k, N, dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        t, j = (ids == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        if case["op"] == "linear":
            y[t, j] = x[t] @ _exact_matrix(st["codes"][e], st["scales"][e], K).T + (st["b"][e].double() if case["bias"] else 0)
            continue
        z = x[t] @ _exact_matrix(st["c1"][e], st["s1"][e], K).T + (st["b1"][e].double() if case["bias"] else 0)
        gate, up = z[:, ::2], z[:, 1::2]
        if case["act"] == "silu":
            h = gate * torch.sigmoid(gate) * up
        elif case["act"] == "gelu":
            h = gate * up * torch.sigmoid(math.sqrt(8 / math.pi) * (gate + 0.044715 * gate ** 3))
        else:
            gate = gate.clamp(max=7.0)
            h = gate * torch.sigmoid(1.702 * gate) * (up.clamp(-7.0, 7.0) + 1)
        y[t, j] = _exact_rounded(h) @ _exact_matrix(st["c2"][e], st["s2"][e], case["I"]).T + (
            st["b2"][e].double() if case["bias"] else 0)
    if case["op"] == "linear":
        return y
    y = (y * torch.where(ids >= 0, st["weights"].double(), 0.0)[..., None]).sum(1)
    return y + st["residual"].double() if case["res"] else y
