"""Cases that time the latent-attention operators against their plain form.

The operators are ``mxfp4_mla_store`` (the latent's RMSNorm, the rotation of
the shared key and of the queries, and the write into the paged cache),
``mxfp4_mla_decode`` (absorbed attention over the paged latent cache) and
``mxfp4_mla_prefill`` (expanded attention of ragged prompts).  ``run`` computes
them with elementary torch operations in 32 bits, or, where ``own`` is true,
with the library's kernels.
"""

from __future__ import annotations

import math

import torch

own = False

L, R = 512, 64          # latent and rotated elements of a cache row
EPS = 1e-6


# ------------------------------------------------------------------- cases
def listed() -> list[dict]:
    return [
        # one decode step of a small batch: four new tokens enter the cache
        dict(name="store step of 4", op="store", T=4, H=64, page=64, interleaved=True, pad=False),
        # a decode step of a graph-captured batch whose tail is padding
        dict(name="store step of 96", op="store", T=96, H=64, page=64, interleaved=True, pad=True),
        # a prompt of 8192 tokens enters the cache (the largest M of the linears' prefill)
        dict(name="store prompt of 8192", op="store", T=8192, H=64, page=64, interleaved=False, pad=False),
        # one user, a short chat: latency
        dict(name="decode 1 x 333", op="decode", S=1, q_len=1, H=64, page=64, longest=333, ragged=False),
        # one user, a long document: the sequence is all there is to split
        dict(name="decode 1 x 131072", op="decode", S=1, q_len=1, H=64, page=64, longest=131072, ragged=False),
        # an ordinary batch with ragged lengths
        dict(name="decode 16 x 4096", op="decode", S=16, q_len=1, H=64, page=64, longest=4096, ragged=True),
        # the largest decode batch of the linears, long ragged contexts
        dict(name="decode 64 x 8192", op="decode", S=64, q_len=1, H=64, page=64, longest=8192, ragged=True),
        # a shard of 16 heads, small pages, three tokens a step (speculation)
        dict(name="decode 32 x 3001 q3 h16", op="decode", S=32, q_len=3, H=16, page=16, longest=3001, ragged=True),
        # two tokens a step of all heads: two blocks of query rows share a sequence
        dict(name="decode 24 x 6000 q2", op="decode", S=24, q_len=2, H=64, page=128, longest=6000, ragged=True),
        # one short prompt
        dict(name="prefill 1 x 77", op="prefill", S=1, H=64, dn=192, dv=256, tokens=77, past=0, causal=True),
        # a batch of ragged prompts, some with earlier context
        dict(name="prefill 6 ragged", op="prefill", S=6, H=64, dn=192, dv=256, tokens=2500, past=3000, causal=True),
        # one prompt of 8192 tokens
        dict(name="prefill 1 x 8192", op="prefill", S=1, H=64, dn=192, dv=256, tokens=8192, past=0, causal=True),
    ]


def _log_int(rng, lo: int, hi: int) -> int:
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng) -> dict:
    op = rng.choice(("store", "decode", "decode", "prefill", "prefill"))
    if op == "store":
        return dict(op=op, T=_log_int(rng, 1, 8192), H=rng.choice((8, 16, 32, 64)), page=rng.choice((16, 32, 64, 128)),
                    interleaved=rng.random() < 0.5, pad=rng.random() < 0.5)
    if op == "decode":
        S = _log_int(rng, 1, 64)
        longest = _log_int(rng, 1, min(131072, 524288 // S))
        return dict(op=op, S=S, q_len=rng.randint(1, 4), H=rng.choice((8, 16, 32, 64)),
                    page=rng.choice((16, 32, 64, 128)), longest=longest, ragged=rng.random() < 0.7)
    S = rng.randint(1, 12)
    tokens = max(S, _log_int(rng, 1, 6000))
    return dict(op=op, S=S, H=rng.choice((8, 16, 32, 64)), dn=rng.choice((64, 128, 192)),
                dv=rng.choice((64, 128, 192, 256)), tokens=tokens, past=rng.choice((0, 0, _log_int(rng, 1, 2000))),
                causal=rng.random() < 0.8)


def _lengths(case: dict) -> list[int]:
    """Lengths of a case's sequences, the same for every seed: the longest,
    and where they are ragged, the others spread evenly below it."""
    S, n = case["S"], case["longest"]
    if not case["ragged"]:
        return [n] * S
    return [max(1, n - (n * 7 * i // (8 * S)) - (i * i) % 5) for i in range(S)]


def _prompts(case: dict) -> tuple[list[int], list[int]]:
    """New tokens and earlier tokens of each prompt of a prefill case."""
    S, T, past = case["S"], case["tokens"], case["past"]
    w = [1 + (3 * i) % 5 for i in range(S)]
    new = [max(1, T * x // sum(w)) for x in w]
    new[0] = max(1, T - sum(new[1:]))
    wp = [(2 * i) % 3 for i in range(S)]
    old = [past * x // max(1, sum(wp)) for x in wp]
    if S == 1:
        old = [past]
    return new, old


# ------------------------------------------------------------------ inputs
def _bf16(g, *shape, scale: float = 1.0):
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(torch.bfloat16)


def prepare(case: dict, seed: int) -> dict:
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)
    dev = "cuda"
    if case["op"] == "store":
        T, H, page = case["T"], case["H"], case["page"]
        most = 16384
        freq = 10000.0 ** (-torch.arange(0, R, 2, device=dev, dtype=torch.float64) / R)
        ang = torch.arange(most, device=dev, dtype=torch.float64)[:, None] * freq
        pages = -(-T // page) + 2                      # page 0 takes no token
        slots = torch.randperm((pages - 1) * page, device=dev, generator=g)[:T] + page
        if case["pad"]:
            slots[T - T // 8:] = -1                    # padding tokens of a captured batch
        return dict(op="store", kv=_bf16(g, T, L + R), q=_bf16(g, T, H, 192 + R)[..., 192:],
                    gamma=(1 + 0.2 * torch.randn(L, device=dev, generator=g)).to(torch.bfloat16),
                    cos_sin=torch.cat((ang.cos(), ang.sin()), 1).float(),
                    positions=torch.randint(0, most, (T,), device=dev, generator=g), slots=slots,
                    cache=_bf16(g, pages, page, L + R), q_out=torch.empty(T, H, R, dtype=torch.bfloat16, device=dev),
                    interleaved=case["interleaved"])
    if case["op"] == "decode":
        S, H, page, q_len = case["S"], case["H"], case["page"], case["q_len"]
        lens = _lengths(case)
        need = [-(-n // page) for n in lens]
        total, width = sum(need), max(need)
        order = torch.randperm(total, device=dev, generator=g).to(torch.int32)
        at = torch.tensor([0] + need[:-1], device=dev).cumsum(0)
        col = torch.arange(width, device=dev)
        idx = at[:, None] + col
        used = col < torch.tensor(need, device=dev)[:, None]
        table = torch.where(used, order[idx.clamp(max=total - 1)], -1).to(torch.int32)
        T = S * q_len
        return dict(op="decode", q_lat=_bf16(g, H, T, L), q_rope=_bf16(g, T, H, R),
                    cache=_bf16(g, total, page, L + R), table=table,
                    lens=torch.tensor(lens, dtype=torch.int32, device=dev), q_len=q_len, scale=(192 + R) ** -0.5,
                    out=torch.empty(H, T, L, dtype=torch.bfloat16, device=dev),
                    lse=torch.empty(T, H, dtype=torch.float32, device=dev))
    new, old = _prompts(case)
    H, dn, dv = case["H"], case["dn"], case["dv"]
    T, N = sum(new), sum(new) + sum(old)
    cu_q = torch.tensor([0] + new, device=dev).cumsum(0).to(torch.int32)
    cu_k = torch.tensor([0] + [a + b for a, b in zip(new, old)], device=dev).cumsum(0).to(torch.int32)
    q = _bf16(g, T, H, dn + R, scale=1.5)
    kv = _bf16(g, N, H, dn + dv)                       # the expanding projection's output, read in place
    return dict(op="prefill", q_nope=q[..., :dn], q_rope=q[..., dn:], k_nope=kv[..., :dn], v=kv[..., dn:],
                k_rope=_bf16(g, N, R), cu_q=cu_q, cu_k=cu_k, causal=case["causal"], scale=(dn + R) ** -0.5,
                out=torch.empty(T, H, dv, dtype=torch.bfloat16, device=dev),
                lse=torch.empty(T, H, dtype=torch.float32, device=dev))


# -------------------------------------------------------------- plain forms
def _rotate(x, cs, interleaved: bool):
    """x [..., R] turned by the angles of cs [..., R] = (cos | sin)."""
    c, s = cs[..., : R // 2], cs[..., R // 2:]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    a, b = x[..., : R // 2], x[..., R // 2:]
    return torch.cat((a * c - b * s, b * c + a * s), -1)


def _store_plain(st: dict):
    kv, cs = st["kv"].float(), st["cos_sin"][st["positions"]]
    lat = kv[:, :L]
    y = lat / torch.sqrt((lat * lat).mean(1, keepdim=True) + EPS) * st["gamma"].float()
    row = torch.cat((y, _rotate(kv[:, L:], cs, st["interleaved"])), 1).to(torch.bfloat16)
    flat = st["cache"].view(-1, L + R)
    keep = st["slots"] >= 0
    # padding tokens write row 0, which no token uses, with what it holds
    flat[torch.where(keep, st["slots"], 0)] = torch.where(keep[:, None], row, flat[:1])
    q = _rotate(st["q"].float(), cs[:, None], st["interleaved"]).to(torch.bfloat16)
    return st["cache"], q


def _softmax_parts(s):
    """exp(s - max), its sum and the max of the last axis; an empty row has sum 0."""
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(s - m)
    return p, p.sum(-1, keepdim=True), m


def _decode_plain(st: dict):
    H, T, _ = st["q_lat"].shape
    S, q_len = st["lens"].shape[0], st["q_len"]
    rows = st["cache"][st["table"].clamp(min=0).long()].flatten(1, 2).float()             # [S, N, L + R]
    N = rows.shape[1]
    at = torch.arange(N, device=rows.device)
    rows = torch.where((at < st["lens"][:, None])[..., None], rows, 0.0)
    q = torch.cat((st["q_lat"].transpose(0, 1), st["q_rope"]), -1).float().view(S, q_len * H, L + R)
    seen = st["lens"][:, None] - q_len + 1 + torch.arange(q_len, device=at.device)        # [S, q_len]
    seen = seen[:, :, None].expand(S, q_len, H).reshape(S, q_len * H, 1)
    s = torch.matmul(q, rows.transpose(1, 2)) * st["scale"]
    p, l, m = _softmax_parts(torch.where(at < seen, s, -math.inf))
    o = torch.matmul(p, rows[..., :L]) / torch.where(l > 0, l, 1.0)
    out = o.view(T, H, L).transpose(0, 1).to(torch.bfloat16)
    return out.contiguous(), (m + torch.log(l)).view(T, H)


def _prefill_plain(st: dict):
    cu_q, cu_k = st["cu_q"].long(), st["cu_k"].long()
    T, N = st["q_nope"].shape[0], st["v"].shape[0]
    t, j = torch.arange(T, device=cu_q.device), torch.arange(N, device=cu_q.device)
    sq, sk = (torch.searchsorted(c, x, right=True) - 1 for c, x in ((cu_q, t), (cu_k, j)))
    see = sq[:, None] == sk
    if st["causal"]:
        last = t - cu_q[sq] + (cu_k[sq + 1] - cu_k[sq]) - (cu_q[sq + 1] - cu_q[sq])       # last visible key
        see = see & ((j - cu_k[sk]) <= last[:, None])
    q = torch.cat((st["q_nope"], st["q_rope"]), -1).float().transpose(0, 1)               # [H, T, dn + R]
    kr = st["k_rope"][:, None].expand(N, st["k_nope"].shape[1], R)
    k = torch.cat((st["k_nope"], kr), -1).float().permute(1, 2, 0)                        # [H, dn + R, N]
    s = torch.matmul(q, k).mul_(st["scale"]).masked_fill_(~see, -math.inf)
    p, l, m = _softmax_parts(s)
    del s
    o = torch.matmul(p, st["v"].float().transpose(0, 1)) / torch.where(l > 0, l, 1.0)
    return o.transpose(0, 1).to(torch.bfloat16).contiguous(), (m + torch.log(l))[..., 0].transpose(0, 1).contiguous()


# ----------------------------------------------------------------- kernels
def _store_own(st: dict):
    from mxfp4_quantized_gemm_gb300 import capi
    kv, q, qo, cache = st["kv"], st["q"], st["q_out"], st["cache"]
    T, H, _ = q.shape
    capi.mxfp4_mla_store(kv, kv.stride(0), st["gamma"], EPS, q, q.stride(0), q.stride(1), qo, qo.stride(0),
                         qo.stride(1), H, st["cos_sin"], st["cos_sin"].shape[0], st["positions"], st["slots"], cache,
                         cache.stride(0), cache.shape[1], cache.shape[0], T, L, R, st["interleaved"])
    return cache, qo


def _decode_own(st: dict):
    from mxfp4_quantized_gemm_gb300 import capi
    ql, qr, cache, table, out = st["q_lat"], st["q_rope"], st["cache"], st["table"], st["out"]
    H, S, q_len = ql.shape[0], st["lens"].shape[0], st["q_len"]
    if "workspace" not in st:                          # kept by the caller, as for the GEMMs
        n = capi.mxfp4_mla_decode_workspace_bytes(S, q_len, H, L, table.shape[1] * cache.shape[1])
        st["workspace"] = torch.empty(max(n, 1), dtype=torch.uint8, device=ql.device)
    ws = st["workspace"]
    capi.mxfp4_mla_decode(ql, ql.stride(1), ql.stride(0), qr, qr.stride(0), qr.stride(1), cache, cache.stride(0),
                          cache.shape[1], cache.shape[0], table, table.stride(0), table.shape[1], st["lens"], out,
                          out.stride(1), out.stride(0), st["lse"], S, q_len, H, L, R, st["scale"], ws, ws.numel())
    return out, st["lse"]


def _prefill_own(st: dict):
    from mxfp4_quantized_gemm_gb300 import capi
    qn, qr, kn, kr, v, out = st["q_nope"], st["q_rope"], st["k_nope"], st["k_rope"], st["v"], st["out"]
    capi.mxfp4_mla_prefill(qn, qn.stride(0), qn.stride(1), qr, qr.stride(0), qr.stride(1), kn, kn.stride(0),
                           kn.stride(1), kr, kr.stride(0), v, v.stride(0), v.stride(1), st["cu_q"], st["cu_k"],
                           st["cu_q"].shape[0] - 1, out, out.stride(0), out.stride(1), st["lse"], qn.shape[0],
                           v.shape[0], qn.shape[1], qn.shape[2], R, v.shape[2], st["scale"], st["causal"])
    return out, st["lse"]


def run(state: dict):
    forms = {"store": (_store_plain, _store_own), "decode": (_decode_plain, _decode_own),
             "prefill": (_prefill_plain, _prefill_own)}[state["op"]]
    return forms[1 if own else 0](state)


# -------------------------------------------------------------------- work
def work(case: dict) -> dict:
    if case["op"] == "store":
        T, H = case["T"], case["H"]
        kept = T - T // 8 if case["pad"] else T
        return {"bytes": T * (L + R) * 2 + kept * (L + R) * 2 + 2 * T * H * R * 2 + T * (R * 4 + 16) + L * 2,
                "flops": T * (4 * L + 3 * R + 3 * H * R)}
    if case["op"] == "decode":
        lens, rows = _lengths(case), case["H"] * case["q_len"]
        return {"bytes": sum(lens) * (L + R) * 2 + case["S"] * (rows * ((L + R) * 2 + L * 2 + 4) + 4)
                + sum(-(-n // case["page"]) for n in lens) * 4, "flops": 2 * rows * sum(lens) * (2 * L + R)}
    new, old = _prompts(case)
    H, dn, dv = case["H"], case["dn"], case["dv"]
    if case["causal"]:
        pairs = sum(a * b + a * (a + 1) // 2 for a, b in zip(new, old))
    else:
        pairs = sum(a * (a + b) for a, b in zip(new, old))
    T, N = sum(new), sum(new) + sum(old)
    return {"bytes": 2 * (T * H * (dn + R + dv) + N * H * (dn + dv) + N * R) + 4 * T * H,
            "flops": 2 * H * pairs * (dn + R + dv)}


# ------------------------------------------------------------ 64-bit values
def exact(case: dict, seed: int):
    """The operators' definitions, sequence by sequence, in 64 bits."""
    st = prepare(case, seed)
    if case["op"] == "store":
        x, cs = st["kv"].double(), st["cos_sin"].double().index_select(0, st["positions"])
        z = torch.complex(cs[:, : R // 2].contiguous(), cs[:, R // 2:].contiguous())

        def turn(u, w):
            if case["interleaved"]:
                return torch.view_as_real(torch.view_as_complex(u.unflatten(-1, (R // 2, 2)).contiguous()) * w).flatten(-2)
            c = torch.complex(u[..., : R // 2].contiguous(), u[..., R // 2:].contiguous()) * w
            return torch.cat((c.real, c.imag), -1)

        rms = (x[:, :L].square().sum(1) / L + EPS).rsqrt()
        cache = st["cache"].double()
        flat = cache.view(-1, L + R)
        keep = (st["slots"] >= 0).nonzero()[:, 0]
        where = st["slots"][keep]
        flat[where, :L] = (x[:, :L] * rms[:, None] * st["gamma"].double())[keep]
        flat[where, L:] = turn(x[:, L:], z)[keep]
        return cache, turn(st["q"].double(), z[:, None])
    if case["op"] == "decode":
        H, T, q_len = st["q_lat"].shape[0], st["q_lat"].shape[1], st["q_len"]
        out = torch.zeros(H, T, L, dtype=torch.float64, device="cuda")
        lse = torch.full((T, H), -math.inf, dtype=torch.float64, device="cuda")
        flat = st["cache"].view(-1, L + R)
        page = case["page"]
        for b, n in enumerate(_lengths(case)):
            j = torch.arange(n, device="cuda")
            rows = flat[st["table"][b].long()[j // page] * page + j % page].double()
            for i in range(q_len):
                t, see = b * q_len + i, n - q_len + 1 + i
                if see <= 0:
                    continue
                q = torch.cat((st["q_lat"][:, t], st["q_rope"][t]), 1).double()
                s = st["scale"] * (q @ rows[:see].T)
                lse[t] = torch.logsumexp(s, 1)
                out[:, t] = torch.softmax(s, 1) @ rows[:see, :L]
        return out, lse
    new, old = _prompts(case)
    H, dv = case["H"], case["dv"]
    out = torch.zeros(sum(new), H, dv, dtype=torch.float64, device="cuda")
    lse = torch.full((sum(new), H), -math.inf, dtype=torch.float64, device="cuda")
    q0 = k0 = 0
    for a, b in zip(new, old):
        n = a + b
        kr = st["k_rope"][k0:k0 + n].double()
        hidden = torch.ones(a, n, dtype=torch.bool, device="cuda").triu(b + 1) if case["causal"] else None
        for h in range(H):
            s = st["q_nope"][q0:q0 + a, h].double() @ st["k_nope"][k0:k0 + n, h].double().T
            s = (s + st["q_rope"][q0:q0 + a, h].double() @ kr.T) * st["scale"]
            if hidden is not None:
                s.masked_fill_(hidden, -math.inf)
            lse[q0:q0 + a, h] = torch.logsumexp(s, 1)
            out[q0:q0 + a, h] = torch.softmax(s, 1) @ st["v"][k0:k0 + n, h].double()
        q0, k0 = q0 + a, k0 + n
    return out, lse
