"""The routed INT4 linear layers as measured workloads: every row of the input picks, beside the
INT4 weight format they share, a second selector of its own -- a low-rank adapter, or an expert.

Operators
  lora     C = A . dequant(W) + s_a (A . La_a^T) . Lb_a^T, a = the row's adapter (or none)
  sort     tokens sorted by expert: row offsets, both row maps and the gathered rows
  experts  the experts' INT4 products on the sorted rows
  combine  the sorted rows back at their tokens, weighted and summed
  grad     the gradients of combine (rows and weights) and of sort

A case is a dict of plain values. `own` false computes a case with elementary torch operations in
32 bits, `own` true through the library's entry points; both read the same state.
"""
import math

import torch

own = False

_T = {"f16": torch.float16, "bf16": torch.bfloat16}

# The work of the largest listed cases, which no drawn case passes.
_MAX_LORA = 2048 * 4096 * 28672
_MAX_WEIGHTS = 8 * 4096 * 14336
_MAX_EXPERTS = 4096 * 4096 * 14336
_MAX_ROWS = 65536 * 4096


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one token of one user's adapter through a fused qkv projection (the 8B decode layer)
        {"name": "lora one token", "op": "lora", "M": 1, "K": 4096, "N": 6144, "group": 128, "sym": 0, "dtype": "f16",
         "rank": 16, "adapters": 8, "rows": "each"},
        # a decode batch, every request with an adapter of its own, two of the rows with none
        {"name": "lora decode batch", "op": "lora", "M": 16, "K": 8192, "N": 10240, "group": 128, "sym": 0,
         "dtype": "bf16", "rank": 32, "adapters": 32, "rows": "each"},
        # a chunk of prompt tokens of a few requests through the gate and up projection
        {"name": "lora prompt chunk", "op": "lora", "M": 2048, "K": 4096, "N": 28672, "group": 128, "sym": 0,
         "dtype": "bf16", "rank": 64, "adapters": 4, "rows": "runs"},
        # routing of a decode batch over many small experts, two padded tokens
        {"name": "sort decode batch", "op": "sort", "T": 16, "k": 4, "E": 64, "H": 2048, "dtype": "f16", "skew": 0.5,
         "pad": 2},
        # routing of a long prompt over many experts
        {"name": "sort long prompt", "op": "sort", "T": 8192, "k": 8, "E": 128, "H": 4096, "dtype": "bf16",
         "skew": 0.5, "pad": 0},
        # one token through two of eight large experts (gate projection)
        {"name": "experts one token", "op": "experts", "T": 1, "k": 2, "E": 8, "K": 4096, "N": 14336, "group": 128,
         "sym": 0, "dtype": "bf16", "skew": 0.0, "pad": 0},
        # an odd-sized batch over many small experts, in small groups
        {"name": "experts batch", "op": "experts", "T": 77, "k": 4, "E": 64, "K": 2048, "N": 1408, "group": 32,
         "sym": 1, "dtype": "f16", "skew": 0.5, "pad": 3},
        # a prompt chunk over eight large experts
        {"name": "experts prompt chunk", "op": "experts", "T": 2048, "k": 2, "E": 8, "K": 4096, "N": 14336,
         "group": 128, "sym": 0, "dtype": "bf16", "skew": 0.5, "pad": 0},
        # one token's expert outputs back
        {"name": "combine one token", "op": "combine", "T": 1, "k": 8, "E": 64, "H": 4096, "dtype": "bf16",
         "skew": 0.0, "pad": 0},
        # a prompt chunk's outputs back, with an odd number of tokens
        {"name": "combine prompt chunk", "op": "combine", "T": 4095, "k": 8, "E": 64, "H": 4096, "dtype": "f16",
         "skew": 0.5, "pad": 31},
        # a small training step's way back through the routing, many choices of narrow rows
        {"name": "grad small step", "op": "grad", "T": 129, "k": 6, "E": 64, "H": 1032, "dtype": "f16", "skew": 0.5,
         "pad": 1},
        # a training step's way back through the routing
        {"name": "grad training step", "op": "grad", "T": 8192, "k": 4, "E": 32, "H": 4096, "dtype": "bf16",
         "skew": 0.5, "pad": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lora", "lora", "experts", "experts", "sort", "combine", "grad"])
    dtype = rng.choice(["f16", "bf16"])
    fmt = {"group": rng.choice([32, 64, 128, 128]), "sym": rng.choice([0, 1]), "dtype": dtype}
    if op == "lora":
        while True:
            M, K, N = _log(rng, 1, 2048), 128 * _log(rng, 4, 64), 128 * _log(rng, 2, 224)
            if M * K * N <= _MAX_LORA:
                break
        rank = 8 * _log(rng, 1, 16)
        return {"op": op, "M": M, "K": K, "N": N, **fmt, "rank": rank, "adapters": _log(rng, 1, 64),
                "rows": rng.choice(["each", "runs"])}
    while True:
        E = _log(rng, 2, 128)
        k = rng.randint(1, min(8, E))
        T = _log(rng, 1, 16384)
        if op == "experts":
            K, N = 128 * _log(rng, 4, 64), 128 * _log(rng, 2, 112)
            if E * K * N <= _MAX_WEIGHTS and T * k * K * N <= _MAX_EXPERTS and T * k <= 65536:
                sizes = {"K": K, "N": N, **fmt}
                break
        else:
            H = 8 * _log(rng, 8, 1024)
            if T * k * H <= _MAX_ROWS:
                sizes = {"H": H, "dtype": dtype}
                break
    return {"op": op, "T": T, "k": k, "E": E, **sizes, "skew": rng.choice([0.0, 0.5, 1.5]),
            "pad": rng.choice([0, 0, T // 8])}


# ------------------------------------------------------------------------------------- inputs
def _pack8(u):
    """Codes 0..15 [..., 8 n, c] -> int32 words [..., n, c], code i of a word in bits 4 i."""
    *lead, K, N = u.shape
    u = u.view(*lead, K // 8, 8, N).to(torch.int64)
    w = torch.zeros(*lead, K // 8, N, dtype=torch.int64, device=u.device)
    for i in range(8):
        w |= u[..., i, :] << (4 * i)
    return _int32(w)


def _int32(w):
    return torch.where(w >= 2**31, w - 2**32, w).to(torch.int32)


def _quantized(K, N, group, sym, gen, dev):
    """Round-to-nearest codes, scales and zeros of a weight ~ N(0, 0.02): the plain packed layout."""
    W = (torch.randn(K, N, generator=gen, device=dev) * 0.02).view(K // group, group, N)
    if sym:
        s = (W.abs().amax(1) / 7).half()
        s = torch.where(s == 0, torch.ones_like(s), s)
        u = torch.clamp(torch.round(W / s.float()[:, None]), -8, 7).to(torch.int32) & 15
        zeros = None
    else:
        lo, hi = W.amin(1).clamp(max=0), W.amax(1).clamp(min=0)
        s = ((hi - lo) / 15).half()
        s = torch.where(s == 0, torch.ones_like(s), s)
        z = torch.clamp(torch.round(-lo / s.float()), 0, 15)
        u = torch.clamp(torch.round(W / s.float()[:, None]) + z[:, None], 0, 15).to(torch.int32)
        zeros = _pack8(z.to(torch.int32).t().contiguous()).t().contiguous()
    return _pack8(u.view(K, N)), s, zeros


def _tiled(codes, scales, zeros, group, sym):
    """The library's tiled buffer of a plain packed weight (uint8): one record per 128 x 128 unit."""
    K, N = codes.shape[0] * 8, codes.shape[1]
    C, T, G = K // 128, N // 128, 128 // group
    w = codes.to(torch.int64) & 0xFFFFFFFF
    if sym:
        w = w ^ 0x88888888
    t = torch.zeros_like(w)
    for p in range(4):
        t |= ((w >> (8 * p)) & 15) << (4 * p)
        t |= ((w >> (8 * p + 4)) & 15) << (16 + 4 * p)
    t = _int32(t).view(C, 4, 4, T, 128).permute(3, 0, 1, 4, 2)                      # [t, c, h, n, w]
    t = torch.stack([t[:, :, h, torch.arange(128, device=w.device) ^ (2 * h)] for h in range(4)], 2)
    # a group of one channel whose codes all equal its zero point keeps scale 0
    u = torch.stack([(w >> (4 * i)) & 15 for i in range(8)], 1).view(K // group, group, N)
    if sym:
        same = (u == 8).all(1)
    else:
        zw = zeros.to(torch.int64) & 0xFFFFFFFF
        z = torch.stack([(zw >> (4 * i)) & 15 for i in range(8)], 2).view(K // group, N)
        same = (u == z[:, None]).all(1)
    s = torch.where(same, torch.zeros_like(scales), scales).view(C, G, T, 128).permute(2, 0, 1, 3).contiguous()
    parts = [t.contiguous().view(T * C, -1).view(torch.uint8), s.view(T * C, -1).view(torch.uint8)]
    if not sym:
        z = zeros.view(C, G, T, 16).permute(2, 0, 1, 3).contiguous()
        parts.append(z.view(T * C, -1).view(torch.uint8))
    return torch.cat(parts, 1).reshape(-1)


def _routing(case, gen, dev):
    """Expert ids [T, k] of a router with unequal experts; the last `pad` tokens are padding (-1)."""
    T, k, E = case["T"], case["k"], case["E"]
    logits = torch.randn(T, E, generator=gen, device=dev) + case["skew"] * torch.randn(E, generator=gen, device=dev)
    top = torch.topk(logits, k, dim=1)
    ids = top.indices.to(torch.int32)
    ids[T - case["pad"]:] = -1
    return ids.contiguous(), torch.softmax(top.values, 1).contiguous()


def _adapters(case, gen, dev):
    """The rows' adapters: "each" deals them out in turn, in random order, every eighth row without
    one; "runs" gives every adapter one run of consecutive rows of uneven length."""
    M, L = case["M"], case["adapters"]
    if case["rows"] == "runs":
        cuts = torch.sort(torch.randint(0, M + 1, (L - 1,), generator=gen, device=dev)).values
        return torch.bucketize(torch.arange(M, device=dev), cuts, right=True).to(torch.int32)
    ids = (torch.arange(M, device=dev) % L)[torch.randperm(M, generator=gen, device=dev)]
    ids[7::8] = -1
    return ids.to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    t = _T[case["dtype"]]
    st = dict(case)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    if case["op"] == "lora":
        M, K, N, r, L = (case[x] for x in ("M", "K", "N", "rank", "adapters"))
        st["codes"], st["scales"], st["zeros"] = _quantized(K, N, case["group"], case["sym"], gen, dev)
        st["tiled"] = _tiled(st["codes"], st["scales"], st["zeros"], case["group"], case["sym"])
        st["A"] = randn(M, K).to(t)
        st["lora_a"] = (randn(L, r, K) / math.sqrt(K)).to(t)
        st["lora_b"] = (randn(L, N, r) * 0.02).to(t)
        st["lora_scale"] = 1.0 + torch.rand(L, generator=gen, device=dev)
        st["row_adapter"] = _adapters(case, gen, dev)
        st["C"] = torch.zeros(M, N, dtype=t, device=dev)
        return st
    ids, weights = _routing(case, gen, dev)
    T, k, E = case["T"], case["k"], case["E"]
    n = T * k
    key = torch.where(ids.view(-1) < 0, E, ids.view(-1)).long()
    counts = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=dev)
    offsets[1:] = torch.cumsum(counts, 0)
    if case["op"] == "experts":
        K, N = case["K"], case["N"]
        plain = [_quantized(K, N, case["group"], case["sym"], gen, dev) for _ in range(E)]
        st["tiled"] = torch.stack([_tiled(c, s, z, case["group"], case["sym"]) for c, s, z in plain])
        st["codes"] = torch.stack([c for c, _, _ in plain])
        st["scales"] = torch.stack([s for _, s, _ in plain])
        st["zeros"] = None if case["sym"] else torch.stack([z for _, _, z in plain])
        st["A"] = randn(n, K).to(t)
        st["offsets"], st["most"] = offsets, max(1, int(counts.max()))
        st["C"] = torch.zeros(n, N, dtype=t, device=dev)
        return st
    H = case["H"]
    order = torch.sort(key, stable=True).indices
    slots = torch.empty_like(key)
    slots[order] = torch.arange(n, device=dev)
    slots = torch.where(key == E, -1, slots).to(torch.int32).view(T, k)
    if case["op"] == "sort":
        st["ids"], st["X"] = ids, randn(T, H).to(t)
        st["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device=dev)
        st["rows"] = torch.zeros(n, dtype=torch.int32, device=dev)
        st["slots"] = torch.zeros(T, k, dtype=torch.int32, device=dev)
        st["Xs"] = torch.zeros(n, H, dtype=t, device=dev)
        return st
    st["slots"], st["weights"], st["Ys"] = slots, weights, randn(n, H).to(t)
    if case["op"] == "combine":
        st["Y"] = torch.zeros(T, H, dtype=t, device=dev)
        return st
    st["dY"], st["dXs"] = randn(T, H).to(t), randn(n, H).to(t)
    st["dYs"] = torch.zeros(n, H, dtype=t, device=dev)
    st["dweights"] = torch.zeros(T, k, dtype=torch.float32, device=dev)
    st["dX"] = torch.zeros(T, H, dtype=t, device=dev)
    return st


# ------------------------------------------------------------------------------------- one pass
def run(st):
    return {"lora": _run_lora, "sort": _run_sort, "experts": _run_experts, "combine": _run_combine,
            "grad": _run_grad}[st["op"]](st)


def _weights(codes, scales, zeros, group, sym):
    """The packed weights [..., K, N] in 32 bits."""
    *lead, Kw, N = codes.shape
    sh = 4 * torch.arange(8, device=codes.device, dtype=torch.int32)
    q = (codes[..., :, None, :] >> sh[:, None]) & 15
    if sym:
        q = (q ^ 8) - 8
    q = q.view(*lead, 8 * Kw // group, group, N)
    if not sym:
        q = q - ((zeros[..., None] >> sh) & 15).view(*lead, 8 * Kw // group, 1, N)
    return (q.float() * scales.float()[..., None, :]).view(*lead, 8 * Kw, N)


def _workspace(st, nbytes):
    """A program's workspace: one buffer, kept between its calls and zeroed once."""
    if "workspace" not in st:
        st["workspace"] = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
    return st["workspace"]


def _run_lora(st):
    M, K, N, r, L = (st[x] for x in ("M", "K", "N", "rank", "adapters"))
    if own:
        from weight_only_int4_07_b200 import native

        ws = st.get("workspace")
        if ws is None:
            ws = _workspace(st, native.w4a16_lora_workspace_bytes(M, N, K, st["group"], r, L))
        return native.w4a16_lora_gemm(st["A"], st["tiled"], N, st["group"], st["sym"], st["lora_a"], st["lora_b"],
                                      st["lora_scale"], st["row_adapter"], C=st["C"], workspace=ws)
    X = st["A"].float()
    base = X @ _weights(st["codes"], st["scales"], st["zeros"], st["group"], st["sym"])
    ids = st["row_adapter"].long()
    # every adapter's rank products, kept where the row has that adapter, times its scale
    low = (X @ st["lora_a"].float().view(L * r, K).t()).view(M, L, r)
    pick = (ids[:, None] == torch.arange(L, device=ids.device)).float() * st["lora_scale"]
    low = (low * pick[:, :, None]).view(M, L * r)
    return (base + low @ st["lora_b"].float().transpose(1, 2).reshape(L * r, N)).to(st["A"].dtype)


def _run_sort(st):
    T, k, E, H = (st[x] for x in ("T", "k", "E", "H"))
    if own:
        from weight_only_int4_07_b200 import native

        ws = st.get("workspace")
        if ws is None:
            ws = _workspace(st, native.w4a16_moe_sort_workspace_bytes(T, k, E))
        return native.w4a16_moe_sort(st["ids"], E, X=st["X"], offsets=st["offsets"], rows=st["rows"],
                                     slots=st["slots"], Xs=st["Xs"], workspace=ws)
    n = T * k
    ids = st["ids"].view(-1).long()
    key = torch.where((ids < 0) | (ids >= E), E, ids)
    order = torch.sort(key, stable=True).indices
    at = torch.arange(n, device=ids.device)
    slots = torch.empty_like(at)
    slots[order] = at
    slots = torch.where(key == E, -1, slots)
    offsets = torch.searchsorted(key[order], torch.arange(E + 1, device=ids.device))
    live = at < offsets[E]
    rows = torch.where(live, order, 0)
    Xs = torch.where(live[:, None], st["X"][rows // k], 0)
    return offsets.to(torch.int32), rows.to(torch.int32), slots.to(torch.int32).view(T, k), Xs


def _run_experts(st):
    n, E, K, N = st["T"] * st["k"], st["E"], st["K"], st["N"]
    if own:
        from weight_only_int4_07_b200 import native

        ws = st.get("workspace")
        if ws is None:
            ws = _workspace(st, native.w4a16_moe_workspace_bytes(n, E, N, K, st["group"]))
        return native.w4a16_moe_gemm(st["A"], st["offsets"], st["tiled"], N, st["group"], st["sym"], C=st["C"],
                                     workspace=ws)
    off = st["offsets"].long()
    at = torch.arange(n, device=off.device)
    live = (at < off[E])[:, None]
    e = torch.searchsorted(off, at, right=True).sub_(1).clamp_(max=E - 1)   # the row's expert
    X = st["A"].float()
    if n <= E:   # fewer rows than experts: each row with its own expert's weights
        W = _weights(st["codes"][e], st["scales"][e], None if st["sym"] else st["zeros"][e], st["group"], st["sym"])
        Y = torch.bmm(X[:, None], W)[:, 0]
    else:        # every expert's rows, padded to the longest run
        W = _weights(st["codes"], st["scales"], st["zeros"], st["group"], st["sym"])
        i = (at - off[e]).clamp(max=st["most"])
        Xp = torch.zeros(E, st["most"] + 1, K, device=off.device)
        Xp[e, torch.where(live[:, 0], i, st["most"])] = X
        Y = torch.bmm(Xp, W)[e, i]
    return torch.where(live, Y, 0).to(st["A"].dtype)


def _run_combine(st):
    if own:
        from weight_only_int4_07_b200 import native

        return native.w4a16_moe_combine(st["Ys"], st["slots"], st["weights"], Y=st["Y"])
    s = st["slots"].long()
    y = torch.where((s >= 0)[:, :, None], st["Ys"][s.clamp(min=0)].float() * st["weights"][:, :, None], 0)
    return y.sum(1).to(st["Ys"].dtype)


def _run_grad(st):
    if own:
        from weight_only_int4_07_b200 import native

        dYs, dweights = native.w4a16_moe_combine_grad(st["dY"], st["Ys"], st["slots"], st["weights"], dYs=st["dYs"],
                                                      dweights=st["dweights"])
        return dYs, dweights, native.w4a16_moe_sort_grad(st["dXs"], st["slots"], dX=st["dX"])
    t, n, H = st["Ys"].dtype, st["T"] * st["k"], st["H"]
    s = st["slots"].long()
    has = (s >= 0)[:, :, None]
    dY = st["dY"].float()[:, None]
    dYs = torch.zeros(n + 1, H, dtype=t, device=s.device)
    dYs[torch.where(s >= 0, s, n)] = (dY * st["weights"][:, :, None]).to(t)
    dweights = torch.where(has, dY * st["Ys"][s.clamp(min=0)].float(), 0).sum(2)
    dX = torch.where(has, st["dXs"][s.clamp(min=0)].float(), 0).sum(1).to(t)
    return dYs[:n], dweights, dX


# ------------------------------------------------------------------------------------- work
def _weight_bytes(K, N, group, sym):
    return K * N // 2 + 2 * N * (K // group) + (0 if sym else N * (K // group) // 2)


def work(case):
    if case["op"] == "lora":
        M, K, N, r, L = (case[x] for x in ("M", "K", "N", "rank", "adapters"))
        rows = M if case["rows"] == "runs" else M - M // 8
        used = min(L, rows)
        return {"bytes": _weight_bytes(K, N, case["group"], case["sym"]) + 2 * M * (K + N) + 2 * used * r * (K + N)
                + 4 * M, "flops": 2 * M * K * N + 2 * rows * r * (K + N)}
    T, k, E = case["T"], case["k"], case["E"]
    rows = (T - case["pad"]) * k
    if case["op"] == "experts":
        K, N = case["K"], case["N"]
        used = E * (1 - (1 - k / E) ** (T - case["pad"]))   # experts with a row, for even routing
        return {"bytes": used * _weight_bytes(K, N, case["group"], case["sym"]) + 2 * rows * (K + N) + 4 * (E + 1),
                "flops": 2 * rows * K * N}
    H = case["H"]
    if case["op"] == "sort":
        return {"bytes": 2 * H * (T - case["pad"] + rows) + 4 * (2 * T * k + rows + E + 1), "flops": T * k}
    if case["op"] == "combine":
        return {"bytes": 2 * H * (rows + T) + 8 * T * k, "flops": 2 * rows * H}
    return {"bytes": 2 * H * (3 * rows + 2 * T) + 12 * T * k, "flops": 4 * rows * H}


# ------------------------------------------------------------------------------------- 64 bits
def _dequant64(codes, scales, zeros, group, sym):
    """w[8 j + i, n] = (q - z) s of one plain packed weight, nibble by nibble, in 64 bits."""
    Kw, N = codes.shape
    W = torch.empty(8 * Kw, N, dtype=torch.float64, device=codes.device)
    for i in range(8):
        q = torch.bitwise_and(torch.bitwise_right_shift(codes, 4 * i), 0xF).double()
        if sym:
            q = torch.where(q > 7, q - 16, q)
        W[i::8] = q
    if not sym:
        z = torch.empty(zeros.shape[0], N, dtype=torch.float64, device=codes.device)
        for i in range(8):
            z[:, i::8] = torch.bitwise_and(torch.bitwise_right_shift(zeros, 4 * i), 0xF).double()
        W -= z.repeat_interleave(group, 0)
    return W.mul_(scales.double().repeat_interleave(group, 0))


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "lora":
        X = st["A"].double()
        Y = X @ _dequant64(st["codes"], st["scales"], st["zeros"], case["group"], case["sym"])
        for a in range(case["adapters"]):
            m = torch.nonzero(st["row_adapter"] == a).view(-1)
            Y[m] += float(st["lora_scale"][a]) * (X[m] @ st["lora_a"][a].double().t()) @ st["lora_b"][a].double().t()
        return Y
    if case["op"] == "experts":
        off = st["offsets"].tolist()
        Y = torch.zeros(st["A"].shape[0], case["N"], dtype=torch.float64, device=st["A"].device)
        for e in range(case["E"]):
            if off[e + 1] > off[e]:
                W = _dequant64(st["codes"][e], st["scales"][e], None if case["sym"] else st["zeros"][e],
                               case["group"], case["sym"])
                Y[off[e]:off[e + 1]] = st["A"][off[e]:off[e + 1]].double() @ W
        return Y
    if case["op"] == "sort":
        # rows of expert e: the flat choices that name it, in order
        flat, k = st["ids"].view(-1), case["k"]
        lists = [torch.nonzero(flat == e).view(-1) for e in range(case["E"])]
        order = torch.cat(lists)
        Xs = torch.zeros(flat.numel(), case["H"], dtype=torch.float64, device=flat.device)
        Xs[:order.numel()] = st["X"].double()[torch.div(order, k, rounding_mode="floor")]
        return None, None, None, Xs
    s, w = st["slots"], st["weights"].double()
    Ys = st["Ys"].double()
    if case["op"] == "combine":
        Y = torch.zeros(case["T"], case["H"], dtype=torch.float64, device=s.device)
        for j in range(case["k"]):
            m = torch.nonzero(s[:, j] >= 0).view(-1)
            Y[m] += w[m, j, None] * Ys[s[m, j].long()]
        return Y
    dY, dXs = st["dY"].double(), st["dXs"].double()
    dYs, dw, dX = torch.zeros_like(Ys), torch.zeros_like(w), torch.zeros_like(dY)
    for j in range(case["k"]):
        m = torch.nonzero(s[:, j] >= 0).view(-1)
        at = s[m, j].long()
        dYs[at] = w[m, j, None] * dY[m]
        dw[m, j] = (dY[m] * Ys[at]).sum(1)
        dX[m] += dXs[at]
    return dYs, dw, dX
