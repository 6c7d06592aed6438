"""Measured cases of the operators of a full-attention layer: rotary positions with their gradient, the
paged cache (8-bit or not) as it is written and read back, and the attention of new tokens over it, for
prompts, chunks and single tokens.

``own`` False computes an operator in its plain form (elementary torch operations in fp32, angles in
fp64); True calls the library.  ``new`` are the new tokens of each sequence and ``ctx`` the tokens that
its cache holds before them.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn
THETA = 10000.0
ORIGINAL = 4096  # positions that the frequencies were trained for, where they are scaled


# ---------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one token of one request, queries and keys in one call: latency
        {"name": "rope_token", "op": "rope", "T": 1, "H": 40, "D": 128, "R": 128, "inter": False, "scaling": "none",
         "far": 4096, "type": "bf16"},
        # a prompt at far positions of a scaled context, half of each head rotated
        {"name": "rope_prompt_far", "op": "rope", "T": 8192, "H": 40, "D": 128, "R": 64, "inter": True,
         "scaling": "yarn", "far": 1 << 20, "type": "bf16"},
        # a training step's positions, forward and gradient, a quarter of each head rotated
        {"name": "rope_train", "op": "rope_train", "T": 16384, "H": 18, "D": 256, "R": 64, "inter": False,
         "scaling": "none", "far": 4096, "type": "bf16"},
        # one token of each request of a padded batch goes into an 8-bit cache
        {"name": "write_step_b64", "op": "write", "T": 64, "H": 8, "D": 128, "P": 16, "pages": 320, "type": "bf16",
         "cache": "e4m3"},
        # a prompt goes into an 8-bit cache
        {"name": "write_prompt", "op": "write", "T": 8192, "H": 8, "D": 128, "P": 64, "pages": 160, "type": "bf16",
         "cache": "e4m3"},
        # a long prompt's cache is read back
        {"name": "read_prompt", "op": "read", "T": 16384, "H": 8, "D": 128, "P": 16, "pages": 1100, "type": "bf16",
         "cache": "e4m3"},
        # one token of one request after a long context: one row and a long axis
        {"name": "attn_step_b1_long", "op": "attn_step", "new": "1", "ctx": "131071", "Hq": 32, "Hk": 8, "D": 128,
         "P": 64, "causal": True, "window": 0, "type": "bf16", "cache": "bf16"},
        # one token of each request of a padded batch, contexts of all lengths, 8-bit cache
        {"name": "attn_step_b32_q8", "op": "attn_step", "new": ",".join(["1"] * 32),
         "ctx": "0,17,63,64,255,300,511,777,1000,1023,1500,2047,2048,2500,3001,3500,4095,4500,5000,5555,6001,7000,"
                "8191,9000,10000,11111,12345,14000,16383,20000,-1,-1", "Hq": 32, "Hk": 8, "D": 128, "P": 16,
         "causal": True, "window": 0, "type": "bf16", "cache": "e4m3"},
        # a serving step: chunks of prompts beside single tokens
        {"name": "attn_chunk_mixed", "op": "attn", "new": "1,1,1,512,33,1,2048,1,7",
         "ctx": "900,4000,77,1024,5000,16000,0,2222,333", "Hq": 32, "Hk": 8, "D": 128, "P": 16, "causal": True,
         "window": 0, "type": "bf16", "cache": "bf16"},
        # a long prompt's second chunk
        {"name": "attn_prompt", "op": "attn", "new": "8192", "ctx": "8192", "Hq": 32, "Hk": 8, "D": 128, "P": 64,
         "causal": True, "window": 0, "type": "bf16", "cache": "bf16"},
        # wide heads over an 8-bit cache, sliding window
        {"name": "attn_window_d256_q8", "op": "attn", "new": "1000,24,3000", "ctx": "0,4321,1500", "Hq": 16, "Hk": 2,
         "D": 256, "P": 32, "causal": True, "window": 1024, "type": "bf16", "cache": "e4m3"},
        # cross attention to an encoder's cached states of other lengths, full precision
        {"name": "attn_cross_f32", "op": "attn", "new": "777,5,130", "ctx": "300,1,77", "Hq": 12, "Hk": 12, "D": 64,
         "P": 16, "causal": False, "window": 0, "type": "f32", "cache": "f32"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope_train", "write", "read", "attn_step", "attn_step", "attn", "attn"])
    kind = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("rope"):
        D = rng.choice([64, 80, 128, 192, 256])
        H = rng.randint(1, 48)
        return {"op": op, "T": _log_int(rng, 1, min(32768, (1 << 25) // (H * D))), "H": H, "D": D,
                "R": rng.choice([D, D // 2, D // 4]), "inter": rng.random() < 0.5,
                "scaling": rng.choice(["none", "linear", "ntk", "yarn"]), "far": _log_int(rng, 64, 1 << 22),
                "type": kind}
    P = rng.choice([16, 32, 64, 128])
    cache = rng.choice([kind, "e4m3"])
    if op in ("write", "read"):
        H, D = rng.randint(1, 16), rng.choice([64, 80, 128, 192, 256])
        T = _log_int(rng, 1, min(16384, (1 << 25) // (H * D)))
        return {"op": op, "T": T, "H": H, "D": D, "P": P, "pages": T // P + 1 + _log_int(rng, 1, 64), "type": kind,
                "cache": cache}
    Hk = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 8])
    c = {"op": op, "Hq": Hk * G, "Hk": Hk, "D": rng.choice([64, 128, 256]), "P": P, "causal": True, "window": 0,
         "type": kind, "cache": cache}
    if op == "attn_step":
        n = _log_int(rng, 1, 48)
        longest = min(131072, (1 << 26) // (n * Hk * c["D"]))  # (the whole batch's cache: half a GB at most)
        ctx = [_log_int(rng, 1, longest) - 1 for _ in range(n)]
        if n >= 8:
            ctx[-1] = -1
        return dict(c, new=",".join(["1"] * n), ctx=",".join(map(str, ctx)),
                    window=rng.choice([0, 0, _log_int(rng, 16, 4096)]))
    n = rng.randint(1, 6)
    most = 512 if kind == "f32" else 2048
    new = [_log_int(rng, 1, most) for _ in range(n)]
    ctx = [_log_int(rng, 1, 4 * most) - 1 for _ in range(n)]
    causal = rng.random() < 0.75
    while len(new) > 1 and sum(a * (a + b) for a, b in zip(new, ctx)) * c["Hq"] * c["D"] > 1 << 38:
        new.pop()
        ctx.pop()
    return dict(c, new=",".join(map(str, new)), ctx=",".join(map(str, ctx)), causal=causal,
                window=rng.choice([0, 0, _log_int(rng, 16, 4096)]) if causal else 0)


# --------------------------------------------------------------------------------------- inputs

def _ints(text):
    return [int(n) for n in text.split(",")]


def _seqs(case):
    """(new tokens, keys) of each sequence.  Keys: context and new tokens of a causal call, the context (an
    encoder's states) otherwise; a context of -1 is a row that pads the batch: no keys."""
    new, ctx = _ints(case["new"]), _ints(case["ctx"])
    return new, [max(c, 0) if not case["causal"] else (0 if c < 0 else c + n) for n, c in zip(new, ctx)]


def _freqs(case):
    """Angles a position [R/2] in fp64, scaled for a context `factor` times the original one, and the factor
    on the rotated values."""
    R, kind = case["R"], case["scaling"]
    i = torch.arange(R // 2, dtype=torch.float64)
    factor = max(1.0, case["far"] / ORIGINAL)
    if kind == "ntk" and R > 2:
        return (THETA * factor ** (R / (R - 2))) ** (-2 * i / R), 1.0
    f = THETA ** (-2 * i / R)
    if kind == "linear":
        return f / factor, 1.0
    if kind == "yarn":
        # pairs that turn more than 32 times within the original length keep their angle, less than once: divided
        def at(turns):
            return R * math.log(ORIGINAL / (turns * 2 * math.pi)) / (2 * math.log(THETA))

        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), R - 1)
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _e4m3(x):
    """(values, scales): a scale for each row of x (fp32)."""
    scale = x.abs().amax(-1).clamp(min=1e-12) / 448
    return (x / scale[..., None]).clamp(-448, 448).to(E4M3), scale


def _cache(case, gen, pages, heads):
    """A cache of random rows; 8-bit ones as values and scales."""
    out = {}
    for name in ("k", "v"):
        x = torch.randn(pages, heads, case["P"], case["D"], generator=gen, device=DEV)
        if case["cache"] == "e4m3":
            out[name + "c"], out[name + "s"] = _e4m3(x)
        else:
            out[name + "c"], out[name + "s"] = x.to(TYPES[case["cache"]]), None
        del x
    return out


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op, t = case["op"], TYPES[case["type"]]
    s = {"case": dict(case)}
    if op.startswith("rope"):
        T, H, D = case["T"], case["H"], case["D"]
        qkv = torch.randn(T, H * D + 256, generator=gen, device=DEV).to(t)  # a projection: queries, keys, values
        s["x"] = qkv[:, :H * D].view(T, H, D)
        start = int(torch.randint(0, max(1, case["far"] - T), (1,), generator=gen, device=DEV))
        s["pos"] = torch.arange(start, start + T, device=DEV, dtype=torch.int32)
        freqs, s["mag"] = _freqs(case)
        s["freqs"] = freqs.to(DEV)
        if op == "rope_train":
            s["dy"] = torch.randn(T, H, D, generator=gen, device=DEV).to(t)
        if own:
            import gated_delta_rule_29_amd as g

            f, s["mag"] = g.rope_freqs(case["R"], THETA, scaling=None if case["scaling"] == "none" else case["scaling"],
                                       factor=max(1.0, case["far"] / ORIGINAL), original=ORIGINAL)
            s["table"] = g.rope_table(f, DEV)
        return s
    if op in ("write", "read"):
        T, H, D, P, pages = case["T"], case["H"], case["D"], case["P"], case["pages"]
        s.update(_cache(case, gen, pages, H))
        # tokens in order in pages that are taken from all over the cache; a part-filled first page
        order = torch.randperm(pages, generator=gen, device=DEV)
        first = int(torch.randint(0, min(P, pages * P - T + 1), (1,), generator=gen, device=DEV))
        at = torch.arange(first, first + T, device=DEV)
        if T <= 64:  # a decoding batch: one token of each request, so each in another place
            at = torch.randperm(pages * P, generator=gen, device=DEV)[:T]
        s["slots"] = (order[at // P] * P + at % P).to(torch.int32)
        if 8 <= T <= 64:
            s["slots"][-(T // 8):] = -1  # rows that pad the batch
        if op == "write":
            qkv = torch.randn(T, 3 * H * D, generator=gen, device=DEV).to(t)
            s["k"] = qkv[:, H * D:2 * H * D].view(T, H, D)
            s["v"] = qkv[:, 2 * H * D:].view(T, H, D)
        return s
    new, keys = _seqs(case)
    P = case["P"]
    need = [-(-n // P) for n in keys]
    pages = sum(need) + 3
    s.update(_cache(case, gen, pages, case["Hk"]))
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(new), max(1, max(need))), -1, dtype=torch.int32, device=DEV)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    s["table"] = table
    s["lens"] = torch.tensor(keys, dtype=torch.int32, device=DEV)
    s["q"] = torch.randn(sum(new), case["Hq"], case["D"], generator=gen, device=DEV).to(t)
    if op == "attn":
        s["q"] = s["q"][None]  # a packed batch
        s["cu_host"] = torch.tensor([0] + new, dtype=torch.int32).cumsum(0).to(torch.int32)
        s["cu"] = s["cu_host"].to(DEV)
    return s


# ---------------------------------------------------------------------------------- plain forms

def _rotate(x, s, sign):
    case = s["case"]
    R, h = case["R"], case["R"] // 2
    angle = s["pos"].double()[:, None] * s["freqs"]
    c, n = (s["mag"] * torch.cos(angle)).float()[:, None], (sign * s["mag"] * torch.sin(angle)).float()[:, None]
    y = x.float().contiguous()
    a, b = (y[..., 0:R:2], y[..., 1:R:2]) if case["inter"] else (y[..., :h], y[..., h:R])
    u, w = a * c - b * n, a * n + b * c
    if case["inter"]:
        y[..., 0:R:2], y[..., 1:R:2] = u, w
    else:
        y[..., :h], y[..., h:R] = u, w
    return y.to(x.dtype)


def _plain_rope(s):
    out = {"y": _rotate(s["x"], s, 1.0)}
    if s["case"]["op"] == "rope_train":
        out["dx"] = _rotate(s["dy"], s, -1.0)
    return out


def _plain_write(s):
    P = s["case"]["P"]
    live = (s["slots"] >= 0).nonzero()[:, 0]
    at = s["slots"].long()[live]
    page, place = at // P, at % P
    out = {}
    for name in ("k", "v"):
        x, cache = s[name][live], s[name + "c"]
        if s[name + "s"] is None:
            cache[page, :, place] = x
        else:
            q, scale = _e4m3(x.float())
            # (torch has no indexed store of 8-bit floats: the same bytes)
            cache.view(torch.uint8)[page, :, place] = q.view(torch.uint8)
            s[name + "s"][page, :, place] = scale
            out[name + "_scale"] = s[name + "s"]
        out[name + "_cache"] = cache
    return out


def _gather(s, name, page, place):
    """Rows [.., Hk, D] of the cache in fp32."""
    if s[name + "s"] is None:
        return s[name + "c"][page, :, place].float()
    rows = s[name + "c"].view(torch.uint8)[page, :, place].view(E4M3).float()
    return rows * s[name + "s"][page, :, place][..., None]


def _plain_read(s):
    P, t = s["case"]["P"], TYPES[s["case"]["type"]]
    at = s["slots"].long().clamp(min=0)
    live = (s["slots"] >= 0)[:, None, None]
    return {n: torch.where(live, _gather(s, n, at // P, at % P), 0.0).to(t) for n in ("k", "v")}


def _attend(q, k, v, seen):
    """q [.., M, D], k and v [.., L, D], seen [.., M, L] (or what broadcasts): outputs, 0 for rows that see nothing."""
    z = torch.matmul(q, k.transpose(-1, -2)).mul_(q.shape[-1] ** -0.5)
    z.masked_fill_(~seen, -math.inf)
    top = z.amax(-1, keepdim=True).clamp(min=-1e30)
    p = z.sub_(top).exp_()
    return torch.matmul(p, v) / p.sum(-1, keepdim=True).clamp(min=1e-30)


def _plain_steps(s):
    """All rows at once, as many as keep the gathered keys within a few GB."""
    case = s["case"]
    Hk, D, P, G = case["Hk"], case["D"], case["P"], case["Hq"] // case["Hk"]
    lens, table = s["lens"].long(), s["table"].long().clamp(min=0)
    at = torch.arange(table.shape[1] * P, device=DEV)
    step = max(1, (1 << 29) // (at.numel() * Hk * D))
    out = []
    for r in range(0, len(lens), step):
        page, place = table[r:r + step][:, at // P], (at % P).expand(table[r:r + step].shape[0], -1)
        k, v = (_gather(s, n, page, place).transpose(1, 2) for n in ("k", "v"))
        n = lens[r:r + step, None]
        seen = at < n
        if case["window"]:
            seen &= at >= n - case["window"]
        q = s["q"][r:r + step].float().view(-1, Hk, G, D)
        o = _attend(q, k, v, seen[:, None, None, :])
        out.append(torch.where(n[:, :, None] > 0, o.reshape(-1, Hk * G, D), 0.0))
    return {"o": torch.cat(out).to(s["q"].dtype)}


def _plain_chunks(s):
    case = s["case"]
    Hk, D, P, G = case["Hk"], case["D"], case["P"], case["Hq"] // case["Hk"]
    new, keys = _seqs(case)
    queries = s["q"][0]
    o = torch.zeros(queries.shape, device=DEV)
    t0 = 0
    for i, (n, L) in enumerate(zip(new, keys)):
        if L:
            at = torch.arange(L, device=DEV)
            page = s["table"][i].long()[at // P]
            k, v = (_gather(s, name, page, at % P).transpose(0, 1).contiguous() for name in ("k", "v"))
            step = max(1, (1 << 28) // (L * Hk * G))
            for r in range(0, n, step):
                q = queries[t0 + r:t0 + min(n, r + step)].float()
                m = q.shape[0]
                q = q.view(m, Hk, G, D).permute(1, 2, 0, 3).reshape(Hk, G * m, D)
                if case["causal"]:
                    pos = L - n + r + torch.arange(m, device=DEV)[:, None]
                    seen = at <= pos
                    if case["window"]:
                        seen &= at > pos - case["window"]
                else:
                    seen = torch.ones(m, L, dtype=torch.bool, device=DEV)
                part = _attend(q, k, v, seen.repeat(G, 1))
                o[t0 + r:t0 + r + m] = part.view(Hk, G, m, D).permute(2, 0, 1, 3).reshape(m, Hk * G, D)
        t0 += n
    return {"o": o.to(s["q"].dtype)[None]}


# ------------------------------------------------------------------------------ the library's calls

def _own(s):
    import gated_delta_rule_29_amd as g

    case = s["case"]
    op = case["op"]
    if op.startswith("rope"):
        how = dict(interleaved=case["inter"], magnitude=s["mag"])
        out = {"y": g.rope_fwd(s["x"], s["pos"], s["table"], **how)}
        if op == "rope_train":
            out["dx"] = g.rope_bwd(s["dy"], s["pos"], s["table"], **how)
        return out
    scales = dict(k_scale=s["ks"], v_scale=s["vs"])
    if op == "write":
        g.kv_cache_write(s["k"], s["v"], s["kc"], s["vc"], s["slots"], **scales)
        out = {"k_cache": s["kc"], "v_cache": s["vc"]}
        if s["ks"] is not None:
            out.update(k_scale=s["ks"], v_scale=s["vs"])
        return out
    if op == "read":
        return g.kv_cache_read(s["kc"], s["vc"], s["slots"], dtype=TYPES[case["type"]], **scales)
    args = (s["q"], s["kc"], s["vc"], s["table"], s["lens"])
    if op == "attn_step":
        return {"o": g.paged_attn_step(*args, window=case["window"], **scales)}
    return g.paged_attn_fwd_varlen(*args, s["cu"], causal=case["causal"], window=case["window"],
                                   cu_seqlens_host=s["cu_host"], **scales)


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op.startswith("rope"):
        return _plain_rope(state)
    if op in ("write", "read"):
        return _plain_write(state) if op == "write" else _plain_read(state)
    return _plain_steps(state) if op == "attn_step" else _plain_chunks(state)


# ------------------------------------------------------------------------------------- the work

def _span(case, n, L):
    """(visible pairs of query token and key, keys that any of them sees) of a sequence."""
    if not case["causal"]:
        return n * L, L
    w = case["window"] or L
    lo = L - n  # position of the first new token
    pairs = sum(min(p + 1, w) for p in range(max(lo, 0), L)) if L else 0
    return pairs, min(L, w + n - 1)


def work(case):
    e = 2 if case["type"] == "bf16" else 4
    op, D = case["op"], case["D"]
    if op.startswith("rope"):
        n = case["T"] * case["H"]
        k = 2 if op == "rope_train" else 1
        return {"bytes": k * (2 * n * D * e + 4 * case["T"]), "flops": k * 3 * n * case["R"]}
    c, extra = (1, 4) if case["cache"] == "e4m3" else (2 if case["cache"] == "bf16" else 4, 0)
    if op in ("write", "read"):
        n = 2 * case["T"] * case["H"]
        return {"bytes": n * (D * (e + c) + extra) + 4 * case["T"], "flops": n * D * (3 if extra else 1)}
    new, keys = _seqs(case)
    spans = [_span(case, n, L) for n, L in zip(new, keys)]
    return {"bytes": 2 * sum(new) * case["Hq"] * D * e + 2 * sum(k for _, k in spans) * case["Hk"] * (D * c + extra)
            + 4 * sum(-(-k // case["P"]) for _, k in spans),
            "flops": 4 * D * case["Hq"] * sum(p for p, _ in spans)}


# ------------------------------------------------------------------- the definitions, in 64 bits

def _exact_turned(x, s, back):
    """Pairs as complex numbers, turned by their angle."""
    case = s["case"]
    R = case["R"]
    x = x.double()
    head, rest = x[..., :R], x[..., R:]
    pairs = head.unflatten(-1, (R // 2, 2)) if case["inter"] else head.unflatten(-1, (2, R // 2)).transpose(-1, -2)
    z = torch.view_as_complex(pairs.contiguous())
    angle = torch.outer(s["pos"].double(), s["freqs"])
    z = z * torch.polar(torch.full_like(angle, s["mag"]), -angle if back else angle)[:, None]
    pairs = torch.view_as_real(z)
    head = pairs.flatten(-2) if case["inter"] else pairs.transpose(-1, -2).flatten(-2)
    return torch.cat([head, rest], -1)


def _exact_cache(case, s):
    P, D = case["P"], case["D"]
    slots = s["slots"].tolist()
    if case["op"] == "write":
        out = {}
        rows = torch.tensor([r for r, k in enumerate(slots) if k >= 0], device=DEV)
        to = torch.tensor([k for k in slots if k >= 0], device=DEV)
        for n in ("k", "v"):
            pages, H = s[n + "c"].shape[:2]
            flat = s[n + "c"].to(torch.float64).transpose(1, 2).reshape(pages * P, H, D)
            x = s[n].double()[rows]
            if s[n + "s"] is not None:
                sc = s[n + "s"].double().transpose(1, 2).reshape(pages * P, H)
                size = torch.clamp(x.abs().max(-1).values, min=1e-12) / 448
                sc[to] = size
                x = x / size[..., None]
                out[n + "_scale"] = sc.view(pages, P, H).transpose(1, 2)
            flat[to] = x
            out[n + "_cache"] = flat.view(pages, P, H, D).transpose(1, 2)
        return out
    out = {}
    at = torch.tensor(slots, device=DEV)
    for n in ("k", "v"):
        pages, H = s[n + "c"].shape[:2]
        flat = s[n + "c"].to(torch.float64)
        if s[n + "s"] is not None:
            flat = flat * s[n + "s"].double()[..., None]
        flat = flat.transpose(1, 2).reshape(pages * P, H, D)
        out[n] = torch.where((at >= 0)[:, None, None], flat[at.clamp(min=0)], 0.0)
    return out


def _exact_attn(case, s):
    """Head by head, each query's weights over the keys that it sees."""
    new, keys = _seqs(case)
    D, P, G = case["D"], case["P"], case["Hq"] // case["Hk"]
    q = s["q"].double().view(-1, case["Hq"], D)
    o = torch.zeros_like(q)
    t0 = 0
    for i, (n, L) in enumerate(zip(new, keys)):
        pages = s["table"][i, :-(-L // P)].long()
        for h in range(case["Hk"] if L else 0):
            k, v = (s[m + "c"][:, h].view(torch.uint8)[pages].view(E4M3).double() if s[m + "s"] is not None
                    else s[m + "c"][:, h][pages].double() for m in ("k", "v"))
            if s["ks"] is not None:
                k, v = k * s["ks"][:, h][pages].double()[..., None], v * s["vs"][:, h][pages].double()[..., None]
            k, v = k.reshape(-1, D)[:L], v.reshape(-1, D)[:L]
            block = max(1, (1 << 26) // L)
            for g in range(h * G, h * G + G):
                for a in range(0, n, block):
                    b = min(n, a + block)
                    z = q[t0 + a:t0 + b, g] @ k.T / math.sqrt(D)
                    if case["causal"]:
                        ago = torch.arange(L - n + a, L - n + b, device=DEV)[:, None] - torch.arange(L, device=DEV)
                        hidden = ago < 0
                        if case["window"]:
                            hidden |= ago >= case["window"]
                        z[hidden] = -math.inf
                    w = torch.softmax(z, -1)
                    o[t0 + a:t0 + b, g] = torch.nan_to_num(w) @ v  # a row without keys: 0
        t0 += n
    return {"o": o.view(s["q"].shape)}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("rope"):
        out = {"y": _exact_turned(s["x"], s, False)}
        if op == "rope_train":
            out["dx"] = _exact_turned(s["dy"], s, True)
        return out
    return _exact_cache(case, s) if op in ("write", "read") else _exact_attn(case, s)
