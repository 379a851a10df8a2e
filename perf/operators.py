"""The attention operators of a caller's own target model, as cases to measure.

A caller that verifies drafts with its own target runs, in every layer of it,
the rotary embedding, the append of new keys and values to a paged cache and
the attention of the new tokens over that cache.  Each case is one call of one
of these operators: in its plain form (elementary torch operations in 32 bits)
or, with `own` set, through block_diffusion_speculative_hiddens_gb300.ops.

Sizes come from this repository's workloads (32 query and 8 or 4 KV heads of
128, 16 and 2 heads of 64; blocks of 16; contexts of 512 to 32,768; batches of
1, 4 and 64) and from the ranges between them.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
SCALINGS = {  # the long-context scalings, by kind: factor and the length that the model was trained at
    "none": None,
    "linear": {"kind": "linear", "factor": 4.0},
    "ntk": {"kind": "ntk", "factor": 4.0},
    "yarn": {"kind": "yarn", "factor": 4.0, "original_len": 32768, "beta_fast": 32.0, "beta_slow": 1.0},
    "llama3": {"kind": "llama3", "factor": 8.0, "original_len": 8192, "low_freq_factor": 1.0,
               "high_freq_factor": 4.0},
}


def _rope(name, rows, hq, hkv, d, rd, interleaved, scaling, dtype, pos, packed, backward=False, theta=1e6):
    return {"name": name, "op": "rope", "rows": rows, "hq": hq, "hkv": hkv, "d": d, "rd": rd,
            "interleaved": interleaved, "scaling": scaling, "dtype": dtype, "pos": pos, "packed": packed,
            "backward": backward, "theta": theta}


def _append(name, b, n_lo, n_hi, ctx_lo, ctx_hi, hq, hkv, d, rd, interleaved, scaling, dtype, page, theta=1e6):
    return {"name": name, "op": "append", "b": b, "n_lo": n_lo, "n_hi": n_hi, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi,
            "hq": hq, "hkv": hkv, "d": d, "rd": rd, "interleaved": interleaved, "scaling": scaling, "dtype": dtype,
            "page": page, "theta": theta}


def _attention(name, b, n_lo, n_hi, ctx_lo, ctx_hi, hq, hkv, d, dtype, page=64, causal=True, window=0):
    return {"name": name, "op": "attention", "b": b, "n_lo": n_lo, "n_hi": n_hi, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi,
            "hq": hq, "hkv": hkv, "d": d, "dtype": dtype, "page": page, "causal": causal, "window": window}


def listed():
    return [
        # one request's verify block: 16 tokens, the smallest call of a decoding loop
        _rope("rope, a verify block", 16, 32, 8, 128, 128, False, "none", "bf16", 2048, False),
        # a long prompt, odd length, half of each head rotated in adjacent pairs, out of a fused QKV projection
        _rope("rope, a long prompt", 8191, 32, 8, 128, 64, True, "yarn", "f16", 120000, True),
        # a decoding step of 64 requests without speculation: one token each
        _append("append, one token each", 64, 1, 1, 512, 4096, 32, 8, 128, 128, False, "none", "bf16", 64),
        # prompts of several requests, behind contexts that end inside pages
        _append("append, prompt chunks", 5, 700, 2301, 0, 9000, 32, 8, 128, 128, False, "llama3", "f16", 64, 5e5),
        # the verify step of one request: the headline workload's block and context
        _attention("attention, a verify block", 1, 16, 16, 2048, 2048, 32, 8, 128, "bf16"),
        # a decoding step of the batched workload: one token each, ragged contexts
        _attention("attention, one token each", 64, 1, 1, 512, 4096, 32, 8, 128, "bf16"),
        # the verify step of the long-context workload
        _attention("attention, long verify blocks", 4, 16, 16, 32750, 32768, 32, 4, 128, "f16"),
        # a non-causal block over its context, as a block drafter attends
        _attention("attention, blocks, no mask", 24, 16, 16, 30, 2000, 16, 2, 64, "f16", 64, False),
        # a chunk of a long prompt over the cache of the chunks before it
        _attention("attention, a prompt chunk", 1, 2048, 2048, 30001, 30001, 32, 8, 128, "bf16"),
        # prompts of several requests with and without contexts, heads of 64
        _attention("attention, ragged prompts", 7, 1, 1900, 0, 700, 16, 2, 64, "f16", 16),
        # a layer with a sliding window
        _attention("attention, a window", 2, 3500, 4001, 500, 1001, 32, 8, 128, "bf16", 64, True, 1024),
        # a whole long prompt
        _attention("attention, a long prompt", 1, 8192, 8192, 0, 0, 32, 8, 128, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    heads = rng.choice([(32, 8, 128), (32, 4, 128), (16, 4, 128), (8, 1, 128), (4, 4, 128), (16, 2, 64), (8, 2, 64),
                        (28, 4, 128), (15, 5, 64), (24, 2, 128)])
    hq, hkv, d = heads
    dtype, page = rng.choice(["bf16", "f16"]), rng.choice([16, 32, 64, 64, 128])
    scaling = rng.choice(sorted(SCALINGS))
    inter, rd = rng.random() < 0.5, rng.choice([d, d, d // 2, d // 4])
    theta = rng.choice([1e4, 5e5, 1e6])
    op = rng.choice(["rope", "append", "attention", "attention", "attention"])
    if op == "rope":
        c = _rope("", _log(rng, 1, 8000), hq, hkv, d, rd, inter, scaling, dtype, _log(rng, 1, 1000000),
                  rng.random() < 0.5, rng.random() < 0.3, theta)
    elif op == "append":
        b = _log(rng, 1, 64)
        n = _log(rng, 1, max(2, 8000 // b))
        ctx = _log(rng, 1, 9000)
        c = _append("", b, rng.randint(1, n), n, rng.randint(0, ctx), ctx, hq, hkv, d, rd, inter, scaling, dtype,
                    page, theta)
    else:
        kind = rng.choice(["one", "block", "prompt"])
        if kind == "one":
            b = _log(rng, 1, 64)
            n_lo = n_hi = 1
            ctx = _log(rng, 16, min(32768, 260000 // b))
        elif kind == "block":
            b = _log(rng, 1, 32)
            n_lo, n_hi = rng.randint(1, 4), rng.randint(4, 40)
            ctx = _log(rng, 16, min(32768, 130000 // b))
        else:
            b = _log(rng, 1, 6)
            n_hi = _log(rng, 64, 4000 // b)
            n_lo = rng.randint(1, n_hi)
            ctx = _log(rng, 1, 16000 // b)
        causal = rng.random() < 0.8
        window = _log(rng, 16, 4096) if causal and rng.random() < 0.3 else 0
        c = _attention("", b, n_lo, n_hi, rng.randint(0, ctx), ctx, hq, hkv, d, dtype, page, causal, window)
    del c["name"]
    return c


def _spread(lo, hi, b, stride):
    """b whole numbers over [lo, hi], both ends among them where b > 1, in a mixed order."""
    if b == 1:
        return [hi]
    order = [(i * stride) % b for i in range(b)] if math.gcd(stride, b) == 1 else list(range(b))
    return [lo + (hi - lo) * i // (b - 1) for i in order]


def _lengths(case):
    n = _spread(case["n_lo"], case["n_hi"], case["b"], 7)
    ctx = _spread(case["ctx_lo"], case["ctx_hi"], case["b"], 11)
    return n, ctx


def _frequencies(case):
    """(angle per position of every rotated pair in 64 bits, factor of cos and sin)."""
    rd, theta, s = case["rd"], case["theta"], SCALINGS[case["scaling"]]
    i = torch.arange(rd // 2, dtype=torch.float64)
    kind = "none" if s is None else s["kind"]
    if kind == "ntk":
        theta = theta * s["factor"] ** (rd / (rd - 2.0))
    f = theta ** (-2.0 * i / rd)
    if kind == "linear":
        f = f / s["factor"]
    elif kind == "llama3":
        turns = s["original_len"] * f / (2 * math.pi)  # turns over the trained length
        mix = ((turns - s["low_freq_factor"]) / (s["high_freq_factor"] - s["low_freq_factor"])).clamp(0, 1)
        f = f * (mix + (1 - mix) / s["factor"])
    elif kind == "yarn":
        def at(beta):  # the pair that makes `beta` turns over the trained length
            return rd * math.log(s["original_len"] / (beta * 2 * math.pi)) / (2 * math.log(theta))
        lo, hi = max(math.floor(at(s["beta_fast"])), 0), min(math.ceil(at(s["beta_slow"])), rd - 1)
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = f * (1 - ramp) + f / s["factor"] * ramp
    return f, 0.1 * math.log(s["factor"]) + 1.0 if kind == "yarn" else 1.0


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dt)

    st = {"case": case}
    if case["op"] != "attention":
        freq, st["factor"] = _frequencies(case)
        st["freq"] = freq.cuda()
        if own:
            from block_diffusion_speculative_hiddens_gb300 import ops
            st["plan"] = ops.RopePlan(case["rd"], case["theta"], interleaved=case["interleaved"],
                                      scaling=SCALINGS[case["scaling"]])
    if case["op"] == "rope":
        rows = case["rows"]
        if case["packed"]:  # views of the fused projection's output
            qkv = randn(rows, hq + 2 * hkv, d)
            st["q"], st["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv]
        else:
            st["q"], st["k"] = randn(rows, hq, d), randn(rows, hkv, d)
        start = torch.randint(0, case["pos"] + 1, (1,), generator=g, device="cuda")
        st["positions"] = (start + torch.arange(rows, device="cuda")).to(torch.int32)
        return st

    n, ctx = _lengths(case)
    page, b = case["page"], case["b"]
    need = [-(-(x + y) // page) for x, y in zip(n, ctx)]
    total = sum(need)
    pages = total + 3
    # contiguous pages of a free list in random order, as a pool that has served for a while gives them
    ids = torch.randperm(pages, generator=g, device="cuda")[:total].to(torch.int32)
    table = torch.full((b, max(need)), -1, dtype=torch.int32, device="cuda")
    row = torch.repeat_interleave(torch.arange(b, device="cuda"), torch.tensor(need, device="cuda"))
    first = torch.tensor([sum(need[:i]) for i in range(b)], device="cuda")
    table[row, torch.arange(total, device="cuda") - first[row]] = ids
    cu = [sum(n[:i]) for i in range(b + 1)]
    st.update(table=table, cu=torch.tensor(cu, dtype=torch.int32, device="cuda"),
              ctx=torch.tensor(ctx, dtype=torch.int32, device="cuda"))
    t = cu[-1]
    if case["op"] == "append":
        st["k_pool"] = torch.zeros(pages, page, hkv, d, dtype=dt, device="cuda")
        st["v_pool"] = torch.zeros(pages, page, hkv, d, dtype=dt, device="cuda")
        qkv = randn(t, hq + 2 * hkv, d)
        st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        st["k_pool"], st["v_pool"] = randn(pages, page, hkv, d), randn(pages, page, hkv, d)
        st["q"] = randn(t, hq, d) * 1.5
    if own:
        from block_diffusion_speculative_hiddens_gb300 import ops
        st["cache"] = ops.PagedCache(st["k_pool"], st["v_pool"], table)
    return st


# ---- the plain forms

def _rotate(x, positions, freq, factor, rd, interleaved, backward=False):
    angle = positions.double()[:, None] * freq  # 64 bits: far positions make thousands of turns
    cos, sin = (torch.cos(angle) * factor).float()[:, None], (torch.sin(angle) * factor).float()[:, None]
    if backward:
        sin = -sin
    x = x.float()
    if interleaved:
        a, c = x[..., 0:rd:2], x[..., 1:rd:2]
        r = torch.stack((a * cos - c * sin, a * sin + c * cos), -1).flatten(-2)
    else:
        a, c = x[..., :rd // 2], x[..., rd // 2:rd]
        r = torch.cat((a * cos - c * sin, a * sin + c * cos), -1)
    return torch.cat((r, x[..., rd:]), -1)


def _rows(st):
    """Each row's sequence and its place in it."""
    cu = st["cu"].long()
    r = torch.arange(st["q"].shape[0], device="cuda")
    b = torch.searchsorted(cu, r, right=True) - 1
    return b, r - cu[b]


def _plain_attention(st):
    c = st["case"]
    hq, hkv, d, page = c["hq"], c["hkv"], c["d"], c["page"]
    n, ctx = st["cu"].diff().long(), st["ctx"].long()
    pages = st["table"].clamp(min=0).long()
    b, length = pages.shape[0], pages.shape[1] * page
    k = st["k_pool"][pages].reshape(b, length, hkv, d).permute(0, 2, 3, 1).float()
    v = st["v_pool"][pages].reshape(b, length, hkv, d).permute(0, 2, 1, 3).float()
    seq, i = _rows(st)
    most = c["n_hi"]
    q = torch.zeros(b, most, hq, d, device="cuda")
    q[seq, i] = st["q"].float()
    q = q.reshape(b, most, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)
    s = torch.matmul(q, k) * (1.0 / math.sqrt(d))
    s = s.reshape(b, hkv, hq // hkv, most, length)
    key = torch.arange(length, device="cuda")
    pos = ctx[:, None] + torch.arange(most, device="cuda")
    seen = key < (ctx + n)[:, None, None]
    if c["causal"]:
        seen = seen & (key <= pos[..., None])
    if c["window"]:
        seen = seen & (key > pos[..., None] - c["window"])
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e30))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(b, hkv, -1, length), v).reshape(b, hkv, hq // hkv, most, d)
    o = o / total.clamp(min=1e-30)
    return o.permute(0, 3, 1, 2, 4).reshape(b, most, hq, d)[seq, i].to(st["q"].dtype)


def run(st):
    c = st["case"]
    if own:
        from block_diffusion_speculative_hiddens_gb300 import ops
        if c["op"] == "rope":
            return ops.rope(st["plan"], st["q"], st["k"], st["positions"], backward=c["backward"])
        if c["op"] == "append":
            q = ops.append(st["cache"], st["k"], st["v"], st["cu"], st["ctx"], plan=st["plan"], q=st["q"])
            return q, st["k_pool"], st["v_pool"]
        return ops.attention(st["cache"], st["q"], st["cu"], st["ctx"], causal=c["causal"], window=c["window"])
    if c["op"] == "attention":
        return _plain_attention(st)
    how = (st["freq"], st["factor"], c["rd"], c["interleaved"])
    dt = st["q"].dtype
    if c["op"] == "rope":
        return tuple(_rotate(st[x], st["positions"], *how, backward=c["backward"]).to(dt) for x in "qk")
    b, i = _rows(st)
    pos = st["ctx"].long()[b] + i
    at = st["table"].long()[b, pos // c["page"]], pos % c["page"]
    st["k_pool"][at] = _rotate(st["k"], pos, *how).to(dt)
    st["v_pool"][at] = st["v"]
    return _rotate(st["q"], pos, *how).to(dt), st["k_pool"], st["v_pool"]


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "rope":
        values = case["rows"] * (hq + hkv) * d
        return {"bytes": 4 * values + 4 * case["rows"], "flops": 3 * case["rows"] * (hq + hkv) * case["rd"]}
    n, ctx = _lengths(case)
    t, b = sum(n), case["b"]
    if case["op"] == "append":
        pages = sum((y + x - 1) // case["page"] - y // case["page"] + 1 for x, y in zip(n, ctx))
        return {"bytes": 4 * t * (hq + 2 * hkv) * d + 4 * (2 * b + 1 + pages),
                "flops": 3 * t * (hq + hkv) * case["rd"]}
    keys = pairs = 0
    w = case["window"]
    for x, y in zip(n, ctx):
        keys += min(x + y, x + w - 1) if w else x + y
        if not case["causal"]:
            pairs += x * (x + y)
        elif not w:
            pairs += x * y + x * (x + 1) // 2
        else:  # row i sees min(y + i + 1, w) keys
            grow = min(max(w - y, 0), x)
            pairs += grow * y + grow * (grow + 1) // 2 + (x - grow) * w
    pages = sum(-(-(x + y) // case["page"]) for x, y in zip(n, ctx))
    return {"bytes": 4 * t * hq * d + 4 * keys * hkv * d + 4 * (2 * b + 1 + pages), "flops": 4 * pairs * hq * d}


# ---- the definitions, in 64 bits

def _turned(x, pos, case, sign):
    """Rotation as a product of complex numbers, pair by pair, from each scaling's definition."""
    rd, s = case["rd"], SCALINGS[case["scaling"]]
    kind = "none" if s is None else s["kind"]
    z = x.double()
    out = z.clone()
    for i in range(rd // 2):
        w, amp = case["theta"] ** (-2.0 * i / rd), 1.0
        if kind == "linear":
            w /= s["factor"]
        elif kind == "ntk":
            w = (case["theta"] * s["factor"] ** (rd / (rd - 2.0))) ** (-2.0 * i / rd)
        elif kind == "llama3":
            wave = 2 * math.pi / w
            long_wave, short_wave = s["original_len"] / s["low_freq_factor"], s["original_len"] / s["high_freq_factor"]
            if wave > long_wave:
                w = w / s["factor"]
            elif wave >= short_wave:
                m = (s["original_len"] / wave - s["low_freq_factor"]) / (s["high_freq_factor"] - s["low_freq_factor"])
                w = (1 - m) * w / s["factor"] + m * w
        elif kind == "yarn":
            edge = [rd * math.log(s["original_len"] / (beta * 2 * math.pi)) / (2 * math.log(case["theta"]))
                    for beta in (s["beta_fast"], s["beta_slow"])]
            lo, hi = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), rd - 1)
            m = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            w = (1 - m) * w + m * w / s["factor"]
            amp = 1.0 + 0.1 * math.log(s["factor"])
        u, v = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rd // 2)
        unit = torch.polar(torch.full_like(pos, amp, dtype=torch.float64), sign * w * pos.double())[:, None]
        turned = torch.complex(z[..., u], z[..., v]) * unit
        out[..., u], out[..., v] = turned.real, turned.imag
    return out


def exact(case, seed):
    global own
    was, own = own, False  # the inputs alone
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "rope":
        sign = -1.0 if case["backward"] else 1.0
        return tuple(_turned(st[x], st["positions"], case, sign) for x in "qk")
    n, ctx = _lengths(case)
    page, hq, hkv, d = case["page"], case["hq"], case["hkv"], case["d"]
    group = hq // hkv
    out = torch.zeros(sum(n), hq, d, dtype=torch.float64, device="cuda")
    kp, vp = st["k_pool"], st["v_pool"]
    if case["op"] == "append":
        kp, vp = kp.double(), vp.double()
    row = 0
    for b in range(case["b"]):
        rows = slice(row, row + n[b])
        row += n[b]
        pos = torch.arange(ctx[b], ctx[b] + n[b], device="cuda")
        ids = st["table"][b, :-(-(ctx[b] + n[b]) // page)].long()
        if case["op"] == "append":
            out[rows] = _turned(st["q"][rows], pos, case, 1.0)
            kp[ids[pos // page], pos % page] = _turned(st["k"][rows], pos, case, 1.0)
            vp[ids[pos // page], pos % page] = st["v"][rows].double()
            continue
        keys = torch.arange(ctx[b] + n[b], device="cuda")
        k, v = (x[ids].flatten(0, 1)[:len(keys)].double() for x in (kp, vp))
        hidden = torch.zeros(n[b], len(keys), dtype=torch.bool, device="cuda")
        if case["causal"]:
            hidden |= keys[None] > pos[:, None]
        if case["window"]:
            hidden |= pos[:, None] - keys[None] >= case["window"]
        for h in range(hq):
            s = st["q"][rows, h].double() @ k[:, h // group].T / math.sqrt(d)
            s[hidden] = -math.inf
            out[rows, h] = torch.softmax(s, -1) @ v[:, h // group]
    return out if case["op"] == "attention" else (out, kp, vp)
