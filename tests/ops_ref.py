"""Plain 64-bit definitions of the caller-target operators, for the tests:
loops over sequences, no paging shortcuts, written from the formulas."""
import math

import torch


def frequencies(rd, theta, scaling=None):
    """Angles per position of the rd/2 pairs (float64 list) and the amplitude."""
    s = dict(scaling or {"kind": "none"})
    kind, f = s["kind"], s.get("factor", 1.0)
    out, amp = [], 1.0
    for i in range(rd // 2):
        w = theta ** (-2.0 * i / rd)
        if kind == "linear":
            w = w / f
        elif kind == "ntk":
            w = (theta * f ** (rd / (rd - 2.0))) ** (-2.0 * i / rd)
        elif kind == "factors":
            w = w / s["factors"][i]
            amp = s.get("attention_factor", 1.0)
        elif kind == "yarn":
            def pair(beta):
                return rd * math.log(s["original_len"] / (beta * 2 * math.pi)) / (2 * math.log(theta))
            lo = max(math.floor(pair(s.get("beta_fast", 32))), 0)
            hi = min(math.ceil(pair(s.get("beta_slow", 1))), rd - 1)
            m = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            w = (1 - m) * w + m * w / f
            amp = s.get("attention_factor", 0.1 * math.log(f) + 1.0)
        elif kind == "llama3":
            wave, lf, hf, n = 2 * math.pi / w, s.get("low_freq_factor", 1), s.get("high_freq_factor", 4), s["original_len"]
            if wave > n / lf:
                w = w / f
            elif wave >= n / hf:
                m = (n / wave - lf) / (hf - lf)
                w = (1 - m) * w / f + m * w
        out.append(w)
    return out, amp


def rotate(x, positions, rd, freq, amp, interleaved, backward=False):
    """x [rows, heads, dim] in float64; also the sum of magnitudes behind each value."""
    x = x.double()
    y, mag = x.clone(), x.abs()
    pos = positions.double()
    for i in range(rd // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rd // 2)
        c, s = torch.cos(pos * freq[i])[:, None] * amp, torch.sin(pos * freq[i])[:, None] * amp
        if backward:
            s = -s
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
        mag[..., a] = mag[..., b] = (x[..., a].abs() + x[..., b].abs()) * amp
    return y, mag


def rotate_tolerance(y, mag, dtype):
    """One rounding to dtype, and behind it in float32: cos, sin (angle off by
    2^-24 of a half turn, the function's two last places) and three roundings."""
    half = torch.finfo(dtype).eps / 2
    return half * y.abs() + 16 * 2.0 ** -24 * mag + 2.0 ** -25


def attention(q, k, v, pos0, kv_len, causal, window, scale):
    """One sequence: q [n, hq, D], k, v [keys, hkv, D] (positions 0..): out and
    lse in float64, and what the tolerance needs."""
    n, hq, _ = q.shape
    hkv = k.shape[1]
    q, k, v = q.double(), k[:max(kv_len, 0)].double(), v[:max(kv_len, 0)].double()
    keys = torch.arange(k.shape[0], device=q.device)
    pos = pos0 + torch.arange(n, device=q.device)
    see = torch.ones(n, len(keys), dtype=torch.bool, device=q.device)
    if causal:
        see &= keys[None] <= pos[:, None]
    if window > 0:
        see &= keys[None] > pos[:, None] - window
    out = torch.zeros_like(q)
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device=q.device)
    mag = torch.zeros_like(q)                       # sum_j p_j |v_j|
    ds = torch.zeros(n, hq, dtype=torch.float64, device=q.device)  # largest sum |q||k| scale of a seen key
    some = see.any(-1)
    for h in range(hq):
        g = h // (hq // hkv)
        if not some.any():
            break
        s = (q[:, h] @ k[:, g].T * scale).masked_fill(~see, -math.inf)[some]
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - m)
        l = p.sum(-1, keepdim=True)
        out[some, h] = p @ v[:, g] / l
        mag[some, h] = p @ v[:, g].abs() / l
        lse[some, h] = (m + torch.log(l))[:, 0]
        ds[some, h] = (q[:, h].abs() @ k[:, g].abs().T * abs(scale)).masked_fill(~see, 0)[some].amax(-1)
    return out, lse, mag, ds, see.sum(-1)


def attention_tolerance(out, lse, mag, ds, seen, dtype, dim, vmax):
    """Per value.  A score is a sum of dim products in float32 (dim 2^-24 of the
    sum of magnitudes, doubled for the base-2 scale): `es`.  Every probability is
    off by that and by its rounding to dtype; f16 ones below 2^-14 by 2^-25 of
    the largest; the sums by n 2^-24; the output by its own rounding."""
    half = torch.finfo(dtype).eps / 2
    n = seen.double()[:, None]
    es = 2 * (dim + 4) * 2.0 ** -24 * ds + 2.0 ** -21
    tol_out = half * out.abs() + (half + 2 * es + 4 * n * 2.0 ** -24)[..., None] * mag + 2.0 ** -25
    if dtype == torch.float16:
        tol_out = tol_out + (n * 2.0 ** -25 * vmax)[..., None]
    tol_lse = 2 * es + 4 * n * 2.0 ** -24 + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0)
    return tol_out, tol_lse
