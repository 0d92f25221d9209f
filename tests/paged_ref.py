"""Plain 64-bit forms of rotary positions, the append to an 8-bit paged cache
and the attention over it, one sequence and one head at a time, and the error
bounds their tests use."""
import math

import torch

F8 = torch.float8_e4m3fn
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}   # half a step, relative
FLOOR = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}  # ... of subnormals
SCALE_FLOOR = 2.0 ** -60
CUDA = "cuda"


def inv_freq(rot, theta=1e4):
    return torch.tensor([theta ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64, device=CUDA)


def rotate(x, pos, f, interleaved=False, amp=1.0, transpose=False):
    """x [tokens, heads, dim] in float64, rotated; and a bound on the fp32
    kernel's error before its last rounding.  The angle reaches sincospi
    rounded to fp32 in half turns (half a step of at most 1: 2^-25 pi radians
    under 2^-23), cos and sin carry at most 2 more steps of 2^-24 each, amp and
    each of the two products one: under 6 * 2^-24 of |a| + |b|, twice 2^-23 for
    the angle; 2^-21 covers their sum."""
    x = x.double()
    half = f.numel()
    ang = pos.double()[:, None, None] * f
    c, s = amp * torch.cos(ang), amp * torch.sin(ang) * (-1.0 if transpose else 1.0)
    i = torch.arange(half, device=x.device)
    a_at, b_at = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a, b = x[..., a_at], x[..., b_at]
    y, err = x.clone(), torch.zeros_like(x)
    y[..., a_at], y[..., b_at] = a * c - b * s, b * c + a * s
    e = (a.abs() + b.abs()) * abs(amp) * 2.0 ** -21
    err[..., a_at], err[..., b_at] = e, e
    return y, err


def values(codes, scale):
    """[pages, heads, size, dim] values of codes and scales, float64."""
    return codes.double() * scale.double()[:, :, None, None]


def cached(codes, scale, table_row, length, head):
    """The first `length` cached rows of one sequence and head, float64."""
    size = codes.shape[2]
    n = -(-length // size)
    pg = table_row[:n].long()
    return values(codes.view(torch.int8)[pg].view(codes.dtype), scale[pg])[:, head].reshape(-1, codes.shape[3])[:length]


def attention(q, kc, vc, ks, vs, q_off, kv_len, table, causal, scale, skip_pages=()):
    """(out, lse, out_bound, lse_bound) in float64 of every row of a sequence.

    Bounds, for a row with softmax weights p: the fp32 score of a key is off by
    at most D 2^-24 sum |q k| scale (the products are exact, D additions), by
    2^-23 of the largest |x| handled in log2 units (three roundings of x), and
    exp2 and log2 by 2^-21 together; all enter as a relative error of p.  p is
    rounded once to fp16 (2^-11), the output once to its type; the normaliser
    carries the same relative errors as p, so they count twice."""
    n, hq, d = q.shape
    hkv = kc.shape[1]
    out = torch.zeros(n, hq, d, dtype=torch.float64, device=q.device)
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device=q.device)
    ob, lb = torch.zeros_like(out), torch.zeros_like(lse)
    off, lens = q_off.tolist(), kv_len.tolist()
    bad = torch.tensor(sorted(skip_pages), dtype=torch.int64, device=q.device)
    size = kc.shape[2]
    for s, L in enumerate(lens):
        r0, r1 = off[s], off[s + 1]
        if r1 == r0 or L == 0:
            continue
        row_pages = table[s]
        j = torch.arange(L, device=q.device)
        ok_page = (row_pages >= 0) & (row_pages < kc.shape[0])
        if bad.numel():
            ok_page &= ~torch.isin(row_pages.long(), bad)
        key_ok = ok_page[j // size]
        pages = torch.where(ok_page, row_pages, 0)
        seen = (L - (r1 - r0) + torch.arange(r1 - r0, device=q.device) + 1) if causal else torch.full((r1 - r0,), L, device=q.device)
        vis = (j[None, :] < seen[:, None]) & key_ok[None, :]
        for h in range(hkv):
            k, v = cached(kc, ks, pages, L, h), cached(vc, vs, pages, L, h)
            sv = vs.double()[pages.long(), h].clamp(min=SCALE_FLOOR)[j // size]
            for e in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                x = q[r0:r1, e].double()
                z = (x @ k.T) * scale
                za = (x.abs() @ k.abs().T) * scale
                z = torch.where(vis, z, torch.full_like(z, -math.inf))
                l = torch.logsumexp(z, -1)
                none = ~vis.any(-1)
                p = torch.where(none[:, None] | ~vis, torch.zeros_like(z), torch.exp(z - l[:, None]))
                out[r0:r1, e] = torch.where(none[:, None], torch.zeros_like(out[r0:r1, e]), p @ torch.where(key_ok[:, None], v, 0.0))
                lse[r0:r1, e] = torch.where(none, torch.full_like(l, -math.inf), l)
                big = (za.masked_fill(~vis, 0.0) * math.log2(math.e) + torch.log2(sv).abs()[None, :].masked_fill(~vis, 0.0)).amax(-1)
                rel = d * 2.0 ** -24 * za.masked_fill(~vis, 0.0).amax(-1) + big * 2.0 ** -23 + 2.0 ** -21
                lb[r0:r1, e] = rel + 2.0 ** -22 * torch.where(none, torch.zeros_like(l), l.abs())
                o = out[r0:r1, e]
                mag = p @ torch.where(key_ok[:, None], v, 0.0).abs()
                # fp16 loses weights 2^-33 of the reference at most: their count times the largest value
                tiny = 2.0 ** -33 * L * (v.abs().amax() if L else 0.0)
                ob[r0:r1, e] = mag * (2.0 ** -11 + 2 * rel[:, None]) * 1.01 + o.abs() * HALF[q.dtype] * 1.01 + FLOOR[q.dtype] + tiny * p.amax(-1)[:, None]
    return out, lse, ob, lb


def make_table(lens, size, n_extra=3, seed=0):
    """A block table [n_seq, width] whose pages are scattered over a pool; unused entries are -1."""
    g = torch.Generator().manual_seed(seed)
    per = [-(-n // size) for n in lens]
    width, pool = max(max(per, default=0), 1), sum(per) + n_extra
    perm = torch.randperm(pool, generator=g).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(per):
        table[i, :n] = perm[at:at + n]
        at += n
    return table.to(CUDA), pool


def make_cache(pool, heads, size, dim, fmt, seed=0, order="head"):
    """Random codes and scales; order "slot" lays pages out as [slot][head]."""
    g = torch.Generator(device=CUDA).manual_seed(seed)
    shape = (pool, heads, size, dim)

    def codes():
        x = torch.randn(*shape, generator=g, device=CUDA)
        x = (x * 32).clamp(-127, 127).round().to(torch.int8) if fmt == "int8" else (x * 72).clamp(-448, 448).to(F8)
        if order == "slot":
            x = x.view(torch.int8).transpose(1, 2).contiguous().transpose(1, 2).view(x.dtype)
        return x

    def scales():
        s = torch.exp2(0.5 * torch.randn(pool, heads, generator=g, device=CUDA)) * (0.8 / (32 if fmt == "int8" else 72))
        return s if fmt == "int8" else torch.exp2(torch.ceil(torch.log2(s)))

    return codes(), codes(), scales(), scales()


def i32(v):
    return torch.tensor(list(v), dtype=torch.int32, device=CUDA)


def offsets(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return i32(out)
