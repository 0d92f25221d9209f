"""The operators around the 8-bit paged KV cache, as they are measured.

Three operators that a serving loop calls one after the other in every layer:

  rope    rotary positions on a [tokens, heads, head_dim] tensor: half or
          interleaved pairs, the whole head or its first part, frequencies
          scaled for long contexts, and the transposed rotation (the gradient);
  append  new keys and values into a paged cache of 8-bit codes with one scale
          for each page and KV head, the keys rotated on the way;
  attend  ragged queries over that cache: single tokens, branch rows over a
          shared prefix, causal chunks.

`own` chooses between the package's kernels and the plain forms below, which
use elementary torch operations in 32 bits (angles in 64).
"""
import math
import random

import numpy as np
import torch

own = False

_F8 = torch.float8_e4m3fn
_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # q and k heads of one projection (12 + 2 heads of 128), one token of each of 64 requests
        dict(name="rope one token x64", op="rope", tokens=64, heads=14, dim=128, rot=128, pairs="half", dtype="f16",
             theta=1e6, scaling="none", factor=1.0, far=32768, transpose=False, extra=0),
        # q and k heads (28 + 4) of a long document's prefill, wavelength-scaled frequencies, far positions
        dict(name="rope 8192 far", op="rope", tokens=8192, heads=32, dim=128, rot=128, pairs="half", dtype="f16",
             theta=1e6, scaling="bands", factor=8.0, far=1000000, transpose=False, extra=0),
        # the gradient of an interleaved rotation of part of the head, rows of a wider fused projection
        dict(name="rope gradient part", op="rope", tokens=5001, heads=20, dim=80, rot=32, pairs="interleaved",
             dtype="bf16", theta=1e4, scaling="ramp", factor=4.0, far=16384, transpose=True, extra=10),
        # one new token of each of 64 running requests (28/4 heads: 4 KV heads), pages of 64
        dict(name="append one token x64", op="append", seqs=64, new=1, spread=0, old=8192, kv_heads=4, dim=128,
             page=64, fmt="e4m3", dtype="f16", pairs="half", rot=128),
        # a batch of prompts prefilled in one pass
        dict(name="append prompts", op="append", seqs=12, new=1200, spread=700, old=0, kv_heads=4, dim=128, page=64,
             fmt="e4m3", dtype="f16", pairs="half", rot=128),
        # answer lines written after cached prefixes, keys already rotated by the projection's epilogue
        dict(name="append lines int8", op="append", seqs=7, new=45, spread=40, old=901, kv_heads=2, dim=64, page=16,
             fmt="int8", dtype="bf16", pairs="none", rot=0),
        # a single request's token over the 901-token prompt of the 28-field request (12/2 heads)
        dict(name="attend one token 901", op="attend", seqs=1, q=1, q_spread=0, kv=901, kv_spread=0, heads=12,
             kv_heads=2, dim=128, page=64, fmt="e4m3", dtype="f16", causal=True, lse=False),
        # batched serving, one token of each of 64 requests with ragged contexts (28/4 heads)
        dict(name="attend one token x64", op="attend", seqs=64, q=1, q_spread=0, kv=8192, kv_spread=4000, heads=28,
             kv_heads=4, dim=128, page=64, fmt="e4m3", dtype="f16", causal=True, lse=False),
        # few very long contexts, one token each
        dict(name="attend one token long int8", op="attend", seqs=3, q=1, q_spread=0, kv=131001, kv_spread=0,
             heads=28, kv_heads=4, dim=128, page=128, fmt="int8", dtype="bf16", causal=True, lse=False),
        # 313 branch rows of one request over its cached prefix, every row seeing all of it (12/2 heads);
        # the log-sum-exp joins them with the branch's own keys
        dict(name="attend branch rows", op="attend", seqs=1, q=313, q_spread=0, kv=901, kv_spread=0, heads=12,
             kv_heads=2, dim=128, page=16, fmt="int8", dtype="f16", causal=False, lse=True),
        # a chunk of 2048 document tokens behind 6144 cached ones, two documents
        dict(name="attend chunk 2048", op="attend", seqs=2, q=2048, q_spread=0, kv=8192, kv_spread=0, heads=28,
             kv_heads=4, dim=128, page=64, fmt="e4m3", dtype="f16", causal=True, lse=False),
        # ragged prompts of odd lengths, heads of 64
        dict(name="attend ragged prompts", op="attend", seqs=9, q=401, q_spread=390, kv=1103, kv_spread=600, heads=14,
             kv_heads=2, dim=64, page=32, fmt="e4m3", dtype="bf16", causal=True, lse=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("rope", "append", "attend", "attend"))
    if op == "rope":
        dim = rng.choice((64, 80, 96, 128, 256))
        rot = dim if rng.random() < 0.5 else 2 * rng.randint(4, dim // 2)
        dtype = rng.choice(("f16", "bf16", "f32"))
        heads = rng.randint(1, 40)
        most = max(1, min(8192, 8192 * 32 * 128 * 2 // (heads * dim * _SIZE[dtype])))
        return dict(op="rope", tokens=_log(rng, 1, most), heads=heads, dim=dim, rot=rot,
                    pairs=rng.choice(("half", "interleaved")), dtype=dtype, theta=rng.choice((1e4, 5e5, 1e6)),
                    scaling=rng.choice(("none", "linear", "base", "bands", "ramp")), factor=rng.choice((2.0, 4.0, 8.0)),
                    far=_log(rng, 1000, 1000000), transpose=rng.random() < 0.3, extra=rng.choice((0, 0, 3)))
    if op == "append":
        fmt = rng.choice(("e4m3", "e4m3", "int8"))
        dim = rng.choice((64, 128))
        seqs = _log(rng, 1, 64)
        new = _log(rng, 1, max(1, 14000 // seqs))
        rotated = fmt == "e4m3"  # int8 codes are compared exactly, so those keys come rotated
        return dict(op="append", seqs=seqs, new=new, spread=rng.randint(0, new - 1), old=_log(rng, 1, 8192) - 1,
                    kv_heads=rng.choice((1, 2, 4)), dim=dim, page=rng.choice((16, 32, 64, 128)), fmt=fmt,
                    dtype=rng.choice(("f16", "bf16", "f32")),
                    pairs=rng.choice(("half", "interleaved")) if rotated else "none",
                    rot=(dim if rng.random() < 0.5 else 2 * rng.randint(4, dim // 2)) if rotated else 0)
    dim = rng.choice((64, 128, 128))
    kv_heads = rng.choice((1, 2, 4))
    heads = kv_heads * rng.choice((1, 2, 4, 6, 7, 8, 16))
    seqs = _log(rng, 1, 64)
    q = 1 if rng.random() < 0.5 else _log(rng, 1, 2048)
    most_q = max(1, 4096 // seqs)
    q = min(q, most_q)
    # under the largest listed cases: 268 M cached channels of keys, 66 G products of a query row, a key and a channel
    most_kv = min(131001, 268 * 10**6 // (seqs * kv_heads * dim), 66 * 10**9 // (seqs * q * heads * dim))
    kv = _log(rng, min(most_kv, max(1, q)), max(most_kv, 2))
    return dict(op="attend", seqs=seqs, q=q, q_spread=rng.randint(0, q - 1), kv=kv, kv_spread=rng.randint(0, kv // 2),
                heads=heads, kv_heads=kv_heads, dim=dim, page=rng.choice((16, 32, 64, 128)),
                fmt=rng.choice(("e4m3", "int8")), dtype=rng.choice(("f16", "bf16")), causal=rng.random() < 0.7,
                lse=rng.random() < 0.5)


def _lens(mean, spread, n, salt):
    """n lengths in mean +- spread that depend on the case alone, the first one mean + spread."""
    r = random.Random(1000003 * mean + 1009 * spread + 31 * n + salt)
    return [mean + spread] + [max(0, mean + r.randint(-spread, spread)) for _ in range(n - 1)]


def _case_lens(case):
    if case["op"] == "append":
        new = _lens(case["new"], case["spread"], case["seqs"], 1)
        old = _lens(case["old"], case["old"] // 2, case["seqs"], 2)
        return new, [n + o for n, o in zip(new, old)]
    return (_lens(case["q"], case["q_spread"], case["seqs"], 3), _lens(case["kv"], case["kv_spread"], case["seqs"], 4))


# ------------------------------------------------------------------ frequencies
def _inv_freq(rot, theta, scaling, factor, far):
    """Radians per position of each pair, in 64 bits, and the amplitude factor."""
    half = rot // 2
    i = np.arange(half, dtype=np.float64)
    orig = max(1.0, far / factor)
    if scaling == "base" and rot > 2:
        theta = theta * factor ** (rot / (rot - 2.0))
    f = theta ** (-2.0 * i / rot)
    amp = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "bands":  # wavelengths under orig / 4 stay, those over orig are stretched, a blend between
        turns = orig * f / (2.0 * math.pi)
        s = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        f = (1.0 - s) * f / factor + s * f
    elif scaling == "ramp":  # pairs that turn over 32 times stay, those under once are stretched, a ramp between
        at = lambda turns: rot * math.log(orig / (turns * 2.0 * math.pi)) / (2.0 * math.log(theta))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        r = np.clip((i - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
        f = f / factor * r + f * (1.0 - r)
        amp = 0.1 * math.log(factor) + 1.0
    return f, amp


def _turns(f):
    """The frequencies as fractions of a turn per position, in units of 2^-64."""
    whole = [int(round(x / (2.0 * math.pi) * 2.0 ** 64)) % (1 << 64) for x in f.tolist()]
    return torch.from_numpy(np.array(whole, dtype=np.uint64).view(np.int64)).cuda()


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _offsets(lens):
    return _i32(np.concatenate([[0], np.cumsum(lens)]).tolist())


def _pages(g, lens, page):
    """A block table with the pages of every sequence scattered over the pool, and the pool's size."""
    per = [-(-n // page) for n in lens]
    width = max(max(per), 1)
    n_pages = sum(per) + 3
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    start = torch.tensor(np.concatenate([[0], np.cumsum(per)[:-1]]), device="cuda")
    at = start[:, None] + torch.arange(width, device="cuda")[None, :]
    table = perm[at.clamp(max=n_pages - 1)].contiguous()
    return table, n_pages


def _codes(g, shape, fmt):
    """Cached codes: the values of a page fill the format's range up to its largest."""
    x = _randn(g, *shape)
    return (x * 32.0).clamp(-127, 127).round().to(torch.int8) if fmt == "int8" else (x * 72.0).clamp(-448, 448).to(_F8)


def _scales(g, shape, fmt, size):
    """Scales that give the codes a spread of about `size`, different for each page and head."""
    s = torch.exp2(0.4 * _randn(g, *shape)) * (size / (32.0 if fmt == "int8" else 72.0))
    return s if fmt == "int8" else torch.exp2(torch.ceil(torch.log2(s)))


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "rope":
        f, amp = _inv_freq(case["rot"], case["theta"], case["scaling"], case["factor"], case["far"])
        wide = _randn(g, case["tokens"], case["heads"] + case["extra"], case["dim"]).to(_DT[case["dtype"]])
        pos = torch.randint(0, case["far"], (case["tokens"],), generator=g, device="cuda", dtype=torch.int32)
        return dict(op="rope", x=wide[:, :case["heads"]], pos=pos, freqs=_turns(f), amp=amp, rot=case["rot"],
                    interleaved=case["pairs"] == "interleaved", transpose=case["transpose"])
    q_lens, kv_lens = _case_lens(case)
    hkv, d, page, fmt = case["kv_heads"], case["dim"], case["page"], case["fmt"]
    table, n_pages = _pages(g, kv_lens, page)
    shape = (n_pages, hkv, page, d)
    state = dict(op=case["op"], fmt=fmt, page=page, q_off=_offsets(q_lens), kv_len=_i32(kv_lens), table=table,
                 max_q=max(q_lens), max_kv=max(kv_lens), k_cache=_codes(g, shape, fmt), v_cache=_codes(g, shape, fmt),
                 k_scale=_scales(g, (n_pages, hkv), fmt, 0.8), v_scale=_scales(g, (n_pages, hkv), fmt, 0.8))
    n = sum(q_lens)
    if case["op"] == "append":
        dt = _DT[case["dtype"]]
        qkv = _randn(g, n, 4 * hkv, d)  # the fused projection: keys and values are slices of its rows
        qkv[:, :, ::17] *= 4.0          # a few channels stand out, as in trained decoders
        qkv = qkv.to(dt)
        f, _ = _inv_freq(max(case["rot"], 2), 1e6, "none", 1.0, 1)
        state.update(k=qkv[:, 2 * hkv:3 * hkv], v=qkv[:, 3 * hkv:], rot=case["rot"],
                     freqs=_turns(f) if case["rot"] else None, interleaved=case["pairs"] == "interleaved")
        return state
    state.update(q=(2.0 * _randn(g, n, case["heads"], d)).to(_DT[case["dtype"]]), causal=case["causal"],
                 lse=case["lse"], scale=1.0 / math.sqrt(d))
    return state


# ------------------------------------------------------------------ plain forms
def _cos_sin(pos, freqs):
    """cos and sin [tokens, pairs] from angles kept in 64 bits."""
    phase = pos.to(torch.int64)[:, None] * freqs[None, :]  # wraps: whole turns drop out
    angle = phase.to(torch.float64) * (2.0 * math.pi / 2.0 ** 64)
    return torch.cos(angle).float(), torch.sin(angle).float()


def _rotate(x, pos, freqs, interleaved, amp, transpose):
    """The rotation of x's first 2 * len(freqs) channels, in 32 bits."""
    rot = 2 * freqs.numel()
    x = x.float()
    cos, sin = _cos_sin(pos, freqs)
    cos, sin = (cos * amp)[:, None, :], (sin * amp)[:, None, :]
    if transpose:
        sin = -sin
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((y, x[..., rot:]), dim=-1)


def _places(s):
    """Sequence, page and slot of every new token, and its position."""
    n = s["k"].shape[0]
    t = torch.arange(n, device="cuda")
    seq = torch.searchsorted(s["q_off"][1:].contiguous(), t.to(torch.int32), right=True)
    pos = s["kv_len"][seq].to(torch.int64) - s["q_off"][seq + 1] + t
    return s["table"][seq, pos // s["page"]].to(torch.int64), pos % s["page"], pos


def _take(cache, at):
    """cache[at] as bytes, for index tensors and slices: 8-bit floats are moved as integers."""
    return cache.view(torch.int8)[at].view(cache.dtype)


def _store(s, x, cache, scale, pages, slots):
    """New rows x [tokens, heads, dim] (32 bits) into one of the two caches."""
    int8 = s["fmt"] == "int8"
    fit = lambda c: (c.round().clamp(-127, 127) if int8 else c.clamp(-448, 448)).to(cache.dtype)  # noqa: E731
    amax = torch.zeros_like(scale).index_reduce_(0, pages, x.abs().amax(-1), "amax")
    if int8:
        want = amax / 127.0
    else:  # the next power of two: codes of another scale move by whole exponents
        part, power = torch.frexp(amax / 448.0)
        want = torch.ldexp(torch.ones_like(amax), power - (part == 0.5).to(power.dtype))
    want = want.clamp(min=2.0 ** -60)
    touched = torch.zeros(scale.shape[0], dtype=torch.bool, device="cuda").index_fill_(0, pages, True)
    # every sequence has new tokens here, and old ones share a page with them only in its first page of this call
    start = (s["kv_len"] - (s["q_off"][1:] - s["q_off"][:-1])).to(torch.int64)
    row = torch.arange(start.numel(), device="cuda")
    first, held = s["table"][row, start // s["page"]].to(torch.int64), start % s["page"]
    has = torch.zeros_like(scale).index_copy_(0, first, (held > 0).float()[:, None].expand(-1, scale.shape[1]).contiguous())
    old = scale.clone()
    new = torch.where(has > 0, torch.maximum(old, want), want)
    scale.copy_(torch.where(touched[:, None], new, old))
    before = _take(cache, first)
    after = fit(before.float() * (old[first] / scale[first])[:, :, None, None])
    keep = (torch.arange(s["page"], device="cuda")[None, :] < held[:, None])[:, None, :, None]
    raw = cache.view(torch.int8)
    raw[first] = torch.where(keep, after.view(torch.int8), before.view(torch.int8))
    raw.permute(0, 2, 1, 3)[pages, slots] = fit(x * (1.0 / scale[pages])[:, :, None]).view(torch.int8)


def _plain_append(s):
    pages, slots, pos = _places(s)
    k = s["k"].float() if s["freqs"] is None else _rotate(s["k"], pos, s["freqs"], s["interleaved"], 1.0, False)
    _store(s, k, s["k_cache"], s["k_scale"], pages, slots)
    _store(s, s["v"].float(), s["v_cache"], s["v_scale"], pages, slots)


def _plain_attend(s):
    page, q = s["page"], s["q"]
    n_seq, hkv, d, hq = s["kv_len"].numel(), s["k_cache"].shape[1], q.shape[2], q.shape[1]
    grp, mq, width = hq // hkv, s["max_q"], -(-s["max_kv"] // page)
    table = s["table"][:, :width].to(torch.int64)
    rows = lambda c, sc: (_take(c, table).float() * sc[table][..., None, None]).permute(0, 2, 1, 3, 4).reshape(n_seq, hkv, width * page, d)  # noqa: E731
    k, v = rows(s["k_cache"], s["k_scale"]), rows(s["v_cache"], s["v_scale"])
    n_q = s["q_off"][1:] - s["q_off"][:-1]
    i = torch.arange(mq, device="cuda")
    at = (s["q_off"][:-1, None] + i[None, :]).clamp(max=max(q.shape[0] - 1, 0)).to(torch.int64)
    x = q[at].float().reshape(n_seq, mq, hkv, grp, d).permute(0, 2, 3, 1, 4).reshape(n_seq, hkv, grp * mq, d)
    z = torch.matmul(x, k.transpose(-1, -2)).mul_(s["scale"]).view(n_seq, hkv, grp, mq, width * page)
    seen = s["kv_len"][:, None] - n_q[:, None] + i[None, :] + 1 if s["causal"] else s["kv_len"][:, None].expand(n_seq, mq)
    hide = torch.arange(width * page, device="cuda")[None, None, :] >= seen[:, :, None]
    z.masked_fill_(hide[:, None, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    none = torch.isinf(m)
    z.sub_(torch.where(none, 0.0, m)).exp_()
    total = z.sum(-1, keepdim=True)
    y = torch.matmul(z.view(n_seq, hkv, grp * mq, width * page), v).view(n_seq, hkv, grp, mq, d)
    y = y / torch.where(none, 1.0, total)
    t = torch.arange(q.shape[0], device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["q_off"][1:].contiguous(), t, right=True)
    place = (t - s["q_off"][seq]).to(torch.int64)
    out = y.permute(0, 3, 1, 2, 4).reshape(n_seq, mq, hq, d)[seq, place].to(q.dtype)
    if not s["lse"]:
        return out
    lse = (m + torch.log(total))[..., 0].permute(0, 3, 1, 2).reshape(n_seq, mq, hq)[seq, place]
    return out, lse


def run(state):
    s = state
    if s["op"] == "rope":
        if own:
            from constrained_decoding_gb300 import paged
            return paged.pcd_k_rope(s["x"], s["freqs"], s["pos"], interleaved=s["interleaved"], amp=s["amp"],
                                    transpose=s["transpose"])
        return _rotate(s["x"], s["pos"], s["freqs"], s["interleaved"], s["amp"], s["transpose"]).to(s["x"].dtype)
    if s["op"] == "append":
        if own:
            from constrained_decoding_gb300 import paged
            paged.pcd_k_kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["q_off"],
                                  s["kv_len"], s["table"], freqs=s["freqs"], interleaved=s["interleaved"])
        else:
            _plain_append(s)
        return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    if own:
        from constrained_decoding_gb300 import paged
        return paged.pcd_k_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["q_off"],
                                           s["kv_len"], s["table"], max_kv=s["max_kv"], causal=s["causal"],
                                           scale=s["scale"], return_lse=s["lse"])
    return _plain_attend(s)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"]
        return dict(bytes=2 * n * case["dim"] * _SIZE[case["dtype"]] + 4 * case["tokens"] + 4 * case["rot"],
                    flops=3 * n * case["rot"])
    q_lens, kv_lens = _case_lens(case)
    hkv, d, page = case["kv_heads"], case["dim"], case["page"]
    if case["op"] == "append":
        n = sum(q_lens) * hkv * d
        pages = sum(-(-l // page) - (l - q) // page for q, l in zip(q_lens, kv_lens) if q)
        return dict(bytes=2 * n * (_SIZE[case["dtype"]] + 1) + pages * (8 * hkv + 4), flops=3 * n + 6 * n)
    cached = sum(kv_lens) * hkv * d * 2 + sum(-(-l // page) for l in kv_lens) * (8 * hkv + 4)
    rows = sum(q_lens) * case["heads"]
    if case["causal"]:
        pairs = sum(max(0, l - q + i + 1) for q, l in zip(q_lens, kv_lens) for i in range(q))
    else:
        pairs = sum(q * l for q, l in zip(q_lens, kv_lens))
    return dict(bytes=cached + 2 * rows * d * 2 + (4 * rows if case["lse"] else 0), flops=4 * pairs * case["heads"] * d)


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_turn(x, pos, f, interleaved, amp, sign):
    """Each pair as a complex number times amp * exp(i * sign * pos * f)."""
    half = f.numel()
    x = x.double()
    first = torch.arange(half, device="cuda") * (2 if interleaved else 1)
    second = first + (1 if interleaved else half)
    z = torch.polar(torch.full_like(f, amp).expand(pos.numel(), half), sign * pos.double()[:, None] * f[None, :])
    z = torch.complex(x[..., first], x[..., second]) * z[:, None, :]
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        f, amp = _inv_freq(case["rot"], case["theta"], case["scaling"], case["factor"], case["far"])
        return _exact_turn(s["x"], s["pos"], torch.from_numpy(f).cuda(), s["interleaved"], amp,
                           -1.0 if case["transpose"] else 1.0)
    q_lens, kv_lens = _case_lens(case)
    page = case["page"]
    table = s["table"].cpu().tolist()
    if case["op"] == "append":
        int8 = case["fmt"] == "int8"
        top = 127.0 if int8 else 448.0
        out = []
        for which in "kv":
            codes, scale = s[which + "_cache"].double(), s[which + "_scale"].double()
            at = 0
            for i, (n, l) in enumerate(zip(q_lens, kv_lens)):
                x = s[which][at:at + n].double()
                pos = torch.arange(l - n, l, device="cuda")
                if which == "k" and case["rot"]:
                    f, _ = _inv_freq(case["rot"], 1e6, "none", 1.0, 1)
                    x = _exact_turn(x, pos, torch.from_numpy(f).cuda(), s["interleaved"], 1.0, 1.0)
                at += n
                for p in range((l - n) // page, -(-l // page) if n else 0):
                    lo, hi = max(p * page, l - n), min((p + 1) * page, l)
                    held, rows = lo - p * page, x[lo - (l - n):hi - (l - n)].transpose(0, 1)
                    need = rows.abs().amax((1, 2)) / top
                    need = need if int8 else torch.exp2(torch.ceil(torch.log2(need)))
                    pg = table[i][p]
                    to = torch.maximum(need, scale[pg]) if held else need
                    if held:
                        codes[pg, :, :held] *= (scale[pg] / to)[:, None, None]
                    codes[pg, :, held:held + hi - lo] = rows / to[:, None, None]
                    scale[pg] = to
            out += [None if int8 else codes, scale]
        return out[0], out[2], out[1], out[3]
    hq, hkv, d = case["heads"], case["kv_heads"], case["dim"]
    ys, ls = [], []
    at = 0
    for i, (n, l) in enumerate(zip(q_lens, kv_lens)):
        pg = torch.tensor(table[i][:-(-l // page)], dtype=torch.int64, device="cuda")
        q = s["q"][at:at + n].double().transpose(0, 1)
        at += n
        y = torch.zeros(hq, n, d, dtype=torch.float64, device="cuda")
        ll = torch.full((hq, n), -math.inf, dtype=torch.float64, device="cuda")
        seen = torch.arange(l - n, l, device="cuda") + 1 if case["causal"] else torch.full((n,), l, device="cuda")
        for h in range(hkv if n and l else 0):
            k = (s["k_cache"][pg, h].double() * s["k_scale"][pg, h].double()[:, None, None]).reshape(-1, d)[:l]
            v = (s["v_cache"][pg, h].double() * s["v_scale"][pg, h].double()[:, None, None]).reshape(-1, d)[:l]
            for j in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                z = (q[j] @ k.T) * s["scale"]
                z = torch.where(torch.arange(l, device="cuda")[None, :] < seen[:, None], z, -math.inf)
                lse = torch.logsumexp(z, -1)
                w = torch.where(torch.isinf(lse)[:, None], 0.0, torch.exp(z - lse[:, None]))
                y[j], ll[j] = w @ v, lse
        ys.append(y.transpose(0, 1))
        ls.append(ll.transpose(0, 1))
    out = torch.cat(ys)
    return (out, torch.cat(ls)) if case["lse"] else out
