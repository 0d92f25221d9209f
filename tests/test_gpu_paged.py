"""Rotary positions, the append to an 8-bit paged cache and the attention over
it against plain 64-bit forms (paged_ref), at the sizes, layouts and masks where
they can go wrong."""
import math

import pytest
import torch

import paged_ref as R
from paged_ref import F8, i32, offsets

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def paged():
    from constrained_decoding_gb300 import paged
    return paged


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ------------------------------------------------------------------------ rope
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,heads,dim,rot,inter,transpose", [
    (1, 1, 2, 2, False, False), (1, 14, 128, 128, False, False), (3, 5, 80, 32, True, False),
    (7, 3, 64, 62, False, True), (129, 2, 96, 96, True, True), (33, 32, 128, 64, False, False),
    (2, 40, 256, 256, False, True), (513, 1, 16, 16, False, False), (5, 2, 7, 4, True, False), (17, 4, 128, 2, False, False),
    (9, 3, 40, 24, False, False), (9, 3, 40, 12, True, True), (6, 5, 22, 12, False, True), (6, 9, 22, 6, True, False),
    (2100, 7, 64, 64, False, False),
])
def test_rope(paged, dtype, n, heads, dim, rot, inter, transpose):
    g = gen(n * 131 + heads)
    x = torch.randn(n, heads, dim, generator=g, device="cuda").to(DT[dtype])
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (n,), generator=g, device="cuda", dtype=torch.int32)
    pos[0] = 2 ** 31 - 1
    freqs, amp = paged.pcd_rope_freqs(rot, 1e4)
    y = paged.pcd_k_rope(x, freqs.cuda(), pos, interleaved=inter, amp=1.25, transpose=transpose)
    # the 64-bit angle at such positions: from the turn fractions, as integers
    turns = (pos.cpu().to(torch.int64)[:, None] * freqs[None, :]).double() * 2.0 ** -64
    ref, err = torch.empty(0), torch.empty(0)
    outs = [R.rotate(x[t:t + 1], torch.ones(1, device="cuda"), (turns[t] * 2 * math.pi).cuda(), inter, 1.25, transpose)
            for t in range(n)]
    ref, err = torch.cat([o[0] for o in outs]), torch.cat([o[1] for o in outs])
    bound = err + ref.abs() * R.HALF[DT[dtype]] * 1.001 + R.FLOOR[DT[dtype]]
    assert amp == 1.0 and y.dtype == x.dtype and y.shape == x.shape
    assert torch.all((y.double() - ref).abs() <= bound)
    assert torch.equal(y[..., rot:], x[..., rot:])


def test_rope_views_positions_and_in_place(paged):
    """Slices of a fused projection, outputs with strides of their own, x
    itself, base positions, and unaligned rows."""
    g = gen(3)
    freqs, _ = paged.pcd_rope_freqs(64, 1e6)
    f = R.inv_freq(64, 1e6)
    dev = freqs.cuda()
    wide = torch.randn(9, 10, 64, generator=g, device="cuda").half()
    q, k = wide[:, :6], wide[:, 6:8]
    base = torch.arange(9, device="cuda") + 40
    for x in (q, k):
        want, err = R.rotate(x, base, f)
        bound = err + want.abs() * R.HALF[x.dtype] * 1.001 + R.FLOOR[x.dtype]
        out = torch.full((9, 20, 64), 7.0, dtype=torch.float16, device="cuda")[:, ::2][:, :x.shape[1]]
        y = paged.pcd_k_rope(x, dev, base=40, out=out)
        assert y is out and torch.all((y.double() - want).abs() <= bound)
        flat = torch.zeros(9 * 64 * x.shape[1] + 3, dtype=torch.float16, device="cuda")
        odd = flat[3:].view(9, x.shape[1], 64)      # rows that start at 2-byte boundaries only
        odd.copy_(x)
        assert torch.equal(paged.pcd_k_rope(odd, dev, base=40), y)
    keep = wide.clone()
    yq = paged.pcd_k_rope(q, dev, base=40)
    assert paged.pcd_k_rope(q, dev, base=40, out=q) is q
    assert torch.equal(q, yq) and torch.equal(wide[:, 6:], keep[:, 6:])
    # side by side in one buffer: another head range of the same rows
    paged.pcd_k_rope(wide[:, 6:8], dev, base=40, out=wide[:, 8:10])
    assert torch.equal(wide[:, 8:10], paged.pcd_k_rope(k, dev, base=40)) and torch.equal(k, keep[:, 6:8])
    same = paged.pcd_k_rope(keep, None)
    assert torch.equal(same, keep)
    assert paged.pcd_k_rope(keep[:0], dev).shape == (0, 10, 64)


def test_rope_gradient(paged):
    """The transposed rotation is the gradient: against differences of <w, y>
    along directions, and it undoes the rotation at amp 1."""
    g = gen(8)
    freqs, amp = paged.pcd_rope_freqs(48, 1e4, "ramp", 4.0, 4096.0)
    dev = freqs.cuda()
    pos = torch.randint(0, 16384, (11,), generator=g, device="cuda", dtype=torch.int32)
    x, w, u = (torch.randn(11, 3, 80, generator=g, device="cuda") for _ in range(3))
    for inter in (False, True):
        run = lambda t, tr=False, a=amp: paged.pcd_k_rope(t, dev, pos, interleaved=inter, amp=a, transpose=tr)  # noqa: E731
        grad = run(w, True)
        # linear in x: the difference quotient over any step is the derivative
        diff = ((run(x + u).double() - run(x - u).double()) * w.double()).sum() / 2
        got = (grad.double() * u.double()).sum()
        # 2640 elements: each side off by 2^-21 of |w| |u| times amp, and x +- u rounds by 2^-24
        bound = 2.0 ** -20 * amp * ((w.double().abs() * (x.abs() + u.abs()).double()).sum() + (w.abs() * u.abs()).double().sum()) * 2
        assert abs(float(diff - got)) <= float(bound)
        back = run(run(x, False, 1.0), True, 1.0)
        assert torch.all((back - x).abs() <= 2.0 ** -19 * (x.abs().amax()))


@pytest.mark.parametrize("scaling", ["none", "linear", "base", "bands", "ramp"])
def test_rope_freqs(paged, scaling):
    """The frequencies of every scaling, recomputed."""
    rot, theta, factor, orig = 128, 5e5, 8.0, 8192.0
    freqs, amp = paged.pcd_rope_freqs(rot, theta, scaling, factor, orig)
    got = [(v % 2 ** 64) / 2 ** 64 * 2 * math.pi for v in freqs.tolist()]
    assert amp == pytest.approx(0.1 * math.log(8.0) + 1 if scaling == "ramp" else 1.0, rel=1e-6)
    for i, v in enumerate(got):
        f = theta ** (-2 * i / rot)
        if scaling == "linear":
            f /= factor
        elif scaling == "base":
            f = (theta * factor ** (rot / (rot - 2))) ** (-2 * i / rot)
        elif scaling == "bands":
            t = orig * f / (2 * math.pi)
            f = f if t >= 4 else f / factor if t <= 1 else f / factor * (4 - t) / 3 + f * (t - 1) / 3
        elif scaling == "ramp":
            lo = max(math.floor(rot * math.log(orig / (32 * 2 * math.pi)) / (2 * math.log(theta))), 0)
            hi = min(math.ceil(rot * math.log(orig / (2 * math.pi)) / (2 * math.log(theta))), rot - 1)
            r = min(max((i - lo) / (hi - lo), 0), 1)
            f = f / factor * r + f * (1 - r)
        assert v == pytest.approx(f, rel=1e-12)


# ---------------------------------------------------------------------- append
def append_case(fmt, dtype, page, dim, heads, new, old, rot, inter, order="head", seed=0):
    lens = [a + b for a, b in zip(new, old)]
    table, pool = R.make_table(lens, page, seed=seed)
    kc, vc, ks, vs = R.make_cache(pool, heads, page, dim, fmt, seed, order)
    n = sum(new)
    g = gen(seed + 5)
    rows = torch.randn(n + 2, 4 * heads, dim, generator=g, device="cuda") * torch.exp2(
        3 * torch.randn(n + 2, 1, 1, generator=g, device="cuda"))
    rows = rows.to(DT[dtype])
    return table, kc, vc, ks, vs, rows[:, 2 * heads:3 * heads], rows[:, 3 * heads:], offsets(new), i32(lens), n


def check_append(before, after, scale_before, scale_after, x, x_err, new, lens, table, fmt):
    """Codes and scales of one of the two caches after the call.  A code is
    within half a step of its value: 2^-4 of it (e4m3; 2^-10 of the scale where
    it is subnormal) or half a scale (int8), plus what the rotation may be off;
    1.001 covers the fp32 division."""
    size, heads = before.shape[2], before.shape[1]
    top = 127.0 if fmt == "int8" else 448.0
    written = torch.zeros(before.shape[:3], dtype=torch.bool, device="cuda")
    touched = torch.zeros(before.shape[:2], dtype=torch.bool, device="cuda")
    at = 0
    for s, (n, L) in enumerate(zip(new, lens)):
        for p in range((L - n) // size, -(-L // size) if n else 0):
            lo, hi = max(p * size, L - n), min((p + 1) * size, L)
            pg, held = int(table[s, p]), lo - p * size
            xr, er = x[at + lo - (L - n):at + hi - (L - n)], x_err[at + lo - (L - n):at + hi - (L - n)]
            written[pg, :, :held + hi - lo] = True
            touched[pg] = True
            for h in range(heads):
                am = xr[:, h].abs().amax()
                sc, old = scale_after[pg, h].double(), scale_before[pg, h].double()
                tol = (er[:, h].amax() / top + am / top * 2.0 ** -22)
                if fmt == "int8":
                    need_lo = need_hi = am / top
                else:
                    need_lo, need_hi = (torch.exp2(torch.ceil(torch.log2((am + d * top) / top))) for d in (-tol, tol))
                need_lo, need_hi = need_lo.clamp(min=R.SCALE_FLOOR), need_hi.clamp(min=R.SCALE_FLOOR)
                if held:
                    need_lo, need_hi = torch.maximum(need_lo, old), torch.maximum(need_hi, old)
                assert need_lo - tol <= sc <= need_hi + tol, (pg, h, float(sc), float(need_lo), float(need_hi))
                got = after[pg, h, held:held + hi - lo].double() * sc
                v = xr[:, h]
                step = sc / 2 if fmt == "int8" else torch.maximum(v.abs() * 2.0 ** -4, sc * 2.0 ** -10)
                assert torch.all((got - v).abs() <= step * 1.001 + er[:, h])
                if held:
                    was, now = before[pg, h, :held].double() * old, after[pg, h, :held].double() * sc
                    if sc == old:
                        assert torch.equal(was, now)
                    elif fmt == "int8":
                        assert torch.all((was - now).abs() <= sc / 2 * 1.001)
                    else:  # by a power of two: exact unless the code became subnormal
                        fine = was.abs() >= sc * 2.0 ** -6
                        assert torch.equal(was[fine], now[fine])
                        assert torch.all((was - now).abs() <= sc * 2.0 ** -10)
        at += n
    same = ~written[..., None].expand_as(before.view(torch.int8))
    assert torch.equal(before.view(torch.int8)[same], after.view(torch.int8)[same])
    assert torch.equal(scale_before[~touched], scale_after[~touched])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype,page,dim,heads,new,old,rot,inter,order", [
    ("f16", 64, 128, 4, [1] * 9, [0, 1, 63, 64, 65, 127, 128, 500, 901], 128, False, "head"),
    ("f32", 16, 64, 2, [1, 17, 0, 33, 16, 15, 45], [0, 5, 40, 15, 16, 17, 0], 64, True, "head"),
    ("bf16", 128, 128, 1, [300, 1, 0, 128], [0, 200, 0, 128], 32, False, "slot"),
    ("f16", 32, 64, 3, [31, 32, 33, 100], [1, 31, 32, 33], 0, False, "slot"),
    ("bf16", 16, 128, 2, [70], [3], 126, False, "head"),
    ("f32", 64, 64, 1, [64, 65], [0, 0], 18, True, "head"),
    ("f16", 16, 64, 6, [2500, 40], [7, 0], 48, False, "head"),     # several heads of a page to a CTA, the last group short
    ("bf16", 32, 64, 5, [5000], [0], 64, True, "slot"),
    ("bf16", 128, 128, 2, [300, 129, 1, 2], [0, 127, 200, 254], 54, False, "slot"),  # pairs that end inside a chunk
    ("f16", 64, 128, 3, [190, 64], [33, 64], 12, True, "head"),
    ("f32", 32, 64, 2, [75], [5], 2, False, "head"),
])
def test_append(paged, fmt, dtype, page, dim, heads, new, old, rot, inter, order):
    table, kc, vc, ks, vs, k, v, q_off, kv_len, n = append_case(fmt, dtype, page, dim, heads, new, old, rot, inter, order, seed=page + dim)
    before = [t.clone() for t in (kc, vc, ks, vs)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    freqs = paged.pcd_rope_freqs(rot, 1e6)[0].cuda() if rot else None
    paged.pcd_k_kv_append(k, v, kc, vc, ks, vs, q_off, kv_len, table, freqs=freqs, interleaved=inter, err=err)
    assert int(err) == 0
    pos = torch.cat([torch.arange(o, o + m, device="cuda") for m, o in zip(new, old)])
    x, e = k[:n].double(), torch.zeros_like(k[:n].double())
    if rot:
        x, e = R.rotate(k[:n], pos, R.inv_freq(rot, 1e6), inter)
    lens = [a + b for a, b in zip(new, old)]
    check_append(before[0], kc, before[2], ks, x, e, new, lens, table, fmt)
    check_append(before[1], vc, before[3], vs, v[:n].double(), torch.zeros_like(x), new, lens, table, fmt)


def test_append_given_positions(paged):
    """Keys rotated at positions of their own (branch tokens after a prefix)."""
    new, old = [5, 9], [20, 0]
    table, kc, vc, ks, vs, k, v, q_off, kv_len, n = append_case("e4m3", "f16", 16, 64, 2, new, old, 64, False)
    pos = torch.randint(-9, 10 ** 6, (n + 2,), generator=gen(1), device="cuda", dtype=torch.int32)
    before = [t.clone() for t in (kc, ks)]
    paged.pcd_k_kv_append(k, v, kc, vc, ks, vs, q_off, kv_len, table, freqs=paged.pcd_rope_freqs(64, 1e4)[0].cuda(), amp=1.5,
                          pos=pos)
    x, e = R.rotate(k[:n], pos[:n], R.inv_freq(64, 1e4), amp=1.5)
    check_append(before[0], kc, before[1], ks, x, e, new, [25, 9], table, "e4m3")


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_token_by_token(paged, fmt):
    """A page filled one token at a time holds what the whole prompt in one
    call gives: the scales are equal, the codes too for e4m3 (codes that were
    made subnormal by a later, larger row may be a step off), and for int8 each
    of the at most 16 rescalings rounds by half a scale."""
    table, kc, vc, ks, vs, k, v, q_off, kv_len, n = append_case(fmt, "f16", 16, 128, 2, [40], [0], 128, False)
    freqs = paged.pcd_rope_freqs(128, 1e6)[0].cuda()
    kc2, vc2, ks2, vs2 = (t.clone() for t in (kc, vc, ks, vs))
    paged.pcd_k_kv_append(k, v, kc, vc, ks, vs, q_off, kv_len, table, freqs=freqs)
    for t in range(n):
        paged.pcd_k_kv_append(k[t:t + 1], v[t:t + 1], kc2, vc2, ks2, vs2, i32([0, 1]), i32([t + 1]), table, freqs=freqs)
    used = table[0].long()
    assert torch.equal(ks[used], ks2[used]) and torch.equal(vs[used], vs2[used])
    for a, b, sc in ((kc, kc2, ks), (vc, vc2, vs)):
        x, y = (R.values(t, sc)[used].transpose(1, 2).reshape(-1, 2, 128)[:n] for t in (a, b))
        s = sc.double()[used].repeat_interleave(16, 0)[:n, :, None]
        if fmt == "e4m3":
            fine = (x.abs() >= s * 2.0 ** -6) & (y.abs() >= s * 2.0 ** -6)
            assert torch.equal(x[fine], y[fine]) and torch.all((x - y).abs() <= s * 2.0 ** -9 * 1.001)
        else:
            assert torch.all((x - y).abs() <= 8.5 * s)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_zeros_nan_and_infinity(paged, fmt):
    """A block of zeros reads as zeros; a NaN or infinity shows in its own
    block's scale and in no other's; the next owner of the page starts anew."""
    table, kc, vc, ks, vs, k, v, q_off, kv_len, n = append_case(fmt, "f32", 16, 64, 2, [48], [0], 0, False)
    k, v = k.clone(), v.clone()
    k[:16] = 0
    k[20, 1, 3] = float("nan")
    v[40, 0, 0] = float("inf")
    paged.pcd_k_kv_append(k, v, kc, vc, ks, vs, q_off, kv_len, table)
    p = table[0].long().tolist()
    assert torch.all(R.values(kc, ks)[p[0]] == 0) and torch.all(ks[p[0]] == R.SCALE_FLOOR)
    assert torch.isnan(ks[p[1], 1]) and torch.isfinite(ks[p[1], 0]) and torch.isfinite(ks[p[2]]).all()
    assert not torch.isfinite(vs[p[2], 0]) and torch.isfinite(vs[p[2], 1]) and torch.isfinite(vs[p[1]]).all()
    paged.pcd_k_kv_append(k[:16], v[:16], kc, vc, ks, vs, i32([0, 16]), i32([32]), table)
    assert torch.isfinite(ks[p[1]]).all()


def test_append_out_of_range(paged):
    """Pages outside the pool, lengths beyond the table or below the new rows,
    and offsets past the rows are skipped and reported; the rest is written."""
    def fresh():
        return append_case("int8", "f16", 16, 64, 1, [4, 20, 4], [0, 0, 30], 0, False)

    def call(change):
        table, kc, vc, ks, vs, k, v, q_off, kv_len, n = fresh()
        args = dict(table=table, q_off=q_off, kv_len=kv_len)
        change(args)
        before = kc.clone()
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        paged.pcd_k_kv_append(k, v, kc, vc, ks, vs, args["q_off"], args["kv_len"], args["table"], err=err)
        wrote = [bool((kc[fresh()[0][s][:2].clamp(min=0).long()] != before[fresh()[0][s][:2].clamp(min=0).long()]).any()) for s in (0, 2)]
        return int(err), wrote

    assert call(lambda a: None) == (0, [True, True])
    assert call(lambda a: a["table"][1].fill_(10 ** 6)) == (5, [True, True])
    assert call(lambda a: a["table"][1].fill_(-1)) == (5, [True, True])
    assert call(lambda a: a["kv_len"][1:2].fill_(10 ** 6)) == (5, [True, True])
    assert call(lambda a: a["kv_len"][1:2].fill_(19)) == (5, [True, True])
    assert call(lambda a: a["kv_len"][1:2].fill_(-2 ** 31)) == (5, [True, True])
    assert call(lambda a: a["q_off"][3:].fill_(2 ** 31 - 1))[0] == 5
    assert call(lambda a: a["q_off"][1:2].fill_(-7))[0] == 5


# ------------------------------------------------------------------- attention
def attend_case(fmt, dtype, page, dim, heads, kv_heads, q_lens, kv_lens, seed=0, order="head", q_size=2.0):
    table, pool = R.make_table(kv_lens, page, seed=seed)
    kc, vc, ks, vs = R.make_cache(pool, kv_heads, page, dim, fmt, seed, order)
    q = (q_size * torch.randn(sum(q_lens), heads, dim, generator=gen(seed + 1), device="cuda")).to(DT[dtype])
    return q, kc, vc, ks, vs, offsets(q_lens), i32(kv_lens), table


def check_attend(got, lse, ref):
    out, l, ob, lb = ref
    assert torch.isfinite(got).all()
    worst = ((got.double() - out).abs() / ob.clamp(min=1e-300)).amax()
    assert torch.all((got.double() - out).abs() <= ob), float(worst)
    if lse is not None:
        none = torch.isinf(l)
        assert torch.equal(torch.isneginf(lse), none)
        assert torch.all((lse.double() - l).abs()[~none] <= lb[~none])


CASES = [
    # page, dim, heads, kv_heads, q_lens, kv_lens, order
    (64, 128, 12, 2, [1], [901], "head"),
    (16, 64, 4, 2, [1], [1], "head"),
    (64, 128, 28, 4, [1, 1, 1, 1, 1], [1, 63, 64, 65, 1000], "head"),
    (32, 128, 8, 8, [1, 0, 1, 1], [100, 50, 0, 31], "slot"),
    (16, 128, 16, 1, [2, 1, 3], [17, 16, 15], "head"),
    (128, 64, 32, 1, [1, 1], [129, 4000], "head"),
    (64, 128, 12, 2, [47], [47], "head"),
    (32, 64, 14, 2, [130, 5, 0, 77], [130, 300, 90, 33], "slot"),
    (16, 128, 28, 4, [33, 64, 1], [700, 64, 5], "head"),
    (64, 64, 128, 1, [3], [200], "head"),
    (128, 128, 5, 5, [200], [90], "head"),
    (64, 128, 6, 2, [300, 129], [1337, 640], "head"),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("fmt,dtype", [("e4m3", "f16"), ("int8", "f16"), ("e4m3", "bf16"), ("int8", "bf16")])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(paged, case, fmt, dtype, causal):
    page, dim, heads, kv_heads, q_lens, kv_lens, order = CASES[case]
    a = attend_case(fmt, dtype, page, dim, heads, kv_heads, q_lens, kv_lens, case, order)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, lse = paged.pcd_k_paged_attention(*a, causal=causal, return_lse=True, err=err)
    assert int(err) == 0
    check_attend(got, lse, R.attention(*a, causal, dim ** -0.5))
    # how the keys are cut into ranges is not what is computed
    for hint in (0, 1, max(kv_lens), 10 ** 6):
        check_attend(paged.pcd_k_paged_attention(*a, causal=causal, max_kv=hint), None, R.attention(*a, causal, dim ** -0.5))


@pytest.mark.parametrize("n_seq,q_len", [(70, 1), (3, 1), (1100, 1), (40, 3)])
def test_attention_many_sequences(paged, n_seq, q_len):
    """Ragged contexts of many sequences, some of them empty."""
    r = torch.Generator().manual_seed(n_seq)
    kv = [int(x) for x in torch.randint(0, 300, (n_seq,), generator=r)]
    ql = [int(x) for x in torch.randint(0, q_len + 1, (n_seq,), generator=r)]
    a = attend_case("e4m3", "f16", 16, 64, 4, 2, ql, kv, 5)
    got, lse = paged.pcd_k_paged_attention(*a, return_lse=True)
    check_attend(got, lse, R.attention(*a, True, 64 ** -0.5))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("fmt,dtype,page,dim,heads,kv_heads,q_lens,kv_lens", [
    ("e4m3", "f16", 16, 128, 7, 1, [18, 1, 7], [1409, 129, 256]),    # 126, 7 and 49 rows; odd and even numbers of blocks
    ("int8", "bf16", 64, 64, 12, 2, [21, 13, 0, 20], [1281, 1100, 50, 19]),
    ("e4m3", "bf16", 128, 128, 8, 2, [32, 8, 31, 9], [4500, 128, 385, 0]),  # exactly a tile; one block; no keys
    ("int8", "f16", 32, 64, 5, 1, [1, 60, 1, 1], [1153, 700, 257, 1]),  # 300 rows among short items
])
def test_attention_one_tile_of_rows(paged, fmt, dtype, page, dim, heads, kv_heads, q_lens, kv_lens, causal):
    """33 to 128 rows a sequence and KV head: the key blocks of an item go to
    two pipelines in turn, whose states are joined."""
    a = attend_case(fmt, dtype, page, dim, heads, kv_heads, q_lens, kv_lens, 6)
    want = R.attention(*a, causal, dim ** -0.5)
    for hint in (max(kv_lens), 5000, 10 ** 6):  # several ranges of keys, and more ranges than blocks
        got, lse = paged.pcd_k_paged_attention(*a, causal=causal, max_kv=hint, return_lse=True)
        check_attend(got, lse, want)


def test_attention_one_tile_of_rows_masks(paged):
    """Rows that see no key of the odd blocks, or none at all, beside rows that
    do; a poisoned scale in an odd block reaches only the rows that see it."""
    q_len, L = 100, 190  # row i sees 91 + i keys: rows 0 .. 37 none of block 1
    a = list(attend_case("e4m3", "f16", 16, 128, 1, 1, [q_len, 110], [L, 60], 2))
    kw = dict(max_kv=5000, return_lse=True)
    got, lse = paged.pcd_k_paged_attention(*a, **kw)
    check_attend(got, lse, R.attention(*a, True, 128 ** -0.5))
    assert torch.isinf(lse[q_len:q_len + 50]).all() and torch.all(got[q_len:q_len + 50] == 0)
    for t in (3, 4):
        keep = a[t]
        a[t] = a[t].clone()
        a[t][a[7][0, 8].long(), 0] = float("nan")  # keys 128 .. 143
        bad, _ = paged.pcd_k_paged_attention(*a, **kw)
        assert torch.equal(bad[:38], got[:38]) and torch.isnan(bad[38:q_len]).all() and torch.equal(bad[q_len:], got[q_len:])
        a[t] = keep


@pytest.mark.parametrize("q_len", [1, 40])
def test_attention_scales_far_apart(paged, q_len):
    """Blocks whose value scales lie 2^40 apart, weights that fall by 2^-60,
    scales of zero, and the largest scores."""
    q, kc, vc, ks, vs, q_off, kv_len, table = attend_case("int8", "f16", 16, 128, 7, 1, [q_len], [400], 3)
    vs[:] = torch.exp2(torch.randint(-20, 20, vs.shape, generator=gen(2), device="cuda").float())
    vs[table[0, 3].long()] = 0.0
    ks[:] *= torch.exp2(torch.randint(-4, 3, ks.shape, generator=gen(3), device="cuda").float())
    a = (q, kc, vc, ks, vs, q_off, kv_len, table)
    vs_ref = vs.clamp(max=2.0 ** 7)
    a = (q, kc, vc, ks, vs_ref, q_off, kv_len, table)
    got, lse = paged.pcd_k_paged_attention(*a, return_lse=True)
    check_attend(got, lse, R.attention(*a, True, 128 ** -0.5))


@pytest.mark.parametrize("q_len", [2, 60])
def test_attention_nan_stays_where_it_is_seen(paged, q_len):
    """Poisoned blocks, and codes and scales behind the last token, reach only
    rows that see them."""
    q, kc, vc, ks, vs, q_off, kv_len, table = attend_case("e4m3", "f16", 16, 64, 4, 2, [q_len, 1], [q_len + 16, 70], 3)
    L = q_len + 16
    used = table[0, (L - 1) // 16].long()
    tail = L % 16
    for t in (kc, vc):  # slots behind the last token, as NaN and largest codes
        if tail:
            t.view(torch.int8)[used, :, tail:] = 0x7f
        for p in range(kc.shape[0]):
            if p not in table.flatten().tolist():
                t.view(torch.int8)[p] = -1
    free = [p for p in range(kc.shape[0]) if p not in table.flatten().tolist()]
    ks[free] = float("nan")
    vs[free] = float("nan")
    a = (q, kc, vc, ks, vs, q_off, kv_len, table)
    clean = paged.pcd_k_paged_attention(*a)
    check_attend(clean, None, R.attention(*a, True, 64 ** -0.5))
    for t in (ks, vs):   # the second sequence's first block, head 1
        keep = t.clone()
        t[table[1, 0].long(), 1] = float("nan")
        got = paged.pcd_k_paged_attention(*a)
        assert torch.equal(got[:q_len], clean[:q_len]) and torch.equal(got[q_len:, :2], clean[q_len:, :2])
        assert torch.isnan(got[q_len:, 2:]).all()
        t.copy_(keep)
    last = table[0, (L - 1) // 16].long()      # a block that only the last rows of sequence 0 see
    ks[last, 0] = float("nan")
    got = paged.pcd_k_paged_attention(*a)
    first_row = max(0, (L - 1) // 16 * 16 - (L - q_len))
    assert torch.equal(got[:first_row], clean[:first_row]) and torch.isnan(got[first_row:q_len, :2]).all()
    assert torch.equal(got[:, 2:], clean[:, 2:])
    ks[last, 0] = 1.0
    vs[last, 1] = float("inf")
    got = paged.pcd_k_paged_attention(*a)
    assert torch.equal(got[:first_row], clean[:first_row]) and torch.isnan(got[first_row:q_len, 2:]).all()
    vs[last, 1] = float("nan")
    got = paged.pcd_k_paged_attention(*a)
    assert torch.equal(got[:first_row], clean[:first_row]) and torch.isnan(got[first_row:q_len, 2:]).all()


@pytest.mark.parametrize("q_len", [1, 50])
def test_attention_out_of_range(paged, q_len):
    """Pages outside the pool are not seen; a length beyond the table reads as
    no tokens; offsets past the rows leave the rows alone.  All are reported."""
    a = list(attend_case("int8", "f16", 16, 64, 4, 2, [q_len, q_len, q_len], [90, 120, 70], 3))
    table = a[7].clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    a[7] = table.clone()
    a[7][1, 2], a[7][1, 5] = -5, 2 ** 31 - 1
    got, lse = paged.pcd_k_paged_attention(*a, return_lse=True, err=err)
    assert int(err) == 5
    check_attend(got, lse, R.attention(*a, True, 0.125))
    a[7] = table
    for wrong in (10 ** 6, -1, 2 ** 31 - 1):
        err.zero_()
        a[6] = i32([90, wrong, 70])
        got, lse = paged.pcd_k_paged_attention(*a, return_lse=True, err=err)
        assert int(err) == 5
        a[6] = i32([90, 0, 70])
        check_attend(got, lse, R.attention(*a, True, 0.125))
    a[6] = i32([90, 120, 70])
    err.zero_()
    bad = a[:5] + [i32([0, q_len, 2 * q_len, 2 ** 31 - 1])] + a[6:]
    got = paged.pcd_k_paged_attention(*bad, err=err)
    good = R.attention(*a, True, 0.125)
    assert int(err) == 5
    check_attend(got[:2 * q_len], None, [t[:2 * q_len] for t in good])


@pytest.mark.parametrize("q_len", [1, 30])
def test_attention_rows_behind_the_last_sequence(paged, q_len):
    """Padding rows are not written, nor the gaps of strided queries and outputs."""
    q, kc, vc, ks, vs, q_off, kv_len, table = attend_case("e4m3", "bf16", 32, 64, 6, 2, [q_len, q_len], [100, 333], 1)
    n = 2 * q_len
    wide = torch.zeros(n + 5, 9, 64, dtype=q.dtype, device="cuda")
    wide[:n, 1:7] = q
    out = torch.full((n + 5, 12, 64), 3.0, dtype=q.dtype, device="cuda")
    res, lse = paged.pcd_k_paged_attention(wide[:, 1:7], kc, vc, ks, vs, q_off, kv_len, table, out=out[:, ::2], return_lse=True)
    check_attend(res[:n], lse[:n], R.attention(q, kc, vc, ks, vs, q_off, kv_len, table, True, 0.125))
    assert torch.all(out[:, 1::2] == 3) and torch.all(out[n:] == 3)


@pytest.mark.parametrize("q_len", [1, 30, 200])
def test_attention_unaligned_rows(paged, q_len):
    """Queries and outputs whose rows start at 2-byte boundaries only."""
    for dtype in ("f16", "bf16"):
        q, *rest = attend_case("e4m3", dtype, 32, 128, 6, 2, [q_len, 1], [q_len + 300, 77], 4)
        flat = torch.zeros(q.numel() + 3, dtype=q.dtype, device="cuda")
        odd = flat[3:].view(q.shape)
        odd.copy_(q)
        out = torch.zeros(q.numel() + 1, dtype=q.dtype, device="cuda")[1:].view(q.shape)
        got = paged.pcd_k_paged_attention(odd, *rest, out=out)
        assert got is out and torch.equal(got, paged.pcd_k_paged_attention(q, *rest))


@pytest.mark.parametrize("q_len,kv,hint", [(1, 901, None), (1, 9000, None), (3, 20000, None), (20, 4000, None), (300, 500, 1), (300, 500, 9000)])
def test_attention_in_place(paged, q_len, kv, hint):
    """The output over the queries, in every way a call is cut up."""
    q, *rest = attend_case("int8", "f16", 64, 128, 14, 2, [q_len, q_len], [kv, kv // 2], 4)
    want = paged.pcd_k_paged_attention(q, *rest, max_kv=hint)
    assert paged.pcd_k_paged_attention(q, *rest, max_kv=hint, out=q) is q and torch.equal(q, want)


def test_two_streams_at_once(paged):
    """Calls that overlap on two streams, each with its own workspace, and a
    page that two sequences share for reading."""
    a = attend_case("int8", "f16", 64, 128, 28, 4, [1] * 6, [20000, 9000, 1, 500, 20000, 64], 2)
    b = attend_case("e4m3", "bf16", 16, 64, 14, 2, [90, 3], [400, 700], 3)
    a[-1][4] = a[-1][0]
    want = [paged.pcd_k_paged_attention(*a), paged.pcd_k_paged_attention(*b)]
    assert not torch.equal(want[0][0], want[0][4])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(6):
        for k, args in enumerate((a, b)):
            with torch.cuda.stream(streams[k]):
                got[k].append(paged.pcd_k_paged_attention(*args))
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(x, want[k]) for x in got[k])


def test_attention_long_cache(paged):
    """Pages beyond 2^31 bytes of the pool, and a long context against the same
    keys near the start of the pool."""
    page, dim = 128, 128
    pool = 2 ** 31 // (page * dim) + 4200
    kc = torch.zeros(pool, 1, page, dim, dtype=torch.int8, device="cuda")
    vc = torch.zeros_like(kc)
    ks, vs = torch.full((pool, 1), 0.02, device="cuda"), torch.full((pool, 1), 0.02, device="cuda")
    n = 4100
    kc[-n:] = torch.randint(-127, 128, (n, 1, page, dim), generator=gen(0), device="cuda", dtype=torch.int8)
    vc[-n:] = torch.randint(-127, 128, (n, 1, page, dim), generator=gen(1), device="cuda", dtype=torch.int8)
    table = torch.arange(pool - n, pool, device="cuda", dtype=torch.int32)[None]
    L = n * page - 77
    q = torch.randn(1, 7, dim, generator=gen(2), device="cuda").half()
    got, lse = paged.pcd_k_paged_attention(q, kc, vc, ks, vs, i32([0, 1]), i32([L]), table, return_lse=True)
    check_attend(got, lse, R.attention(q, kc, vc, ks, vs, i32([0, 1]), i32([L]), table, True, dim ** -0.5))
    low = [t[-n:].clone() for t in (kc, vc, ks, vs)]
    again = paged.pcd_k_paged_attention(q, *low, i32([0, 1]), i32([L]), table - (pool - n))
    assert torch.equal(again, got)


# ----------------------------------------------------------- as they are used
def run_layer(paged, q, k, v, cache, q_off, kv_len, table, freqs, pos, scratch=None):
    qr = paged.pcd_k_rope(q, freqs, pos)
    paged.pcd_k_kv_append(k, v, *cache, q_off, kv_len, table, freqs=freqs)
    return paged.pcd_k_paged_attention(qr, *cache, q_off, kv_len, table, scratch=scratch)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_prefill_then_tokens(paged, fmt):
    """Prompts of three requests, then five tokens each: rotate, append, attend,
    against unquantised attention in 64 bits.  With unit-variance keys and
    values an 8-bit code is off by at most 2^-4 of the value (e4m3) or 1/254 of
    the block's largest (int8, under 6 here, times up to 1.5 for rescalings):
    a score by sqrt(D) times that at the very worst over random signs; the
    outputs of softmax averages stay within 0.1, where a misplaced token or
    angle gives differences of order 1."""
    lens, steps, hq, hkv, d, page = [200, 33, 64], 5, 6, 2, 128, 64
    table, pool = R.make_table([n + steps for n in lens], page, seed=4)
    cache = R.make_cache(pool, hkv, page, d, fmt, 1)
    freqs = paged.pcd_rope_freqs(d, 1e6)[0].cuda()
    f = R.inv_freq(d, 1e6)
    g = gen(6)
    full = [[torch.randn(n + steps, h, d, generator=g, device="cuda").half() for h in (hq, hkv, hkv)] for n in lens]
    outs = [[] for _ in lens]
    spans = [[(0, n) for n in lens]] + [[(n + t, n + t + 1) for n in lens] for t in range(steps)]
    for span in spans:
        q, k, v = (torch.cat([full[s][w][a:b] for s, (a, b) in enumerate(span)]) for w in range(3))
        pos = torch.cat([torch.arange(a, b, device="cuda", dtype=torch.int32) for a, b in span])
        o = run_layer(paged, q, k, v, cache, offsets([b - a for a, b in span]), i32([b for _, b in span]), table, freqs, pos)
        at = 0
        for s, (a, b) in enumerate(span):
            outs[s].append(o[at:at + b - a])
            at += b - a
    for s, n in enumerate(lens):
        pos = torch.arange(n + steps, device="cuda")
        q, k = R.rotate(full[s][0], pos, f)[0], R.rotate(full[s][1], pos, f)[0]
        z = torch.einsum("ihd,jhd->hij", q, k.repeat_interleave(hq // hkv, 1)) * d ** -0.5
        z = z.masked_fill(pos[None, :, None] < pos[None, None, :], -math.inf)
        want = torch.einsum("hij,jhd->ihd", torch.softmax(z, -1), full[s][2].double().repeat_interleave(hq // hkv, 1))
        err = (torch.cat(outs[s]).double() - want).abs()
        assert err.amax() < (0.35 if fmt == "e4m3" else 0.12) and err.mean() < (0.02 if fmt == "e4m3" else 0.01)


def test_captured_and_replayed(paged):
    """One token's layer in a CUDA graph, replayed with new inputs and lengths
    in the same buffers, equals the calls made one by one; two graphs with
    scratch of their own do not disturb one another."""
    lens, hq, hkv, d, page = [300, 5], 12, 2, 128, 16
    table, pool = R.make_table([n + 8 for n in lens], page, seed=4)
    freqs = paged.pcd_rope_freqs(d, 1e6)[0].cuda()
    g = gen(6)
    q, k, v = (torch.randn(2, h, d, generator=g, device="cuda").half() for h in (hq, hkv, hkv))
    q_off, kv_len = offsets([1, 1]), i32([n + 1 for n in lens])
    pos = kv_len - 1
    caches = [R.make_cache(pool, hkv, page, d, "e4m3", 1) for _ in range(3)]
    for c in caches[1:]:
        for a, b in zip(c, caches[0]):
            a.view(torch.uint8).copy_(b.view(torch.uint8))
    need = paged.pcd_k_paged_attention_scratch_bytes(2, 2, hq, hkv, d, table.shape[1] * page)
    scr = [torch.empty(max(need, 1), dtype=torch.uint8, device="cuda") for _ in range(2)]
    run_layer(paged, q, k, v, caches[0], q_off, kv_len, table, freqs, pos)
    graphs, res = [], []
    side = torch.cuda.Stream()
    for i in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            res.append(run_layer(paged, q, k, v, caches[1 + i], q_off, kv_len, table, freqs, pos, scr[i]))
        graphs.append(gr)
    for gr in graphs:
        gr.replay()
    torch.cuda.synchronize()
    for step in range(4):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        kv_len.add_(1)
        pos.add_(1)
        want = run_layer(paged, q, k, v, caches[0], q_off, kv_len, table, freqs, pos)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(res[0], want) and torch.equal(res[1], want)
    for a, b in zip(caches[0], caches[1]):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_side_stream_and_repeatability(paged):
    """On a side stream the calls wait for what that stream was given, and the
    same call gives the same bits every time."""
    a = attend_case("e4m3", "f16", 64, 128, 28, 4, [1] * 5 + [37], [4000, 1, 77, 2048, 900, 500], 2)
    want = paged.pcd_k_paged_attention(*a)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        big = torch.randn(4096, 4096, device="cuda")
        q = torch.zeros_like(a[0])
        for _ in range(20):
            big = big @ big * 1e-4
        q.copy_(a[0])
        got = [paged.pcd_k_paged_attention(q, *a[1:]) for _ in range(3)]
    side.synchronize()
    assert all(torch.equal(x, want) for x in got)
