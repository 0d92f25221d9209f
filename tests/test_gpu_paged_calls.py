"""Calls of rotary positions and the 8-bit paged cache as their documentation
allows them and programs make them: block tables cut out of wider ones, bad
offsets and lengths beside good ones, outputs in odd places."""
import math
import os
import subprocess
import sys

import pytest
import torch

import paged_ref as R
from paged_ref import i32, offsets
from test_gpu_paged import append_case, attend_case, check_append, check_attend, gen, paged  # noqa: F401

pytestmark = pytest.mark.gpu


# -------------------------------------------------------------- table slices
def in_wider(table, left, fill):
    """The same table as the last columns of one that is `left` entries wider: its last row ends with the storage."""
    big = torch.full((table.shape[0], left + table.shape[1]), fill, dtype=torch.int32, device="cuda")
    big[:, left:] = table
    return big[:, left:]


@pytest.mark.parametrize("q_len,hint", [(1, None), (3, 20000), (20, None), (60, 20000), (300, 1)])
def test_attention_table_slice(paged, q_len, hint):  # noqa: F811
    """A column slice gives what its own columns say: a length beyond them
    reads as no tokens and is reported, also where the wider table goes on."""
    lens = [310, 400, 330]
    a = list(attend_case("e4m3", "f16", 16, 128, 7, 1, [q_len] * 3, lens, 3))
    want = paged.pcd_k_paged_attention(*a, max_kv=hint)
    table = a[7]
    a[7] = in_wider(table, 9, 0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = paged.pcd_k_paged_attention(*a, max_kv=hint, err=err)
    assert int(err) == 0 and torch.equal(got, want)
    width = table.shape[1] * 16
    for s in (1, 2):
        for wrong in (width + 1, width + 9 * 16):
            bad = list(lens)
            bad[s] = wrong
            a[6] = i32(bad)
            err.zero_()
            got, l = paged.pcd_k_paged_attention(*a, max_kv=hint, return_lse=True, err=err)
            assert int(err) == 5
            a[6] = i32([0 if i == s else n for i, n in enumerate(lens)])
            check_attend(got, l, R.attention(*a, True, 128 ** -0.5))
            a[6] = i32(lens)


@pytest.mark.parametrize("rot", [0, 64, 54])
def test_append_table_slice(paged, rot):  # noqa: F811
    """New rows go to the pages of the slice; a length beyond it writes nothing
    and is reported, whatever pages stand in the columns behind."""
    new, old = [4, 20, 5], [40, 60, 59]
    table, kc, vc, ks, vs, k, v, q_off, kv_len, n = append_case("int8", "f16", 16, 64, 2, new, old, rot, False)
    freqs = paged.pcd_rope_freqs(rot, 1e6)[0].cuda() if rot else None
    start = [t.clone() for t in (kc, vc, ks, vs)]
    want = [t.clone() for t in start]
    paged.pcd_k_kv_append(k, v, *want, q_off, kv_len, table, freqs=freqs)
    sliced = in_wider(table, 3, 0)  # page 0 stands behind every row's end but the last
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = [t.clone() for t in start]
    paged.pcd_k_kv_append(k, v, *got, q_off, kv_len, sliced, freqs=freqs, err=err)
    assert int(err) == 0 and all(torch.equal(a, b) for a, b in zip(got, want))
    for s in (0, 2):
        lens = kv_len.clone()
        lens[s] = table.shape[1] * 16 + 2
        err.zero_()
        got = [t.clone() for t in start]
        paged.pcd_k_kv_append(k, v, *got, q_off, lens, sliced, freqs=freqs, err=err)
        assert int(err) == 5
        first = (old[s]) // 16
        mine = table[s, first:-(-(old[s] + new[s]) // 16)].long()
        expect = [t.clone() for t in want]
        for t, b in zip(expect, start):
            t[mine] = b[mine]  # nothing of this sequence was written, all of the others'
        assert all(torch.equal(a, b) for a, b in zip(got, expect))


# ---------------------------------------------------------------- bad offsets
# rows and hints that make every way a call is cut up: clusters, stretches, one and two tiles with ranges of keys and without
CUTS = [(1, 400), (1, 20000), (3, 20000), (10, 20000), (10, 1), (60, 20000), (60, 1)]
FAR = 2 ** 31 - 1


def bad_offsets(q):
    """Offsets of three sequences of q rows with something wrong in them, and what becomes of each third of the rows:
    its sequence's output (g), left alone (-), or another sequence's (?)."""
    n = 3 * q
    return [([0, q, 2 * q, FAR], "gg-"), ([0, q, 2 * q, n + 1], "gg-"), ([0, q, -7, n], "g--"), ([0, q, FAR, n], "g--"),
            ([-3, q, 2 * q, n], "-gg"), ([-9, -8, -8, n], "---"), ([0, 0, 2 * q, FAR], "??-"), ([0, 2 * q, q, n], "???")]


@pytest.mark.parametrize("q_len,hint", CUTS)
@pytest.mark.parametrize("empty", [0, 40])
def test_bad_offsets_are_reported(paged, q_len, hint, empty):  # noqa: F811
    """Every offset that is out of range or decreases is reported by the append
    and by the attention, however the call is cut up; good ones are not, empty
    sequences among them."""
    lens = [310, 400, 330]
    a = list(attend_case("e4m3", "f16", 16, 128, 7, 1, [q_len] * 3, lens, 3))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    k = torch.randn(3 * q_len, 1, 128, generator=gen(1), device="cuda").half()
    kv_len = i32(lens + [5] * empty)
    table = torch.cat([a[7], a[7][:1].expand(empty, -1)]).contiguous()
    good = [0, q_len, 2 * q_len, 3 * q_len]
    for off in [good, [FAR] * 4] + [b for b, _ in bad_offsets(q_len)]:
        q_off = i32(off + off[-1:] * empty)
        want = 0 if len(set(off)) == 1 or off == good else 5
        err.zero_()
        paged.pcd_k_paged_attention(a[0], *a[1:5], q_off, kv_len, table, max_kv=hint, err=err)
        assert int(err) == want, off
        err.zero_()
        paged.pcd_k_kv_append(k, k, *[t.clone() for t in a[1:5]], q_off, kv_len, table, err=err)
        assert int(err) == want, off


def attend_raw(paged, a, out, lse, max_kv, scratch, err, causal=True):  # noqa: F811
    """The C call on the caller's own output, log-sum-exp and workspace."""
    q, kc, vc, ks, vs, q_off, kv_len, table = a
    c, _, _, _, dim = paged._pages(kc, vc, ks, vs)
    rc = paged._lib.pcd_k_paged_attention(
        c, q.data_ptr(), out.data_ptr(), lse.data_ptr(), 3 if q.dtype == torch.float16 else 2, q.shape[1], *q.stride()[:2],
        *out.stride()[:2], q_off.data_ptr(), kv_len.data_ptr(), table.data_ptr(), kv_len.numel(), q.shape[0], table.shape[1],
        max_kv, causal, dim ** -0.5, scratch.data_ptr(), scratch.numel(), err.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0


@pytest.mark.parametrize("q_len,hint", CUTS)
@pytest.mark.parametrize("dim,empty", [(64, 0), (128, 0), (128, 40)])
def test_attention_leaves_skipped_rows(paged, q_len, hint, dim, empty):  # noqa: F811
    """Rows of sequences with bad offsets keep what stood in the output and the
    log-sum-exp, although the workspace holds states of an earlier call."""
    lens = [310, 400, 330]
    n = 3 * q_len
    a = list(attend_case("e4m3", "f16", 32, dim, 7, 1, [q_len] * 3 + [0] * empty, lens + [9] * empty, 3))
    size = paged.pcd_k_paged_attention_scratch_bytes(n, 3 + empty, 7, 1, dim, hint)
    scratch = torch.zeros(max(size, 16), dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(args, poison=None):
        out = torch.full_like(args[0], 7.0)
        lse = torch.full((n, 7), 7.0, device="cuda")
        if poison is not None:
            scratch.view(torch.int32)[:] = poison
        err.zero_()
        attend_raw(paged, args, out, lse, hint, scratch, err)
        return out, lse

    ref = R.attention(*a, True, dim ** -0.5)
    good = run(a)
    check_attend(*good, ref)
    assert int(err) == 0
    for off, becomes in bad_offsets(q_len):
        for poison in (None, 0x3f800000, 0x00010000):  # states left by the good call; ones; small counts
            run(a)
            out, lse = run(a[:5] + [i32(off + off[-1:] * empty)] + a[6:], poison)
            assert int(err) == 5
            for s, what in enumerate(becomes):
                rows = slice(s * q_len, (s + 1) * q_len)
                if what == "-":
                    assert torch.all(out[rows] == 7) and torch.all(lse[rows] == 7), off
                elif what == "g" and not (empty and torch.all(out[rows] == 7)):  # (of many, a search may miss its neighbours)
                    check_attend(out[rows], lse[rows], [t[rows] for t in ref])
    # offsets that decrease: what is written is a sequence's own
    out, lse = run(a[:5] + [i32([0, 2 * q_len, q_len, n] + [n] * empty)] + a[6:], 0x3f800000)
    assert int(err) == 5
    first = R.attention(a[0][:2 * q_len], *a[1:5], i32([0, 2 * q_len]), a[6][:1], a[7][:1], True, dim ** -0.5)
    last = R.attention(a[0][q_len:], *a[1:5], i32([0, 2 * q_len]), a[6][2:3], a[7][2:3], True, dim ** -0.5)
    for rows, want, at in ((slice(0, q_len), first, 0), (slice(2 * q_len, n), last, q_len)):
        w, l, ob, lb = (t[at:at + q_len] for t in want)
        kept = (out[rows] == 7).all(-1) & (lse[rows] == 7)
        assert torch.all(kept[..., None] | ((out[rows].double() - w).abs() <= ob)) and torch.all(kept | ((lse[rows].double() - l).abs() <= lb))


# ------------------------------------------------------------------- odd places
@pytest.mark.parametrize("strides", [(192, 128), (128, 192), (64, 200), (200, 64)])
def test_outputs_that_interleave(paged, strides):  # noqa: F811
    """Rows of an output that lie between one another without meeting, not all
    of them one axis within the other."""
    n, heads, dim = 3, 2, 64
    x = torch.randn(n, heads, dim, generator=gen(5), device="cuda").half()
    freqs = paged.pcd_rope_freqs(64, 1e6)[0].cuda()
    buf = torch.full((2048,), 7.0, dtype=torch.float16, device="cuda")
    out = buf.as_strided((n, heads, dim), (*strides, 1))
    assert torch.equal(paged.pcd_k_rope(x, freqs, out=out), paged.pcd_k_rope(x, freqs))
    q, *rest = attend_case("e4m3", "f16", 16, dim, heads, 1, [n], [90], 3)
    assert torch.equal(paged.pcd_k_paged_attention(q, *rest, out=out), paged.pcd_k_paged_attention(q, *rest))
    untouched = torch.ones_like(buf, dtype=torch.bool)
    untouched.as_strided((n, heads, dim), (*strides, 1))[:] = False
    assert torch.all(buf[untouched] == 7)


def test_append_to_caches_in_odd_places(paged):  # noqa: F811
    """Caches cut out of pools that hold other things between their rows, or
    whose pages and heads lie between one another."""
    new, old = [40, 17], [0, 30]
    table, kc, vc, ks, vs, k, v, q_off, kv_len, n = append_case("int8", "f16", 16, 64, 2, new, old, 0, False)
    pool = kc.shape[0]
    want = [t.clone() for t in (kc, vc, ks, vs)]
    paged.pcd_k_kv_append(k, v, *want, q_off, kv_len, table)

    def check(kd, vd):
        kd.copy_(kc), vd.copy_(vc)
        s = [ks.clone(), vs.clone()]
        paged.pcd_k_kv_append(k, v, kd, vd, *s, q_off, kv_len, table)
        assert all(torch.equal(a, b) for a, b in zip((kd, vd, *s), want))

    both = torch.zeros(pool, 2, 16, 2, 128, dtype=torch.int8, device="cuda")  # [page][k, v][slot][head], wide rows
    check(*(both[:, i, :, :, 64:].transpose(1, 2) for i in range(2)))
    pair = torch.zeros(pool, 2, 16, 128, dtype=torch.int8, device="cuda")  # keys and values side by side in a row
    check(pair[..., :64], pair[..., 64:])
    flat = torch.zeros(2, 16 * 192 * pool, dtype=torch.int8, device="cuda")  # slots of three heads' width, heads between
    check(*(f.as_strided((pool, 2, 16, 64), (16 * 192, 64, 192, 1)) for f in flat))


def test_output_beside_the_input(paged):  # noqa: F811
    """The output in the other half of the input's heads, and in every second
    token's rows: places of their own, though the rows lie between one another."""
    freqs = paged.pcd_rope_freqs(64, 1e6)[0].cuda()
    q, *rest = attend_case("int8", "f16", 16, 64, 4, 2, [9, 3], [90, 30], 3)
    n = q.shape[0]
    for shape, cut in (((n, 4, 128), lambda b, i: b[..., 64 * i:64 * i + 64]), ((2 * n, 4, 64), lambda b, i: b[i::2]),
                       ((n, 8, 64), lambda b, i: b[:, i::2]), ((n, 4, 160), lambda b, i: b[..., 80 * i:80 * i + 64])):
        for i in (0, 1):
            buf = torch.full(shape, 7.0, dtype=q.dtype, device="cuda")
            x, y = cut(buf, i), cut(buf, 1 - i)
            x.copy_(q)
            assert torch.equal(paged.pcd_k_rope(x, freqs, out=y), paged.pcd_k_rope(q, freqs)) and torch.equal(x, q)
            assert torch.equal(paged.pcd_k_paged_attention(x, *rest, out=y), paged.pcd_k_paged_attention(q, *rest))
            assert torch.equal(x, q)


@pytest.mark.parametrize("base", [2 ** 31 - 4, 2 ** 31 - 1, -2 ** 31, -5])
@pytest.mark.parametrize("inter", [False, True])
def test_rope_base_at_the_ends(paged, base, inter):  # noqa: F811
    """Positions base + row that pass 2^31, or start at -2^31."""
    n = 9
    x = torch.randn(n, 3, 64, generator=gen(2), device="cuda")
    freqs, _ = paged.pcd_rope_freqs(64, 1e4)
    y = paged.pcd_k_rope(x, freqs.cuda(), base=base, interleaved=inter)
    for t in range(n):
        turns = torch.tensor([((base + t) * int(f)) % 2 ** 64 / 2 ** 64 for f in freqs.tolist()], dtype=torch.float64, device="cuda")
        want, err = R.rotate(x[t:t + 1], torch.ones(1, device="cuda"), turns * 2 * math.pi, inter)
        assert torch.all((y[t:t + 1].double() - want).abs() <= err + want.abs() * R.HALF[x.dtype] * 1.001)


def test_rope_base_refused(paged):  # noqa: F811
    x = torch.zeros(2, 1, 64, device="cuda")
    freqs = paged.pcd_rope_freqs(64, 1e4)[0].cuda()
    for base in (2 ** 31, -2 ** 31 - 1, 2 ** 32, 2 ** 70):
        with pytest.raises(ValueError):
            paged.pcd_k_rope(x, freqs, base=base)


def test_sizes_beyond_c_ints(paged):  # noqa: F811
    """More rows than a C int counts are refused, not taken by their low bits."""
    freqs = paged.pcd_rope_freqs(2, 1e4)[0].cuda()
    for n in (2 ** 31, 2 ** 32 + 1):
        with pytest.raises(ValueError):
            paged.pcd_k_rope(torch.zeros(1, 1, 2, device="cuda").expand(n, 1, 2), freqs)
        with pytest.raises(ValueError):
            paged.pcd_k_rope(torch.zeros(1, 1, 2, device="cuda").expand(1, n, 2), freqs)
        q, *cache, q_off, kv_len, table = attend_case("int8", "f16", 16, 64, 2, 2, [1], [20], 3)
        many = q.expand(n, 2, 64)
        with pytest.raises(ValueError):
            paged.pcd_k_paged_attention(many, *cache, q_off, kv_len, table)
        with pytest.raises(ValueError):
            paged.pcd_k_kv_append(many, many, *cache, q_off, kv_len, table)
        with pytest.raises(ValueError):
            paged.pcd_k_paged_attention_scratch_bytes(n, 1, 2, 2, 64, 100)


def test_rows_that_require_a_gradient(paged):  # noqa: F811
    """No call records a gradient: rows that want one are refused, and taken
    detached or where gradients are off."""
    freqs = paged.pcd_rope_freqs(64, 1e6)[0].cuda()
    q, *cache, q_off, kv_len, table = attend_case("int8", "f16", 16, 64, 2, 2, [3], [20], 3)
    want = paged.pcd_k_rope(q, freqs), paged.pcd_k_paged_attention(q, *cache, q_off, kv_len, table)
    leaf = q.clone().requires_grad_()
    rows = leaf * 1.0
    for x in (leaf, rows):
        with pytest.raises(ValueError, match="gradient"):
            paged.pcd_k_rope(x, freqs)
        with pytest.raises(ValueError, match="gradient"):
            paged.pcd_k_rope(q, freqs, out=x)
        with pytest.raises(ValueError, match="gradient"):
            paged.pcd_k_paged_attention(x, *cache, q_off, kv_len, table)
        for k, v in ((x, q), (q, x)):
            with pytest.raises(ValueError, match="gradient"):
                paged.pcd_k_kv_append(k, v, *cache, q_off, kv_len, table)
        assert torch.equal(paged.pcd_k_rope(x.detach(), freqs), want[0])
        with torch.no_grad():
            assert torch.equal(paged.pcd_k_paged_attention(x, *cache, q_off, kv_len, table), want[1])
    with torch.inference_mode():
        assert torch.equal(paged.pcd_k_rope(leaf, freqs), want[0])


# --------------------------------------------------------------------- failures
def test_attention_wait_timeout():
    """Under a 1 ns wait limit a failed pipeline's rows are NaN and reported,
    and the others right (in a child process: the limit is the process's)."""
    import paged_timeout_worker as wk
    env = {**os.environ, "PCD_WAIT_LIMIT_MS": "0.000001"}
    r = subprocess.run([sys.executable, wk.__file__], env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "other calls ok" in r.stdout, r.stdout
    print(r.stdout)


# ----------------------------------------------------------------------- scales
@pytest.mark.parametrize("dtype,lo,hi", [("f16", -33, 7), ("bf16", -20, 20), ("bf16", -60, 40)])
@pytest.mark.parametrize("q_len,hint", CUTS)
def test_attention_value_scales_far_apart(paged, q_len, hint, dtype, lo, hi):  # noqa: F811
    """Blocks whose value scales lie 2^40 and 2^100 apart, in falling, rising
    and random order, beside blocks of scale zero and sharp scores.  The bounds
    are those of every other call: a weight's share of O that fp16 loses is
    2^-33 of the largest, and fp32 weights of under 2^-126, which the normaliser
    would miss, lie 2^-134 below the largest times its scale, so 2^-34 below its
    softmax weight at 2^100."""
    q, kc, vc, ks, vs, q_off, kv_len, table = attend_case("int8", dtype, 16, 128, 7, 1, [q_len, q_len], [400, 250], 3)
    ks *= torch.exp2(torch.randint(-4, 4, ks.shape, generator=gen(3), device="cuda").float())
    pages = table[0, :25].long()
    for order in ("falls", "rises", "random"):
        e = torch.linspace(hi, lo, 25, device="cuda").round() if order != "random" else \
            torch.randint(lo, hi + 1, (25,), generator=gen(2), device="cuda").float()
        vs[:] = 2.0 ** lo
        vs[pages, 0] = torch.exp2(e.flip(0) if order == "rises" else e)
        vs[pages[3]] = 0.0
        a = (q, kc, vc, ks, vs, q_off, kv_len, table)
        for causal in (True, False):
            got, lse = paged.pcd_k_paged_attention(*a, max_kv=hint, causal=causal, return_lse=True)
            check_attend(got, lse, R.attention(*a, causal, 128 ** -0.5))
