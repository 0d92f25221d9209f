"""Refusals of the calls of rotary positions and the 8-bit paged cache that
depend on how several arguments go together, and sizes the host computes: no GPU
is needed."""
import ctypes

import pytest

from test_paged_refusals import BASE, INVALID, append, attend, lib, pages, rope  # noqa: F401


# ------------------------------------------------------------- table slices
def append_cols(lib, stride, width, n=4):
    return lib.pcd_k_kv_append_cols(ctypes.byref(pages()), BASE, BASE, 3, 128, 64, 128, 64, BASE, BASE, BASE, 2, n, stride, width,
                                    BASE, 64, 0, 1.0, None, None, None)


def attend_cols(lib, stride, width, n=4):
    return lib.pcd_k_paged_attention_cols(ctypes.byref(pages()), BASE, 2 * BASE, None, 3, 4, 256, 64, 256, 64, BASE, BASE, BASE,
                                          2, n, stride, width, 64, 1, 0.125, None, 0, None, None)


@pytest.mark.parametrize("stride,width", [(4, 5), (4, -1), (-1, -1), (0, 1), (-4, 0)])
def test_table_slices_refused(lib, stride, width):  # noqa: F811
    for call in (append_cols, attend_cols):
        assert call(lib, stride, width) == INVALID and lib.pcd_last_error()
        assert call(lib, 4, 3, n=0) == 0


# -------------------------------------------------------- rows that share a place
@pytest.mark.parametrize("tok,head,heads", [(64, 64, 2), (128, 64, 3), (64, 128, 2), (96, 64, 2), (100, 164, 2), (160, 96, 3), (128, 190, 2)])
def test_outputs_whose_rows_overlap(lib, tok, head, heads):  # noqa: F811
    """Each stride alone holds a row, together they put two rows in one place."""
    assert rope(lib, yt=tok, yh=head, heads=heads, xt=64 * heads, y=1 << 40) == INVALID
    assert b"strides of y overlap" in lib.pcd_last_error()
    assert attend(lib, ot=tok, oh=head, hq=2 * heads, out=1 << 40) == INVALID
    assert b"strides of out overlap" in lib.pcd_last_error()


@pytest.mark.parametrize("kw", [
    dict(page_stride=64), dict(page_stride=1024), dict(head_stride=64), dict(head_stride=512), dict(token_stride=128),
    dict(page_stride=1024 + 16), dict(page_stride=64, head_stride=64 * 8), dict(page_stride=128, head_stride=64, token_stride=192),
])
def test_append_refuses_caches_whose_rows_overlap(lib, kw):  # noqa: F811
    assert append(lib, pages(**kw)) == INVALID
    assert b"cache: strides overlap" in lib.pcd_last_error()


@pytest.mark.parametrize("kw", [
    dict(v=BASE + 16), dict(v=BASE + 48), dict(v=BASE - 48), dict(v=BASE + 1024), dict(v=BASE + 2048 * 7 + 1024), dict(v=BASE - 2048 * 7),
    dict(token_stride=128, head_stride=2048, page_stride=4096, v=BASE + 48), dict(v=BASE + 2048 * 8 - 16),
    dict(v_scale=BASE + 4), dict(v_scale=BASE + 4 * 15), dict(v_scale=BASE - 4 * 15),
    dict(page_size=32, n_pages=3, n_kv_heads=5, head_stride=64, token_stride=320, page_stride=320 * 32, v=BASE + 2 * 10240 + 320 * 31 + 64 * 4 + 48),
])
def test_append_refuses_keys_over_values(lib, kw):  # noqa: F811
    """Keys and values, or their scales, that share some places."""
    assert append(lib, pages(**kw)) == INVALID
    assert b"one place" in lib.pcd_last_error()


@pytest.mark.parametrize("kw", [dict(y=BASE + 2 * 32), dict(y=BASE + 2 * 128), dict(y=BASE - 2 * 64), dict(y=BASE + 2 * 64, heads=1),
                                dict(xt=256, yt=256, xh=128, yh=128, y=BASE + 2 * 48), dict(xt=256, yt=256, xh=128, yh=128, y=BASE + 2 * 208)])
def test_views_of_equal_strides_that_meet(lib, kw):  # noqa: F811
    if kw.get("heads") == 1:
        kw = dict(kw, xt=64, yt=64)
    assert rope(lib, **kw) == INVALID
    assert b"overlap without" in lib.pcd_last_error()


# ------------------------------------------------------------------ frequencies
@pytest.mark.parametrize("scaling", ["bands", "ramp"])
@pytest.mark.parametrize("orig,lo,hi", [(1.0, 1.0, 32.0), (6.0, 1.0, 4.0), (40.0, 8.0, 9.0), (6.3, 1.0, 32.0), (1e9, 1.0, 32.0), (1e300, 1.0, 2.0)])
def test_frequencies_at_the_ends_of_the_scalings(lib, scaling, orig, lo, hi):  # noqa: F811
    """Pairs that turn at least hi times over the length stay, those that turn
    at most lo times are divided by the factor, for lengths so short that even
    the first pair is among these and so long that all stay."""
    import math

    from constrained_decoding_gb300 import paged
    rot, theta, factor = 32, 1e4, 8.0
    freqs, _ = paged.pcd_rope_freqs(rot, theta, scaling, factor, orig, lo, hi)
    for i, v in enumerate(freqs.tolist()):
        f = theta ** (-2 * i / rot)
        turns = orig * f / (2 * math.pi)
        got = (v % 2 ** 64) / 2 ** 64 * 2 * math.pi
        # the ramp's ends are rounded outwards to whole pairs: only pairs beyond those are at an end for sure
        step = theta ** (2 / rot) if scaling == "ramp" and turns < orig / (2 * math.pi) else 1.0
        if turns >= hi * step:
            assert got == pytest.approx(f, rel=1e-12), i
        elif turns * step <= lo:
            assert got == pytest.approx(f / factor, rel=1e-12), i
        else:
            assert f / factor * (1 - 1e-12) <= got <= f * (1 + 1e-12), i


# -------------------------------------------------------------------- workspace
@pytest.mark.parametrize("n_tok,heads,kv_heads,max_kv", [(8192, 64, 8, 131072), (4096, 64, 8, 1 << 20), (4096, 64, 8, 131072), (65536, 128, 8, 1 << 20)])
def test_long_prompts_need_no_workspace(lib, n_tok, heads, kv_heads, max_kv):  # noqa: F811
    """Where the query rows alone fill the GPU, ranges of keys would cost
    hundreds of MB for no time."""
    assert lib.pcd_k_paged_attention_scratch_bytes(n_tok, 1, heads, kv_heads, 128, max_kv) == 0


def test_workspace_is_bounded(lib):  # noqa: F811
    b = lib.pcd_k_paged_attention_scratch_bytes
    assert b(1024, 1, 64, 8, 128, 131072) > 0  # few rows: ranges of keys
    for n_tok in (64, 313, 1000, 1024, 2048, 3000, 5000, 20000):
        for n_seq in (1, 3, 17):
            for heads, kv_heads in ((8, 8), (28, 4), (64, 8), (128, 1)):
                for max_kv in (900, 8192, 131072, 1 << 20, 1 << 31):
                    if n_tok * heads // kv_heads > 32 * n_seq:
                        assert b(n_tok, n_seq, heads, kv_heads, 128, max_kv) <= 1 << 29
