"""What the calls of rotary positions and the 8-bit paged cache refuse, checked
on the host before any GPU call: no GPU is needed."""
import ctypes

import pytest
import torch

INVALID, SHAPE = -1, -8
BASE = 1 << 20  # stands for device memory: a refused call touches none


@pytest.fixture(scope="module")
def lib():
    from constrained_decoding_gb300.build import build
    build()
    import constrained_decoding_gb300 as pkg
    return pkg.load()


def rope(lib, **kw):
    a = dict(x=BASE, y=2 * BASE, dtype=3, n=4, heads=2, dim=64, xt=128, xh=64, yt=128, yh=64, f=BASE, rot=64, inter=0,
             amp=1.0, pos=BASE, base=0, tr=0)
    a.update(kw)
    return lib.pcd_k_rope(*a.values(), None)


def pages(**kw):
    from constrained_decoding_gb300 import _decls as D
    a = dict(k=BASE, v=2 * BASE, k_scale=BASE, v_scale=3 * BASE, page_stride=2 * 16 * 64, head_stride=16 * 64, token_stride=64,
             n_pages=8, page_size=16, n_kv_heads=2, head_dim=64, format=1)
    a.update(kw)
    return D.pcd_kv_pages(**a)


def append(lib, cache=None, **kw):
    c = cache or pages()
    a = dict(k=BASE, v=BASE, dtype=3, kt=128, kh=64, vt=128, vh=64, q_off=BASE, kv_len=BASE, table=BASE, n_seq=2, n=4, ts=4,
             f=BASE, rot=64, inter=0, amp=1.0, pos=None, err=None)
    a.update(kw)
    return lib.pcd_k_kv_append(ctypes.byref(c), *a.values(), None)


def attend(lib, cache=None, **kw):
    c = cache or pages()
    a = dict(q=BASE, out=2 * BASE, lse=None, dtype=3, hq=4, qt=256, qh=64, ot=256, oh=64, q_off=BASE, kv_len=BASE, table=BASE,
             n_seq=2, n=4, ts=4, max_kv=64, causal=1, scale=0.125, scratch=None, sb=0, err=None)
    a.update(kw)
    return lib.pcd_k_paged_attention(ctypes.byref(c), *a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(dtype=0), dict(dtype=9), dict(n=-1), dict(heads=-1), dict(dim=0), dict(dim=1025), dict(rot=63), dict(rot=66),
    dict(rot=-2), dict(rot=0), dict(f=None), dict(f=BASE + 4), dict(amp=float("nan")), dict(amp=float("inf")), dict(x=None),
    dict(y=None), dict(x=BASE + 1), dict(pos=BASE + 2), dict(xt=-1), dict(yh=-64), dict(yh=63), dict(yt=63),
    dict(y=BASE + 2), dict(y=BASE + 128), dict(y=BASE, yt=256), dict(y=BASE, yh=128, yt=256),
    dict(n=2 ** 30, heads=4, dim=64, xt=256, yt=256, y=2 ** 50),
])
def test_rope_refuses(lib, kw):
    assert rope(lib, **kw) == INVALID
    assert lib.pcd_last_error()


def test_rope_takes_empty_calls(lib):
    assert rope(lib, n=0, x=None, y=None) == 0 and rope(lib, heads=0, x=None, y=None) == 0


@pytest.mark.parametrize("kw", [
    dict(rot=0), dict(rot=7), dict(theta=1.0), dict(theta=float("nan")), dict(theta=float("inf")), dict(scaling=5), dict(scaling=-1),
    dict(scaling=1, factor=0.5), dict(scaling=1, factor=float("inf")), dict(scaling=2, rot=2), dict(scaling=3, orig=0.0),
    dict(scaling=3, lo=0.0), dict(scaling=4, lo=4.0, hi=4.0), dict(scaling=4, hi=float("inf")), dict(scaling=4, orig=float("nan")),
])
def test_rope_freqs_refuses(lib, kw):
    a = dict(rot=8, theta=1e4, scaling=0, factor=4.0, orig=4096.0, lo=1.0, hi=8.0)
    a.update(kw)
    out = (ctypes.c_int64 * 4)(*[7] * 4)
    assert lib.pcd_rope_freqs(*a.values(), out, None) == INVALID
    assert list(out) == [7] * 4 and lib.pcd_last_error()


def test_rope_freqs_without_gpu(lib):
    from constrained_decoding_gb300 import paged
    f, amp = paged.pcd_rope_freqs(8, 1e4)
    assert amp == 1.0
    for i, v in enumerate(f.tolist()):
        assert v / 2.0 ** 64 * 6.283185307179586 == pytest.approx(1e4 ** (-i / 4), rel=1e-12)
    with pytest.raises(ValueError):
        paged.pcd_rope_freqs(8, 1e4, "wide")
    with pytest.raises(paged.PCDError) as e:
        paged.pcd_rope_freqs(7, 1e4)
    assert e.value.code == INVALID and "rot_dim" in str(e.value)


BAD_PAGES = [
    dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None), dict(k=BASE + 8), dict(v=BASE + 1), dict(k_scale=BASE + 2),
    dict(page_size=8), dict(page_size=48), dict(page_size=256), dict(page_size=0), dict(n_pages=0), dict(n_kv_heads=0),
    dict(n_kv_heads=70000), dict(format=0), dict(format=3), dict(page_stride=2056), dict(head_stride=1032), dict(token_stride=72),
    dict(token_stride=48), dict(token_stride=0), dict(token_stride=-64), dict(token_stride=(1 << 24) + 16), dict(head_stride=0), dict(page_stride=0),
]


@pytest.mark.parametrize("kw", BAD_PAGES)
def test_cache_refused(lib, kw):
    for call in (append, attend):
        assert call(lib, pages(**kw)) == INVALID
        assert lib.pcd_last_error()


@pytest.mark.parametrize("dim", [16, 32, 80, 96, 192, 256])
def test_head_dims_refused(lib, dim):
    c = pages(head_dim=dim, token_stride=256, head_stride=4096, page_stride=8192)
    assert append(lib, c) == SHAPE and attend(lib, c) == SHAPE


@pytest.mark.parametrize("kw", [
    dict(dtype=0), dict(n=-1), dict(n_seq=-1), dict(ts=-1), dict(q_off=None), dict(kv_len=None), dict(table=None),
    dict(q_off=BASE + 2), dict(kv_len=BASE + 1), dict(table=BASE + 3), dict(k=None), dict(v=None), dict(k=BASE + 1), dict(v=BASE + 1),
    dict(kt=-1), dict(vh=-1), dict(rot=66), dict(rot=5), dict(rot=0), dict(f=None), dict(f=BASE + 4), dict(pos=BASE + 1),
    dict(err=BASE + 2), dict(amp=float("nan")),
])
def test_append_refuses(lib, kw):
    assert append(lib, **kw) == INVALID
    assert lib.pcd_last_error()


@pytest.mark.parametrize("kw", [dict(v=BASE), dict(v_scale=BASE)])
def test_append_refuses_keys_and_values_in_one_place(lib, kw):
    assert append(lib, pages(**kw)) == INVALID
    assert b"one place" in lib.pcd_last_error()


@pytest.mark.parametrize("kw", [
    dict(dtype=1), dict(dtype=7), dict(hq=0), dict(hq=3), dict(hq=258), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(max_kv=-1), dict(n=2 ** 29, max_kv=0), dict(q=None), dict(out=None), dict(q=BASE + 1),
    dict(out=BASE + 1), dict(lse=BASE + 2), dict(err=BASE + 1), dict(qt=-1), dict(oh=-64), dict(oh=63), dict(ot=63), dict(n=-1),
    dict(n_seq=-1), dict(ts=-1), dict(q_off=None), dict(kv_len=None), dict(table=None), dict(table=BASE + 2),
    dict(max_kv=100000, ts=10000, scratch=None), dict(max_kv=100000, ts=10000, scratch=BASE, sb=64),
    dict(max_kv=100000, ts=10000, scratch=BASE + 8, sb=1 << 40),
    dict(out=BASE, ot=512), dict(out=BASE, oh=128, ot=512), dict(out=BASE + 128), dict(out=BASE - 256, qt=256, ot=512),
])
def test_attention_refuses(lib, kw):
    assert attend(lib, **kw) == INVALID
    assert lib.pcd_last_error()


def test_binding_packs_the_struct_of_the_header(lib):
    """The binding's packed pcd_kv_pages has the layout of its declaration."""
    from constrained_decoding_gb300 import _decls as D
    from constrained_decoding_gb300 import paged
    vals = (11, 12, 13, 14, 21, 22, 23, 31, 32, 33, 34, 35)
    raw = paged._PAGES.pack(*vals)
    assert len(raw) == ctypes.sizeof(D.pcd_kv_pages)
    c = D.pcd_kv_pages.from_buffer_copy(raw)
    assert tuple(getattr(c, n) for n, _ in D.pcd_kv_pages._fields_) == vals


def test_empty_calls(lib):
    assert append(lib, n=0, k=None, v=None) == 0 and append(lib, n_seq=0, n=3) == 0
    assert attend(lib, n=0, q=None, out=None) == 0 and attend(lib, n_seq=0) == 0


def test_scratch_sizes(lib):
    b = lib.pcd_k_paged_attention_scratch_bytes
    assert b(0, 1, 4, 2, 64, 100) == 0 and b(4, 0, 4, 2, 64, 100) == 0 and b(4, 1, 3, 2, 64, 100) == 0
    assert b(4, 1, 4, 2, 64, -1) == 0 and b(4, 1, 4, 2, 64, 16) == 0
    assert b(1, 1, 4, 2, 64, 100000) > 0


def test_binding_refuses_host_tensors(lib):
    from constrained_decoding_gb300 import paged
    x = torch.zeros(2, 2, 64, dtype=torch.float16)
    c = torch.zeros(3, 2, 16, 64, dtype=torch.int8)
    s = torch.ones(3, 2)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        paged.pcd_k_rope(x, None)
    with pytest.raises(ValueError):
        paged.pcd_k_kv_append(x, x, c, c, s, s, i, i[:1], i[None])
    with pytest.raises(ValueError):
        paged.pcd_k_paged_attention(x, c, c, s, s, i, i[:1], i[None])
