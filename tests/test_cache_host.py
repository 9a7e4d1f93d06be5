"""The paged 4-bit cache without a GPU: sizes, seeds and workspaces from the host
entry points, and every refusal that is made before anything is enqueued."""
import ctypes as C

import pytest

import kv_cache_compression_04_b200 as kvc
from kv_cache_compression_04_b200 import build

FAKE = 0x7F0000000000  # never dereferenced: nothing is enqueued without a GPU
GOLDEN = 0x9E3779B97F4A7C15
OK_ARGS = kvc.KVC_ERR_CUDA  # what a call that passes its checks ends with here


@pytest.fixture(scope="module", autouse=True)
def L():
    import torch
    if torch.cuda.is_available():
        pytest.skip("the accepted calls would be enqueued on fake pointers")
    build.build()
    return kvc.lib()


def desc(**over):
    f = dict(layers=2, kv_heads=8, head_dim=128, bits=4, group_size=64, quant=kvc.KVC_QUANT_ASYM,
             signs=kvc.KVC_SIGNS_GLOBAL, first_layer=0, sign_seed=7, page_tokens=16, reserved=0,
             num_pages=100, pool=FAKE)
    f.update(over)
    block = 16 * (128 // 2 + 2 * 4)
    f.setdefault("stride_head", block)
    f.setdefault("stride_kv", block * 8)
    f.setdefault("stride_page", block * 16)
    f.setdefault("stride_layer", block * 1600)
    d = kvc.kvc_cache_desc()
    for k, v in f.items():
        setattr(d, k, v)
    return d


def rows(**over):
    f = dict(dtype=kvc.KVC_BF16, reserved=0, tokens=5, k=FAKE, v=FAKE, k_stride_layer=5120,
             k_stride_token=1024, k_stride_head=128, v_stride_layer=5120, v_stride_token=1024,
             v_stride_head=128, slots=FAKE)
    f.update(over)
    r = kvc.kvc_cache_rows()
    for k, v in f.items():
        setattr(r, k, v)
    return r


def attn(**over):
    f = dict(dtype=kvc.KVC_BF16, q_per_kv=4, n_requests=3, max_q=1, causal=1, window=0, scale=0.1,
             reserved=0, q_tokens=3, q_starts=None, seq_lens=FAKE, page_table=FAKE,
             page_table_pages=10, page_table_stride=10, q=FAKE, q_stride_layer=3 * 4096,
             q_stride_token=4096, q_stride_head=128, out=FAKE, out_stride_layer=3 * 4096,
             out_stride_token=4096, out_stride_head=128, lse=None)
    f.update(over)
    t = kvc.kvc_cache_attn()
    for k, v in f.items():
        setattr(t, k, v)
    return t


INVALID, UNSUPPORTED, CAPACITY = kvc.KVC_ERR_INVALID_ARG, kvc.KVC_ERR_UNSUPPORTED, kvc.KVC_ERR_CAPACITY
BAD_SHAPES = [(dict(layers=-1), INVALID), (dict(kv_heads=-1), INVALID), (dict(num_pages=-1), INVALID),
              (dict(first_layer=-1), INVALID), (dict(reserved=1), INVALID), (dict(page_tokens=0), INVALID),
              (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=256), UNSUPPORTED), (dict(bits=8), UNSUPPORTED),
              (dict(group_size=16), UNSUPPORTED), (dict(head_dim=64, group_size=128), UNSUPPORTED),
              (dict(quant=kvc.KVC_QUANT_FP4), UNSUPPORTED), (dict(signs=2), UNSUPPORTED),
              (dict(page_tokens=24), UNSUPPORTED), (dict(page_tokens=65552), UNSUPPORTED),
              (dict(num_pages=1 << 31), UNSUPPORTED), (dict(num_pages=1 << 28), UNSUPPORTED),
              (dict(layers=1 << 20), UNSUPPORTED)]
BAD_POOLS = [(dict(pool=None), INVALID), (dict(pool=FAKE + 8), INVALID), (dict(stride_head=1160), INVALID),
             (dict(stride_page=8), INVALID), (dict(stride_kv=4), INVALID), (dict(stride_layer=24), INVALID)]


@pytest.mark.parametrize("d,g", [(128, 128), (128, 64), (128, 32), (64, 64), (64, 32)])
@pytest.mark.parametrize("page", [16, 48, 65536])
def test_block_bytes(d, g, page):
    assert kvc.kvc_cache_block_bytes(desc(head_dim=d, group_size=g, page_tokens=page)) == \
        page * (d // 2 + d // g * 4)


@pytest.mark.parametrize("over,why", BAD_SHAPES)
def test_bad_descriptions(over, why):
    c = desc(**over)
    assert kvc.kvc_cache_block_bytes(c) == 0 and kvc.kvc_cache_stream_seed(c) == 0
    assert kvc.kvc_cache_load_workspace_bytes(c, [4]) == 0
    assert kvc.kvc_cache_attend_workspace_bytes(c, attn()) == 0
    assert kvc.kvc_cache_write(c, rows(), FAKE, None) == why
    assert kvc.kvc_cache_read(c, rows(), FAKE, None) == why
    assert kvc.kvc_cache_load(FAKE, 1 << 20, c, [4], FAKE, FAKE, 1 << 30, None) == why
    assert kvc.kvc_cache_attend(c, attn(), FAKE, 1 << 40, FAKE, None) == why


@pytest.mark.parametrize("over,why", BAD_POOLS)
def test_bad_pools(over, why):
    c = desc(**over)
    assert kvc.kvc_cache_block_bytes(c) > 0  # the pool is not looked at
    assert kvc.kvc_cache_write(c, rows(), FAKE, None) == why
    assert kvc.kvc_cache_read(c, rows(), FAKE, None) == why
    assert kvc.kvc_cache_load(FAKE, 1 << 20, c, [4], FAKE, FAKE, 1 << 30, None) == why
    assert kvc.kvc_cache_attend(c, attn(), FAKE, 1 << 40, FAKE, None) == why


def test_null_descriptions(L):
    assert L.kvc_cache_block_bytes(None) == 0 and L.kvc_cache_stream_seed(None) == 0
    assert L.kvc_cache_write(None, C.byref(rows()), FAKE, None) == INVALID
    assert L.kvc_cache_read(C.byref(desc()), None, FAKE, None) == INVALID
    assert L.kvc_cache_attend(C.byref(desc()), None, FAKE, 1 << 40, FAKE, None) == INVALID
    assert L.kvc_cache_load(FAKE, 1 << 20, C.byref(desc()), None, 1, FAKE, FAKE, 1 << 30, None) == INVALID
    assert L.kvc_cache_status_clear(None, None) == INVALID
    assert L.kvc_cache_status_clear(FAKE + 2, None) == INVALID


@pytest.mark.parametrize("over,why", [
    (dict(reserved=1), INVALID), (dict(tokens=-1), INVALID), (dict(tokens=1 << 31), INVALID),
    (dict(dtype=2), UNSUPPORTED), (dict(k=None), INVALID), (dict(v=FAKE + 8), INVALID),
    (dict(k_stride_token=1028), INVALID), (dict(v_stride_head=4), INVALID),
    (dict(k_stride_layer=12), INVALID), (dict(slots=None), INVALID), (dict(slots=FAKE + 4), INVALID)])
def test_bad_rows(over, why):
    for call in (kvc.kvc_cache_write, kvc.kvc_cache_read):
        assert call(desc(), rows(), FAKE, None) == OK_ARGS
        assert call(desc(), rows(), None, None) == OK_ARGS
        assert call(desc(), rows(**over), FAKE, None) == why
        assert call(desc(), rows(), FAKE + 1, None) == INVALID


def test_nothing_to_do():
    """No tokens, layers, heads or requests: accepted, whatever the other pointers are."""
    for c, r in ((desc(), rows(tokens=0, k=None, v=None, slots=None)),
                 (desc(layers=0, pool=None), rows(k=None)), (desc(kv_heads=0, pool=None), rows(slots=None))):
        assert kvc.kvc_cache_write(c, r, None, None) == kvc.KVC_OK
        assert kvc.kvc_cache_read(c, r, None, None) == kvc.KVC_OK
    for c, t in ((desc(), attn(n_requests=0, q=None, seq_lens=None, page_table=None)),
                 (desc(), attn(q_tokens=0, q_starts=FAKE, out=None)), (desc(layers=0, pool=None), attn(q=None)),
                 (desc(kv_heads=0, pool=None), attn(out=None))):
        assert kvc.kvc_cache_attend(c, t, None, 0, None, None) == kvc.KVC_OK


@pytest.mark.parametrize("over,why", [
    (dict(reserved=1), INVALID), (dict(n_requests=-1), INVALID),
    (dict(n_requests=kvc.KVC_MAX_REQUESTS + 1, q_tokens=5000), INVALID), (dict(max_q=0), INVALID),
    (dict(causal=2), INVALID), (dict(window=-1), INVALID), (dict(window=4, causal=0), INVALID),
    (dict(q_tokens=-1), INVALID), (dict(q_tokens=(1 << 24) + 1), INVALID), (dict(q_tokens=2), INVALID),
    (dict(page_table_pages=-1), INVALID), (dict(page_table_pages=1 << 31), INVALID),
    (dict(page_table_stride=-1), INVALID), (dict(dtype=3), UNSUPPORTED), (dict(q_per_kv=0), UNSUPPORTED),
    (dict(q_per_kv=65), UNSUPPORTED)])
def test_bad_attention_shapes(over, why):
    assert kvc.kvc_cache_attend_workspace_bytes(desc(), attn(**over)) == 0
    assert kvc.kvc_cache_attend(desc(), attn(**over), FAKE, 1 << 40, FAKE, None) == why


@pytest.mark.parametrize("over", [
    dict(q=None), dict(q=FAKE + 2), dict(out=FAKE + 8), dict(q_stride_token=4100), dict(q_stride_head=4),
    dict(out_stride_layer=2), dict(seq_lens=None), dict(seq_lens=FAKE + 2), dict(q_starts=FAKE + 1),
    dict(page_table=None), dict(page_table=FAKE + 2), dict(lse=FAKE + 2)])
def test_bad_attention_pointers(over):
    assert kvc.kvc_cache_attend(desc(), attn(), FAKE, 1 << 40, FAKE, None) == OK_ARGS
    assert kvc.kvc_cache_attend(desc(), attn(**over), FAKE, 1 << 40, FAKE, None) == INVALID


def test_attention_workspace():
    """One record per unit and per warp of the launch (few rows) or CTA (blocks of 128), of
    cols x (4 + head_dim) floats, and the prefixes, shapes, fragments or block numbers."""
    for max_q, qpk, cols, blocks, extra in ((1, 4, 4, 3, 2560), (2, 4, 8, 3, 2560), (1, 9, 16, 3, 2560),
                                            (8, 4, 16, 6, 2560), (9, 4, 128, 3 + 27 * 4 // 128, 160)):
        t = attn(max_q=max_q, q_per_kv=qpk, q_tokens=3 * max_q, q_starts=FAKE)
        units = 2 * 8 * blocks
        rec = (units + extra) * cols * 132 * 4
        got = kvc.kvc_cache_attend_workspace_bytes(desc(), t)
        assert rec < got <= rec + units * (18000 if cols <= 16 else 68000) + 4096
        assert kvc.kvc_cache_attend(desc(), t, FAKE, got, FAKE, None) == OK_ARGS
        assert kvc.kvc_cache_attend(desc(), t, FAKE, got - 1, FAKE, None) == CAPACITY
        assert kvc.kvc_cache_attend(desc(), t, None, got, FAKE, None) == INVALID
        assert kvc.kvc_cache_attend(desc(), t, FAKE + 8, got, FAKE, None) == INVALID
        assert kvc.kvc_cache_attend(desc(), t, FAKE, got, FAKE + 2, None) == INVALID
    assert kvc.kvc_cache_attend(desc(), attn(page_table_pages=0, page_table=None), FAKE, 1 << 40, FAKE,
                                None) == OK_ARGS
    # units that 32 bits do not count
    many = desc(layers=1 << 10, kv_heads=1 << 12)
    assert kvc.kvc_cache_attend_workspace_bytes(many, attn(n_requests=1024, q_tokens=1024)) == 0
    assert kvc.kvc_cache_attend(many, attn(n_requests=1024, q_tokens=1024), FAKE, 1 << 60, FAKE,
                                None) == UNSUPPORTED


def test_load_workspace_and_refusals():
    seq = [1000, 0, 513]
    meta = -(-2 * 2 * 8 * sum(seq) * 8 // 16384)
    got = kvc.kvc_cache_load_workspace_bytes(desc(), seq)
    assert meta * 16384 < got <= meta * 16384 + 4096
    call = kvc.kvc_cache_load
    assert call(FAKE, 1 << 20, desc(), seq, FAKE, FAKE, got, None) == OK_ARGS
    assert call(FAKE, 1 << 20, desc(), seq, FAKE, FAKE, got - 1, None) == CAPACITY
    assert call(None, 1 << 20, desc(), seq, FAKE, FAKE, got, None) == INVALID
    assert call(FAKE + 8, 1 << 20, desc(), seq, FAKE, FAKE, got, None) == INVALID
    assert call(FAKE, 1 << 20, desc(), seq, None, FAKE, got, None) == INVALID
    assert call(FAKE, 1 << 20, desc(), seq, FAKE + 4, FAKE, got, None) == INVALID
    assert call(FAKE, 1 << 20, desc(), seq, FAKE, FAKE + 8, got, None) == INVALID
    assert call(FAKE, 1 << 20, desc(), seq, FAKE, None, got, None) == INVALID
    assert call(FAKE, 1 << 20, desc(), [5, -1], FAKE, FAKE, got, None) == INVALID
    assert call(FAKE, 1 << 20, desc(), [1] * 1025, FAKE, FAKE, 1 << 40, None) == INVALID
    assert call(FAKE, 1 << 20, desc(), [1 << 30, 1 << 30], FAKE, FAKE, 1 << 40, None) == UNSUPPORTED
    assert call(FAKE, 1 << 20, desc(), [], None, FAKE, got, None) == OK_ARGS  # (the header is checked)


def test_stream_seed():
    per = kvc.KVC_SIGNS_PER_VECTOR
    assert kvc.kvc_cache_stream_seed(desc(first_layer=3)) == 7
    assert kvc.kvc_cache_stream_seed(desc(signs=per)) == 7
    got = kvc.kvc_cache_stream_seed(desc(signs=per, first_layer=3, sign_seed=2 ** 64 - 5))
    assert got == (2 ** 64 - 5 + 3 * 2 * 8 * 2 * GOLDEN) % 2 ** 64
    got = kvc.kvc_cache_stream_seed(desc(signs=per, first_layer=3, head_dim=64))
    assert got == (7 + 3 * 2 * 8 * GOLDEN) % 2 ** 64


def test_paged_cache_refuses_in_python():
    """Descriptions that no block fits, and pools that are not on a GPU."""
    import torch
    with pytest.raises(kvc.KvcError):
        kvc.PagedCache(1, 2, 96, 4)
    with pytest.raises(kvc.KvcError):
        kvc.PagedCache(1, 2, 128, 4, page_tokens=20)
    with pytest.raises(ValueError):
        kvc.PagedCache(1, 2, 128, 4, pool=torch.zeros(1, 4, 2, 2, 16 * 68, dtype=torch.uint8))


def test_packed_structures():
    """The bytes that PagedCache's calls pass are the structures'."""
    a = rows(dtype=1, tokens=1 << 20, slots=FAKE + 64)
    assert bytes(a) == kvc._ROWS.pack(1, 0, 1 << 20, FAKE, FAKE, 5120, 1024, 128, 5120, 1024, 128, FAKE + 64)
    t = attn(dtype=1, window=5, scale=0.25, q_starts=FAKE + 4, lse=FAKE + 8)
    assert bytes(t) == kvc._ATTN.pack(1, 4, 3, 1, 1, 5, 0.25, 0, 3, FAKE + 4, FAKE, FAKE, 10, 10, FAKE,
                                      3 * 4096, 4096, 128, FAKE, 3 * 4096, 4096, 128, FAKE + 8)
