"""The paged 4-bit cache in use on the GPU: streams loaded into pages against the
decoder, the forms for few and for many rows against each other, what bad numbers
on the device do, captured calls, other streams, and the calls together."""
import numpy as np
import pytest
import torch

import cache_ref as ref
import kv_cache_compression_04_b200 as kvc
from kvc_testutil import chunk_table
from test_gpu_cache import HALF, KINDS, make, rows, run_attend, slots_for

pytestmark = pytest.mark.gpu

CORRUPT, NONFINITE, RANGE = kvc.KVC_ERR_CORRUPT, kvc.KVC_ERR_NONFINITE, kvc.KVC_ERR_RANGE


def status_of(c):
    """The cache's status word, cleared."""
    try:
        c.check()
    except kvc.KvcError as e:
        return e.status
    return kvc.KVC_OK


def dev(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def cache_values(c, slots):
    """What the slots hold, in 64 bits: [L, 2, H, N, d], and the spreads."""
    d = c.desc
    sg = ref.signs(d.sign_seed, d.signs, d.layers, d.kv_heads, d.head_dim, d.first_layer)
    pool = c.pool.cpu().numpy()
    x = ref.values(pool, slots, sg, d.head_dim, d.group_size, d.page_tokens)
    return x, ref.spreads(*ref.rows_of(pool, slots, d.head_dim, d.group_size, d.page_tokens), d.group_size)


def close(c, slots, q, got, qpk, limits, scale, dtype, but=()):
    """Attention over the slots in 64 bits, with run_attend's bound; but: (query, head)
    pairs that are not compared."""
    x, spread = cache_values(c, slots)
    o, _, mag, size = ref.attend(x, q.double().cpu().numpy(), qpk, scale, limits, spread)
    ds = 2.0 ** -18 * size + 2.0 ** -20
    tol = HALF[dtype] * np.abs(o) + (2 * ds + 2.0 ** -11)[..., None] * mag * 1.01 + 1e-7
    bad = np.abs(got.double().cpu().numpy() - o) - tol
    for i, j in but:
        bad[:, i, j] = 0
    assert (bad <= 0).all(), bad.max()


# ---------------------------------------------------------------- load --
def stream_of(kv, g, seed, lossless, quant, signs):
    codec = kvc.Codec(4, g, seed, lossless, quant, signs)
    desc = kvc.dense_desc(kv)
    out, ws, n = codec.compress(desc)
    back = torch.empty_like(kv)
    codec.decompress(out, int(n.item()), kvc.dense_desc(back), ws)
    return out, int(n.item()), back


def narrow_meta(L, H, T, d, g, seed, signs):
    """Rows whose scales and zeros are nearly the same in every vector: their meta
    chunks are stored eliminated, their codes are not."""
    rng = np.random.default_rng(4)
    y = rng.uniform(-1, 1, (L, 2, H, T, d // g, g))
    y[..., 0], y[..., 1] = -1, 1
    x = y.reshape(L, 2, H, T, d) @ ref.hadamard(d) / d * ref.signs(seed, signs, L, H, d)[:, :, :, None]
    return torch.from_numpy(x * 8).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("d,g", KINDS)
@pytest.mark.parametrize("lossless,quant,signs,T", [(0, 0, 0, 77), (1, 1, 1, 600), (2, 0, 1, 1), (0, 1, 0, 2000)])
def test_load_is_the_decoder(d, g, lossless, quant, signs, T):
    L, H, page, seed = 2, 3, 32, 99
    gen = torch.Generator(device="cuda").manual_seed(T)
    kv = torch.randn(L, 2, H, T, d, generator=gen, device="cuda").to(torch.bfloat16)
    buf, n, back = stream_of(kv, g, seed, lossless, quant, signs)
    pages = -(-T // page) + 2
    c = make(d, g, L, H, pages, page, quant, signs, seed)
    s = slots_for(T, pages, page)
    before = c.pool.cpu().numpy().copy()
    c.load(buf, n, torch.from_numpy(s).cuda(), [T], check=True)
    k, v = c.read(torch.from_numpy(s).cuda())
    for i, x in enumerate((k, v)):
        assert torch.equal(x.transpose(1, 2).view(torch.int16), back[:, i].view(torch.int16))
    other = np.setdiff1d(np.arange(pages * page), s)
    after = c.pool.cpu().numpy()
    for a, b in zip(ref.rows_of(after, other, d, g, page), ref.rows_of(before, other, d, g, page)):
        assert np.array_equal(a, b)


@pytest.mark.parametrize("d,g", [(128, 32), (128, 128), (64, 64)])
@pytest.mark.parametrize("lossless", [0, 1])
def test_load_of_eliminated_meta(d, g, lossless):
    L, H, T, signs, seed = 1, 2, 3000, 1, 5
    kv = narrow_meta(L, H, T, d, g, seed, signs)
    buf, n, back = stream_of(kv, g, seed, lossless, 0, signs)
    vectors = L * 2 * H * T
    n_code, n_meta = -(-vectors * d // 2 // 16384), -(-vectors * (d // g) * 4 // 16384)
    host = buf[:n].cpu().numpy()
    sizes = chunk_table(host, n_code + n_meta)[0][n_code:]
    assert host[11] & 1 == 0 and (sizes[:-1] != 16384).any(), sizes
    c = make(d, g, L, H, T // 16 + 2, 16, 0, signs, seed)
    at = dev(slots_for(T, T // 16 + 2, 16).tolist(), torch.int64)
    c.load(buf, n, at, [T], check=True)
    k, v = c.read(at)
    for i, x in enumerate((k, v)):
        assert torch.equal(x.transpose(1, 2).view(torch.int16), back[:, i].view(torch.int16))


def test_load_some_layers_and_skipped_tokens():
    """A stream of layers 1 and 2 alone, with the seed whose diagonals are theirs; tokens
    without a slot, slots outside the pool."""
    d, g, H, T, page = 128, 64, 2, 50, 16
    c = make(d, g, 4, H, 5, page, 0, 1, seed=31)
    view = c[1:3]
    kv = torch.randn(2, 2, H, T, d, device="cuda").to(torch.bfloat16)
    buf, n, back = stream_of(kv, g, kvc.kvc_cache_stream_seed(view.desc), 0, 0, 1)
    s = slots_for(T, 5, page)
    s[::7] = -1
    before = c.pool.cpu().numpy().copy()
    view.load(buf, n, torch.from_numpy(s).cuda(), [T], check=True)
    after = c.pool.cpu().numpy()
    assert np.array_equal(after[[0, 3]], before[[0, 3]])
    keep = np.flatnonzero(s >= 0)
    k, v = view.read(torch.from_numpy(s[keep]).cuda())
    for i, x in enumerate((k, v)):
        assert torch.equal(x.transpose(1, 2).view(torch.int16), back[:, i][:, :, keep].view(torch.int16))
    s[3] = 5 * page
    with pytest.raises(kvc.KvcError):
        view.load(buf, n, torch.from_numpy(s).cuda(), [T], check=True)
    assert status_of(c) == kvc.KVC_OK  # its status word is its own


def test_load_refuses_other_streams():
    """A stream of other shapes, groups, signs or seeds, or cut short, says so."""
    d, g, L, H, T = 128, 64, 1, 2, 40
    kv = torch.randn(L, 2, H, T, d, device="cuda").to(torch.bfloat16)
    c = make(d, g, L, H, 4, 16, 0, 0, seed=3)
    at = dev(slots_for(T, 4, 16).tolist(), torch.int64)
    good, n, _ = stream_of(kv, g, 3, 0, 0, 0)
    c.load(good, n, at, [T], check=True)
    for buf, size, lens in ((good, n - 1, [T]), (good, 40, [T]), (good, n, [T - 1]), (good, n, [T - 5, 5]),
                            (stream_of(kv, g, 4, 0, 0, 0)[0], n, [T]),
                            (stream_of(kv, 128, 3, 0, 0, 0)[0], None, [T]),
                            (stream_of(kv, g, 3, 0, 0, 1)[0], n, [T]),
                            (stream_of(torch.zeros(1, 2, 2, 2048, d, dtype=torch.bfloat16, device="cuda"),
                                       g, 3, 0, 0, 0)[0], None, [2048])):
        slots = at[:sum(lens)] if sum(lens) <= T else dev([-1] * sum(lens), torch.int64)
        with pytest.raises(kvc.KvcError):
            c.load(buf, buf.numel() if size is None else size, slots, lens, check=True)
    c.load(torch.zeros(64, dtype=torch.uint8, device="cuda"), 0, at, [T])  # unread: nothing raises


# ------------------------------------------------------- rows and forms --
@pytest.mark.parametrize("d,g,L,H,n", [(128, 128, 2, 16, 9001), (128, 32, 2, 16, 9001), (64, 64, 2, 8, 4801),
                                       (64, 32, 1, 16, 4801), (128, 64, 2, 16, 9001)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_many_rows_are_few_rows(d, g, L, H, n, dtype):
    """Calls with enough blocks of 32 tokens per SM take another form: the same bytes,
    and the same rows, as calls of a few tokens each."""
    page, sms = 32, torch.cuda.get_device_properties(0).multi_processor_count
    assert L * 2 * H * -(-n // 32) >= (120 if d == 128 else 28) * sms
    pages = -(-n // page) + 1
    a, b = (make(d, g, L, H, pages, page, int(g == 64), 1, seed=8, fill=0) for _ in range(2))
    gen = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn(L, n, H, d, generator=gen, device="cuda").to(dtype)
    v = (torch.randn(L, n, H, d, generator=gen, device="cuda") * 3).to(dtype)
    k[0, 5, 1, 3] = float("nan")
    v[-1, n - 1, 0, 0] = float("inf")
    s = slots_for(n, pages, page)
    s[::11] = -1
    s[1000] = pages * page
    at = torch.from_numpy(s).cuda()
    a.write(k, v, at)
    assert status_of(a) in (CORRUPT, NONFINITE)
    step = 500
    for i in range(0, n, step):
        b.write(k[:, i:i + step], v[:, i:i + step], at[i:i + step])
    status_of(b)
    assert torch.equal(a.pool, b.pool)
    got = [torch.full((L, n, H, d), 5.0, dtype=dtype, device="cuda") for _ in range(4)]
    a.read(at, got[0], got[1])
    assert status_of(a) == CORRUPT
    for i in range(0, n, step):
        a.read(at[i:i + step], got[2][:, i:i + step], got[3][:, i:i + step])
    assert status_of(a) == CORRUPT
    for x, y in zip(got[:2], got[2:]):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))
        assert (x[:, ::11] == 5).all() and (x[:, 1000] == 5).all()
    assert torch.isnan(got[0][0, 5, 1]).all() and torch.isnan(got[1][-1, n - 1, 0]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_rows_that_cannot_be_stored(dtype):
    """NaN, infinities, and (bf16) ranges past fp16's: the row reads as NaN, others as they
    would; the first error stays until it is read."""
    d, g, n = 128, 64, 20
    c = make(d, g, 1, 2, 3, 16)
    k, v = rows(1, n, 2, d, dtype)
    clean = make(d, g, 1, 2, 3, 16)
    at = dev(slots_for(n, 3, 16).tolist(), torch.int64)
    clean.write(k, v, at)
    k[0, 3, 0, 7] = float("inf")
    v[0, 4, 1, 100] = float("nan")
    c.write(k, v, at)
    want = {(0, 3, 0), (1, 4, 1)}
    if dtype == torch.bfloat16:
        v[0, 9, 0] = 1e30
        want.add((1, 9, 0))
        assert status_of(c) == NONFINITE
        c.write(k[:, 9:10], v[:, 9:10], at[9:10])
        assert status_of(c) == RANGE
    else:
        assert status_of(c) == NONFINITE
    assert status_of(c) == kvc.KVC_OK
    got, good = c.read(at), clean.read(at)
    c.check()
    for kv in range(2):
        for i in range(n):
            for h in range(2):
                if (kv, i, h) in want:
                    assert torch.isnan(got[kv][0, i, h]).all()
                else:
                    assert torch.equal(got[kv][0, i, h], good[kv][0, i, h])


def test_slots_outside_the_pool():
    d, g, n = 64, 32, 9
    c = make(d, g, 1, 2, 2, 16)
    before = c.pool.clone()
    k, v = rows(1, n, 2, d)
    for bad in (32, 2 ** 31, 2 ** 32 + 1, 2 ** 62):
        c.write(k, v, dev([bad] * n, torch.int64))
        assert status_of(c) == CORRUPT
        out = torch.full((1, n, 2, d), 2.0, device="cuda", dtype=torch.bfloat16)
        c.read(dev([bad] * n, torch.int64), out, out.clone())
        assert status_of(c) == CORRUPT and (out == 2).all()
    c.write(k, v, dev([-1] * (n - 1) + [-2 ** 62], torch.int64))
    assert status_of(c) == kvc.KVC_OK and torch.equal(c.pool, before)
    s = dev(list(range(8)) + [40], torch.int64)
    c.write(k, v, s)  # the others are written
    assert status_of(c) == CORRUPT
    e = make(d, g, 1, 2, 2, 16)
    e.write(k[:, :8], v[:, :8], s[:8])
    assert torch.equal(c.pool, e.pool)
    # without a status word
    r = kvc.kvc_cache_rows(kvc.KVC_BF16, 0, n, k.data_ptr(), v.data_ptr(), *(0, 2 * d, d) * 2, s.data_ptr())
    assert kvc.kvc_cache_write(c.desc, r, None, torch.cuda.current_stream().cuda_stream) == kvc.KVC_OK
    torch.cuda.synchronize()
    assert status_of(c) == kvc.KVC_OK
    # the same slot read many times
    y = c.read(dev([3] * 40, torch.int64))[0]
    assert torch.equal(y, y[:, :1].expand_as(y))
    c.write(k[:, :0], v[:, :0], dev([], torch.int64))
    assert c.read(dev([], torch.int64))[0].shape == (1, 0, 2, d)


def test_high_offsets():
    """Pages past 2^32 bytes from the pool's start, in a pool that is not contiguous."""
    d, g, H, page = 128, 128, 2, 512
    block = ref.block_bytes(d, g, page)
    pages = (2 ** 32 + 2 ** 28) // (2 * H * block) + 2
    big = torch.empty(pages * 2 * H * block + 4096, dtype=torch.uint8, device="cuda")
    pool = big[:pages * 2 * H * block].view(1, pages, H, 2, block).transpose(2, 3)  # heads outside kv
    c = kvc.PagedCache(1, H, d, pages, page_tokens=page, group=g, sign_seed=1, pool=pool)
    small = make(d, g, 1, H, 2, page, seed=1)
    n = 700
    k, v = rows(1, n, H, d)
    t = np.arange(n)
    far = np.where(t < page, (pages - 1) * page, (pages - 7) * page - page) + t
    c.write(k, v, torch.from_numpy(far).cuda())
    small.write(k, v, torch.from_numpy(t).cuda())
    for x, y in zip(c.read(torch.from_numpy(far).cuda()), small.read(torch.from_numpy(t).cuda())):
        assert torch.equal(x, y)
    for asked in (1, 4, 100):  # 2, 8 and 200 rows
        q = torch.randn(1, asked, 2 * H, d, device="cuda").to(torch.bfloat16)
        st = dev([0, asked])
        a = c.attend(q, dev([[pages - 1, pages - 7]]), dev([n]), q_starts=st, max_q=asked)
        b = small.attend(q, dev([[0, 1]]), dev([n]), q_starts=st, max_q=asked)
        assert torch.equal(a, b) and a.abs().sum() > 0
    c.check()


# ------------------------------------------------------------ attention --
@pytest.mark.parametrize("d,g", KINDS)
@pytest.mark.parametrize("qpk,asked,causal,window", [
    (4, 5, True, 0), (8, 4, True, 21), (16, 3, True, 21), (12, 4, False, 0),  # 20 .. 48 rows
    (7, 7, True, 0), (64, 1, True, 0), (3, 90, True, 33), (8, 33, False, 0)])  # 49 .. 270: blocks of 128
def test_attend_many_rows(d, g, qpk, asked, causal, window):
    lens = [170, 1, 64, 65, 300]
    c = make(d, g, 1, 2, 64, 16, signs=1)
    run_attend(c, lens, [min(asked, n) for n in lens], qpk, torch.float16, window, causal, pad=2)


@pytest.mark.parametrize("d,g", KINDS)
@pytest.mark.parametrize("qpk,asked,window", [(4, 1, 0), (8, 1, 9), (16, 1, 0), (4, 6, 7), (8, 20, 0)])
def test_hidden_slots_may_hold_large_numbers(d, g, qpk, asked, window):
    """Scales and zeros of 65504 in slots that no query sees cost no precision."""
    c = make(d, g, 1, 1, 6, 16, fill=0)
    c.pool.view(torch.int16).fill_(0x7BFF)
    run_attend(c, [37 + asked], [asked], qpk, torch.float16, window=window)


@pytest.mark.parametrize("asked", [1, 6, 40])  # 4, 24 and 160 rows
def test_attend_marks_requests_that_are_out_of_range(asked):
    d, g, H, qpk, page = 128, 64, 2, 4, 16
    c = make(d, g, 1, H, 20, page)
    n = 64
    k, v = rows(1, 4 * n, H, d)
    c.write(k, v, torch.arange(4 * n, device="cuda"))
    tab = torch.arange(16, dtype=torch.int32, device="cuda").view(4, 4)
    q = torch.randn(1, 4 * asked, H * qpk, d, device="cuda").to(torch.bfloat16)
    starts = dev([i * asked for i in range(5)])
    good = c.attend(q, tab, dev([n] * 4), q_starts=starts, max_q=asked)
    c.check()

    def run(lens, st, **kw):
        out = torch.full_like(q, 3.0)
        lse = torch.full(q.shape[:3], 3.0, device="cuda")
        c.attend(q, tab, dev(lens), q_starts=dev(st), max_q=asked, out=out, lse=lse, **kw)
        return out, lse, status_of(c)

    for lens in ([n, n + 1, n, n], [n, -1, n, n], [n, 2 ** 31 - 1, n, n], [n, -2 ** 31, n, n]):
        out, lse, st = run(lens, starts.tolist())
        assert st == CORRUPT
        b = slice(asked, 2 * asked)
        assert (out[:, b] == 3).all() and (lse[:, b] == 3).all()
        out[:, b] = good[:, b]
        assert torch.equal(out, good)
    # more queries than max_q; past q's rows
    out, lse, st = run([n] * 4, [0, asked, 2 * asked, 3 * asked, 4 * asked + 1])
    assert st == CORRUPT and (out[:, 3 * asked:] == 3).all() and torch.equal(out[:, :3 * asked], good[:, :3 * asked])
    if asked > 1:
        out, _, st = run([n] * 4, [0, asked + 1, 2 * asked, 3 * asked, 4 * asked])
        assert st == CORRUPT and (out[:, :asked + 1] == 3).all()
        assert torch.equal(out[:, 2 * asked:], good[:, 2 * asked:])
    # decreasing, negative: an error and no more
    assert run([n] * 4, [0, 3 * asked, 2 * asked, 4 * asked, 4 * asked])[2] == CORRUPT
    assert run([n] * 4, [-5, asked, 2 * asked, 3 * asked, 4 * asked])[2] == CORRUPT
    assert run([n] * 4, [2 ** 31 - 1] * 5)[2] == CORRUPT
    assert run([n] * 4, starts.tolist())[2] == kvc.KVC_OK


@pytest.mark.parametrize("asked", [1, 2, 6, 40])
def test_attend_leaves_out_pages_outside_the_pool(asked):
    d, g, H, qpk, page, n = 128, 32, 1, 4, 32, 150
    c = make(d, g, 1, H, 6, page)
    k, v = rows(1, n, H, d)
    c.write(k, v, torch.arange(n, device="cuda"))
    q = torch.randn(1, asked, qpk, d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    for bad in (6, -1, 2 ** 31 - 1, -2 ** 31):
        out = c.attend(q.cuda(), dev([[0, bad, 2, 3, 4]]), dev([n]), q_starts=dev([0, asked]),
                       max_q=asked, causal=False)
        assert status_of(c) == CORRUPT
        slots = np.setdiff1d(np.arange(n), np.arange(page, 2 * page))
        close(c, slots, q, out, qpk, [(0, n - page)] * asked, d ** -0.5, torch.bfloat16)
    out = c.attend(q.cuda(), dev([[9] * 5]), dev([n]), q_starts=dev([0, asked]), max_q=asked)
    assert status_of(c) == CORRUPT and (out == 0).all()  # no page left
    # a bad page that no row sees is not looked at
    c.attend(q.cuda(), dev([[9, 1, 2, 3, 4]]), dev([n]), q_starts=dev([0, asked]), max_q=asked, window=20)
    assert status_of(c) == kvc.KVC_OK


@pytest.mark.parametrize("d,g", KINDS)
@pytest.mark.parametrize("asked", [1, 4, 12, 60])
@pytest.mark.parametrize("which", [0, 1])
def test_nan_rows_reach_the_queries_that_see_them(d, g, asked, which):
    H, qpk, n, at = 1, 4, 100, 90
    c = make(d, g, 1, H, 8, 16)
    kv = rows(1, n, H, d)
    c.write(*kv, torch.arange(n, device="cuda"))
    q = torch.randn(1, asked, qpk, d, device="cuda").to(torch.bfloat16)
    tab, st = dev([list(range(7))]), dev([0, asked])
    kv[which][0, at, 0, 5] = float("nan")
    c.write(*kv, torch.arange(n, device="cuda"))
    assert status_of(c) == NONFINITE
    lse = torch.empty(1, asked, qpk, device="cuda")
    out = c.attend(q, tab, dev([n]), q_starts=st, max_q=asked, lse=lse)
    c.check()
    see = [n - asked + i >= at for i in range(asked)]
    assert torch.isnan(out[0, see]).all()
    assert which == 1 or torch.isnan(lse[0, see]).all()  # (lse does not depend on values)
    blind = asked - sum(see)
    if blind:
        close(c, np.arange(n), q[:, :blind], out[:, :blind], qpk,
              [(0, n - asked + i + 1) for i in range(blind)], d ** -0.5, torch.bfloat16)


@pytest.mark.parametrize("asked", [1, 3, 8, 50])
def test_nonfinite_queries_stay_in_their_rows(asked):
    d, g, n = 128, 128, 80
    c = make(d, g, 1, 1, 6, 16)
    c.write(*rows(1, n, 1, d), torch.arange(n, device="cuda"))
    q = torch.randn(1, asked, 4, d, device="cuda").to(torch.bfloat16)
    tab, st = dev([list(range(5))]), dev([0, asked])
    fine = q.clone()
    q[0, 0, 1, 3] = float("nan")
    q[0, asked - 1, 2, 9] = float("inf")
    out = c.attend(q, tab, dev([n]), q_starts=st, max_q=asked)
    c.check()
    odd = [(0, 1), (asked - 1, 2)]
    assert all(torch.isnan(out[0, i, j]).all() for i, j in odd)
    out.nan_to_num_(0.0)
    close(c, np.arange(n), fine, out, 4, [(0, n - asked + i + 1) for i in range(asked)], d ** -0.5,
          torch.bfloat16, odd)
    assert (out != 0).sum() >= (asked * 4 - 2) * d * 0.9


@pytest.mark.parametrize("asked", [1, 5, 70])
def test_strided_queries_tables_and_outputs(asked):
    d, g, H, qpk, n, R = 64, 32, 2, 4, 90, 3
    c = make(d, g, 2, H, 20, 16)
    c.write(*rows(2, n, H, d), torch.arange(n, device="cuda"))
    tab = torch.arange(6, dtype=torch.int32, device="cuda").expand(R, 6)     # one table for all
    wide = torch.full((R, 9), 77, dtype=torch.int32, device="cuda")
    wide[:, 2:8] = tab
    q = torch.randn(2, R * asked, H * qpk, d, device="cuda").to(torch.bfloat16)
    lens, st = dev([n, n - 9, 1]), dev([0, asked, 2 * asked, 3 * asked])
    want = c.attend(q, tab.contiguous(), lens, q_starts=st, max_q=asked)
    qs = torch.randn(R * asked, 2, 3 * H * qpk, d, device="cuda").to(torch.bfloat16)
    qs[:, :, H * qpk:2 * H * qpk] = q.transpose(0, 1)
    out = torch.full_like(qs, 6.0)
    view = out.transpose(0, 1)[:, :, :H * qpk]
    for t in (tab, wide[:, 2:8]):
        view.fill_(6.0)
        c.attend(qs.transpose(0, 1)[:, :, H * qpk:2 * H * qpk], t, lens, q_starts=st, max_q=asked, out=view)
        c.check()
        assert torch.equal(view, want) and (out[:, :, H * qpk:] == 6).all()
    # a length past the slice's own columns is out of range, whatever its stride is
    c.attend(q, wide[:, 2:8], dev([97, n, n]), q_starts=st, max_q=asked)
    assert status_of(c) == CORRUPT


@pytest.mark.parametrize("asked", [1, 2, 9, 60])
def test_captured_calls_follow_their_lengths(asked):
    """write, attend and read in two graphs that are replayed in turn, beside eager calls."""
    d, g, H, qpk, page, R = 128, 64, 2, 4, 16, 2
    c, e = (make(d, g, 1, H, 2 * 40, page, fill=0) for _ in range(2))
    tab = torch.arange(2 * 40, dtype=torch.int32, device="cuda").view(R, 40)
    graphs = []
    for x in range(2):
        t = dict(k=torch.zeros(1, R * asked, H, d, dtype=torch.bfloat16, device="cuda"),
                 q=torch.zeros(1, R * asked, H * qpk, d, dtype=torch.bfloat16, device="cuda"),
                 slots=torch.zeros(R * asked, dtype=torch.int64, device="cuda"), lens=dev([0, 0]),
                 st=dev([0, asked, 2 * asked]), ko=torch.zeros(1, R * asked, H, d, dtype=torch.float16, device="cuda"))
        t["vo"] = torch.zeros_like(t["ko"])
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            c.write(t["k"], t["k"], t["slots"])
            t["out"] = c.attend(t["q"], tab, t["lens"], q_starts=t["st"], max_q=asked)
            c.read(t["slots"], t["ko"], t["vo"])
        graphs.append((gr, t))
    e.attend(t["q"], tab, dev([0, 0]), q_starts=t["st"], max_q=asked)
    at = [0, 200]
    for step in range(6):
        gr, t = graphs[step % 2]
        k = torch.randn(1, R * asked, H, d, device="cuda").to(torch.bfloat16)
        q = torch.randn(1, R * asked, H * qpk, d, device="cuda").to(torch.bfloat16)
        s = np.concatenate([r * 640 + at[r] + np.arange(asked) for r in range(R)])
        at = [x + asked for x in at]
        for name, x in (("k", k), ("q", q), ("slots", dev(s.tolist(), torch.int64)), ("lens", dev(at))):
            t[name].copy_(x)
        gr.replay()
        e.write(k, k, t["slots"])
        want = e.attend(q, tab, dev(at), q_starts=t["st"], max_q=asked)
        assert torch.equal(t["out"], want)
        assert torch.equal(t["ko"], e.read(t["slots"], dtype=torch.float16)[0]) and torch.equal(t["vo"], t["ko"])
    c.check()
    e.check()


def test_other_streams_threads_and_repeats():
    """The same calls on three streams at once and from two threads: each call's result is
    the same, bit for bit."""
    import threading
    d, g, H, qpk, n = 128, 128, 2, 4, 2000
    c = make(d, g, 1, H, 130, 16)
    c.write(*rows(1, n, H, d), torch.arange(n, device="cuda"))
    tab = torch.arange(125, dtype=torch.int32, device="cuda").view(1, -1)
    qs = [torch.randn(1, m, H * qpk, d, device="cuda").to(torch.bfloat16) for m in (1, 6, 100)]
    st = [dev([0, m]) for m in (1, 6, 100)]
    want = [c.attend(q, tab, dev([n]), q_starts=s, max_q=q.shape[1]) for q, s in zip(qs, st)]
    lens = dev([n])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for i in range(12):
        s = streams[i % 3]
        outs.append((i // 3 % 3, c.attend(qs[i // 3 % 3], tab, lens, q_starts=st[i // 3 % 3],
                                          max_q=qs[i // 3 % 3].shape[1], stream=s)))
    torch.cuda.synchronize()
    for i, o in outs:
        assert torch.equal(o, want[i])
    got = {}

    def work(i):
        got[i] = [c.attend(qs[x % 3], tab, lens, q_starts=st[x % 3], max_q=qs[x % 3].shape[1]) for x in range(30)]

    kv = torch.randn(1, 2, H, 16, d, device="cuda").to(torch.bfloat16)
    buf, nbytes, _ = stream_of(kv, g, 11, 0, 0, 0)
    free = torch.arange(128 * 16, 129 * 16, device="cuda")  # a page of no request

    def load():
        try:
            for _ in range(30):
                c.load(buf, nbytes, free, [16], check=True)
            got["load"] = True
        except kvc.KvcError as e:
            got["load"] = e

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)] + [threading.Thread(target=load)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[x % 3]) for x, o in enumerate(got[i]))
    assert got["load"] is True
    c.check()


def test_python_refusals():
    c = make(128, 64, 2, 2, 4, 16)
    k = torch.zeros(2, 3, 2, 128, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(2, 3, 8, 128, dtype=torch.bfloat16, device="cuda")
    s, tab, lens = dev([0, 1, 2], torch.int64), dev([[0], [1], [2]]), dev([1, 1, 1])
    for call in (lambda: c.write(k, k[:, :2], s), lambda: c.write(k, k.half(), s), lambda: c.write(k, k, s.int()),
                 lambda: c.write(k[:1], k[:1], s), lambda: c.write(k.transpose(2, 3), k, s),
                 lambda: c.read(s, k), lambda: c.write(k.cpu(), k, s), lambda: c[0:2:2],
                 lambda: c.attend(q[:1], tab, lens), lambda: c.attend(q[:, :, :7], tab, lens),
                 lambda: c.attend(q, tab.long(), lens), lambda: c.attend(q, tab[:2], lens),
                 lambda: c.attend(q, tab, lens, q_starts=lens), lambda: c.attend(q, tab, lens, out=q.half()),
                 lambda: c.attend(q, tab, lens, lse=torch.zeros(2, 3, 8, device="cuda", dtype=torch.bfloat16)),
                 lambda: c.load(torch.zeros(8, dtype=torch.uint8, device="cuda"), 64, s, [3]),
                 lambda: c.load(torch.zeros(64, dtype=torch.uint8, device="cuda"), 64, s, [4])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: c.write(k.float(), k.float(), s), lambda: c.attend(q.float(), tab, lens),
                 lambda: c.attend(q, tab, lens, max_q=0), lambda: c.attend(q, tab, lens, window=-1),
                 lambda: c.attend(q, tab, lens, window=5, causal=False),
                 lambda: c.attend(q[:, :2], tab, lens)):
        with pytest.raises(kvc.KvcError):
            call()
    for i in (2, -3):
        with pytest.raises(IndexError):
            c[i]
    assert c[-1].desc.first_layer == 1 and c[0:0].desc.layers == 0
    assert status_of(c) == kvc.KVC_OK


@pytest.mark.parametrize("d,g", [(128, 64), (64, 32)])
def test_the_calls_together(d, g):
    """A prompt's cache arrives as a stream, goes into pages, a piece of prompt and then
    single tokens follow; each step's attention against 64 bits."""
    L, H, qpk, page, seed, T = 2, 2, 4, 16, 21, 75
    c = make(d, g, L, H, 14, page, signs=1, seed=seed)
    kv = torch.randn(L, 2, H, T, d, device="cuda").to(torch.bfloat16)
    buf, n, back = stream_of(kv, g, seed, 1, 0, 1)
    order = np.random.default_rng(1).permutation(14)
    tab = dev([order.tolist()])
    where = lambda a, b: order[np.arange(a, b) // page] * page + np.arange(a, b) % page
    c.load(buf, n, torch.from_numpy(where(0, T)).cuda(), [T], check=True)
    at = T
    for m in (40, 1, 5, 1):
        k = torch.randn(L, m, H, d, device="cuda").to(torch.bfloat16)
        v = torch.randn(L, m, H, d, device="cuda").to(torch.bfloat16)
        q = torch.randn(L, m, H * qpk, d, device="cuda").to(torch.bfloat16)
        out = torch.empty_like(q)
        for l in range(L):  # a layer at a time, as a model goes
            view = c[l]
            view.write(k[l:l + 1], v[l:l + 1], torch.from_numpy(where(at, at + m)).cuda())
            view.attend(q[l:l + 1], tab, dev([at + m]), q_starts=dev([0, m]), max_q=m, out=out[l:l + 1])
        at += m
        close(c, where(0, at), q, out, qpk, [(0, at - m + i + 1) for i in range(m)], d ** -0.5, torch.bfloat16)
    rk, rv = c.read(torch.from_numpy(where(0, at)).cuda())
    c.check()
    assert torch.equal(rk[:, :T].transpose(1, 2), back[:, 0]) and torch.equal(rv[:, :T].transpose(1, 2), back[:, 1])
