"""The paged 4-bit cache on the GPU: written codes and meta bit for bit against
the codec's oracle, reads against the oracle's decoder, loads against the
stream's codes, attention against 64-bit arithmetic on the stored values."""
import numpy as np
import pytest
import torch

import cache_ref as ref
import kv_cache_compression_04_b200 as kvc
import oracle

pytestmark = pytest.mark.gpu

KINDS = [(128, 128), (128, 64), (128, 32), (64, 64), (64, 32)]
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def make(d=128, g=128, layers=1, heads=2, pages=12, page=16, quant=0, signs=0, seed=11, fill=None):
    pool = torch.randint(0, 256, (layers, pages, 2, heads, ref.block_bytes(d, g, page)),
                         dtype=torch.uint8, generator=torch.Generator().manual_seed(5))
    if fill is not None:
        pool.fill_(fill)
    return kvc.PagedCache(layers, heads, d, pages, page_tokens=page, group=g, sign_seed=seed,
                          quant=quant, signs=signs, pool=pool.cuda())


def rows(layers, n, heads, d, dtype=torch.bfloat16, seed=0):
    """bf16 values (fp16 holds them too) with uneven channel scales."""
    rng = np.random.default_rng(seed)
    scale = np.exp(rng.standard_normal((layers, 1, heads, d)) * 0.7)
    x = [ref.bf16(np.clip(rng.standard_normal((layers, n, heads, d)) * s, -60, 60))
         for s in (scale, 1.0)]
    return [t.to(dtype).cuda() for t in x]


def slots_for(n, pages, page, seed=0):
    order = np.random.default_rng(seed).permutation(pages)
    t = np.arange(n)
    return order[t // page] * page + t % page


def expected_rows(k, v, g, quant, seed, per_vector, first_layer=0):
    """The oracle's codes [L, 2, H, N, d/2] and meta bytes for rows [L, N, H, d]."""
    L, n, H, d = k.shape
    codes = np.empty((L, 2, H, n, d // 2), np.uint8)
    meta = np.empty((L, 2, H, n, d // g * 4), np.uint8)
    for l in range(L):
        for kv, t in enumerate((k, v)):
            for h in range(H):
                x = t[l, :, h].float().cpu().to(torch.bfloat16).view(torch.uint16).numpy()
                i = ((first_layer + l) * 2 + kv) * H + h
                st, c, m = oracle.quantize_vectors(np.ascontiguousarray(x), 4, g,
                                                   ref.diagonal_seed(seed, per_vector, i, d), quant)
                assert st == oracle.OK
                codes[l, kv, h], meta[l, kv, h] = c, m
    return codes, meta


@pytest.mark.parametrize("d,g", KINDS)
@pytest.mark.parametrize("quant,signs,dtype,n,page,layers,heads", [
    (0, 0, torch.bfloat16, 1, 16, 1, 1), (1, 1, torch.float16, 37, 32, 2, 3),
    (0, 1, torch.bfloat16, 65, 48, 1, 2), (1, 0, torch.bfloat16, 16, 16, 3, 1)])
def test_write_is_the_codec(d, g, quant, signs, dtype, n, page, layers, heads):
    pages = (n + page - 1) // page + 3
    c = make(d, g, layers, heads, pages, page, quant, signs, seed=2 ** 63 + 9)
    before = c.pool.cpu().numpy().copy()
    k, v = rows(layers, n, heads, d, dtype)
    s = slots_for(n, pages, page)
    c.write(k, v, torch.from_numpy(s).cuda())
    c.check()
    after = c.pool.cpu().numpy()
    codes, meta = ref.rows_of(after, s, d, g, page)
    want_c, want_m = expected_rows(k, v, g, quant, 2 ** 63 + 9, signs)
    assert np.array_equal(codes, want_c)
    assert np.array_equal(meta, want_m)
    # every other slot as it was
    other = np.setdiff1d(np.arange(pages * page), s)
    for a, b in zip(ref.rows_of(after, other, d, g, page), ref.rows_of(before, other, d, g, page)):
        assert np.array_equal(a, b)


@pytest.mark.parametrize("d,g", KINDS)
@pytest.mark.parametrize("quant,signs", [(0, 0), (1, 1)])
def test_read_is_the_decoder(d, g, quant, signs):
    layers, heads, n, page, pages = 2, 3, 45, 32, 4
    c = make(d, g, layers, heads, pages, page, quant, signs)
    k, v = rows(layers, n, heads, d)
    s = slots_for(n, pages, page)
    at = torch.from_numpy(s).cuda()
    c.write(k, v, at)
    got = c.read(at)
    half = c.read(at, dtype=torch.float16)
    c.check()
    pool = c.pool.cpu().numpy()
    codes, meta = ref.rows_of(pool, s, d, g, page)
    x = ref.values(pool, s, ref.signs(11, signs, layers, heads, d), d, g, page)
    y = np.abs(ref.grid_values(codes, meta, g)).sum(-1)[..., None] / d
    for kv in range(2):
        for l in range(layers):
            for h in range(heads):
                i = (l * 2 + kv) * heads + h
                want = oracle.dequantize_vectors(codes[l, kv, h], meta[l, kv, h], d, 4, g,
                                                 ref.diagonal_seed(11, signs, i, d), quant)
                assert np.array_equal(got[kv][l, :, h].cpu().view(torch.uint16).numpy(), want)
        # fp16: half a step, and log2(d) + 1 fp32 roundings of sums of at most sum |y| / d
        w = np.moveaxis(x[:, kv], 1, 2)
        tol = 2.0 ** -11 * np.abs(w) + 2.0 ** -25 + 8 * 2.0 ** -24 * np.moveaxis(y[:, kv], 1, 2)
        assert (np.abs(half[kv].double().cpu().numpy() - w) <= tol).all()


def test_strides_padding_and_views():
    """Slices of a fused projection, skipped tokens, one layer of several, rows left alone."""
    d, g, heads, n, pages = 128, 64, 2, 33, 4
    c = make(d, g, 3, heads, pages, 16, signs=1, seed=77)
    before = c.pool.cpu().numpy().copy()
    qkv = torch.randn(1, n, 5 * heads, d, device="cuda").to(torch.bfloat16)
    k, v = qkv[:, :, 2 * heads:3 * heads], qkv[:, :, 4 * heads:]
    s = slots_for(n, pages, 16)
    s[::4] = -1
    at = torch.from_numpy(s).cuda()
    c[1].write(k, v, at)
    out = torch.full((1, n, 3 * heads, d), 7.0, dtype=torch.bfloat16, device="cuda")
    c[1:2].read(at, out[:, :, :heads], out[:, :, heads:2 * heads])
    c.check()
    after = c.pool.cpu().numpy()
    assert np.array_equal(after[[0, 2]], before[[0, 2]])
    keep = s >= 0
    want = expected_rows(k[:, keep], v[:, keep], g, 0, 77, True, first_layer=1)
    got = ref.rows_of(after[1:2], s[keep], d, g, 16)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    out = out.float().cpu().numpy()
    assert (out[:, ~keep] == 7).all() and (out[:, :, 2 * heads:] == 7).all()
    x = ref.values(after[1:2], s[keep], ref.signs(77, True, 1, heads, d, 1), d, g, 16)
    assert np.abs(out[:, keep][:, :, :heads] - np.moveaxis(x[:, 0], 1, 2)).max() < 0.05


def run_attend(c, lens, asked, qpk, dtype, window=0, causal=True, pad=0, lse=True, seed=3,
               scale=None, max_q=None, table=None, k_scale=1.0):
    """Fills the cache's requests with written rows and compares attention with 64 bits."""
    d, g, H, L, page = (c.desc.head_dim, c.desc.group_size, c.desc.kv_heads, c.desc.layers,
                        c.desc.page_tokens)
    per = [-(-n // page) for n in lens]
    order = np.random.default_rng(seed).permutation(c.desc.num_pages)
    tab = np.full((len(lens), max(per + [1])), -1, np.int32)
    at, slots = 0, []
    for r, n in enumerate(per):
        tab[r, :n] = order[at:at + n]
        t = np.arange(lens[r])
        slots.append(tab[r, t // page].astype(np.int64) * page + t % page)
        at += n
    every = np.concatenate(slots)
    if every.size:
        k, v = rows(L, every.size, H, d, seed=seed)
        c.write(k * k_scale, v, torch.from_numpy(every).cuda())
    starts = np.concatenate(([0], np.cumsum(asked))).astype(np.int32)
    total = int(starts[-1]) + pad
    q = torch.randn(L, total, H * qpk, d, generator=torch.Generator().manual_seed(seed))
    q = q.to(dtype)
    out = torch.full(q.shape, 9.0, dtype=dtype, device="cuda")
    ls = torch.full(q.shape[:3], 9.0, device="cuda") if lse else None
    scale = d ** -0.5 if scale is None else scale
    one = all(m == 1 for m in asked) and pad == 0
    c.attend(q.cuda(), torch.from_numpy(tab if table is None else table).cuda(),
             torch.tensor(lens, dtype=torch.int32).cuda(),
             q_starts=None if one else torch.from_numpy(starts).cuda(),
             max_q=max_q or max(list(asked) + [1]), out=out, lse=ls, scale=scale, causal=causal,
             window=window)
    c.check()
    pool, sg = c.pool.cpu().numpy(), None
    sg = ref.signs(c.desc.sign_seed, c.desc.signs, L, H, d, c.desc.first_layer)
    got, got_l = out.double().cpu().numpy(), ls.double().cpu().numpy() if lse else None
    for r, n in enumerate(lens):
        m = asked[r]
        x = ref.values(pool, slots[r], sg, d, g, page)
        hi = [max(0, n - m + i + 1) if causal else n for i in range(m)]
        limits = [(max(0, h - window) if window else 0, h) for h in hi]
        rowsl = slice(starts[r], starts[r + 1])
        spread = ref.spreads(*ref.rows_of(pool, slots[r], d, g, page), g)
        o, l, mag, size = ref.attend(x, q[:, rowsl].double().numpy(), qpk, scale, limits, spread)
        # Scores: the fp16 parts of the transformed query leave 2^-22 of its largest
        # channel, sums of up to 8 terms per group and the products' sums in fp32
        # a few 2^-24 more: 2^-18 of sum |q||y| covers them. Weights are then off by that
        # and by exp2's 2^-22, and rounded to fp16 once; the rounded weight multiplies the
        # centred codes, so a relative e of it moves a channel by up to e * spread, the rest
        # by e |v|. out is off by half a step of its type more.
        ds = 2.0 ** -18 * size + 2.0 ** -20
        tol = HALF[dtype] * np.abs(o) + (2 * ds + 2.0 ** -11)[..., None] * mag * 1.01 + 1e-7
        assert np.isfinite(got[:, rowsl]).all()
        bad = np.abs(got[:, rowsl] - o) - tol
        assert (bad <= 0).all(), (r, n, m, bad.max(), np.unravel_index(bad.argmax(), bad.shape))
        if lse:
            empty = np.isneginf(l)
            assert np.array_equal(empty, np.isneginf(got_l[:, rowsl]))
            diff = np.abs(np.where(empty, 0, got_l[:, rowsl]) - np.where(empty, 0, l))
            assert (diff <= ds + 2.0 ** -21 * np.abs(np.where(empty, 0, l))).all(), diff.max()
    if pad:
        assert (got[:, -pad:] == 9).all() and (not lse or (got_l[:, -pad:] == 9).all())
    return got


@pytest.mark.parametrize("d,g", KINDS)
@pytest.mark.parametrize("qpk,asked", [(1, 1), (3, 1), (4, 1), (8, 1), (7, 2), (16, 1), (5, 9)])
def test_attend_kinds(d, g, qpk, asked):
    lens = [70, 1, 16, 17, 300]
    c = make(d, g, 1, 2, 64, 16, quant=qpk % 2, signs=asked % 2)
    run_attend(c, lens, [min(asked, n) for n in lens], qpk, torch.bfloat16)


@pytest.mark.parametrize("lens,asked,qpk,page,window,causal", [
    ([0], [1], 4, 16, 0, True),                       # nothing cached
    ([5, 0, 33], [1, 1, 1], 2, 16, 0, True),          # an empty request among others
    ([1], [1], 1, 32, 0, True),
    ([3, 40], [5, 0], 4, 16, 0, True),                # more queries than keys; a request without any
    ([100, 64, 63], [3, 3, 3], 4, 48, 20, True),      # window inside, at and over tile ends
    ([100, 64], [7, 7], 8, 16, 1, True),              # a window of the own key alone
    ([100, 31], [6, 2], 4, 16, 0, False),
    ([2000], [1], 6, 256, 0, True),
    ([2000, 1999], [1, 1], 8, 64, 500, True),
    ([130], [130], 2, 16, 0, True),                   # a whole prompt
    ([700, 90, 5], [300, 90, 1], 4, 16, 0, True),
    ([400], [200], 3, 32, 77, True)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_attend_lengths(lens, asked, qpk, page, window, causal, dtype):
    pages = sum(-(-n // page) for n in lens) + 2
    c = make(128, 64, 1, 2, pages, page)
    run_attend(c, lens, asked, qpk, dtype, window, causal)


def test_attend_layers_padding_many_requests():
    rng = np.random.default_rng(8)
    lens = [int(x) for x in rng.integers(0, 90, 150)]
    c = make(64, 32, 2, 3, sum(-(-n // 16) for n in lens) + 5, 16, signs=1)
    run_attend(c, lens, [1] * 150, 4, torch.bfloat16, pad=3)
    run_attend(c, lens, [min(n, 2) for n in lens], 2, torch.float16, pad=1, lse=False)


def test_attend_sharp_and_flat_scores():
    """Running maxima that rise late and by much; all scores alike."""
    c = make(128, 128, 1, 2, 80, 16)
    run_attend(c, [1200], [1], 4, torch.float16, scale=3.0)
    run_attend(c, [1200], [1], 8, torch.float16, scale=3.0)
    run_attend(c, [1200], [2], 8, torch.float16, scale=0.0)


def test_hidden_slots_may_hold_anything():
    """NaN scales past a request's end and before its window change nothing."""
    c = make(128, 128, 1, 1, 6, 16, fill=0xFF)  # every meta word a NaN
    run_attend(c, [37], [1], 4, torch.bfloat16)
    c = make(128, 32, 1, 1, 6, 16, fill=0xFF)
    run_attend(c, [37], [3], 8, torch.bfloat16, window=9)
