"""The paged 4-bit cache on the GPU where its calls could go wrong unseen: streams whose
requests are cut elsewhere, errors of a load that nobody waits for, values that no query
should see by their size, and the largest lengths."""
import numpy as np
import pytest
import torch

import cache_ref as ref
import kv_cache_compression_04_b200 as kvc
from test_gpu_cache import KINDS, make, rows, slots_for
from test_gpu_cache_use import CORRUPT, cache_values, close, dev, narrow_meta, status_of, stream_of

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- load --
def paged_stream(lens, L, H, d, g, seed):
    """A stream of several requests, and what it decodes to: rows [L, 2, H, tokens, d]."""
    page, T = 16, sum(lens)
    per = [-(-n // page) for n in lens]
    pool = torch.randn(L, sum(per) + 1, 2, H, page, d, device="cuda").to(torch.bfloat16)
    table = torch.zeros(len(lens), max(per + [1]), dtype=torch.int32)
    at, rows = 0, []
    for r, n in enumerate(per):
        table[r, :n] = torch.arange(at, at + n)
        t = torch.arange(lens[r])
        rows.append((at + t // page) * page + t % page)
        at += n
    table = table.cuda()
    codec = kvc.Codec(4, g, seed)
    out, ws, n = codec.compress(kvc.paged_desc(pool, table, lens))
    back = torch.zeros_like(pool)
    codec.decompress(out, int(n.item()), kvc.paged_desc(back, table, lens), ws)
    rows = torch.cat(rows).cuda()
    x = back.permute(0, 2, 3, 1, 4, 5).reshape(L, 2, H, -1, d)[:, :, :, rows]
    return out, int(n.item()), x


@pytest.mark.parametrize("lens,other", [
    ([10, 30], [30, 10]), ([10, 0, 30], [10, 30, 0]), ([5, 5, 5], [5, 4, 6]),
    ([3] * 400 + [7] * 624, [3] * 399 + [7, 3] + [7] * 623), ([40], None), ([0, 17], None)])
def test_load_compares_the_length_of_every_request(lens, other):
    """Requests of the stream cut elsewhere than the caller's: refused, nothing is stored."""
    L, H, d, g = 1, 2, 128, 64
    buf, n, x = paged_stream(lens, L, H, d, g, 11)
    T = sum(lens)
    pages = -(-T // 16) + 1
    c = make(d, g, L, H, pages, 16)
    at = torch.from_numpy(slots_for(T, pages, 16)).cuda()
    if other is not None:
        before = c.pool.clone()
        with pytest.raises(kvc.KvcError) as e:
            c.load(buf, n, at, other, check=True)
        assert e.value.status == CORRUPT and torch.equal(c.pool, before)
    c.load(buf, n, at, lens, check=True)
    for i, y in enumerate(c.read(at)):
        assert torch.equal(y.transpose(1, 2).view(torch.int16), x[:, i].view(torch.int16))


def test_a_load_that_nobody_waits_for_leaves_its_error():
    """Of the header, of a slot, of an eliminated meta chunk: in the cache's status word;
    with check=True in the exception alone."""
    d, g, L, H, T, seed = 128, 32, 1, 2, 3000, 5
    kv = narrow_meta(L, H, T, d, g, seed, 1)
    buf, n, _ = stream_of(kv, g, seed, 0, 0, 1)
    pages = T // 16 + 2
    c = make(d, g, L, H, pages, 16, 0, 1, seed)
    at = torch.from_numpy(slots_for(T, pages, 16)).cuda()
    c.load(buf, n, at, [T])
    assert status_of(c) == kvc.KVC_OK
    c.load(buf, n - 1, at, [T])  # cut short
    assert status_of(c) == CORRUPT and status_of(c) == kvc.KVC_OK
    far = at.clone()
    far[77] = pages * 16
    c.load(buf, n, far, [T])
    assert status_of(c) == CORRUPT
    n_code = -(-L * 2 * H * T * d // 2 // 16384)
    odd = buf.clone()
    entry = odd[64 + 8 * n_code: 72 + 8 * n_code]
    assert int(entry[0]) + 256 * int(entry[1]) < 16384  # the first meta chunk is eliminated
    entry[0], entry[1] = 8, 0                           # shorter than its bitmap
    c.load(odd, n, at, [T])
    assert status_of(c) == CORRUPT
    for bad, slots in ((odd, at), (buf, far)):
        with pytest.raises(kvc.KvcError):
            c.load(bad, n, slots, [T], check=True)
        assert status_of(c) == kvc.KVC_OK


def test_a_captured_load_leaves_its_error():
    d, g, L, H, T = 64, 64, 2, 2, 50
    kv = torch.randn(L, 2, H, T, d, device="cuda").to(torch.bfloat16)
    buf, n, back = stream_of(kv, g, 11, 0, 0, 0)
    c = make(d, g, L, H, 6, 16)
    at = torch.from_numpy(slots_for(T, 6, 16)).cuda()
    c.load(buf, n, at, [T])  # (its kernels are known to the device)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.load(buf, n, at, [T])
    c.pool.zero_()
    graph.replay()
    c.check()
    k, v = c.read(at)
    assert torch.equal(k.transpose(1, 2), back[:, 0]) and torch.equal(v.transpose(1, 2), back[:, 1])
    buf[40] ^= 1  # another sign seed
    graph.replay()
    assert status_of(c) == CORRUPT
    buf[40] ^= 1
    graph.replay()
    assert status_of(c) == kvc.KVC_OK


# ----------------------------------------------------------- attention --
@pytest.mark.parametrize("d,g", KINDS)
@pytest.mark.parametrize("asked", [1, 2, 9, 60])
@pytest.mark.parametrize("size", [2.0 ** -12, 2.0 ** -17])
def test_zero_values_among_small_ones(d, g, asked, size):
    """Rows of zeros (padding that a model left in) beside values of 1e-4 and less."""
    n, qpk = 200, 4
    c = make(d, g, 1, 1, 14, 16)
    k, v = rows(1, n, 1, d)
    v = v * size
    v[:, ::3] = 0
    c.write(k, v, torch.arange(n, device="cuda"))
    q = torch.randn(1, asked, qpk, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    out = c.attend(q.cuda(), torch.arange(13, dtype=torch.int32, device="cuda")[None], dev([n]),
                   q_starts=dev([0, asked]), max_q=asked) / size
    c.check()
    x, spread = cache_values(c, np.arange(n))
    o, _, mag, s = ref.attend(x, q.double().numpy(), qpk, d ** -0.5,
                              [(0, n - asked + i + 1) for i in range(asked)], spread)
    tol = 2.0 ** -8 * np.abs(o) + (2 * (2.0 ** -18 * s + 2.0 ** -20) + 2.0 ** -11)[..., None] * mag * 1.01
    bad = np.abs(out.double().cpu().numpy() - o / size) - tol / size
    assert (bad <= 1e-7).all(), bad.max()


@pytest.mark.parametrize("d,g", KINDS)
def test_values_of_blocks_of_128_are_rounded_once(d, g):
    """One key per request, seen by 80 rows: out is that value, its transformed channels
    rounded to fp16 once (times a power of two), the inverse transform in fp32 and one more
    rounding. Channels far from zero whose steps are fractions of an fp16 step show a rounding
    of z + 8 s of its own."""
    R, asked, qpk, page = 24, 20, 4, 16
    c = make(d, g, 1, 1, R, page, signs=1, fill=0)
    rng = np.random.default_rng(d + g)
    at = np.arange(R) * page
    # codes at random; zeros of 1 .. 2 and scales of odd multiples of 2^-14: z + 8 s lies
    # halfway between fp16 values
    host = c.pool.cpu().numpy()
    cb, mb = d // 2, d // g * 4
    t = host.reshape(R, 2, 16 * (cb + mb))
    t[:, :, :cb] = rng.integers(0, 256, (R, 2, cb))
    meta = np.zeros((R, 2, d // g, 2), np.float16)
    meta[..., 0] = (2 * rng.integers(0, 8, meta.shape[:-1]) + 1) * 2.0 ** -14
    meta[..., 1] = 1 + rng.integers(0, 500, meta.shape[:-1]) * 2.0 ** -10
    t[:, :, 16 * cb:16 * cb + mb] = meta.view(np.uint8).reshape(R, 2, mb)
    c.pool.copy_(torch.from_numpy(host))
    q = torch.randn(1, R * asked, qpk, d, device="cuda").half()
    out = c.attend(q, torch.arange(R, dtype=torch.int32, device="cuda")[:, None], dev([1] * R),
                   q_starts=dev([asked * i for i in range(R + 1)]), max_q=asked, causal=False)
    c.check()
    codes, m = ref.rows_of(c.pool.cpu().numpy(), at, d, g, page)
    y = ref.grid_values(codes, m, g)[0, 1, 0]  # [R, d]; its fp16 grid: 2^-10 of the power of two below 8 z
    y16 = (y / 8).astype(np.float16).astype(np.float64) * 8
    assert np.abs(y16 - y).max() > 2.0 ** -9
    sg = ref.signs(11, 1, 1, 1, d)[0, 1, 0]
    want = (y16 @ ref.hadamard(d) / d * sg).repeat(asked * qpk, 0).reshape(R * asked, qpk, d)
    # half a step of the output; the weight's exponent (2^-21 of it); fp32: the merge's weights,
    # 1 / (L d) and seven sums, of sum |y| / d
    tol = (2.0 ** -11 + 2.0 ** -21) * np.abs(want) + 2.0 ** -25 + 10 * 2.0 ** -24 * np.abs(y).mean(-1).max()
    bad = np.abs(out[0].double().cpu().numpy() - want) - tol
    assert (bad <= 0).all(), bad.max()


@pytest.mark.parametrize("qpk,asked", [(4, 1), (8, 1), (8, 3), (16, 3), (4, 30)])
@pytest.mark.parametrize("n", [2 ** 31 - 1, 2 ** 31 - 14, 2 ** 31 - 16, 2 ** 31 - 40])
def test_the_longest_requests(qpk, asked, n):
    """Lengths up to 2^31 - 1, of which a window shows the last tokens: a page that stands in
    every entry of the table."""
    d, g, page, window = 64, 64, 65536, 45
    c = make(d, g, 1, 1, 1, page, fill=0)
    m = 300  # the page's last slots
    at = torch.arange(page - m, page, device="cuda")
    c.write(*rows(1, m, 1, d), at)
    q = torch.randn(1, asked, qpk, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    tab = torch.zeros(1, 2 ** 31 // page, dtype=torch.int32, device="cuda")
    out = c.attend(q.cuda(), tab, dev([n]), q_starts=dev([0, asked]), max_q=asked, window=window)
    c.check()
    end = m - (2 ** 31 - n)  # the length, counted from the first of those slots
    lim = [(end - asked + i + 1 - window, end - asked + i + 1) for i in range(asked)]
    close(c, at.cpu().numpy(), q, out, qpk, lim, d ** -0.5, torch.bfloat16)


@pytest.mark.parametrize("d,g", [(128, 128), (128, 32), (64, 64)])
@pytest.mark.parametrize("asked", [1, 2, 6, 12, 60])     # 4 .. 240 rows: every form
@pytest.mark.parametrize("at", [3, 90, 95])  # in tiles that all queries see in full, and in the last one
def test_lse_does_not_depend_on_values(d, g, asked, at):
    """A value stored as NaN makes out NaN for the queries that see it and changes no lse."""
    H, qpk, n = 1, 4, 97
    c = make(d, g, 1, H, 8, 16)
    kv = rows(1, n, H, d)
    c.write(*kv, torch.arange(n, device="cuda"))
    q = torch.randn(1, asked, qpk, d, device="cuda").to(torch.bfloat16)
    tab, st = dev([list(range(7))]), dev([0, asked])
    lse, want = (torch.empty(1, asked, qpk, device="cuda") for _ in range(2))
    fine = c.attend(q, tab, dev([n]), q_starts=st, max_q=asked, lse=want)
    c.check()
    kv[1][0, at, 0, 5] = float("nan")
    c.write(*kv, torch.arange(n, device="cuda"))
    assert status_of(c) == kvc.KVC_ERR_NONFINITE
    out = c.attend(q, tab, dev([n]), q_starts=st, max_q=asked, lse=lse)
    c.check()
    see = torch.tensor([n - asked + i >= at for i in range(asked)])
    assert torch.isnan(out[0, see]).all()
    # (the weights' common power of two may differ: one rounding of a sum of a few units, and exp2's)
    assert (lse - want).abs().max() <= 2.0 ** -18
    assert torch.isfinite(out[0, ~see]).all() and torch.isfinite(fine).all()


def ranged(kind, n, d, rng):
    """Keys along one direction u, whose scores against u-like queries are `score` (times
    the softmax's scale), and values of very different sizes."""
    u = rng.standard_normal(d)
    score, size = rng.uniform(-2, 2, n), np.full(n, 2.0 ** -13)
    if kind == "first" or kind == "last":  # a huge value of no weight, before or after the others
        i = 1 if kind == "first" else n - 2
        score[i], size[i] = -60, 2.0 ** 12
    elif kind == "slight":                 # whose weight makes it count as much as another
        score[n // 2], size[n // 2] = -16, 2.0 ** 12
    elif kind == "rising":                 # scores rise by 2^90 while sizes fall
        score, size = np.linspace(-32, 32, n), 2.0 ** np.linspace(12, -13, n)
    elif kind == "falling":
        score, size = np.linspace(32, -32, n), 2.0 ** np.linspace(-13, 12, n)
    elif kind == "mixed":
        score, size = rng.uniform(-40, 8, n), 2.0 ** rng.uniform(-13, 12, n)
    k = score[:, None] * u / (u @ u) * d ** 0.5
    return u, k, size[:, None] * rng.standard_normal((n, d))


@pytest.mark.parametrize("kind", ["first", "last", "slight", "rising", "falling", "mixed"])
@pytest.mark.parametrize("d,g,qpk,asked,window", [
    (128, 128, 4, 1, 0), (128, 32, 8, 1, 0), (64, 32, 7, 1, 0), (128, 64, 4, 4, 70), (64, 64, 8, 2, 0),
    (128, 128, 4, 30, 0), (128, 64, 8, 20, 0), (128, 32, 4, 40, 90), (64, 64, 4, 40, 0), (64, 32, 64, 1, 0)])
@pytest.mark.parametrize("n", [130, 700])
def test_values_of_very_different_sizes(kind, d, g, qpk, asked, window, n):
    """Scales of visible values up to 2^25 apart, with any weights, cost no precision: the
    same bound as everywhere."""
    rng = np.random.default_rng(n)
    c = make(d, g, 1, 1, n // 16 + 2, 16)
    u, k, v = ranged(kind, n, d, rng)
    c.write(ref.bf16(k)[None, :, None].cuda(), ref.bf16(v)[None, :, None].cuda(), torch.arange(n, device="cuda"))
    q = torch.from_numpy(u + 0.02 * rng.standard_normal((1, asked, qpk, d))).to(torch.bfloat16).cuda()
    out = torch.empty_like(q)
    c.attend(q, torch.arange(n // 16 + 1, dtype=torch.int32, device="cuda")[None], dev([n]), out=out,
             q_starts=dev([0, asked]), max_q=asked, window=window)
    c.check()
    lim = [(max(0, n - asked + i + 1 - window) if window else 0, n - asked + i + 1) for i in range(asked)]
    close(c, np.arange(n), q, out, qpk, lim, d ** -0.5, torch.bfloat16)


@pytest.mark.parametrize("d,g", [(128, 128), (128, 32), (64, 64)])
@pytest.mark.parametrize("asked", [2, 6, 50])
def test_zero_values_beside_one_that_is_not_finite(d, g, asked):
    """The last tiles hold zeros and, in the last token, a value stored as NaN: the queries
    before it get what the other values weigh."""
    n, qpk = 164, 4
    c = make(d, g, 1, 1, 12, 16)
    k, v = rows(1, n, 1, d)
    v[:, 100:] = 0
    v[0, n - 1, 0, 3] = float("nan")
    c.write(k, v, torch.arange(n, device="cuda"))
    assert status_of(c) == kvc.KVC_ERR_NONFINITE
    q = torch.randn(1, asked, qpk, d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    out = c.attend(q.cuda(), torch.arange(11, dtype=torch.int32, device="cuda")[None], dev([n]),
                   q_starts=dev([0, asked]), max_q=asked)
    c.check()
    assert torch.isnan(out[0, -1]).all()
    close(c, np.arange(n), q[:, :-1], out[:, :-1], qpk, [(0, n - asked + i + 1) for i in range(asked - 1)],
          d ** -0.5, torch.bfloat16)


@pytest.mark.parametrize("kind", ["first", "last", "slight", "rising", "falling", "mixed"])
@pytest.mark.parametrize("d,g,qpk,asked", [(128, 128, 4, 1), (128, 32, 8, 1), (64, 64, 7, 2), (128, 64, 4, 20),
                                           (64, 32, 4, 30)])
def test_values_of_very_different_sizes_in_long_segments(kind, d, g, qpk, asked):
    """The same where a warp (or block) goes through all of a request's keys itself: many
    requests and heads that share them."""
    n, L, H, R = 700, 2, 16, 24
    rng = np.random.default_rng(n + d + g)
    c = make(d, g, L, H, n // 16 + 2, 16)
    u, k, v = ranged(kind, n, d, rng)
    c.write(*(ref.bf16(x)[None, :, None].expand(L, n, H, d).contiguous().cuda() for x in (k, v)),
            torch.arange(n, device="cuda"))
    one = torch.from_numpy(u + 0.02 * rng.standard_normal((1, asked, qpk, d))).to(torch.bfloat16)
    q = one.repeat(L, R, H, 1).cuda()
    tab = torch.arange(n // 16 + 1, dtype=torch.int32, device="cuda").expand(R, -1)
    out = c.attend(q, tab, dev([n] * R), q_starts=dev([asked * i for i in range(R + 1)]), max_q=asked)
    c.check()
    x, spread = (t[:1, :, :1] for t in cache_values(c, np.arange(n)))
    o, _, mag, size = ref.attend(x, one.double().numpy(), qpk, d ** -0.5,
                                 [(0, n - asked + i + 1) for i in range(asked)], spread)
    ds = 2.0 ** -18 * size + 2.0 ** -20
    tol = 2.0 ** -8 * np.abs(o) + (2 * ds + 2.0 ** -11)[..., None] * mag * 1.01 + 1e-7
    got = out.double().cpu().numpy().reshape(L, R, asked, H, qpk, d)
    bad = np.abs(got - o[0][None, None, :, None]) - tol[0][None, None, :, None]
    assert (bad <= 0).all(), bad.max()


@pytest.mark.parametrize("d,g", [(128, 128), (128, 32), (64, 64)])
@pytest.mark.parametrize("asked", [1, 2, 9, 60])
@pytest.mark.parametrize("n,at", [(192, 70), (192, 0), (190, 185)])
def test_a_zero_value_with_nearly_all_the_weight(d, g, asked, n, at):
    """One key's score is 17 above the others', its value zeros: what is left keeps its
    precision, though the values beside it are all alike."""
    qpk, rng = 4, np.random.default_rng(d + at)
    c = make(d, g, 1, 1, 13, 16)
    u = rng.standard_normal(d)
    score = rng.uniform(-0.5, 0.5, n)
    score[at] = 17
    k, v = score[:, None] * u / (u @ u) * d ** 0.5, rng.standard_normal((n, d)) * 2.0 ** 6
    v[at] = 0
    c.write(ref.bf16(k)[None, :, None].cuda(), ref.bf16(v)[None, :, None].cuda(), torch.arange(n, device="cuda"))
    q = torch.from_numpy(u + 0.02 * rng.standard_normal((1, asked, qpk, d))).to(torch.bfloat16).cuda()
    out = c.attend(q, torch.arange(12, dtype=torch.int32, device="cuda")[None], dev([n]),
                   q_starts=dev([0, asked]), max_q=asked) * 2.0 ** 12
    c.check()
    x, spread = cache_values(c, np.arange(n))
    x[:, 1] *= 2.0 ** 12
    spread[:, 1] *= 2.0 ** 12
    o, _, mag, size = ref.attend(x, q.double().cpu().numpy(), qpk, d ** -0.5,
                                 [(0, n - asked + i + 1) for i in range(asked)], spread)
    ds = 2.0 ** -18 * size + 2.0 ** -20
    tol = 2.0 ** -8 * np.abs(o) + (2 * ds + 2.0 ** -11)[..., None] * mag * 1.01 + 1e-7
    bad = np.abs(out.double().cpu().numpy() - o) - tol
    assert (bad <= 0).all(), bad.max()


@pytest.mark.parametrize("size", [1.0, 2.0 ** -9, 2.0 ** -18, 0.0])
@pytest.mark.parametrize("d,g,qpk,asked", [(128, 128, 4, 1), (128, 32, 8, 1), (64, 64, 4, 8), (128, 64, 4, 40)])
def test_lse_keeps_its_precision_whatever_the_values_are(d, g, qpk, asked, size):
    """lse against 64 bits, with values of any size and none: the scores' bound and a
    rounding or two of lse itself."""
    n, rng = 150, np.random.default_rng(3)
    c = make(d, g, 1, 1, 11, 16)
    k, v = rows(1, n, 1, d)
    k = k * 0.25  # small scores: lse is near ln n, and the scores' bound small
    c.write(k, v * size, torch.arange(n, device="cuda"))
    q = torch.from_numpy(rng.standard_normal((1, asked, qpk, d)) * 0.25).to(torch.bfloat16)
    lse = torch.empty(q.shape[:3], device="cuda")
    c.attend(q.cuda(), torch.arange(10, dtype=torch.int32, device="cuda")[None], dev([n]),
             q_starts=dev([0, asked]), max_q=asked, lse=lse)
    c.check()
    x, spread = cache_values(c, np.arange(n))
    _, l, _, s = ref.attend(x, q.double().numpy(), qpk, d ** -0.5, [(0, n - asked + i + 1) for i in range(asked)], spread)
    # the sum of n exponentials, each off by exp2's 2^-22 and its argument's rounding (2^-24 of at
    # most 64): 2^-18 in all; two roundings of a result below 8
    assert (np.abs(lse.double().cpu().numpy() - l) <= 2.0 ** -18 * s + 2.0 ** -18 + 2.0 ** -21).all()


def test_waiting_calls_leave_a_capture_alone():
    """check() and load(check=True) wait: under capture they refuse, and the graph goes on."""
    d, g, L, H, T = 64, 64, 1, 2, 50
    kv = torch.randn(L, 2, H, T, d, device="cuda").to(torch.bfloat16)
    buf, n, back = stream_of(kv, g, 11, 0, 0, 0)
    c = make(d, g, L, H, 6, 16)
    at = torch.from_numpy(slots_for(T, 6, 16)).cuda()
    c.load(buf, n, at, [T], check=True)
    c.pool.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError):
            c.load(buf, n, at, [T], check=True)
        with pytest.raises(ValueError):
            c.check()
        c.load(buf, n, at, [T])
    graph.replay()
    c.check()
    k, v = c.read(at)
    assert torch.equal(k.transpose(1, 2), back[:, 0]) and torch.equal(v.transpose(1, 2), back[:, 1])
