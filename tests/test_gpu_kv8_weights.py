"""Attention over the 8-bit paged cache where small softmax weights carry the
output: a key far above the rest whose own value is zero (an attention sink), a
winning page whose value scale is far below another's, pages that only later
rows see.

Bound (`lost` and `near`).  A weight times its page's value scale is rounded to
f16 in units of the largest such product of its tile (of at most 64 tokens at a
multiple of 64), brought to [2^14, 2^15) by a power of two.  Down to 2^-14 in
those units, 2^-28 of the largest, the rounding is 2^-11 relative; below, at
most 2^-25, which is 2^-39 of the largest, and never more than the product
itself.  The rest is as for all attention here: the scores (d + 8 roundings of
2^-24 of their terms) and the exponential (2^-21), twice for numerator and
denominator, fp32 sums, and the output's own rounding, in fp16's smallest
numbers half a step of 2^-24."""
import numpy as np
import pytest

from tests.test_gpu_kv8 import HALF, Setup, i32, starts, tdt

pytestmark = pytest.mark.gpu

TOP = {"int8": 127.0, "e4m3": 448.0}


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available()
    return t


def put(torch, s, k=None, v=None, ks=None, vs=None):
    """Codes [pages, heads, P, d] (uint8) and scales [pages, heads] into the cache and its plain form."""
    n, h, p, d = s.ref.c[0].shape
    if k is not None:
        s.cache.k[0].view(torch.uint8).copy_(torch.from_numpy(k.copy()).cuda())
        s.ref.c[0] = k.copy()
    if v is not None:
        lay = v.reshape(n, h, p // 16, 16, d).transpose(0, 1, 2, 4, 3)
        s.cache.v[0].view(torch.uint8).copy_(torch.from_numpy(np.ascontiguousarray(lay)).cuda())
        s.ref.c[1] = v.copy()
    for w, x, t in ((0, ks, s.cache.k_scale), (1, vs, s.cache.v_scale)):
        if x is not None:
            t[0].copy_(torch.from_numpy(x.astype(np.float32)).cuda())
            s.ref.s[w] = x.astype(np.float32)


def near(s, b, q, out, limit, head, dtype, scale):
    """One query [d] of sequence b that sees `limit` tokens, for key head `head`: |out - exact| within the bound."""
    n, d = limit, s.d
    k, v = (s.ref.tokens(w, s.table[b], n)[:, head] for w in (0, 1))
    vs = np.array([s.ref.s[1][s.table[b, t // s.page], head] for t in range(n)], np.float64)
    x = k @ q * scale
    w = np.exp(x - x.max())
    dot = np.max(np.abs(k) @ np.abs(q)) * abs(scale)
    exact, mag = w @ v / w.sum(), w @ np.abs(v) / w.sum()
    lost = np.zeros(d)
    for t in range(0, n, 64):
        e = slice(t, min(n, t + 64))
        most = (w[e] * vs[e]).max() * TOP[s.kind]
        lost += np.minimum((e.stop - t) * 2.0 ** -39 * most, w[e] @ np.abs(v[e])) / w.sum()
    err = (d + 8) * 2.0 ** -24 * dot + 2.0 ** -21
    lim = np.abs(exact) * HALF[dtype] + mag * (2.0 ** -11 + 2 * err + (n + 64) * 2.0 ** -24) + lost
    lim += 2.0 ** -25 if dtype == "fp16" else 2.0 ** -134
    got = out.double().cpu().numpy()
    # fp16 ends at 65504, and its rounding of anything from 65520 on is an infinity: one is right where a value
    # within the bound lies that far out
    past = np.isinf(got) & (np.abs(exact) + lim >= 65520.0) & (np.sign(got) == np.sign(exact)) & (dtype == "fp16")
    got, exact, lim = got[~past], exact[~past], lim[~past]
    bad = np.abs(got - exact) / lim if got.size else np.zeros(1)
    assert np.all(bad <= 1), (b, float(bad.max()), got[bad.argmax()], exact[bad.argmax()])


@pytest.mark.parametrize("kind,dtype", [("int8", "bf16"), ("int8", "fp16"), ("e4m3", "bf16"), ("e4m3", "fp16")])
@pytest.mark.parametrize("d,page,G,L,sink", [(64, 16, 1, 1000, 0), (64, 32, 4, 20000, 1), (128, 64, 4, 9000, 5000),
                                             (128, 16, 2, 700, 690), (32, 16, 12, 3000, 2999), (16, 128, 16, 700, 300)])
@pytest.mark.parametrize("nats", [14.0, 17.0, 17.5, 24.0, 40.0])
def test_one_key_above_a_heavy_tail(torch, kind, dtype, d, page, G, L, sink, nats):
    """The key at `sink` lies `nats` above the rest and its value is zero, so the
    output is what the small weights make it; scales that bring it near one."""
    s = Setup(torch, kind, 1, d, page, [L], [1], seed=d + page)
    pages = len(s.ref.s[0])
    rng = np.random.default_rng(L)
    one = 127 if kind == "int8" else 126                     # the largest code: 127, or 448
    k = np.zeros((pages, 1, page, d), np.uint8)
    # (d - 1 small random channels: the tail's scores differ by about one)
    small = rng.integers(-3, 4, size=k.shape) if kind == "int8" else None
    k[...] = small.astype(np.int8).view(np.uint8) if kind == "int8" else rng.integers(0, 30, size=k.shape) + 128 * rng.integers(0, 2, size=k.shape)
    k[..., 0] = 0
    at = s.table[0, sink // page], 0, sink % page
    k[at] = 0
    k[at + (0,)] = one
    v = rng.integers(1, 120, size=k.shape).astype(np.uint8)  # positive in both code types
    v[at] = 0
    vs = rng.uniform(0.5, 1.0, size=(pages, 1)) / TOP[kind] * np.exp(nats) / L
    ks = np.full((pages, 1), 1.0 / TOP[kind])
    put(torch, s, k, v, ks, vs)
    q = torch.zeros(1, G, d)
    q[..., 0] = nats
    q[..., 1:] = 6.0 * torch.randn(G, d - 1, generator=torch.Generator().manual_seed(3)) / d ** 0.5
    q = q.to(tdt(torch, dtype))
    out = s.cache.attention(0, q.cuda(), s.batch(torch, False), scale=1.0)
    for h in range(G):
        near(s, 0, q[0, h].double().numpy(), out[0, h], L, 0, dtype, 1.0)
    assert s.cache.status() == 0


@pytest.mark.parametrize("kind,dtype", [("int8", "bf16"), ("int8", "fp16"), ("e4m3", "fp16")])
@pytest.mark.parametrize("d,page,L", [(64, 16, 64), (64, 64, 256), (128, 16, 1500), (32, 32, 5000)])
@pytest.mark.parametrize("below", [12, 16, 18, 20, 30, 60])
def test_winning_page_of_small_values(torch, kind, dtype, d, page, L, below):
    """The tokens that win lie in a page whose value scale is 2^below under the
    others', first or last in the row; the winners' values are near one."""
    for where in (0, (L - 1) // page):
        s = Setup(torch, kind, 1, d, page, [L], [1], seed=below)
        rng = np.random.default_rng(below)
        pages = len(s.ref.s[0])
        win = s.table[0, where]
        k = rng.integers(1, 40, size=(pages, 1, page, d)).astype(np.uint8)
        k[:, :, :, 0] = 0
        k[win, :, :, 0] = 127 if kind == "int8" else 126
        ks = np.full((pages, 1), 0.05 / TOP[kind])
        ks[win] = 1.0 / TOP[kind]
        vs = np.full((pages, 1), 2.0 ** below / TOP[kind])
        vs[win] = 1.0 / TOP[kind]
        put(torch, s, k, None, ks, vs)
        # the others' weights: e^-(0.7 below + 20), so that the winners make the output
        q = torch.zeros(1, 2, d)
        q[..., 0] = 0.7 * below + 20.0
        q[..., 1:] = 0.5 * torch.randn(2, d - 1, generator=torch.Generator().manual_seed(5)) / d ** 0.5
        q = q.to(tdt(torch, dtype))
        out = s.cache.attention(0, q.cuda(), s.batch(torch, False), scale=1.0)
        for h in range(2):
            near(s, 0, q[0, h].double().numpy(), out[0, h], L, 0, dtype, 1.0)
        assert s.cache.status() == 0


@pytest.mark.parametrize("kind,dtype", [("int8", "fp16"), ("e4m3", "bf16")])
@pytest.mark.parametrize("d,page,G,L", [(64, 16, 1, 64), (64, 16, 12, 300), (128, 16, 1, 1500)])
@pytest.mark.parametrize("above,nats", [(115, 80.0), (119, 84.0), (118, 100.0), (100, 60.0)])
def test_scales_that_leave_fp32(torch, kind, dtype, d, page, G, L, above, nats):
    """A page whose values are 2^above times the others' while its tokens lie
    `nats` below, so that both count (or, at 100, it does not): scale and power
    of two together pass fp32's largest number."""
    s = Setup(torch, kind, 1, d, page, [L], [1], seed=above)
    pages = len(s.ref.s[0])
    big = s.table[0, 1]
    rng = np.random.default_rng(above)
    k = np.zeros((pages, 1, page, d), np.uint8)
    k[..., 0] = 127 if kind == "int8" else 126
    k[big, :, :, 0] = 0
    v = rng.integers(1, 120, size=k.shape).astype(np.uint8)
    vs = np.full((pages, 1), 1.0 / TOP[kind])
    vs[big] *= 2.0 ** above
    put(torch, s, k, v, np.full((pages, 1), 1.0 / TOP[kind]), vs)
    q = torch.zeros(1, G, d)
    q[..., 0] = nats
    q = q.to(tdt(torch, dtype))
    out = s.cache.attention(0, q.cuda(), s.batch(torch, False), scale=1.0)
    for h in range(G):
        near(s, 0, q[0, h].double().numpy(), out[0, h], L, 0, dtype, 1.0)
    assert s.cache.status() == 0


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("d,page,G,L", [(64, 16, 1, 70), (128, 16, 12, 300), (32, 64, 4, 2000)])
@pytest.mark.parametrize("scale", [2.0 ** -126, 2.0 ** -120, 2.0 ** 100, 0.0])
def test_scales_at_the_ends_of_fp32(torch, kind, d, page, G, L, scale):
    """Values of 1e-36, of 1e31, and none: one rounding to bf16 like any others."""
    s = Setup(torch, kind, 1, d, page, [L], [1], seed=L)
    rng = np.random.default_rng(L)
    vs = np.full_like(s.ref.s[1], scale)
    vs[rng.random(vs.shape) < 0.5] *= 1.5
    put(torch, s, vs=vs)
    q = (2.0 * torch.randn(1, G, d, generator=torch.Generator().manual_seed(2))).to(torch.bfloat16)
    out = s.cache.attention(0, q.cuda(), s.batch(torch, False))
    for h in range(G):
        near(s, 0, q[0, h].double().numpy(), out[0, h], L, 0, "bf16", d ** -0.5)
    assert s.cache.status() == 0


@pytest.mark.parametrize("kind,dtype,d,L", [("int8", "fp16", 64, 64), ("e4m3", "bf16", 128, 200), ("int8", "bf16", 32, 1500)])
@pytest.mark.parametrize("last", [2.0 ** 25, float("nan"), float("inf"), 0.0])
def test_pages_that_later_rows_see(torch, kind, dtype, d, L, last):
    """The last page holds values 2^25 times the others', a NaN or an infinite
    scale, or none: rows that end before it do not feel it."""
    page, n = 16, 20
    s = Setup(torch, kind, 1, d, page, [L], [n], seed=7)
    vs = s.ref.s[1].copy()
    at = s.table[0, (L - 1) // page]
    vs[at] = vs[at] * last if last == 2.0 ** 25 else last
    put(torch, s, vs=vs)
    q = torch.randn(n, 3, d, generator=torch.Generator().manual_seed(1)).to(tdt(torch, dtype))
    out = s.cache.attention(0, q.cuda(), s.batch(torch, True))
    first = (L - 1) // page * page
    for i in range(n):
        limit = L - n + i + 1
        if limit > first and not np.isfinite(last):
            # (a NaN or infinite scale times a zero code is a NaN, times others a NaN or an infinity)
            assert not torch.isfinite(out[i]).any()
            continue
        for h in range(3):
            near(s, 0, q[i, h].double().numpy(), out[i, h], limit, 0, dtype, d ** -0.5)
    assert s.cache.status() == 0


def test_one_key_above_many_rows(torch):
    """Several sequences and rows, each with its own first token above the rest, in one call."""
    heads, G, d, page, lens, new = 2, 3, 64, 16, [300, 40, 2000, 1], [4, 1, 2, 1]
    s = Setup(torch, "int8", heads, d, page, lens, new, seed=2)
    k, v = s.ref.c[0].copy(), s.ref.c[1].copy()
    for b in range(len(lens)):
        v[s.table[b, 0], :, 0] = 0
        k[s.table[b, 0], :, 0] = 0
        k[s.table[b, 0], :, 0, 0] = 127
    k[..., 0][k[..., 0] != 127] = 0
    put(torch, s, k, v, np.full_like(s.ref.s[0], 0.25 / 127))
    q = torch.randn(sum(new), heads * G, d, generator=torch.Generator().manual_seed(9))
    q[..., 0] = 80.0
    q = q.half()
    out = s.cache.attention(0, q.cuda(), s.batch(torch, True), scale=1.0)
    at = starts(new)
    for b, (n, m) in enumerate(zip(lens, new)):
        for i in range(m):
            for h in range(heads * G):
                near(s, b, q[at[b] + i, h].double().numpy(), out[at[b] + i, h], n - m + i + 1, h // G, "fp16", 1.0)
    assert s.cache.status() == 0
