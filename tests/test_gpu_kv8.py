"""The 8-bit paged key/value cache on the GPU against the plain forms of
tests/kv8_ref.py: codes and scales bit for bit (their definition is a chain of
single fp32 operations), values read back to one 16-bit rounding, attention
within a bound added up from its roundings (`bound` below)."""
import numpy as np
import pytest

from tests import kv8_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available()
    return t


HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


def tdt(torch, dtype):
    return {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]


def i32(torch, v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def starts(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


def make_table(rng, counts, width, pages):
    ids = rng.permutation(pages)[:sum(counts)]
    t = np.full((len(counts), max(1, width)), -1, np.int32)
    at = 0
    for b, n in enumerate(counts):
        t[b, :n] = ids[at:at + n]
        at += n
    return t


class Setup:
    """A cache of one layer whose pages hold random codes, unused ones
    arbitrary bytes (e4m3's NaN among them), beside its plain form."""

    def __init__(self, torch, kind, heads, d, page, lens, new, seed, extra=2, layers=1, layer=0):
        from scratch_decoder_only_b200.kv8 import KV8Cache
        rng = self.rng = np.random.default_rng(seed)
        counts = [-(-n // page) for n in lens]
        pages = sum(counts) + extra
        self.kind, self.lens, self.new, self.page, self.layer = kind, list(lens), list(new), page, layer
        self.table = make_table(rng, counts, max(counts + [1]), pages)
        raw = rng.integers(0, 256, size=(2, layers, pages, heads, page * d), dtype=np.uint8)
        low = 0.01 if kind == "int8" else 0.003
        sc = rng.uniform(low, 3 * low, size=(2, layers, pages, heads)).astype(np.float32)
        # slots in use hold no NaN (and int8 no -128)
        ok = raw[:, layer].reshape(2, pages, heads, -1)
        if kind == "int8":
            ok[ok == 128] = 129
        else:
            used = [ids for b in range(len(lens)) for ids in self.table[b, :counts[b]]]
            sub = ok[:, used]
            sub[(sub & 127) == 127] = 1
            ok[:, used] = sub
        k = raw[0].reshape(layers, pages, heads, page, d)
        v = raw[1].reshape(layers, pages, heads, page // 16, d, 16)
        if kind == "e4m3":
            # slots behind a sequence's end: NaN codes
            for b, n in enumerate(lens):
                if n % page:
                    i, at = self.table[b, counts[b] - 1], n % page
                    k[layer, i, :, at:] = 127
                    vt = v[layer, i].transpose(0, 1, 3, 2).reshape(heads, page, d).copy()
                    vt[:, at:] = 255
                    v[layer, i] = vt.reshape(heads, page // 16, 16, d).transpose(0, 1, 3, 2)
        code = torch.int8 if kind == "int8" else torch.float8_e4m3fn
        dev = [torch.from_numpy(x.copy()).cuda() for x in (k, v, sc[0], sc[1])]
        self.cache = KV8Cache(dev[0].view(code), dev[1].view(code), dev[2], dev[3])
        self.ref = R.Ref(kind, pages, heads, page, d)
        self.ref.load(k[layer], v[layer], sc[0, layer], sc[1, layer])
        self.heads, self.d = heads, d

    def batch(self, torch, ragged=True, table=None, lens=None, new=None, rows=None):
        from scratch_decoder_only_b200.kv8 import KV8Batch
        new = self.new if new is None else new
        t = i32(torch, self.table if table is None else table)
        n = i32(torch, self.lens if lens is None else lens)
        return KV8Batch(t, n, i32(torch, starts(new)), int(sum(new)) if rows is None else rows) if ragged else KV8Batch(t, n)

    def state(self, torch):
        c = self.cache
        u = [x[self.layer].view(torch.uint8).cpu().numpy() for x in (c.k, c.v)]
        n, h, p, d = u[0].shape
        return [u[0], u[1].transpose(0, 1, 2, 4, 3).reshape(n, h, p, d)], [x[self.layer].cpu().numpy() for x in (c.k_scale, c.v_scale)]

    def same(self, torch, lens, table=None):
        """Codes of all tokens in `lens`, and all scales, equal the plain form's."""
        codes, scales = self.state(torch)
        for w in range(2):
            assert np.array_equal(scales[w], self.ref.s[w], equal_nan=True), w
            for b, n in enumerate(lens):
                for j in range(-(-n // self.page)):
                    i, m = self.table[b, j], min(self.page, n - j * self.page)
                    assert np.array_equal(codes[w][i, :, :m], self.ref.c[w][i, :, :m]), (w, b, j)


def values(torch, rng, shape, dtype, scale=1.0):
    x = torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(tdt(torch, dtype))
    return x, x.float().numpy()


# (heads, d, page, tokens before, new tokens): nothing, one token, ends and
# starts on and beside page and 16-token borders, several pages at once
APPENDS = [
    (1, 16, 16, [0, 1, 15, 16, 0], [1, 1, 1, 1, 0]),
    (3, 32, 32, [0, 31, 5, 40], [33, 1, 70, 24]),
    (2, 64, 16, [0, 0, 7, 3, 16], [16, 17, 9, 0, 200]),
    (12, 64, 64, [63, 64, 10, 0], [2, 1, 6, 64]),
    (2, 128, 128, [0, 100, 127, 3], [128, 29, 1, 130]),
    (5, 128, 16, [0, 12], [50, 3]),
    (1, 16, 128, [90, 0], [100, 1]),
]


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,d,page,old,new", APPENDS)
def test_append_and_read(torch, kind, dtype, heads, d, page, old, new):
    lens = [a + b for a, b in zip(old, new)]
    s = Setup(torch, kind, heads, d, page, lens, new, seed=heads * d + page)
    b = s.batch(torch)
    rng = np.random.default_rng(5)
    # keys and values side by side in wider rows, as a fused projection leaves them
    wide = torch.zeros(sum(new), heads * d * 2 + 24, dtype=tdt(torch, dtype), device="cuda")
    k, kf = values(torch, rng, (sum(new), heads, d), dtype, 2.0)
    v, vf = values(torch, rng, (sum(new), heads, d), dtype, 3.0)
    kd = wide[:, 8:8 + heads * d]
    vd = wide[:, 16 + heads * d:16 + 2 * heads * d]
    kd.copy_(k.reshape(sum(new), -1)), vd.copy_(v.reshape(sum(new), -1))
    s.cache.append(0, kd, vd, b)
    at = starts(new)
    for i in range(len(lens)):
        s.ref.append(s.table[i], lens[i], (kf[at[i]:at[i + 1]], vf[at[i]:at[i + 1]]))
    s.same(torch, lens)
    assert s.cache.status() == 0
    # against the values themselves: half a step of the page's scale, or of e4m3's own
    for w, x in ((0, kf), (1, vf)):
        for i in range(len(lens)):
            got = s.ref.tokens(w, s.table[i], lens[i])[lens[i] - new[i]:]
            for j in range(new[i]):
                sc = s.ref.s[w][s.table[i, (lens[i] - new[i] + j) // page]][:, None].astype(np.float64)
                want = x[at[i] + j].astype(np.float64)
                lim = sc / 2 if kind == "int8" else np.maximum(np.abs(want) * 2.0 ** -4, sc * 2.0 ** -10)
                assert np.all(np.abs(got[j] - want) <= lim * (1 + 1e-5)), (w, i, j)
    # read back: all tokens of each sequence
    rb = s.batch(torch, new=lens)
    rk, rv = s.cache.read(0, rb, tdt(torch, dtype))
    for w, r in ((0, rk), (1, rv)):
        want = np.concatenate([s.ref.tokens(w, s.table[i], lens[i]) for i in range(len(lens))])
        # code * scale in fp32 (2^-24), then the 16-bit type's half step
        assert np.all(np.abs(r.double().cpu().numpy() - want) <= np.abs(want) * (HALF[dtype] + 2.0 ** -23) + 2.0 ** -25)
    assert s.cache.status() == 0


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("P,heads,d,dtype", [(16, 2, 64, "bf16"), (32, 3, 16, "fp16"), (64, 1, 128, "bf16"), (128, 5, 32, "fp16")])
def test_append_token_by_token(torch, kind, P, heads, d, dtype):
    """Growing values: the scale of a page rises with most tokens and its codes
    are rounded anew each time; one row per sequence, without starts."""
    s = Setup(torch, kind, heads, d, P, [40, 33, 8], [1, 1, 1], seed=1)
    rng = np.random.default_rng(2)
    for step in range(1, 34):
        lens = [step if n >= step else 0 for n in s.lens]
        live = [i for i, n in enumerate(lens) if n]
        from scratch_decoder_only_b200.kv8 import KV8Batch
        b = KV8Batch(i32(torch, s.table[live]), i32(torch, [lens[i] for i in live]))
        k, kf = values(torch, rng, (len(live), heads, d), dtype, 0.1 * step)
        v, vf = values(torch, rng, (len(live), heads, d), dtype, 4.0 / step)
        s.cache.append(0, k.cuda(), v.cuda(), b)
        for j, i in enumerate(live):
            s.ref.append(s.table[i], lens[i], (kf[j:j + 1], vf[j:j + 1]))
        s.same(torch, lens)
    assert s.cache.status() == 0


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_append_odd_values(torch, kind):
    """Zeros, values whose scale would be below the normal numbers, infinities
    and NaN, also as a page's later token; the sign of zero."""
    P, heads, d = 16, 1, 32
    rows = np.zeros((6, heads, d), np.float32)
    rows[1, 0, :3] = [1e-38, -3e-39, 1e-40]
    rows[2, 0, 5] = np.inf
    rows[3, 0, 7] = np.nan
    rows[4] = 1.0
    rows[5, 0, ::2] = -0.0
    lens, new = [1, 1, 1, 1, 4, 1], [1] * 6
    s = Setup(torch, kind, heads, d, P, lens, new, seed=3)
    x = torch.from_numpy(rows).to(torch.bfloat16)
    s.cache.append(0, x.cuda(), x.cuda(), s.batch(torch, ragged=False))
    for i in range(6):
        s.ref.append(s.table[i], lens[i], (x.float().numpy()[i:i + 1],) * 2)
    s.same(torch, lens)
    sc = s.state(torch)[1][0][:, 0]
    got = [sc[s.table[i, 0]] for i in range(6)]
    assert got[0] == 0 and got[1] == 0 and np.isnan(got[2]) and np.isnan(got[3]) and got[4] > 0 and got[5] == 0
    # a finite token after a NaN one: the page stays NaN; a new page does not
    s.cache.append(0, x[4:5].cuda(), x[4:5].cuda(), s.batch(torch, False, table=s.table[3:4], lens=[2]))
    assert np.isnan(s.state(torch)[1][0][s.table[3, 0], 0])
    s.cache.append(0, x[4:5].cuda(), x[4:5].cuda(), s.batch(torch, False, table=s.table[3:4], lens=[1]))
    assert s.state(torch)[1][0][s.table[3, 0], 0] > 0
    assert s.cache.status() == 0


def bound(out, mag, dot, L, d, dtype):
    """|out - exact| at most: the output's rounding, the weights' rounding to
    f16 (2^-12 of each term; those below f16's normal numbers 2^-25 of the
    largest term), the scores' error x (fp32 sum of d products, q's own f16
    rounding) and the exponential's (2^-21), twice for numerator and denominator, and the fp32 sums."""
    x = (d + 8) * 2.0 ** -24 * dot[..., None] + 2.0 ** -21
    return np.abs(out) * HALF[dtype] + mag * (2.0 ** -11 + 2 * x + (L + 64) * 2.0 ** -24) + 2.0 ** -24


ATTENDS = [
    # heads, G, d, page, tokens, new
    (1, 1, 16, 16, [1, 2, 16, 17, 0], [1, 1, 1, 1, 1]),
    (12, 1, 64, 16, [1, 63, 64, 65, 500], [1] * 5),
    (2, 4, 64, 32, [300, 5, 1, 129], [1] * 4),
    (2, 3, 32, 64, [200, 0, 77], [5, 2, 3]),
    (1, 8, 128, 64, [1000, 31], [1, 1]),
    (2, 5, 128, 128, [400, 130, 3], [4, 1, 3]),
    (1, 1, 64, 128, [90, 260], [33, 40]),
    (3, 2, 16, 32, [700], [17]),
    (1, 12, 64, 16, [50, 51], [1, 1]),
    (1, 40, 32, 16, [20, 400], [1, 1]),
    (1, 16, 128, 64, [300, 40], [1, 1]),
]


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,G,d,page,lens,new", ATTENDS)
def test_attention(torch, kind, dtype, heads, G, d, page, lens, new):
    s = Setup(torch, kind, heads, d, page, lens, new, seed=G * d + page)
    q, qf = values(torch, s.rng, (sum(new), heads * G, d), dtype)
    ragged = new != [1] * len(new)
    out, lse = s.cache.attention(0, q.cuda(), s.batch(torch, ragged), return_lse=True)
    check(torch, s, qf, out, lse, lens, new, dtype)
    assert s.cache.status() == (16 if any(n < m for n, m in zip(lens, new)) else 0)
    again = s.cache.attention(0, q.cuda(), s.batch(torch, True))
    assert torch.equal(again, out) or not ragged
    again = s.cache.attention(0, q.cuda(), s.batch(torch, ragged))
    assert torch.equal(again, out)          # the same bits


def check(torch, s, qf, out, lse, lens, new, dtype, scale=None, skip=()):
    at = starts(new)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for i, (n, m) in enumerate(zip(lens, new)):
        k, v = s.ref.tokens(0, s.table[i], n), s.ref.tokens(1, s.table[i], n)
        if skip:
            keep = [t for t in range(n) if (i, t // s.page) not in skip]
            k, v = k[keep], v[keep]
        else:
            keep = list(range(n))
        limits = [sum(t <= n - m + j for t in keep) for j in range(m)]
        o, e, mag, dot = R.attention(qf[at[i]:at[i + 1]].astype(np.float64), k, v, limits,
                                     s.d ** -0.5 if scale is None else scale)
        g = out[at[i]:at[i + 1]]
        assert np.all(np.abs(g - o) <= bound(o, mag, dot, n, s.d, dtype)), (i, np.max(np.abs(g - o)))
        gl = lse[at[i]:at[i + 1]]
        assert np.array_equal(np.isinf(gl), np.isinf(e)), i
        fin = np.isfinite(e)
        lim = (s.d + 8) * 2.0 ** -24 * dot + 2.0 ** -21 + (n + 64) * 2.0 ** -24 + 2.0 ** -22 * np.abs(np.where(fin, e, 0))
        assert np.all(np.abs(gl[fin] - e[fin]) <= lim[fin]), i


def test_attention_long_split(torch):
    """One long sequence beside short ones: pieces and their merge; an odd length."""
    lens, new = [9001, 3, 0, 1024, 257], [1] * 5
    s = Setup(torch, "int8", 2, 64, 16, lens, new, seed=9)
    q, qf = values(torch, s.rng, (5, 8, 64), "bf16", 2.0)
    out, lse = s.cache.attention(0, q.cuda(), s.batch(torch, False), return_lse=True)
    check(torch, s, qf, out, lse, lens, new, "bf16")
    new = [7, 3, 0, 5, 1]
    s = Setup(torch, "e4m3", 1, 128, 64, lens, new, seed=10)
    q, qf = values(torch, s.rng, (sum(new), 4, 128), "fp16", 2.0)
    out, lse = s.cache.attention(0, q.cuda(), s.batch(torch), return_lse=True)
    check(torch, s, qf, out, lse, lens, new, "fp16")
    assert s.cache.status() == 0


@pytest.mark.parametrize("kind,dtype,heads,G,d,page,lens,new", [
    ("int8", "bf16", 1, 1, 16, 16, [2500], [1]), ("e4m3", "fp16", 2, 3, 32, 32, [1300, 700], [1, 1]),
    ("int8", "fp16", 1, 16, 64, 16, [3000, 40], [1, 1]), ("e4m3", "bf16", 1, 16, 128, 64, [1500, 641], [1, 1]),
    ("int8", "bf16", 2, 4, 32, 64, [900, 1200], [9, 6]), ("e4m3", "bf16", 1, 5, 16, 128, [2000, 0, 77], [8, 0, 5]),
    ("int8", "fp16", 1, 2, 128, 16, [1100], [40])])
def test_attention_long_at_every_width(torch, kind, dtype, heads, G, d, page, lens, new):
    """Runs of tiles that cut jobs, for 8 and for 16 queries a job."""
    s = Setup(torch, kind, heads, d, page, lens, new, seed=G * d + page)
    q, qf = values(torch, s.rng, (sum(new), heads * G, d), dtype, 1.5)
    b = s.batch(torch, new != [1] * len(new))
    out, lse = s.cache.attention(0, q.cuda(), b, return_lse=True)
    check(torch, s, qf, out, lse, lens, new, dtype)
    assert torch.equal(s.cache.attention(0, q.cuda(), b), out)
    assert s.cache.status() == 0


@pytest.mark.parametrize("top,ragged", [(90, False), (90, True), (700, True), (700, False), (1500, True), (1500, False)])
def test_many_sequences(torch, top, ragged):
    """More sequences than threads of a block, empty ones and ones without rows
    among them, for whole jobs (rows of at most 1024 tokens) and for runs; also append and read."""
    rng = np.random.default_rng(top + ragged)
    B, heads, d, P = 300, 2, 32, 16
    lens = [int(n) for n in np.where(rng.random(B) < 0.1, 0, np.exp(rng.uniform(0, np.log(top), B)).astype(int))]
    lens[7] = top
    new = [min(n, int(rng.integers(0, 4))) for n in lens] if ragged else [1] * B
    if ragged:
        new[0], new[-1] = 0, 0
    s = Setup(torch, "int8", heads, d, P, lens, new, seed=3)
    q, qf = values(torch, s.rng, (sum(new), heads * 2, d), "fp16")
    out, lse = s.cache.attention(0, q.cuda(), s.batch(torch, ragged), return_lse=True)
    check(torch, s, qf, out, lse, lens, new, "fp16")
    x, xf = values(torch, s.rng, (sum(new), heads, d), "fp16")
    s.cache.status()
    s.cache.append(0, x.cuda(), x.cuda(), s.batch(torch, ragged))
    at = starts(new)
    for i in range(B):
        m = min(new[i], lens[i])
        s.ref.append(s.table[i], lens[i], (xf[at[i + 1] - m:at[i + 1]],) * 2)
    s.same(torch, lens)
    assert s.cache.status() == (0 if ragged else 16)      # a row for an empty sequence has no place
    k, v = s.cache.read(0, s.batch(torch, True, new=lens), torch.float16)
    want = np.concatenate([s.ref.tokens(1, s.table[i], lens[i]) for i in range(B)])
    assert np.all(np.abs(v.double().cpu().numpy() - want) <= np.abs(want) * (2.0 ** -11 + 2.0 ** -23) + 2.0 ** -25)


@pytest.mark.parametrize("B,ragged", [(4200, True), (4200, False), (9000, True), (1600, True)])
def test_attention_of_many_sequences(torch, B, ragged):
    """A thread's share of the sequences is more than a warp looks at in one step (from 4096 sequences on), or
    more than one in whole jobs (1600 of one head)."""
    rng = np.random.default_rng(B)
    heads, d, P = 1 if B == 1600 else 2, 16, 16
    lens = [int(n) for n in rng.integers(0, 40, size=B)]
    lens[B // 3] = 700
    new = [min(n, int(rng.integers(0, 3))) for n in lens] if ragged else [1] * B
    if B == 1600:
        new = [min(n, 1) if i % 20 == 3 else 0 for i, n in enumerate(lens)]
    s = Setup(torch, "e4m3", heads, d, P, lens, new, seed=4)
    q, qf = values(torch, s.rng, (sum(new), heads * 3, d), "bf16")
    out, lse = s.cache.attention(0, q.cuda(), s.batch(torch, ragged), return_lse=True)
    check(torch, s, qf, out, lse, lens, new, "bf16")


@pytest.mark.parametrize("G,d,B", [(1, 128, 160), (12, 64, 160), (16, 128, 160), (2, 16, 160), (1, 32, 1000)])
def test_many_short_jobs(torch, G, d, B):
    """More whole jobs than blocks of eight warps fit at once: blocks of four; and
    so many that the warps take runs of them."""
    rng = np.random.default_rng(d)
    lens, new = [int(n) for n in rng.integers(0, 120, B)], [1] * B
    s = Setup(torch, "e4m3", 2, d, 32, lens, new, seed=d)
    q, qf = values(torch, s.rng, (B, 2 * G, d), "bf16")
    out, lse = s.cache.attention(0, q.cuda(), s.batch(torch, False), return_lse=True)
    check(torch, s, qf, out, lse, lens, new, "bf16")


def test_attention_of_equal_weights(torch):
    """scale = 0: the mean of the values, whatever the keys."""
    s = Setup(torch, "int8", 2, 64, 16, [100, 700], [1, 1], seed=5)
    q, qf = values(torch, s.rng, (2, 4, 64), "bf16")
    out, lse = s.cache.attention(0, q.cuda(), s.batch(torch, False), scale=0.0, return_lse=True)
    check(torch, s, qf, out, lse, [100, 700], [1, 1], "bf16", scale=0.0)


def test_attention_strides_scale_and_rows_outside(torch):
    """q and out inside wider rows, a scale of its own, rows before the first
    and behind the last sequence: those stay as they were."""
    lens, new = [40, 100], [2, 3]
    s = Setup(torch, "int8", 2, 32, 16, lens, new, seed=4)
    wide = torch.full((9, 200), 7.0, dtype=torch.float16, device="cuda")
    q, qf = values(torch, s.rng, (5, 4, 32), "fp16")
    qd = torch.zeros(9, 160, dtype=torch.float16, device="cuda")
    qd[2:7, 8:136] = q.reshape(5, -1).cuda()
    from scratch_decoder_only_b200.kv8 import KV8Batch
    b = KV8Batch(i32(torch, s.table), i32(torch, lens), i32(torch, [2, 4, 7]), 9)
    out, lse = s.cache.attention(0, qd[:, 8:136], b, scale=-0.3, out=wide[:, 16:144], return_lse=True)
    check(torch, s, qf, wide[2:7, 16:144].reshape(5, 4, 32), lse[2:7], lens, new, "fp16", scale=-0.3)
    assert torch.all(wide[:2] == 7) and torch.all(wide[7:] == 7)
    assert torch.all(wide[:, :16] == 7) and torch.all(wide[:, 144:] == 7)
    # append and read leave them too, and the pages of the skipped rows
    x = torch.randn(9, 2, 32, device="cuda", dtype=torch.float16)
    s.cache.append(0, x, x, b)
    for i in range(2):
        s.ref.append(s.table[i], lens[i], (x.float().cpu().numpy()[[2, 4][i]:[4, 7][i]],) * 2)
    s.same(torch, lens)
    assert s.cache.status() == 0


def test_attention_extreme_scores(torch):
    """Scores of hundreds (one token takes all), huge and tiny queries, value
    scales that differ by 2^20 between pages, a NaN scale, an infinite query."""
    lens, new = [64, 64, 64, 64], [1] * 4
    s = Setup(torch, "int8", 1, 64, 16, lens, new, seed=6)
    sc = s.cache.v_scale.view(-1)
    for b in range(4):
        sc[int(s.table[b, 1])] *= 2.0 ** -20
    s.ref.s[1] = s.cache.v_scale[0].cpu().numpy()
    q = torch.randn(4, 2, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    q[1] *= 300.0
    q[2] *= 1e-37
    q[3, 0, 5] = float("inf")
    out, lse = s.cache.attention(0, q.cuda(), s.batch(torch, False), return_lse=True)
    for b in range(3):
        k, v = s.ref.tokens(0, s.table[b], 64), s.ref.tokens(1, s.table[b], 64)
        o, e, mag, dot = R.attention(q[b:b + 1].double().numpy(), k, v, [64], 64 ** -0.5)
        assert np.all(np.abs(out[b:b + 1].double().cpu().numpy() - o) <= bound(o, mag, dot, 64, 64, "bf16"))
    assert torch.isnan(out[3, 0]).all() and torch.isfinite(out[3, 1]).all() and torch.isnan(lse[3, 0])
    # a page whose scale is NaN reaches the rows that see it, no others
    s.cache.k_scale[0, int(s.table[0, 3]), 0] = float("nan")
    s.cache.v_scale[0, int(s.table[1, 0]), 0] = float("nan")
    lens2 = i32(torch, [48, 64, 64, 64])
    from scratch_decoder_only_b200.kv8 import KV8Batch
    out = s.cache.attention(0, q.cuda(), KV8Batch(i32(torch, s.table), lens2))
    assert torch.isfinite(out[0]).all() and torch.isnan(out[1]).all() and torch.isfinite(out[2]).all()
    out = s.cache.attention(0, q.cuda(), s.batch(torch, False))
    assert torch.isnan(out[0]).all()


def test_attention_dominant_small_page(torch):
    """The tokens that win lie in a page whose value scale is 2^12 below
    another's: the weights keep their bits (relative to that page's values the
    f16 weights lose 2^12 of range, not of precision)."""
    s = Setup(torch, "int8", 1, 64, 16, [64], [1], seed=8)
    s.cache.v_scale[0, int(s.table[0, 0])] *= 2.0 ** -12
    s.cache.k_scale[0, int(s.table[0, 0])] *= 30.0
    s.ref.s = [s.cache.k_scale[0].cpu().numpy(), s.cache.v_scale[0].cpu().numpy()]
    q, qf = values(torch, s.rng, (1, 1, 64), "fp16", 4.0)
    out, lse = s.cache.attention(0, q.cuda(), s.batch(torch, False), return_lse=True)
    check(torch, s, qf, out, lse, [64], [1], "fp16")


def test_bad_pages_and_lengths(torch):
    """Ids outside the pool, lengths beyond the row's pages or below the new
    tokens: those tokens are skipped, the error word says so, nothing else changes."""
    lens, new = [60, 40, 33], [1, 1, 1]
    s = Setup(torch, "int8", 2, 64, 16, lens, new, seed=12)
    bad = s.table.copy()
    bad[0, 1], bad[1, 0], bad[2, 2] = 10 ** 6, -5, len(s.ref.s[0])
    q, qf = values(torch, s.rng, (3, 4, 64), "bf16")
    out, lse = s.cache.attention(0, q.cuda(), s.batch(torch, False, table=bad), return_lse=True)
    check(torch, s, qf, out, lse, lens, new, "bf16", skip={(0, 1), (1, 0), (2, 2)})
    assert s.cache.status() == 32 and s.cache.status() == 0
    before = s.state(torch)
    x = torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    s.cache.append(0, x, x, s.batch(torch, False, table=bad, lens=[17, 1, 33]))
    after = s.state(torch)
    assert all(np.array_equal(a, b) for a, b in zip(before[0] + before[1], after[0] + after[1]))
    assert s.cache.status() == 32
    s.cache.append(0, x, x, s.batch(torch, False, lens=[65, -3, 10 ** 9]))
    after = s.state(torch)
    assert all(np.array_equal(a, b) for a, b in zip(before[0] + before[1], after[0] + after[1]))
    assert s.cache.status() == 16
    out, lse = s.cache.attention(0, q.cuda(), s.batch(torch, False, lens=[60, -3, 33]), return_lse=True)
    assert torch.all(out[1] == 0) and torch.all(torch.isinf(lse[1])) and s.cache.status() == 16
    # three new tokens of which one would lie before the sequence's start
    lens = [2, 40, 33]
    q3, q3f = values(torch, s.rng, (5, 4, 64), "bf16")
    out, lse = s.cache.attention(0, q3.cuda(), s.batch(torch, True, lens=lens, new=[3, 1, 1]), return_lse=True)
    assert torch.all(out[0] == 0) and s.cache.status() == 16
    check(torch, s, q3f, out, lse, lens, [3, 1, 1], "bf16")
    # starts that decrease or leave the rows
    from scratch_decoder_only_b200.kv8 import KV8Batch
    for st in ([0, 3, 2, 5], [-1, 1, 2, 5], [0, 1, 2, 99]):
        s.cache.attention(0, q3.cuda(), KV8Batch(i32(torch, s.table), i32(torch, [60, 40, 33]), i32(torch, st), 5))
        assert s.cache.status() & 64


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_lengths_at_the_ends_of_32_bits(torch, kind):
    """Lengths whose differences with the new tokens pass 32 bits: no token, and the
    word says so, in each form of each call."""
    s = Setup(torch, kind, 2, 32, 16, [40, 20], [1, 1], seed=31)
    before = s.state(torch)
    for new in ([1, 1], [3, 2]):
        n = sum(new)
        x, _ = values(torch, s.rng, (n, 2, 32), "bf16")
        q, _ = values(torch, s.rng, (n, 4, 32), "bf16")
        for low in (-2 ** 31, -2 ** 31 + 1, -2 ** 31 + 16, -2 ** 31 + 17, -1, 0):
            for ragged in (True, False) if new == [1, 1] else (True,):
                b = s.batch(torch, ragged, lens=[low, low], new=new)
                s.cache.append(0, x.cuda(), x.cuda(), b)
                assert s.cache.status() == 16
                s.cache.read(0, b)
                assert s.cache.status() == 16
                out, lse = s.cache.attention(0, q.cuda(), b, return_lse=True)
                assert torch.all(out == 0) and torch.all(lse == -float("inf")) and s.cache.status() == 16
    after = s.state(torch)
    assert all(np.array_equal(a, b) for a, b in zip(before[0] + before[1], after[0] + after[1]))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_read_leaves_rows_of_skipped_tokens(torch, dtype):
    """Rows outside the starts, of tokens before a sequence's first and of bad pages keep what they hold."""
    import ctypes
    from scratch_decoder_only_b200 import gpt as G
    lens, new, rows = [40, 3, 33], [20, 5, 33], 61
    s = Setup(torch, "int8", 3, 32, 16, [40, 5, 33], [20, 5, 33], seed=33)
    table = s.table.copy()
    table[2, 1] = -7
    b = s.batch(torch, True, table=table, lens=lens, new=new, rows=rows)
    out = [torch.full((rows, 96), 7.0, dtype=tdt(torch, dtype), device="cuda") for _ in range(2)]
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert G.load_library().gpt_kv8_read(s.cache._c, 0, b.ref, out[0].data_ptr(), 96, out[1].data_ptr(), 96,
                                         1 if dtype == "bf16" else 2, s.cache._err, stream) == G.GPT_OK
    assert s.cache.status() == 16 | 32
    for w in range(2):
        want = np.full((rows, 3, 32), 7.0, np.float32)
        want[0:20] = s.ref.tokens(w, s.table[0], 40)[20:]
        want[22:25] = s.ref.tokens(w, s.table[1], 3)
        third = s.ref.tokens(w, s.table[2], 33)
        want[25:41], want[57:58] = third[:16], third[32:]
        got = out[w].float().cpu().numpy().reshape(rows, 3, 32)
        kept = want == 7.0
        assert np.all(got[kept] == 7.0)
        # code * scale in fp32, then one rounding (2^-24 and half a step, relative)
        assert np.all(np.abs(got - want) <= np.abs(want) * (HALF[dtype] + 2.0 ** -23))


@pytest.mark.parametrize("heads,d,page,B", [(1, 16, 16, 1500), (3, 32, 16, 1500), (2, 128, 64, 1100), (1, 16, 16, 18000)])
def test_append_of_many_sequences(torch, heads, d, page, B):
    """More sequences than a block has threads, and than their square, some without new tokens."""
    rng = np.random.default_rng(B + d)
    new = rng.integers(0, 6, size=B)
    new[:40] = 0
    new[-1] = page + 1
    lens = new + rng.integers(0, 20, size=B)
    s = Setup(torch, "int8", heads, d, page, lens, new, seed=B)
    x = [values(torch, rng, (int(new.sum()), heads, d), "bf16") for _ in range(2)]
    b = s.batch(torch)
    s.cache.append(0, x[0][0].cuda(), x[1][0].cuda(), b)
    at = starts(new)
    for i in range(B):
        if new[i]:
            s.ref.append(s.table[i], lens[i], (x[0][1][at[i]:at[i + 1]], x[1][1][at[i]:at[i + 1]]))
    s.same(torch, lens)
    got = s.cache.read(0, b)
    for w in range(2):
        want = np.concatenate([s.ref.tokens(w, s.table[i], lens[i])[lens[i] - new[i]:] for i in range(B)])
        # code * scale in fp32 (2^-24), then bf16's half step
        assert np.all(np.abs(got[w].double().cpu().numpy() - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -23) + 2.0 ** -25)
    assert s.cache.status() == 0


def test_empty_calls(torch):
    s = Setup(torch, "int8", 1, 16, 16, [5], [1], seed=1)
    from scratch_decoder_only_b200.kv8 import KV8Batch
    z = torch.zeros(0, 1, 16, dtype=torch.bfloat16, device="cuda")
    for b in (KV8Batch(i32(torch, np.zeros((0, 1))), i32(torch, [])), KV8Batch(i32(torch, s.table), i32(torch, [5]), i32(torch, [0, 0]), 0)):
        s.cache.append(0, z, z, b)
        assert s.cache.read(0, b)[0].shape == (0, 1, 16)
        assert s.cache.attention(0, z, b).shape == (0, 1, 16)
    assert s.cache.status() == 0


def test_layers_and_offsets_past_32_bits(torch):
    """The last pages of a 2-layer cache of 4.5 GB a side: byte offsets beyond 2^32."""
    from scratch_decoder_only_b200.kv8 import KV8Batch, KV8Cache
    n, heads, page, d = 17200, 8, 128, 128
    c = KV8Cache.empty(2, n, heads, d, page=page, kind="int8", n_rows=1, max_pages=4)
    table = np.array([[n - 1, n - 3, 0]], np.int32)
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(300, heads, d, generator=g).to(torch.bfloat16) for _ in range(2))
    b = KV8Batch(i32(torch, table), i32(torch, [300]), i32(torch, [0, 300]), 300)
    c.append(1, k.cuda(), v.cuda(), b)
    assert not c.k[0].view(torch.uint8).any() and not c.k[1, 1:n - 3].view(torch.uint8).any()
    rk, rv = c.read(1, b)
    for got, x in ((rk, k), (rv, v)):
        # half a step of the scale (at most the largest value / 127) and one rounding to bf16
        a = x.float().abs().max()
        assert ((got.float().cpu() - x.float()).abs() <= a / 254 * 1.001 + x.float().abs() * 2.0 ** -7).all()
    q = torch.randn(300, heads, d, generator=g).to(torch.bfloat16)
    out = c.attention(1, q.cuda(), b)
    kk, vv = rk.double().cpu().numpy(), rv.double().cpu().numpy()
    o, _, mag, dot = R.attention(q[-2:].double().numpy(), kk, vv, [299, 300], d ** -0.5)
    # the read-back keys and values carry another rounding: 2^-8 of each product and value
    lim = bound(o, mag, dot, 300, d, "bf16") + mag * (2.0 ** -8 + 2 * 2.0 ** -8 * dot[..., None])
    assert np.all(np.abs(out[-2:].double().cpu().numpy() - o) <= lim)
    assert c.status() == 0


def test_graph_replay_and_streams(torch):
    """A captured append + attention follows the lengths and tables that the
    replay finds; eager calls on another stream at the same time do not disturb it."""
    from scratch_decoder_only_b200.kv8 import KV8Batch, KV8Cache
    g = torch.Generator(device="cuda").manual_seed(1)
    heads, d, B = 4, 64, 6
    def fresh():
        c = KV8Cache.empty(1, 600, heads, d, page=16, n_rows=B, max_pages=80)
        lens = i32(torch, [1, 100, 513, 40, 1200, 17])
        c.extend(lens)
        x = torch.randn(int(lens.sum()), heads, d, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").to(torch.bfloat16)
        c.append(0, x, -x, c.batch(i32(torch, starts(lens.cpu().numpy())), x.shape[0]))
        return c
    xs = torch.randn(5, B, heads, d, generator=g, device="cuda").to(torch.bfloat16)
    one = torch.ones(B, dtype=torch.int32, device="cuda")
    def step(c, b, x):
        c.extend(one)
        c.append(0, x, x, b)
        return c.attention(0, x, b)
    c = fresh()
    b = c.batch()
    want = [step(c, b, x).clone() for x in xs]
    e = fresh()
    be, buf = e.batch(), torch.empty_like(xs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            out = step(e, be, buf)
    torch.cuda.synchronize()
    other = fresh()
    ob = other.batch()
    torch.cuda.synchronize()
    for i, x in enumerate(xs):
        with torch.cuda.stream(side):
            buf.copy_(x)
            graph.replay()
            got = out.clone()
        o2 = step(other, ob, x)          # the default stream, unordered with `side`
        torch.cuda.synchronize()
        assert torch.equal(got, want[i]) and torch.equal(o2, want[i]), i
    assert c.status() == 0 and e.status() == 0 and other.status() == 0


# ---- pages

def pool_state(c):
    return c.table.cpu().numpy(), c.lens.cpu().numpy(), c.ref.cpu().numpy()


def same_pool(c, p):
    for got, want in zip(pool_state(c), (p.t, p.lens, p.ref)):
        assert np.array_equal(got, want)


def stamp(torch, c, rng):
    """Random bytes in every page, so that each copy shows."""
    for t in (c.k, c.v):
        u = t.view(torch.uint8)
        u.copy_(torch.from_numpy(rng.integers(0, 120, size=u.shape, dtype=np.uint8)).cuda())
    for t in (c.k_scale, c.v_scale):
        t.copy_(torch.from_numpy(rng.random(t.shape, dtype=np.float32)).cuda())


def buffers(torch, c):
    return [t.view(torch.uint8).cpu().numpy().copy() if t.dtype != torch.float32 else t.cpu().numpy().copy()
            for t in (c.k, c.v, c.k_scale, c.v_scale)]


@pytest.mark.parametrize("rows,max_pages,pages,page,heads,d,layers", [
    (1, 1, 1, 16, 1, 16, 1), (5, 7, 20, 16, 3, 32, 2), (40, 12, 333, 32, 2, 64, 3), (9, 40, 261, 64, 8, 64, 1),
    (3, 5, 9, 128, 5, 128, 2)])
def test_pages_against_plain_form(torch, rows, max_pages, pages, page, heads, d, layers):
    """Random calls of all kinds, bad arguments among them, each compared."""
    from scratch_decoder_only_b200.kv8 import KV8Cache
    rng = np.random.default_rng(rows * pages)
    c = KV8Cache.empty(layers, pages, heads, d, page=page, kind="e4m3", n_rows=rows, max_pages=max_pages)
    p = R.Pool(rows, max_pages, pages, page)
    stamp(torch, c, rng)
    bufs = buffers(torch, c)
    for step in range(60):
        what = rng.choice(["extend", "extend", "fork", "free", "compact"])
        bits = 0
        if what == "extend":
            add = rng.integers(0, 2 * page, size=rows) * (rng.random(rows) < 0.5)
            if rng.random() < 0.2:
                add[rng.integers(rows)] = rng.choice([-1, max_pages * page + 1, 2 ** 31 - 1])
            c.extend(i32(torch, add))
            bits = p.extend(add.astype(np.int64))
        elif what == "fork":
            n = int(rng.integers(1, 8))
            src, dst = rng.integers(0, rows, size=n), rng.integers(0, rows, size=n)
            if rng.random() < 0.2:
                src[0], dst[-1] = rng.choice([-1, rows]), rng.choice([-7, rows, 10 ** 9])
            got = c.fork(i32(torch, src), i32(torch, dst))
            done, copies, bits = p.fork(src, dst)
            assert np.array_equal(got.cpu().numpy(), done), step
            for a, z in copies:
                for t in bufs:
                    t[:, z] = t[:, a]
        elif what == "free":
            ids = rng.integers(0, rows, size=int(rng.integers(1, 4)))
            if rng.random() < 0.2:
                ids[0] = rng.choice([-1, rows])
            c.free(i32(torch, ids))
            bits = p.free(ids)
        else:
            n, copies = p.compact()
            assert int(c.compact()) == n
            for a, z in copies:
                for t in bufs:
                    t[:, z] = t[:, a]
        same_pool(c, p)
        assert c.status() == bits, (step, what)
        for got, want in zip(buffers(torch, c), bufs):
            assert np.array_equal(got, want), (step, what)


def test_pages_of_a_large_pool(torch):
    """More rows than threads of a block and more pages than one pass of its
    threads over their slice: the ranks carry over; then the pool runs out."""
    from scratch_decoder_only_b200.kv8 import KV8Cache
    rng = np.random.default_rng(4)
    rows, max_pages, pages = 2500, 64, 70001
    c = KV8Cache.empty(1, pages, 1, 16, page=16, n_rows=rows, max_pages=max_pages)
    p = R.Pool(rows, max_pages, pages, 16)
    for _ in range(3):
        add = rng.integers(0, 400, size=rows)
        c.extend(i32(torch, add))
        bits = p.extend(add)
        same_pool(c, p)
        assert c.status() == bits
        out = np.unique(rng.integers(0, rows, size=rows // 2))
        c.free(i32(torch, out))
        p.free(out)
        same_pool(c, p)
    empty = np.nonzero(p.lens == 0)[0]
    src = rng.integers(0, rows, size=len(empty))
    got = c.fork(i32(torch, src), i32(torch, empty))
    done, _, bits = p.fork(src, empty)
    assert np.array_equal(got.cpu().numpy(), done) and c.status() == bits
    same_pool(c, p)
    n, _ = p.compact()
    assert int(c.compact()) == n
    same_pool(c, p)
    add = np.full(rows, 1000)
    c.extend(i32(torch, add))
    assert p.extend(add) == c.status() != 0
    same_pool(c, p)


def test_pages_of_the_most_rows(torch):
    """16384 rows: as much shared memory as a call can ask for."""
    from scratch_decoder_only_b200.kv8 import KV8Cache
    rng = np.random.default_rng(6)
    rows, pages = 16384, 40009
    c = KV8Cache.empty(1, pages, 1, 16, page=16, n_rows=rows, max_pages=5)
    p = R.Pool(rows, 5, pages, 16)
    for _ in range(2):
        add = rng.integers(0, 40, size=rows)
        c.extend(i32(torch, add))
        assert p.extend(add) == c.status()
        same_pool(c, p)
        out = np.unique(rng.integers(0, rows, size=rows))
        c.free(i32(torch, out))
        p.free(out)
    empty = np.nonzero(p.lens == 0)[0]
    src = rng.integers(0, rows, size=len(empty))
    got = c.fork(i32(torch, src), i32(torch, empty))
    done, _, bits = p.fork(src, empty)
    assert np.array_equal(got.cpu().numpy(), done) and c.status() == bits
    same_pool(c, p)


def test_python_refusals(torch):
    """What the binding refuses before a call."""
    from scratch_decoder_only_b200.kv8 import KV8Batch, KV8Cache, KV8Pool
    c = KV8Cache.empty(1, 8, 2, 64, n_rows=3, max_pages=4)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    b = c.batch()
    bad = [lambda: c.append(0, x.float(), x.float()), lambda: c.append(0, x, x.half()), lambda: c.append(0, x[:2], x[:2]),
           lambda: c.append(0, x.cpu(), x), lambda: c.append(0, x.transpose(0, 1).contiguous().transpose(0, 1), x),
           lambda: c.append(0, x[:, :, ::2], x), lambda: c.attention(0, x[0, 0], b), lambda: c.attention(0, x, b, out=x[:1]),
           lambda: c.attention(0, x, b, out=torch.zeros_like(x).half()), lambda: c.read(0, b, torch.float32),
           lambda: KV8Batch(c.table, c.lens[:2]), lambda: KV8Batch(c.table, c.lens, c.lens), lambda: KV8Batch(c.table.long(), c.lens),
           lambda: KV8Batch(c.table, c.lens, rows=4), lambda: KV8Batch(c.table.cpu(), c.lens),
           lambda: KV8Cache(c.k, c.v[:, :4], c.k_scale, c.v_scale), lambda: KV8Cache(c.k.cpu(), c.v.cpu(), c.k_scale, c.v_scale),
           lambda: KV8Cache(c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale, c.v_scale),
           lambda: KV8Cache(c.k, c.v, c.k_scale.half(), c.v_scale), lambda: KV8Cache(c.k, c.v, c.k_scale, c.v_scale).batch(),
           lambda: KV8Cache(c.k, c.v, c.k_scale, c.v_scale).compact(), lambda: KV8Cache(c.k, c.v, c.k_scale, c.v_scale, c.table, c.lens, c.ref[:4]),
           lambda: c.extend(c.lens[:2]), lambda: c.extend(c.lens.long()), lambda: c.fork(c.lens, c.lens[:1]), lambda: c.free(c.lens.cpu()),
           lambda: KV8Pool(c.table, c.lens[:1], c.ref, 16)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    from scratch_decoder_only_b200.gpt import GPTError
    for f in (lambda: c.append(1, x, x), lambda: c.attention(0, torch.zeros(3, 3, 64, dtype=torch.bfloat16, device="cuda"), b),
              lambda: c.attention(0, x, b, scale=float("nan"))):
        with pytest.raises(GPTError):
            f()
    assert c.status() == 0 and not c.k.view(torch.uint8).any()


def test_free_of_pages_nobody_holds(torch):
    """A table that names a free page, one outside the pool or one page twice:
    reference counts do not fall below zero."""
    from scratch_decoder_only_b200.kv8 import KV8Cache
    c = KV8Cache.empty(1, 8, 1, 16, page=16, n_rows=2, max_pages=4)
    c.table.copy_(i32(torch, [[3, 99, 3, -1], [-1] * 4]))
    c.lens.copy_(i32(torch, [48, 0]))
    c.ref[3] = 1
    c.free(i32(torch, [0, 1, 0]))
    assert c.status() == 32 and not c.ref.any() and not c.lens.any() and bool((c.table == -1).all())


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_serving_run(torch, kind):
    """Prompts in, forked into continuations that then differ, one finished,
    the pool compacted in between: every step's attention equals that of a cache
    of its own per sequence which saw the same tokens."""
    from scratch_decoder_only_b200.kv8 import KV8Batch, KV8Cache
    heads, G, d, P, L = 2, 2, 64, 16, 2
    g = torch.Generator(device="cuda").manual_seed(11)
    rnd = lambda *n: torch.randn(*n, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    c = KV8Cache.empty(L, 64, heads, d, page=P, kind=kind, n_rows=7, max_pages=8)
    prompts = [37, 16]
    c.extend(i32(torch, prompts + [0] * 5))
    x = rnd(L, 2, sum(prompts), heads, d)
    b = KV8Batch(c.table[:2], c.lens[:2], i32(torch, starts(prompts)), sum(prompts))
    for layer in range(L):
        c.append(layer, x[layer, 0], x[layer, 1], b)
    parent = [0, 1, 0, 0, 1, 1, 0]
    c.fork(i32(torch, parent[2:]), i32(torch, [2, 3, 4, 5, 6]))
    own = [KV8Cache.empty(L, 8, heads, d, page=P, kind=kind, n_rows=1, max_pages=8) for _ in parent]
    at = starts(prompts)
    for r, a in enumerate(parent):
        own[r].extend(i32(torch, [prompts[a]]))
        for layer in range(L):
            own[r].append(layer, *(x[layer, w, at[a]:at[a + 1]] for w in (0, 1)), own[r].batch(i32(torch, [0, prompts[a]]), prompts[a]))
    alive = list(range(7))
    for step in range(24):
        if step == 9:
            c.free(i32(torch, [2, 1]))
            alive = [0, 3, 4, 5, 6]
        if step == 12:
            assert int(c.compact()) == int((c.ref > 0).sum())
            assert int((c.ref[:int((c.ref > 0).sum())] == 0).sum()) == 0
        add = np.zeros(7, np.int32)
        add[alive] = 1
        c.extend(i32(torch, add))
        rows = torch.tensor(alive, device="cuda")
        one = KV8Batch(c.table[rows], c.lens[rows])
        y = rnd(L, 3, len(alive), heads * G, d)
        for layer in range(L):
            k, v, q = y[layer, 0][:, :heads].contiguous(), y[layer, 1][:, :heads].contiguous(), y[layer, 2]
            c.append(layer, k, v, one)
            out = c.attention(layer, q, one)
            for j, r in enumerate(alive):
                if layer == 0:
                    own[r].extend(i32(torch, [1]))
                own[r].append(layer, k[j:j + 1], v[j:j + 1])
                assert torch.equal(own[r].attention(layer, q[j:j + 1])[0], out[j]), (step, layer, r)
    assert c.status() == 0 and all(o.status() == 0 for o in own)
    c.free(i32(torch, alive))
    assert not c.ref.any() and not c.lens.any()
