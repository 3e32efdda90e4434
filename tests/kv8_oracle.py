"""The oracle's model with keys and values as the 8-bit paged cache holds them,
for the tests of parallel sampling, and the check of drawn tokens against it.

Each key and value is rounded to the model's 16 bits and then quantised by the
plain form in tests/kv8_ref.py, page by page as the decoding appends them; a
token behind the prompt reads the codes as they are once it is appended, the
prompt's own tokens read 16-bit keys and values.  What is left between these
logits and the GPU's is the 16-bit arithmetic, and the codes that it tips over a
rounding border.

How far a logit may be off, in fp16 (`SPREAD`, in standard deviations of the
row's logits).  A few roundings of 2^-11 (rms 2^-11 / sqrt 3 each) leave keys and
values 0.1 % off.  A code flips with a chance of that difference over the code's
step and is then a step off, so the mean square is difference x step: with steps
of 9 % of the value (e4m3) and 1/127 of a page's largest, 2.6 % of a typical
value (int8), 0.85 % and 0.46 % in the root mean square.  Keys and values of two
layers added as independent errors, three times over: 5 % and 2.8 %, and 0.5 % for
three times the arithmetic's own 0.15 %."""
import numpy as np

from oracle import gpt_oracle as O
from tests import kv8_ref as R

PAGE = 16
SPREAD = {"int8": 0.035, "e4m3": 0.055}


def cached_attention(kind, Tp, mistake=None):
    """In place of the oracle's attention [rows, heads, T, d].  `mistake` plants one, to show that the check sees it."""
    def f(q, k, v, seg):
        n, H, T, d = q.shape
        q, k, v = (x.astype(np.float16).astype(np.float64) for x in (q, k, v))
        o = np.empty_like(q)
        pages = -(-T // PAGE)
        for r in range(n):
            p = O.attention_probs(q[r][:, :Tp], k[r][:, :Tp], O.allowed_mask(np.zeros(Tp, int)))
            o[r][:, :Tp] = p @ v[r][:, :Tp]
            ref = R.Ref(kind, pages, H, PAGE, d)
            rows = [x[r].transpose(1, 0, 2).astype(np.float32) for x in (k, v)]
            ref.append(np.arange(pages), Tp, [x[:Tp] for x in rows])
            if mistake == "last page not copied" and r % 2 and Tp % PAGE:
                for w in range(2):
                    ref.c[w][Tp // PAGE] = 0
            for t in range(Tp, T):
                ref.append(np.arange(pages), t + 1, [x[t:t + 1] for x in rows])
                kk, vv = (R.value(ref.c[w], kind) * ref.s[w][:, :, None, None].astype(np.float64) for w in range(2))
                kk, vv = (x.transpose(1, 0, 2, 3).reshape(H, pages * PAGE, d)[:, :t + 1] for x in (kk, vv))
                if mistake == "newest token not seen":
                    kk, vv = kk[:, :-1], vv[:, :-1]
                if mistake == "keys of the page before":
                    kk = np.roll(kk, PAGE, axis=1)
                s = np.einsum("hd,htd->ht", q[r][:, t], kk) / np.sqrt(d)
                o[r][:, t] = np.einsum("ht,htd->hd", O.softmax_rows(s), vv)
        return o
    return f


def logits(cfg, params, prompt, out, kind, mistake=None):
    """[n, n_new, vocab]: of one prompt [Tp] and its continuations out [n, n_new], the row that each token was drawn from."""
    n = out.shape[0]
    seq = np.concatenate([np.repeat(prompt[None], n, axis=0), out[:, :-1]], axis=1)
    plain = O.attention_fwd
    O.attention_fwd = cached_attention(kind, len(prompt), mistake)
    try:
        z, _ = O.forward(cfg, params, seq)
    finally:
        O.attention_fwd = plain
    return z.reshape(n, seq.shape[1], -1)[:, len(prompt) - 1:, :cfg.vocab]


def unlike(z, out, uni, temp, spread):
    """Draws [n, n_new] (bool) that no logits within `spread` standard deviations of z's explain.  Logits that differ by
    at most e (at this temperature) move the odds F / (1 - F) of a cumulated weight F by a factor of at most exp(2 e)."""
    x = z / temp
    e = spread * x.std(-1, keepdims=True)
    w = np.exp(x - x.max(-1, keepdims=True))
    c = np.cumsum(w, -1) / w.sum(-1, keepdims=True)
    before = np.concatenate([np.zeros_like(c[..., :1]), c[..., :-1]], -1)

    def moved(F, by):
        a, b = F * np.exp(by), (1 - F) * np.exp(-by)
        return a / (a + b)
    lo, hi = (np.take_along_axis(F, out[..., None].astype(np.int64), -1)[..., 0]
              for F in (moved(before, -e), moved(np.minimum(c, 1.0), e)))
    return (uni < lo - 1e-6) | (uni > hi + 1e-6)
