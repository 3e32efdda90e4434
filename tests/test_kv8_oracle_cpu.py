"""The check of parallel sampling's tokens (tests/kv8_oracle.py) accepts what the
oracle draws itself and rejects planted mistakes.  No GPU needed."""
import numpy as np
import pytest

from oracle import gpt_oracle as O
from scratch_decoder_only_b200 import configs as CF
from tests import kv8_oracle as K
from tests.helpers import ocfg

GPT2 = dict(vocab=500, vocab_padded=512, d_model=128, n_heads=2, d_mlp=512, n_layers=2, max_seq=96, max_batch=12,
            tied=True, precision="fp16", init_std=0.3)
LLAMA = dict(GPT2, arch="llama", d_model=256, n_heads=4, n_kv_heads=2)
TEMP = 0.9


def drawn(spec, kind, Tp, n, n_new):
    cfg = ocfg(CF.ModelConfig(**spec))
    flat = O.init_params(cfg, 3)
    P, C, kvd = O.unflatten(cfg, flat), cfg.d_model, cfg.kv_heads * cfg.head_dim
    for l in range(cfg.n_layers):
        P[f"h{l}.w_qkv"][:C + kvd] *= np.float32(0.25)      # as the GPU tests' models (tame_attention)
    params = flat.astype(np.float16).astype(np.float64)
    rng = np.random.default_rng(Tp)
    prompt, uni = rng.integers(0, cfg.vocab, size=Tp), rng.random((n, n_new))
    out = np.zeros((n, n_new), int)
    for s in range(n_new):
        z = K.logits(cfg, params, prompt, out[:, :s + 1], kind)[:, -1]
        out[:, s] = [O.sample_token(z[i], cfg.vocab, TEMP, 0, 1.0, float(uni[i, s])) for i in range(n)]
    return cfg, params, prompt, uni, out


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("spec", [GPT2, LLAMA])
def test_right_tokens_pass_and_planted_mistakes_do_not(spec, kind):
    cfg, params, prompt, uni, out = drawn(spec, kind, 21, 4, 12)
    z = K.logits(cfg, params, prompt, out, kind)
    bad = lambda z: int(K.unlike(z, out, uni, TEMP, K.SPREAD[kind]).sum())  # noqa: E731
    assert bad(z) == 0
    for mistake in ("last page not copied", "newest token not seen", "keys of the page before"):
        assert bad(K.logits(cfg, params, prompt, out, kind, mistake)) >= 2, mistake
    # logits of another row, and of the position before
    assert bad(np.roll(z, 1, axis=0)) >= 0.2 * out.size and bad(np.roll(z, 1, axis=1)) >= 0.2 * out.size
    # noise as large as the tolerance allows passes
    rng = np.random.default_rng(2)
    e = K.SPREAD[kind] * z.std(-1, keepdims=True)
    assert bad(z + e * rng.choice([-1.0, 1.0], size=z.shape)) == 0


def test_shift_of_a_distribution_is_bounded():
    """`unlike` allows exactly the draws that logits within the tolerance can make: the two that move a border most."""
    rng = np.random.default_rng(5)
    z = 2.0 * rng.standard_normal((1, 1, 50))
    e, t = 0.1 * z.std(), 20
    w = np.exp(z[0, 0])
    for sign in (-1, 1):
        d = np.where(np.arange(50) <= t, sign * e, -sign * e)
        F = (w * np.exp(d))[:t + 1].sum() / (w * np.exp(d)).sum()
        tok = np.array([[t if sign > 0 else t + 1]])      # the border above t, or below t + 1
        inside, outside = (F - 1e-4, F + 1e-4) if sign > 0 else (F + 1e-4, F - 1e-4)
        assert not K.unlike(z, tok, np.array([[inside]]), 1.0, 0.1).any()
        assert K.unlike(z, tok, np.array([[outside]]), 1.0, 0.1).all()
