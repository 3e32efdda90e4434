"""Parallel sampling over the 8-bit paged cache (gpt_sample_parallel) against the
oracle: for every token the oracle computes the logits of the sequence that the
GPU generated (full prefix, no cache, fp64 on the 16-bit-rounded weights).

The GPU's logits differ from those by the model's 16-bit arithmetic (about 1 % of
a logit's spread over the vocabulary for two layers) and by the codes: an int8
code is off by up to 1/254 of its page's largest value, 0.75 % of a typical key
or value for pages of 16 x 64 normal values (largest about 3.3 standard
deviations); an e4m3 one by up to 2^-4 of itself, 2.6 % in the mean square.  Two
layers of keys and values each, added as independent errors and taken three
times over: 5 % of the spread for int8 and 16 % for e4m3."""
import numpy as np
import pytest

from oracle import gpt_oracle as O
from scratch_decoder_only_b200 import configs as CF
from tests.helpers import ocfg, tame_attention

pytestmark = pytest.mark.gpu

SPREAD = {"int8": 0.05, "e4m3": 0.16}
GPT2 = dict(vocab=500, vocab_padded=512, d_model=128, n_heads=2, d_mlp=512, n_layers=2, max_seq=96, max_batch=12,
            tied=True, precision="bf16", init_std=0.3)
LLAMA = dict(GPT2, arch="llama", d_model=256, n_heads=4, n_kv_heads=2, precision="fp16")
SMALL = dict(GPT2, d_model=96, n_heads=6, tied=False)          # heads of 16


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available()
    return t


def dev(torch, a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def make(torch, spec, seed):
    from scratch_decoder_only_b200.gpt import GPT
    mc = CF.ModelConfig(**spec)
    cfg = ocfg(mc)
    model = GPT(mc, seed)
    p32 = tame_attention(model, cfg)
    t = torch.from_numpy(p32).to(torch.bfloat16 if mc.precision == "bf16" else torch.float16)
    return mc, cfg, model, t.double().numpy()


def check(cfg, params, prompt, out, uni, temp, k, p, spread):
    """Every token is the one that the oracle draws with its uniform moved by at
    most the shift of the distribution that logits off by `spread` of their
    standard deviation make (greedy: within twice that of the largest)."""
    B, n, n_new = out.shape
    moved = 0
    for b in range(B):
        seq = np.concatenate([np.repeat(prompt[b:b + 1], n, axis=0), out[b, :, :-1]], axis=1)
        z, _ = O.forward(cfg, params, seq)
        z = z.reshape(n, seq.shape[1], -1)[:, prompt.shape[1] - 1:, :cfg.vocab]
        for i in range(n):
            for s in range(n_new):
                row, got = z[i, s], int(out[b, i, s])
                off = spread * row.std()
                if temp == 0.0:
                    assert row[got] >= row.max() - 2 * off, (b, i, s)
                    continue
                u, off = float(uni[b, i, s]), off / temp
                want = O.sample_token(row, cfg.vocab, temp, k, p, u)
                if got == want:
                    continue
                moved += 1
                lo, hi = (O.sample_token(row, cfg.vocab, temp, k, p, min(max(u + d, 0.0), 1 - 1e-12)) for d in (-off, off))
                assert lo <= got <= hi, (b, i, s, got, want, u)
    return moved


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("spec,B,n,Tp,n_new", [(GPT2, 2, 5, 21, 12), (GPT2, 3, 1, 16, 20), (LLAMA, 1, 12, 33, 9),
                                               (LLAMA, 4, 3, 1, 18), (SMALL, 2, 4, 40, 1), (SMALL, 1, 3, 64, 33)])
def test_parallel_samples_match_oracle(torch, kind, spec, B, n, Tp, n_new):
    mc, cfg, model, params = make(torch, spec, 3 + Tp)
    rng = np.random.default_rng(Tp)
    prompt = rng.integers(0, mc.vocab, size=(B, Tp)).astype(np.int32)
    uni = rng.random((B, n, n_new)).astype(np.float32)
    out = model.sample_parallel(dev(torch, prompt), n_new, n, dev(torch, uni), 0.9, 0, 1.0, kind=kind)
    assert model.status() == 0, model.last_error()
    out = out.cpu().numpy()
    assert out.min() >= 0 and out.max() < mc.vocab
    moved = check(cfg, params, prompt, out, uni, 0.9, 0, 1.0, SPREAD[kind])
    # most draws are far from a border of their distribution
    assert moved <= 0.5 * out.size
    greedy = model.sample_parallel(dev(torch, prompt), n_new, n, dev(torch, uni), 0.0, kind=kind).cpu().numpy()
    assert np.all(greedy == greedy[:, :1])          # the continuations of a prompt read the same cache
    check(cfg, params, prompt, greedy, uni, 0.0, 0, 1.0, SPREAD[kind])
    assert model.status() == 0


def test_other_decoding_is_unchanged_and_calls_repeat(torch):
    """Greedy, sampled and beam decoding give the same before and after, also
    between two parallel calls; the same call twice gives the same tokens, with
    other kinds and shapes between them."""
    mc, cfg, model, _ = make(torch, GPT2, 5)
    rng = np.random.default_rng(1)
    prompt = dev(torch, rng.integers(0, mc.vocab, size=(2, 19)).astype(np.int32))
    uni = dev(torch, rng.random((2, 4, 15)).astype(np.float32))

    def others():
        return [model.greedy_decode(prompt, 15).clone(), model.sample_decode(prompt, 15, uni[:, 0].contiguous(), 0.8, 30, 0.9),
                *model.beam_decode(prompt, 8, 4)]
    first = others()
    a = model.sample_parallel(prompt, 15, 4, uni, 0.8, 30, 0.9)
    second = others()
    model.sample_parallel(prompt, 15, 4, uni, 0.8, 30, 0.9, kind="e4m3")
    model.sample_parallel(prompt[:1].contiguous(), 3, 7, dev(torch, rng.random((1, 7, 3)).astype(np.float32)))
    b = model.sample_parallel(prompt, 15, 4, uni, 0.8, 30, 0.9)
    assert torch.equal(a, b)
    assert all(torch.equal(x, y) for x, y in zip(first, second))
    # one sample each, drawn with the same numbers as the first of four
    one = model.sample_parallel(prompt, 15, 1, uni[:, :1].contiguous(), 0.8, 30, 0.9)
    assert (one[:, 0] == a[:, 0]).float().mean() > 0.5
    assert model.status() == 0


def test_refusals(torch):
    from scratch_decoder_only_b200.gpt import GPT, GPT_ERR_ARG, GPT_ERR_STATE, GPTError
    mc, cfg, model, _ = make(torch, GPT2, 5)
    prompt = torch.zeros((2, 10), dtype=torch.int32, device="cuda")
    uni = torch.zeros((2, 8, 100), device="cuda")
    for args, kw, code in (((4, 7, uni), {}, GPT_ERR_ARG), ((0, 2, uni), {}, GPT_ERR_ARG), ((4, 0, uni), {}, GPT_ERR_ARG),
                           ((88, 2, uni), {}, GPT_ERR_STATE), ((4, 2, uni), dict(temperature=-1.0), GPT_ERR_ARG),
                           ((4, 2, uni), dict(top_p=0.0), GPT_ERR_ARG), ((4, 2, None), {}, GPT_ERR_ARG)):
        with pytest.raises(GPTError) as e:
            model.sample_parallel(prompt, *args, **kw)
        assert e.value.code == code and str(e.value)
    with pytest.raises(ValueError):
        model.sample_parallel(prompt, 4, 2, uni, kind="fp8")
    fp32 = GPT(CF.TINY_BYTE.model, 1)
    with pytest.raises(GPTError) as e:
        fp32.sample_parallel(prompt, 4, 2, uni)
    assert e.value.code == GPT_ERR_ARG
    assert model.status() == 0 and fp32.status() == 0
