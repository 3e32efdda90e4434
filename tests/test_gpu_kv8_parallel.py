"""Parallel sampling over the 8-bit paged cache: the memory it takes, large
batches, and its tokens against the oracle with keys and values quantised as the
cache quantises them."""
import numpy as np
import pytest

from scratch_decoder_only_b200 import configs as CF

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available()
    return t


def test_cache_is_as_large_as_a_call_can_need(torch):
    """A call has 32 rows at most, whatever max_batch is: 2 * layers * 32 * max_seq * heads * head size bytes of codes,
    an eighth of that and more for scales and the rest, and what the first launch of a kernel takes (below 64 MB)."""
    from scratch_decoder_only_b200.gpt import GPT
    mc = CF.ModelConfig(vocab=200, vocab_padded=256, d_model=128, n_heads=2, d_mlp=128, n_layers=2, max_seq=8192, max_batch=128,
                        tied=True, precision="bf16")
    m = GPT(mc, 1)
    prompt = torch.randint(0, 200, (1, 20), dtype=torch.int32, device="cuda")
    uni = torch.rand(1, 4, 3, device="cuda")
    m.sample_decode(prompt, 3, uni[:, 0].contiguous())
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    m.sample_parallel(prompt, 3, 4, uni)
    torch.cuda.synchronize()
    took = before - torch.cuda.mem_get_info()[0]
    codes = 2 * 2 * 32 * 8192 * 128
    assert took <= codes * 1.125 + (64 << 20), took
    assert m.status() == 0


def test_models_of_many_rows(torch):
    """max_batch beyond what a page pool has rows for: a call's own rows are what counts."""
    from scratch_decoder_only_b200.gpt import GPT
    mc = CF.ModelConfig(vocab=60, vocab_padded=64, d_model=32, n_heads=2, d_mlp=64, n_layers=1, max_seq=24, max_batch=16500,
                        tied=True, precision="bf16")
    few = CF.ModelConfig(**{**mc.__dict__, "max_batch": 32})
    prompt = torch.randint(0, 60, (4, 9), dtype=torch.int32, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    uni = torch.rand(4, 8, 12, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    out = []
    for c in (mc, few):
        m = GPT(c, 3)
        out.append(m.sample_parallel(prompt, 12, 8, uni))
        assert m.status() == 0
    assert torch.equal(*out)


GPT2 = dict(vocab=500, vocab_padded=512, d_model=128, n_heads=2, d_mlp=512, n_layers=2, max_seq=96, max_batch=12,
            tied=True, precision="fp16", init_std=0.3)
LLAMA = dict(GPT2, arch="llama", d_model=256, n_heads=4, n_kv_heads=2)
SMALL = dict(GPT2, d_model=96, n_heads=6, tied=False)          # heads of 16


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("spec,B,n,Tp,n_new", [(GPT2, 2, 5, 21, 12), (GPT2, 3, 1, 16, 20), (LLAMA, 1, 12, 33, 9),
                                               (LLAMA, 4, 3, 1, 18), (SMALL, 2, 4, 40, 1), (SMALL, 1, 3, 64, 33)])
def test_tokens_follow_the_quantised_cache(torch, kind, spec, B, n, Tp, n_new):
    """Every token is one that logits near the oracle's draw with its uniform, the oracle's keys and values quantised as
    the cache quantises them (the bound and what it rejects: tests/kv8_oracle.py, tests/test_kv8_oracle_cpu.py).
    Greedy: a logit within the bound of the largest."""
    from tests import kv8_oracle as K
    from tests.test_gpu_kv8_decode import dev, make
    mc, cfg, model, params = make(torch, spec, 3 + Tp)
    rng = np.random.default_rng(100 + Tp)
    prompt = rng.integers(0, mc.vocab, size=(B, Tp)).astype(np.int32)
    uni = rng.random((B, n, n_new)).astype(np.float32)
    temp = 0.9
    out = model.sample_parallel(dev(torch, prompt), n_new, n, dev(torch, uni), temp, 0, 1.0, kind=kind).cpu().numpy()
    greedy = model.sample_parallel(dev(torch, prompt), n_new, n, dev(torch, uni), 0.0, kind=kind).cpu().numpy()
    assert model.status() == 0, model.last_error()
    assert out.min() >= 0 and out.max() < mc.vocab
    for b in range(B):
        z = K.logits(cfg, params, prompt[b], out[b], kind)
        bad = K.unlike(z, out[b], uni[b].astype(np.float64), temp, K.SPREAD[kind])
        assert not bad.any(), (b, np.argwhere(bad))
        if out[b].size >= 48:
            # the same tokens against another position's logits: the check would see it
            assert K.unlike(np.roll(z, 1, axis=1), out[b], uni[b].astype(np.float64), temp, K.SPREAD[kind]).sum() >= 2
        z = K.logits(cfg, params, prompt[b], greedy[b], kind)
        got = np.take_along_axis(z, greedy[b][..., None].astype(np.int64), -1)[..., 0]
        assert np.all(got >= z.max(-1) - 2 * K.SPREAD[kind] * z.std(-1)), b
