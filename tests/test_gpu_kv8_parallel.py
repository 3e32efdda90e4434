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
