"""Host side of the 8-bit paged cache: refusals before anything is enqueued, and
checks of the plain forms that the GPU tests compare with.  No GPU needed."""
import ctypes

import numpy as np
import pytest

from scratch_decoder_only_b200 import gpt as G
from tests import kv8_ref as R


@pytest.fixture(scope="module")
def lib():
    import os
    from scratch_decoder_only_b200 import build
    if not os.path.exists(G.LIB_PATH):
        build.build()
    return G.load_library()


# device addresses that no call of this file may come to use
def cache(**kw):
    d = dict(kind=0, n_layers=2, n_pages=10, n_kv_heads=2, head_dim=64, page=16, k=4096, v=8192, k_scale=64, v_scale=128)
    d.update(kw)
    return G.gpt_kv8_cache(**d)


def batch(**kw):
    d = dict(start=256, lens=512, table=1024, B=3, max_pages=4, ld_table=4, rows=5)
    d.update(kw)
    return G.gpt_kv8_batch(**d)


def pool(**kw):
    d = dict(table=1024, lens=512, ref=256, n_rows=3, max_pages=4, ld_table=4, n_pages=10, page=16)
    d.update(kw)
    return G.gpt_kv8_pool(**d)


BAD_CACHE = [dict(kind=2), dict(n_layers=0), dict(n_pages=0), dict(n_kv_heads=0), dict(n_kv_heads=2000),
             dict(head_dim=48), dict(head_dim=256), dict(page=8), dict(page=48), dict(page=256), dict(k=None), dict(v=None),
             dict(k_scale=None), dict(v_scale=None), dict(k=4104), dict(v=8193), dict(k_scale=66),
             dict(n_pages=2 ** 30, n_kv_heads=8, page=128, head_dim=128)]
BAD_BATCH = [dict(B=-1), dict(rows=-1), dict(max_pages=0), dict(ld_table=3), dict(lens=None), dict(table=None),
             dict(start=None), dict(max_pages=2 ** 28, ld_table=2 ** 28), dict(rows=2 ** 29)]
BAD_POOL = [dict(table=None), dict(lens=None), dict(ref=None), dict(n_rows=0), dict(n_rows=16385), dict(max_pages=0),
            dict(ld_table=3), dict(n_pages=0), dict(n_pages=2 ** 25), dict(page=20)]


def refused(lib, rc):
    assert rc == G.GPT_ERR_ARG
    assert lib.gpt_last_error(None).decode()


def calls(lib, c, b, layer=0, dtype=1, x=65536, ld=128, y=131072, heads=4, scale=0.125, ldq=256, work=1 << 20, nwork=1 << 30,
          lse=0):
    r = ctypes.byref
    c, b = c if c is None else r(c), b if b is None else r(b)
    yield lib.gpt_kv8_append(c, layer, b, x, ld, y, ld, dtype, None, None)
    yield lib.gpt_kv8_read(c, layer, b, x, ld, y, ld, dtype, None, None)
    yield lib.gpt_kv8_attention(c, layer, b, x, ldq, heads, dtype, scale, y, ldq, lse, work, nwork, None, None)


@pytest.mark.parametrize("bad", BAD_CACHE)
def test_bad_caches_are_refused(lib, bad):
    for rc in calls(lib, cache(**bad), batch()):
        refused(lib, rc)
    n = ctypes.c_size_t()
    if "k" not in bad and "v" not in bad and "k_scale" not in bad and "v_scale" not in bad:
        c = cache(**bad)
        refused(lib, lib.gpt_kv8_attention_work(ctypes.byref(c), ctypes.byref(batch()), 4, ctypes.byref(n)))
    p, c = pool(), cache(**bad)
    if "n_layers" not in bad:
        refused(lib, lib.gpt_kv8_fork(ctypes.byref(p), ctypes.byref(c), 64, 128, 1, 256, None, None))
        refused(lib, lib.gpt_kv8_compact(ctypes.byref(p), ctypes.byref(c), None, 256, None, None))


@pytest.mark.parametrize("bad", BAD_BATCH)
def test_bad_batches_are_refused(lib, bad):
    for rc in calls(lib, cache(), batch(**bad)):
        refused(lib, rc)


@pytest.mark.parametrize("bad", [dict(layer=2), dict(layer=-1), dict(dtype=0), dict(dtype=3), dict(x=None), dict(y=None),
                                 dict(x=65544), dict(y=131080), dict(ld=124, ldq=252), dict(ld=120, ldq=248)])
def test_bad_matrices_are_refused(lib, bad):
    for rc in calls(lib, cache(), batch(), **bad):
        refused(lib, rc)


@pytest.mark.parametrize("bad", [dict(heads=0), dict(heads=3), dict(heads=-2), dict(scale=float("inf")), dict(scale=float("nan")),
                                 dict(work=None), dict(work=1 << 20 | 8), dict(nwork=8), dict(lse=6)])
def test_bad_attention_calls_are_refused(lib, bad):
    # (rows long enough that scratch is needed)
    refused(lib, list(calls(lib, cache(), batch(max_pages=400, ld_table=400), **bad))[2])


def test_missing_descriptions_are_refused(lib):
    for c, b in ((None, batch()), (cache(), None)):
        for rc in calls(lib, c, b):
            refused(lib, rc)
    n = ctypes.c_size_t()
    refused(lib, lib.gpt_kv8_attention_work(None, ctypes.byref(batch()), 4, ctypes.byref(n)))
    refused(lib, lib.gpt_kv8_attention_work(ctypes.byref(cache()), None, 4, ctypes.byref(n)))
    refused(lib, lib.gpt_kv8_attention_work(ctypes.byref(cache()), ctypes.byref(batch()), 4, None))


@pytest.mark.parametrize("bad", BAD_POOL)
def test_bad_pools_are_refused(lib, bad):
    p, c = ctypes.byref(pool(**bad)), ctypes.byref(cache())
    refused(lib, lib.gpt_kv8_extend(p, 64, None, None))
    refused(lib, lib.gpt_kv8_free(p, 64, 1, None, None))
    refused(lib, lib.gpt_kv8_fork(p, c, 64, 128, 1, 256, None, None))
    refused(lib, lib.gpt_kv8_compact(p, c, None, 256, None, None))


def test_bad_page_calls_are_refused(lib):
    p, c = ctypes.byref(pool()), ctypes.byref(cache())
    refused(lib, lib.gpt_kv8_extend(p, None, None, None))
    refused(lib, lib.gpt_kv8_extend(None, 64, None, None))
    refused(lib, lib.gpt_kv8_free(p, None, 1, None, None))
    refused(lib, lib.gpt_kv8_free(p, 64, -1, None, None))
    for args in ((None, 128, 1, 256), (64, None, 1, 256), (64, 128, 1, None), (64, 128, -1, 256), (64, 128, 16385, 256)):
        refused(lib, lib.gpt_kv8_fork(p, c, *args, None, None))
    refused(lib, lib.gpt_kv8_compact(p, c, None, None, None, None))
    refused(lib, lib.gpt_kv8_compact(p, c, 4, 256, None, None))
    for other in (cache(n_pages=11), cache(page=32)):
        refused(lib, lib.gpt_kv8_fork(p, ctypes.byref(other), 64, 128, 1, 256, None, None))
        refused(lib, lib.gpt_kv8_compact(p, ctypes.byref(other), None, 256, None, None))


def test_empty_calls_enqueue_nothing(lib):
    """No rows or no requests: done, without a device."""
    for b in (batch(B=0, rows=0), batch(rows=0)):
        for rc in calls(lib, cache(), b, x=None, y=None):
            assert rc == G.GPT_OK
    p, c = ctypes.byref(pool()), ctypes.byref(cache())
    assert lib.gpt_kv8_free(p, None, 0, None, None) == G.GPT_OK
    assert lib.gpt_kv8_fork(p, c, None, None, 0, None, None, None) == G.GPT_OK


def test_scratch_is_asked_for_long_rows_only(lib):
    n = ctypes.c_size_t(1)
    def ask(pages, **kw):
        assert lib.gpt_kv8_attention_work(ctypes.byref(cache()), ctypes.byref(batch(max_pages=pages, ld_table=pages, **kw)), 4,
                                          ctypes.byref(n)) == G.GPT_OK
        return n.value
    assert ask(64) == 0                     # 1024 tokens: whole jobs
    assert 0 < ask(65) <= ask(4000)
    assert ask(4000) <= 64 << 20
    # a multiple that keeps the records behind the sums aligned
    assert ask(4000) % 16 == 0


def test_structs_match_the_header(tmp_path):
    import os
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    structs = {n: getattr(G, n) for n in ("gpt_kv8_cache", "gpt_kv8_batch", "gpt_kv8_pool")}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "gpt.h"', "int main(void) {"]
    for n, cls in structs.items():
        lines.append(f'  printf("%zu", sizeof({n}));')
        lines += [f'  printf(" %zu", offsetof({n}, {f}));' for f, _ in cls._fields_]
        lines.append('  printf("\\n");')
    src, exe = tmp_path / "l.c", tmp_path / "l"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    for line, cls in zip(subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines(), structs.values()):
        assert [int(x) for x in line.split()] == [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f, _ in cls._fields_]


# ---- the plain forms

def test_e4m3_codes_are_torchs():
    import torch
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, R.E4M3, equal_nan=True)
    x = np.concatenate([np.linspace(-448, 448, 4001), 2.0 ** np.linspace(-14, 8.8, 999), [0.0, -0.0, 2.0 ** -10, 3 * 2.0 ** -10]])
    x = x.astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.round_code(x, "e4m3"), want)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_plain_append_is_near_its_input(kind):
    rng = np.random.default_rng(0)
    r = R.Ref(kind, 6, 2, 16, 32)
    x = rng.standard_normal((37, 2, 32)).astype(np.float32)
    table = [4, 1, 3]
    at = 0
    for n in (5, 1, 1, 20, 10):
        at += n
        r.append(table, at, (x[at - n:at], x[at - n:at]))
    got = r.tokens(1, table, 37)
    s = r.s[1][table].repeat(16, 0)[:37, :, None]
    # a code rounded anew k times is off by k + 1 half steps at most (five appends)
    lim = 5 * s / 2 if kind == "int8" else 5 * np.maximum(np.abs(x) * 2.0 ** -4, s * 2.0 ** -10) * 1.1
    assert np.all(np.abs(got - x) <= lim)


def test_plain_pool_keeps_its_books():
    rng = np.random.default_rng(1)
    p = R.Pool(7, 6, 25, 16)
    for _ in range(300):
        what = rng.integers(4)
        if what == 0:
            p.extend(rng.integers(0, 30, size=7) * (rng.random(7) < 0.5))
        elif what == 1:
            p.fork(rng.integers(0, 7, size=3), rng.integers(0, 7, size=3))
        elif what == 2:
            p.free(rng.integers(0, 7, size=1))
        else:
            live, _ = p.compact()
            assert np.all(p.ref[:live] > 0) and not p.ref[live:].any()
        held = np.zeros(25, int)
        for r in range(7):
            n = p.count(p.lens[r])
            assert np.all(p.t[r, :n] >= 0) and len(set(p.t[r, :n])) == n
            np.add.at(held, p.t[r, :n], 1)
        assert np.array_equal(held, p.ref)
