"""Seeded random shapes of the serving operators against their plain
definitions: sizes, groupings, pages, windows, types, lengths and masks drawn
together, small enough to be replayed on the host."""
import random

import pytest
import torch

import test_gpu_kv_evict as evict
import test_gpu_paged_attention as paged
import test_gpu_verify_probs as probs

pytestmark = pytest.mark.gpu

sv = pytest.importorskip("speculative_decoding_verification_vocab_gb300")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.load_library()


@pytest.mark.parametrize("seed", range(60))
def test_paged_attention(seed):
    rng = random.Random(seed)
    Hkv, G = rng.choice([1, 1, 2, 3, 5, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 9, 12, 16, 17, 25])
    D, page = rng.choice([64, 64, 128, 256]), rng.choice([1, 3, 8, 16, 16, 20, 32, 48, 64, 100, 256])
    B = rng.choice([1, 1, 2, 3, 7, 20, 140])
    top = max(1, min(6000, 60000 // (B * Hkv)))
    lens = [rng.choice([0, 1, 15, 16, 17, 63, 64, 65, top, rng.randint(0, top), rng.randint(0, top)])
            for _ in range(B)]
    window = rng.choice([0, 0, 1, 5, 16, 100, 1000]) and rng.randint(1, max(1, top))
    sinks = rng.choice([0, 1, 4, 16, 33]) if window else 0
    q, kv, table, n = paged.make(lens, Hkv * G, Hkv, D, page, rng.choice([torch.bfloat16, torch.float16]),
                                 seed, window, sinks, extra_pages=rng.choice([0, 1, 40]),
                                 sigma=rng.choice([0.5, 1.5, 4.0]))
    paged.check(q, kv, table, n, window=window, sinks=sinks, weights=rng.random() < 0.5)


@pytest.mark.parametrize("seed", range(60))
def test_kv_evict(seed):
    rng = random.Random(1000 + seed)
    L, Hkv = rng.choice([1, 1, 2, 3]), rng.choice([1, 2, 3, 8])
    B = rng.choice([1, 2, 5, 17, 60])
    top = max(2, min(20000, 120000 // (L * Hkv * B)))
    lens = [rng.choice([0, 1, top, rng.randint(0, top), rng.randint(0, top)]) for _ in range(B)]
    budget = rng.choice([1, 2, top, top + 9, rng.randint(1, top), rng.randint(1, top)])
    sinks = rng.choice([0, 0, 1, min(4, budget), rng.randint(0, budget)])
    recent = rng.choice([0, 0, min(1, budget - sinks), budget - sinks, rng.randint(0, budget - sinks)])
    dtype, D = rng.choice([(torch.bfloat16, 64), (torch.bfloat16, 128), (torch.float16, 8), (torch.float32, 32),
                           (torch.float32, 5), (torch.int8, 64), (torch.int8, 12)])
    evict.check(*evict.make(L, lens, Hkv, D, rng.choice([1, 7, 16, 16, 64, 100]), dtype, seed,
                            zeros=rng.choice([0.0, 0.2, 0.95]), coarse=rng.random() < 0.4),
                budget, sinks, recent)


@pytest.mark.parametrize("seed", range(60))
def test_verify_probs(seed):
    rng = random.Random(2000 + seed)
    B, N = rng.choice([1, 2, 5, 33]), rng.choice([0, 1, 2, 3, 7, 31, 32, 33, 70])
    top = max(2, 600000 // (B * (N + 1)))
    V = rng.choice([1, 2, 7, 8, 9, 255, 256, 257, rng.randint(1, top), rng.randint(1, top)])
    args = probs.make(B, N, V, rng.choice([torch.float32, torch.bfloat16]), seed, rng.choice([0, 0, 1, 3, 8]),
                      rng.random() < 0.3, sigma=rng.choice([0.5, 2.0, 8.0]), noise=rng.choice([0.0, 0.1, 1.0, 4.0]))
    n = torch.tensor([rng.randint(0, N) for _ in range(B)], dtype=torch.int32) if rng.random() < 0.5 else None
    probs.check(*args, n)


@pytest.mark.parametrize("window", [1, 5, 16, 17, 100, 1000])
@pytest.mark.parametrize("seed", range(4))
def test_paged_attention_windows(window, seed):
    """Windows at the edges of a group and of a tile, against odd pages,
    groupings and first tokens."""
    rng = random.Random(3000 + 10 * window + seed)
    Hkv, G = rng.choice([1, 2, 3]), rng.choice([1, 3, 7, 16, 17])
    D, page = rng.choice([64, 128]), (1, 16, 20, 48)[seed]
    lens = [rng.choice([0, 1, window, window + 1, window + 15, window + 16, rng.randint(1, 2500)])
            for _ in range(rng.choice([1, 4, 40]))]
    sinks = rng.choice([0, 1, 15, 16, 33])
    q, kv, table, n = paged.make(lens, Hkv * G, Hkv, D, page, rng.choice([torch.bfloat16, torch.float16]),
                                 seed, window, sinks)
    paged.check(q, kv, table, n, window=window, sinks=sinks, weights=seed % 2 == 0)
