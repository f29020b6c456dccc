"""Seeded random shapes of the target's operators against their plain definitions,
small enough to be replayed on the host; the prefix attention's workspaces in a
guarded buffer, and its cache in page-locked host memory and in pages of any
length."""
import random

import pytest
import torch

import test_gpu_distill as distill
import test_gpu_prefix_attention as prefix
import test_gpu_token_logprobs as logprobs
from test_gpu_serving_workspace import Guarded

pytestmark = pytest.mark.gpu

sv = pytest.importorskip("speculative_decoding_verification_vocab_gb300")
DEV = "cuda:0"
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.load_library()


@pytest.mark.parametrize("seed", range(40))
def test_prefix_attention(seed):
    rng = random.Random(seed)
    Hkv, G = rng.choice([1, 1, 2, 3, 8]), rng.choice([1, 2, 4, 7, 8, 16])
    D, page = rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 8, 12, 16, 16, 20, 33, 50, 64, 100, 128, 136, 256])
    N, W = rng.choice([1, 1, 2, 5, 40]), rng.choice([1, 2, 4, 17, 40])
    if N * W > 200:
        W = 2
    top = max(1, min(6000, 40000 // (N * Hkv)))
    plens = [rng.choice([0, 1, 127, 128, 129, top, rng.randint(0, top), rng.randint(0, top)]) for _ in range(N)]
    own = max(1, min(300, 20000 // (N * W * Hkv)))
    lens = [rng.choice([0, 1, own, rng.randint(0, own)]) for _ in range(N * W)]
    prefix.check(*prefix.make(plens, lens, Hkv * G, Hkv, D, page, rng.choice([torch.bfloat16, torch.float16]), seed,
                              sigma=rng.choice([0.5, 1.5, 4.0]), extra=rng.choice([0, 1, 9])))


@pytest.mark.parametrize("seed", range(40))
def test_token_logprobs(seed):
    rng = random.Random(1000 + seed)
    V = rng.choice([1, 2, 7, 8, 255, 1000, 4097, rng.randint(1, 9000), rng.randint(1, 150000)])
    B, T = rng.choice([1, 2, 3]), rng.choice([1, 2, 5])
    K = min(V, rng.choice([0, 1, 2, 5, 20, 64, 127, 128]))
    x, tokens = logprobs.make(B, T, V, rng.choice(TYPES), seed, pad=rng.choice([0, 0, 1, 8, 13]),
                              sigma=rng.choice([0.01, 1.0, 3.0, 10.0]))
    rows = None
    if rng.random() < 0.5:
        P = rng.choice([1, 3, 9])
        rows = torch.tensor([[rng.randint(-1, T - 1) for _ in range(P)] for _ in range(B)], dtype=torch.int32)
        tokens = torch.tensor([[rng.randint(-1, V - 1) for _ in range(P)] for _ in range(B)], dtype=torch.int32)
    if rng.random() < 0.3:
        tokens = None
    logprobs.check(x, tokens, rows, K, rng.choice([1.0, 0.3, 2.0]))


@pytest.mark.parametrize("seed", range(40))
def test_distill(seed):
    rng = random.Random(2000 + seed)
    V = rng.choice([1, 2, 7, 8, 255, 1000, 4097, rng.randint(1, 9000), rng.randint(1, 150000)])
    R, K = rng.choice([1, 2, 5, 9]), min(V, rng.choice([1, 2, 5, 20, 64, 127, 128]))
    T, tail, dtype = rng.choice([1.0, 0.5, 2.0]), rng.random() < 0.6, rng.choice(TYPES)
    x, token, value = distill.make(R, V, K, dtype, seed, pad=rng.choice([0, 0, 1, 8, 13]),
                                   noise=rng.choice([0.1, 1.0, 3.0]), T=T, sigma=rng.choice([0.1, 1.0, 3.0]))
    for r in range(R):                       # lists that are not full
        for i in range(rng.choice([0, 0, 1, K])):
            token[r, rng.randint(0, K - 1)] = -1
    w = torch.rand(R, generator=torch.Generator().manual_seed(seed)) if rng.random() < 0.5 else None
    distill.check(x, token, value, w, T, tail)


@pytest.mark.parametrize("fill", [0xFF, 0x00])
@pytest.mark.parametrize("plens,lens,Hq,Hkv,page,D", [
    ([1], [0], 1, 1, 16, 64),
    ([9000], [5, 0], 6, 1, 16, 128),                   # one prefix over the whole card
    ([700, 3], [40] * 64, 16, 4, 20, 64),              # pairs of query tiles
    ([400] * 20, [3] * 20, 8, 2, 32, 128),             # a query tile to a prefix
    ([90] * 3, [2000, 1, 700] * 2, 8, 2, 16, 64),      # own slots cut into shares
    ([50] * 70, [70] * 700, 2, 1, 16, 128),
])
def test_prefix_workspaces(plens, lens, Hq, Hkv, page, D, fill):
    """The bytes the query names are enough, none of them is read before the call
    has written it, and none beside them is written; the later calls' lengths are
    shorter than what the first left behind."""
    N, B = len(plens), len(lens)
    case = prefix.make(plens, lens, Hq, Hkv, D, page, seed=3)
    q, kv, pt, pl, t, n = case
    guard = Guarded(sv.sv_prefix_attention_workspace(B, N, Hq, Hkv, D, page, pt.shape[1], t.shape[1]), fill)
    for cut in (1, 3, 50):
        prefix.check(q, kv, pt, pl // cut, t, n // cut, workspace=guard.ws)
        guard.check_edges()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,W,Hkv,G", [
    (70, 3, 8, 3),        # nine rows to a segment: four, four and one
    (9, 43, 2, 3),        # 129: the second tile has one row
    (1, 259, 1, 9),       # 2331: ten columns, the last of one ragged tile
    (300, 1, 8, 1),       # one row to a segment
])
def test_prefix_many_rows(N, W, Hkv, G, D):
    rng = random.Random(N)
    plens = [rng.choice([0, 1, 40, 129, 300]) for _ in range(N - 1)] + [260]
    lens = [rng.choice([0, 1, 9, 30]) for _ in range(N * W)]
    prefix.check(*prefix.make(plens, lens, Hkv * G, Hkv, D, 16, torch.bfloat16, seed=N))


@pytest.mark.parametrize("page", [1, 4, 12, 16, 33, 50, 100, 128, 136])
@pytest.mark.parametrize("D", [64, 128])
def test_prefix_cache_in_host_memory(page, D):
    q, kv, pt, pl, t, n = prefix.make([500, 130], [20, 0, 1, 70], 8, 2, D, page, seed=page)
    dev = [x.to(DEV) for x in (q, pt, pl, t, n)]
    by_page = kv.transpose(0, 1).contiguous()
    for there in (kv.to(DEV), kv.pin_memory(), by_page.to(DEV).transpose(0, 1), by_page.pin_memory().transpose(0, 1)):
        out = sv.prefix_attention(dev[0], there, *dev[1:], return_lse=True)
        torch.cuda.synchronize()
        prefix.close(*out, q, kv, pt, pl, t, n, D ** -0.5)


def test_distill_in_place_at_the_largest_sizes():
    """In place where a row is cut over the most CTAs, and where the rows are many."""
    x, token, value = distill.make(2, sv.SV_MAX_VOCAB, 128, torch.float32, 1)
    distill.check(x, token, value, torch.tensor([0.5, 2.0]))
    # many rows, a CTA to each where a few rows have more: the same up to the order of
    # the sums, each off by `rel` of its share at most, and a step of the type
    V, K, n = 9001, 128, 3000
    x, token, value = distill.make(3, V, K, torch.bfloat16, 2)
    want = distill.check(x, token, value)
    big = distill.put(x).repeat(n, 1)
    tok, val = distill.put(token).repeat(n, 1), distill.put(value).repeat(n, 1)
    stat = sv.distill_loss(big, tok, val)["stat"]
    other = big.clone()
    r = sv.distill_loss(big, tok, val, out_grad=big)
    sv.distill_grad(other, tok, val, stat, out_grad=other)
    torch.cuda.synchronize()
    rel = 2.0 ** -24 * (3 * 48 + 4 + V / 512 + 24 + 8 + K)
    share = torch.softmax(x.double(), -1)
    share.scatter_add_(1, token.long(), value.double().exp())
    tol = 4 * rel * share + (torch.finfo(torch.bfloat16).eps + 2.0 ** -23) * want["grad"].double().cpu().abs()
    for g in (big, other):
        off = (g.view(n, 3, V).double() - want["grad"].double()).abs().amax(0).cpu()
        assert bool((off <= tol).all())
    assert float((r["loss"].view(n, 3) - want["loss"]).abs().max()) <= 4 * rel * 30


def test_nothing_to_do():
    """No sequences, entries or rows: nothing is launched, empty tensors come back."""
    i32 = dict(dtype=torch.int32, device=DEV)
    before = sv.sv_launch_count()
    kv = torch.zeros(2, 3, 16, 2, 64, dtype=torch.bfloat16, device=DEV)
    out, lse, st = sv.prefix_attention(torch.zeros(0, 4, 64, dtype=torch.bfloat16, device=DEV), kv, torch.zeros(1, 1, **i32),
                                       torch.zeros(1, **i32), torch.zeros(0, 1, **i32), torch.zeros(0, **i32), return_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4) and st.shape == (0,)
    x = torch.zeros(2, 3, 40, device=DEV)
    assert sv.token_logprobs(x[:0], top_k=4)["top_token"].shape == (0, 3, 4)
    assert sv.token_logprobs(x, torch.zeros(2, 0, **i32))["logprob"].shape == (2, 0)
    r = sv.distill_loss(x[0, :0], torch.zeros(0, 2, **i32), torch.zeros(0, 2, device=DEV), grad=True)
    assert r["loss"].shape == (0,) and r["grad"].shape == (0, 40)
    g, st = sv.distill_grad(x[0, :0], torch.zeros(0, 2, **i32), torch.zeros(0, 2, device=DEV), r["stat"])
    assert g.shape == (0, 40) and st.shape == (0,)
    torch.cuda.synchronize()
    assert sv.sv_launch_count() == before


def test_one_of_everything():
    """One sequence without a slot of its own or of a prefix, a vocabulary of one."""
    i32 = dict(dtype=torch.int32, device=DEV)
    kv = torch.full((2, 1, 1, 1, 128), float("nan"), dtype=torch.float16, device=DEV)
    out, lse, st = sv.prefix_attention(torch.ones(1, 1, 128, dtype=torch.float16, device=DEV), kv, torch.full((1, 1), 9, **i32),
                                       torch.zeros(1, **i32), torch.full((1, 1), -3, **i32), torch.zeros(1, **i32), return_lse=True)
    assert not bool(out.any()) and bool(torch.isneginf(lse).all()) and st.tolist() == [0]
    r = sv.token_logprobs(torch.full((1, 1, 1), 3e38, device=DEV), torch.zeros(1, 1, **i32), top_k=1)
    assert r["logprob"].tolist() == [[0.0]] and r["entropy"].tolist() == [[0.0]] and r["top_token"].tolist() == [[[0]]]
    for tail in (True, False):
        r = sv.distill_loss(torch.full((1, 1), -3e38, device=DEV), torch.zeros(1, 1, **i32), torch.zeros(1, 1, device=DEV),
                            tail=tail, grad=True)
        assert r["loss"].tolist() == [0.0] and r["grad"].tolist() == [[0.0]] and r["status"].tolist() == [0]
