"""sv_token_logprobs against the plain definition in 64 bits
(tests/plain_target.py): tokens and status words equal, numbers within what 32
bits account for."""
import math

import numpy as np
import pytest
import torch

import plain_target as plain

pytestmark = pytest.mark.gpu

sv = pytest.importorskip("speculative_decoding_verification_vocab_gb300")
DEV = "cuda:0"
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.load_library()


def slack(x, T):
    """Error of ln l and of an entropy, from the arithmetic.  An exponent y = (x -
    ref) log2(e) / T is off by 3 roundings of itself (difference, product, factor),
    2^-24 |y| each, and by the base-2 exponential's 2^-22; elements of y < -40 do
    not count.  A thread adds at most V / 512 pairs of terms of at least a
    one-CTA row one after the other, a few more joins follow: 2^-24 each.  The
    entropy's sum is off by as much of itself (at most 48 log2 units: 40 and the
    reference's slack of 8) and the difference of the two by both."""
    V = x.shape[-1]
    finite = np.where(np.isfinite(x), x, 0.0).astype(np.float64)
    span = min(40.0, (finite.max() - finite.min()) * 1.4427 / T if V else 0.0)
    rel = 2.0 ** -24 * (3 * (span + 8) * 0.7 + 4 + V / 512 + 24)
    return rel, rel * (2 + 2 * 48 * 0.7)


def check(logits, tokens=None, rows=None, K=0, T=1.0, **kw):
    """logits: CPU tensor [B][T][V] (strides kept); compares every entry."""
    kept = tuple(slice(0, 1) if st == 0 else slice(None) for st in logits.stride())
    dev = torch.empty_strided(logits[kept].size(), logits.stride(), dtype=logits.dtype, device=DEV)
    dev = dev.copy_(logits[kept]).expand(logits.size())
    r = sv.token_logprobs(dev, None if tokens is None else tokens.to(DEV),
                          rows=None if rows is None else rows.to(DEV), top_k=K, temperature=T, **kw)
    torch.cuda.synchronize()
    got = {k: v.cpu().numpy() for k, v in r.items()}
    B, R, V = logits.shape
    P = got["entropy"].shape[1]
    x = logits.float().numpy()
    for b in range(B):
        for p in range(P):
            row = p if rows is None else int(rows[b, p])
            tok = None if tokens is None else int(tokens[b, p])
            at = (b, p, row, tok)
            if row == -1 or tok == -1:
                assert got["entropy"][b, p] == 0 and got["status"][b, p] == 0, at
                assert tokens is None or got["logprob"][b, p] == 0, at
                if K:
                    assert (got["top_token"][b, p] == -1).all() and (got["top_logprob"][b, p] == -np.inf).all()
                continue
            if not 0 <= row < R:
                assert got["status"][b, p] == plain.BAD_ROW and np.isnan(got["entropy"][b, p]), at
                assert tokens is None or np.isnan(got["logprob"][b, p]), at
                if K:
                    assert (got["top_token"][b, p] == -1).all() and np.isnan(got["top_logprob"][b, p]).all()
                continue
            lp, H, top, top_lp, st = plain.token_logprobs(x[b, row], tok, K, T)
            assert got["status"][b, p] == st, (at, got["status"][b, p], st)
            tol, tol_h = slack(x[b, row], T)

            def near(a, w):
                if math.isnan(w) or math.isinf(w):
                    return np.array_equal(np.float32(a), np.float32(w), equal_nan=True)
                return abs(a - w) <= tol + 2.0 ** -22 * abs(w)
            if tok is not None:
                assert near(got["logprob"][b, p], lp), (at, got["logprob"][b, p], lp, tol)
            if math.isnan(H):
                assert np.isnan(got["entropy"][b, p]), at
            else:
                assert abs(got["entropy"][b, p] - H) <= tol_h + 2.0 ** -22 * H, (at, got["entropy"][b, p], H, tol_h)
            if K:
                assert got["top_token"][b, p].tolist() == top, (at, got["top_token"][b, p], top)
                assert all(near(a, w) for a, w in zip(got["top_logprob"][b, p], top_lp)), at
    return got


def make(B, T, V, dtype, seed, pad=0, sigma=3.0):
    g = torch.Generator().manual_seed(seed)
    full = torch.full((B, T, V + pad), float("nan"), dtype=dtype)  # what is between rows is not looked at
    full[..., :V] = (torch.randn(B, T, V, generator=g) * sigma).to(dtype)
    tokens = torch.randint(0, V, (B, T), generator=g, dtype=torch.int32)
    return full[..., :V], tokens


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,T,V,K,pad", [
    (1, 1, 1, 1, 0),
    (2, 3, 5, 5, 0),          # all of the vocabulary listed
    (3, 2, 17, 3, 2),
    (1, 5, 1000, 5, 0),       # the tiny chain
    (2, 2, 1001, 128, 0),     # rows off the 16-byte grid
    (2, 3, 4096, 20, 8),
    (1, 3, 8199, 1, 1),       # a group and 7 elements
    (2, 2, 32000, 64, 0),
    (1, 2, 40001, 127, 63),
    (1, 2, 128256, 20, 0),    # eight CTAs
    (3, 1, 70000, 0, 0),      # no alternatives
])
def test_matches_the_definition(B, T, V, K, pad, dtype):
    logits, tokens = make(B, T, V, dtype, B * V + K, pad)
    check(logits, tokens, K=K)
    check(logits, None, K=K, T=0.7)


@pytest.mark.parametrize("B,T", [(40, 8), (400, 4), (1300, 1)])
def test_many_rows(B, T):
    """From several CTAs to a row to one CTA that takes all of it."""
    logits, tokens = make(B, T, 20011, torch.bfloat16, B)
    dev, tok = logits.to(DEV), tokens.to(DEV)
    r = sv.token_logprobs(dev, tok, top_k=7)
    lp = torch.log_softmax(dev.double(), -1)
    rel, rel_h = slack(logits[0, 0].float().numpy(), 1.0)
    assert int(r["status"].count_nonzero()) == 0
    want = lp.gather(2, tok.long()[..., None])[..., 0]
    assert float(((r["logprob"] - want).abs() - rel - 2.0 ** -22 * want.abs()).max()) <= 0
    H = -(lp.exp() * lp).sum(-1)
    assert float((r["entropy"] - H).abs().max()) <= rel_h + 2.0 ** -22 * 10
    order = dev.float().sort(dim=-1, descending=True, stable=True).indices[..., :7]
    assert torch.equal(r["top_token"].long(), order)
    want = lp.gather(2, order)
    assert float(((r["top_logprob"] - want).abs() - rel - 2.0 ** -22 * want.abs()).max()) <= 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [1, 20, 128])
@pytest.mark.parametrize("V", [3000, 40003, 128256])
def test_orders_that_overflow_the_list(V, K, dtype):
    """Ascending, descending, constant, two-valued and blockwise ascending rows,
    all with many equal elements in 16 bits; the largest at the very ends."""
    i = torch.arange(V, dtype=torch.float64)
    rows = [i / V * 20, -i / V * 20, torch.zeros(V, dtype=torch.float64), (i % 2) * 3.0,
            torch.floor(i / 700), (i * 7919 % V) / V * 9, torch.where(i >= V - K, 5.0, -5.0),
            torch.where(i < K, 5.0, -5.0)]
    logits = torch.stack(rows).to(dtype)[None]
    tokens = torch.tensor([[V - 1, 0, V // 2, 1, V - 1, 3, 0, 0]], dtype=torch.int32)
    check(logits, tokens, K=K)


def test_rounds_outputs_fit_as_they_come():
    """The tokens and path of a round, -1 behind what it emitted."""
    logits, _ = make(4, 9, 5003, torch.bfloat16, 3)
    rows = torch.tensor([[0, 2, 5, -1], [0, -1, -1, -1], [0, 1, 3, 8], [-1, -1, -1, -1]], dtype=torch.int32)
    tokens = torch.tensor([[7, 9, 5002, -1], [-1, -1, -1, -1], [1, 2, 3, 4], [5, 5, 5, 5]], dtype=torch.int32)
    check(logits, tokens, rows, K=3)
    check(logits, None, rows, K=3)
    # more entries than rows, the same row several times
    rows = torch.tensor([[0, 0, 8, 8, 3, 3, 3, 1, 1, 1, 4, 0]] * 4, dtype=torch.int32)
    tokens = torch.arange(48, dtype=torch.int32).view(4, 12)
    check(logits, tokens, rows, K=2)


def test_a_row_that_is_not_asked_for_may_hold_anything():
    logits, tokens = make(3, 4, 1003, torch.float32, 5)
    logits[1, 2] = float("nan")
    logits[2, 0] = float("inf")
    tokens[1, 2] = tokens[2, 0] = -1
    got = check(logits, tokens, K=4)
    assert not got["status"].any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [37, 9001, 128256])
def test_masked_and_extreme_rows(V, dtype):
    g = torch.Generator().manual_seed(V)
    lowest = torch.finfo(dtype).min
    x = (torch.randn(12, V, generator=g) * 2).to(dtype)
    x[0, : V // 2] = -math.inf                 # a half masked
    x[1] = -math.inf                           # nothing left: a fault
    x[2] = lowest                              # masked with the lowest value, all of it: uniform
    x[3] = lowest
    x[3, V // 3] = 1.0                         # one token left
    x[4] = -math.inf
    x[4, V - 1] = 2.0                          # one token, the last; alternatives run out
    x[5, V // 2] = math.nan
    x[6, 0] = math.inf
    x[7, :] = 0.0
    x[7, ::2] = -0.0                           # equal to 0: ties go to the lowest token
    x[8] = torch.finfo(dtype).max
    x[9] = torch.linspace(-60, 60, V).to(dtype)
    x[10, V // 2:] = lowest
    x[11] = -math.inf
    x[11, 0], x[11, V - 1] = lowest, lowest
    tokens = torch.full((1, 12), V // 3, dtype=torch.int32)
    tokens[0, 9] = V
    tokens[0, 10] = -2
    K = min(V, 30)
    got = check(x[None], tokens, K=K)
    assert got["status"][0].tolist()[:9] == [0, 1, 0, 0, 0, 1, 1, 0, 0]
    assert got["top_token"][0, 7].tolist() == list(range(K))


@pytest.mark.parametrize("T", [1e-3, 0.3, 5.0, 1e4])
def test_temperatures(T):
    logits, tokens = make(2, 3, 12345, torch.bfloat16, 9)
    check(logits, tokens, K=9, T=T)


def test_bad_rows_and_tokens():
    logits, _ = make(1, 3, 500, torch.float32, 1)
    rows = torch.tensor([[0, 3, -2, 2, 1]], dtype=torch.int32)
    tokens = torch.tensor([[500, 1, 1, -7, 2]], dtype=torch.int32)
    got = check(logits, tokens, rows, K=2)
    assert got["status"][0].tolist() == [2, 1024, 1024, 2, 0]


def test_strides():
    logits, tokens = make(4, 6, 777, torch.bfloat16, 2, pad=5)
    check(logits[::2, 1::2], tokens[::2, 1::2].contiguous(), K=3)
    one = logits[:1, :1].expand(3, 4, 777)          # broadcast rows
    check(one, tokens[:3, :4].contiguous(), K=3)


def test_streams_capture_and_page_locked_inputs():
    logits, tokens = make(3, 5, 30011, torch.bfloat16, 4)
    dev, tok = logits.to(DEV), tokens.to(DEV)
    want = sv.token_logprobs(dev, tok, top_k=6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sv.token_logprobs(dev, tok, top_k=6, stream=side)
    side.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)
    graph = torch.cuda.CUDAGraph()
    static = dev.clone()
    with torch.cuda.graph(graph):
        got = sv.token_logprobs(static, tok, top_k=6)
    for seed in (5, 6):
        new, _ = make(3, 5, 30011, torch.bfloat16, seed)
        static.copy_(new)
        graph.replay()
        want = sv.token_logprobs(static, tok, top_k=6)
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], want[k]) for k in want)
    host = sv.token_logprobs(static.cpu().pin_memory(), tok, top_k=6)
    torch.cuda.synchronize()
    assert all(torch.equal(host[k], want[k]) for k in want)


def test_two_calls_at_once():
    logits, tokens = make(64, 8, 32000, torch.bfloat16, 8)
    dev, tok = logits.to(DEV), tokens.to(DEV)
    want = sv.token_logprobs(dev, tok, top_k=20)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [sv.token_logprobs(dev, tok, top_k=20, stream=s) for _ in range(5) for s in streams]
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(r[k], want[k]) for k in want)


def test_round_of_the_chain_end_to_end():
    """Verify a chain, then ask for the log probabilities of what it emitted."""
    from speculative_decoding_verification_vocab_gb300 import synth
    vq, dp, d = synth.chain_inputs(synth.CONFIGS[2], seed=1, B=9)
    vq, dp, d = vq.to(DEV), dp.to(DEV), d.to(DEV)
    r = sv.verify_chain(vq, dp, d, seed=3)
    got = sv.token_logprobs(vq, r["tokens"], top_k=2)
    lp = torch.log_softmax(vq.double(), -1)
    some = r["tokens"] >= 0
    want = lp.gather(2, r["tokens"].clamp(min=0).long()[..., None])[..., 0]
    assert float((got["logprob"] - want)[some].abs().max()) <= 1e-4
    assert not got["logprob"][~some].any() and int(got["status"].count_nonzero()) == 0
    q = r["q_prob"]
    a = r["accept_len"]
    for b in range(9):
        n = int(a[b])
        assert torch.allclose(got["logprob"][b, :n].exp(), q[b, :n], atol=1e-5)


def test_largest_vocabulary():
    V = sv.SV_MAX_VOCAB
    g = torch.Generator(device=DEV).manual_seed(1)
    x = (torch.randn(2, 1, V, generator=g, device=DEV) * 3).to(torch.bfloat16)
    tok = torch.tensor([[V - 1], [0]], dtype=torch.int32, device=DEV)
    r = sv.token_logprobs(x, tok, top_k=128)
    lp = torch.log_softmax(x.double(), -1)
    order = x.float().sort(dim=-1, descending=True, stable=True).indices[..., :128]
    assert torch.equal(r["top_token"].long(), order)
    rel, _ = slack(np.array([-40.0, 40.0]), 1.0)
    rel += 2.0 ** -24 * V / 512
    assert float((r["logprob"] - lp.gather(2, tok.long()[..., None])[..., 0]).abs().max()) <= rel + 2.0 ** -22 * 40


def test_offsets_that_pass_32_bits():
    """Rows more than 2^32 bytes, and 2^31 elements, behind the first."""
    V, stride = 1000, (1 << 31) + 24
    buf = torch.zeros(stride + V, dtype=torch.bfloat16, device=DEV)
    x = buf.as_strided((2, 1, V), (stride, V, 1))
    x.copy_(torch.randn(2, 1, V, device=DEV))
    tok = torch.tensor([[5], [999]], dtype=torch.int32, device=DEV)
    r = sv.token_logprobs(x, tok, top_k=4)
    want = sv.token_logprobs(x.contiguous(), tok, top_k=4)
    torch.cuda.synchronize()
    assert all(torch.equal(r[k], want[k]) for k in want)
