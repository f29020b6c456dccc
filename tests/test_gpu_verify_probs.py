"""sv_verify_chain_probs against the plain definition (tests/plain_serving.py,
exact integers): every output is a whole number and has to be equal, whatever
the sizes, strides, types and faults."""
import numpy as np
import pytest
import torch

import plain_serving as plain

pytestmark = pytest.mark.gpu

sv = pytest.importorskip("speculative_decoding_verification_vocab_gb300")
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.load_library()


def make(B, N, V, dtype=torch.float32, seed=0, pad=0, onehot=False, sigma=2.0, noise=0.7):
    """CPU inputs: probabilities of random rows, drafts drawn from the draft rows."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, N + 1, V, generator=g) * sigma
    y = x[:, :N] + noise * torch.randn(B, N, V, generator=g)
    q = torch.zeros(B, N + 1, V + pad, dtype=dtype)
    p = torch.zeros(B, N, V + pad, dtype=dtype)
    q[..., :V] = torch.softmax(x, -1).to(dtype)
    p[..., :V] = torch.softmax(y, -1).to(dtype)
    if N:
        d = torch.multinomial(torch.softmax(y, -1).reshape(B * N, V), 1, generator=g).view(B, N)
    else:
        d = torch.zeros(B, 0)
    ua = torch.rand(B, N, generator=g)
    if onehot:
        ua *= 0.1
    us = torch.rand(B, generator=g)
    return (q[..., :V], None if onehot else p[..., :V], d.to(torch.int32), ua, us)


def run(q, p, d, ua, us, n=None, **kw):
    def dev(t):
        if t is None:
            return None
        if t.dim() == 3 and t.stride(1) != t.shape[2] and t.numel():  # keep the padding
            full = torch.zeros(t.shape[0], t.shape[1], t.stride(1), dtype=t.dtype, device=DEV)
            full[..., :t.shape[2]] = t.to(DEV)
            return full[..., :t.shape[2]]
        return t.to(DEV)
    r = sv.verify_chain_probs(dev(q), dev(p), dev(d), dev(ua), dev(us), n_draft=dev(n), **kw)
    torch.cuda.synchronize()
    return tuple(r[k].cpu().numpy() for k in ("tokens", "accept_len", "status"))


def expect(q, p, d, ua, us, n=None):
    f = lambda t: None if t is None else t.float().numpy()  # noqa: E731
    return plain.verify_probs(f(q), f(p), d.numpy(), ua.numpy(), us.numpy(),
                              None if n is None else n.numpy())


def check(*args, **kw):
    got, want = run(*args, **kw), expect(*args, **kw)
    for a, b, name in zip(got, want, ("tokens", "accept_len", "status")):
        assert np.array_equal(a, b), (name, a[:8], b[:8])
    return want


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,N,V,pad,onehot", [
    (1, 4, 1000, 0, False),      # the tiny chain
    (3, 1, 1, 0, False),         # one token: always accepted, then drawn again
    (5, 3, 2, 6, False),
    (7, 0, 37, 0, False),        # nothing drafted: a bonus draw alone
    (4, 40, 257, 0, False),      # more positions than a warp
    (6, 5, 8192, 0, False),      # one CTA, aligned rows
    (5, 5, 8193, 0, False),      # rows off the 16-byte grid
    (5, 2, 16400, 16, False),    # padded rows
    (4, 3, 40001, 63, True),     # one-hot drafts
    (3, 3, 128256, 0, False),    # eight CTAs
    (2, 2, 300007, 1, True),
])
def test_matches_the_definition(B, N, V, pad, onehot, dtype):
    for seed in range(3):
        check(*make(B, N, V, dtype, seed, pad, onehot, noise=1.5 if seed else 0.3))


def test_ragged_lengths_and_rows_after_them_unread():
    q, p, d, ua, us = make(9, 6, 5003, seed=4)
    n = torch.tensor([0, 1, 2, 3, 4, 5, 6, 6, 0], dtype=torch.int32)
    for b in range(9):   # nothing behind a sequence's own drafts is looked at
        q[b, n[b] + 1:] = float("nan")
        p[b, n[b]:] = float("nan")
        d[b, n[b]:] = -5
        ua[b, n[b]:] = float("nan")
    want = check(q, p, d, ua, us, n)
    assert not want[2].any()
    check(q, p, d, ua, us, torch.tensor([0, 1, -1, 3, 7, 5, 6, 6, 0], dtype=torch.int32))


def test_acceptance_at_the_border_is_exact():
    """u p(d) against q(d) where they are equal or one unit apart."""
    V = 64
    q = torch.full((4, 2, V), 1.0 / V)
    p = torch.full((4, 1, V), 1.0 / V)
    q[:, 0, 5], p[:, 0, 5] = 0.1, 0.3
    d = torch.full((4, 1), 5, dtype=torch.int32)
    u = np.float32(np.float64(np.float32(0.1)) / np.float64(np.float32(0.3)))
    ua = torch.tensor([[u], [np.nextafter(u, np.float32(0))], [np.nextafter(u, np.float32(1))], [0.0]])
    want = check(q, p, d, ua, torch.tensor([0.0, 0.5, 0.999999, 0.25]))
    assert want[1][1] == 1 and want[1][2] == 0 and want[1][3] == 1
    # equality rejects: u = 1/2, p = 1/2, q = 1/4
    q[:, 0, 5], p[:, 0, 5] = 0.25, 0.5
    assert not check(q, p, d, torch.full((4, 1), 0.5), torch.full((4,), 0.5))[1].any()


def test_draws_at_cdf_borders():
    """Thresholds on and beside the borders of a CDF of exact powers of two."""
    V = 4096
    q = torch.full((8, 1, V), 1.0 / V)
    us = torch.tensor([0.0, 1 / V, 2 / V, 0.5, 1 - 1 / V, 1 - 2.0 ** -24, 2.0 ** -149, 2.0 ** -126])
    w = check(q, None, torch.zeros(8, 0, dtype=torch.int32), torch.zeros(8, 0), us)
    assert w[0][:6, 0].tolist() == [0, 1, 2, V // 2, V - 1, V - 1]
    # leading and trailing zeros are never drawn
    q[:, 0, :100] = 0
    q[:, 0, -100:] = 0
    w = check(q, None, torch.zeros(8, 0, dtype=torch.int32), torch.zeros(8, 0), us)
    assert w[0].min() == 100 and w[0].max() == V - 101


def test_tiny_and_denormal_weights():
    q = torch.zeros(4, 1, 1000)
    q[0, 0, 7] = 2.0 ** -60
    q[1, 0, 7], q[1, 0, 900] = 2.0 ** -62, 2.0 ** -61
    q[2, 0, 3] = 2.0 ** -63        # below the grid: no mass at all
    q[3, 0, 3] = 1e-40
    w = check(q, None, torch.zeros(4, 0, dtype=torch.int32), torch.zeros(4, 0),
              torch.full((4,), 0.9))
    assert w[0][:, 0].tolist() == [7, 900, -1, -1] and w[2].tolist() == [0, 0, 1, 1]


@pytest.mark.parametrize("V", [500, 20000, 70001])
def test_residual_without_mass_draws_from_q(V):
    """q <= p everywhere: the residual is empty and the correction comes from q."""
    q, p, d, ua, us = make(6, 3, V, seed=9)
    p[:, 1] = (q[:, 1] * 1.5).clamp(max=1.0)
    ua[:, 0], ua[:, 1] = 0.0, 0.9999
    want = check(q, p, d, ua, us)
    assert (want[2] == plain.RESID_ZERO).any()
    # one-hot: q is the point mass on a rejected token's neighbour / on itself
    q = torch.zeros(2, 2, V)
    q[0, 0, 3] = 1.0
    q[1, 0, 4] = 0.5
    d = torch.full((2, 1), 4, dtype=torch.int32)
    want = check(q, None, d, torch.full((2, 1), 0.75), torch.tensor([0.2, 0.8]))
    assert want[0][:, 0].tolist() == [3, 4] and want[2].tolist() == [0, plain.RESID_ZERO]


def test_zero_draft_probability_is_accepted_and_flagged():
    q, p, d, ua, us = make(4, 3, 300, seed=2)
    p[2, 0, d[2, 0]] = 0
    p[3, 0, d[3, 0]] = -0.0
    q[1, 0, 0] = -0.0                      # a negative zero is a zero
    ua[:, 0] = 0.999
    want = check(q, p, d, ua, us)
    assert want[2][2] & plain.P_ZERO and want[1][2] >= 1


@pytest.mark.parametrize("V", [100, 40000])
def test_faults(V):
    nan, inf = float("nan"), float("inf")
    for seed, (where, value) in enumerate([("q", nan), ("q", inf), ("q", -0.25), ("q", 2.0),
                                           ("p", nan), ("p", -inf), ("p", 3.0), ("sum", 0.0)]):
        q, p, d, ua, us = make(6, 2, V, seed=seed)
        ua[:, 0], ua[:, 1] = 0.0, torch.tensor([0.0, 0.999, 0.5, 0.0, 0.999, 0.3])
        q[:, 0] = q[:, 0].clamp(min=1e-30)
        if where == "q":
            q[0, 2, V - 1] = q[1, 1, V // 2] = q[2, 0, 1] = value
            q[3, 2, 0] = value
        elif where == "p":
            p[0, 1, V - 1] = p[1, 1, V // 2] = p[4, 1, 0] = value
        else:
            q[0, 2], q[3, 2] = 0.0, 1.9           # no mass; a sum far above 2
        check(q, p, d, ua, us)
    q, p, d, ua, us = make(8, 2, V, seed=77)
    d[0, 0], d[1, 1], d[2, 0] = -1, V, 2 ** 31 - 1
    us[3], us[4], us[5] = 1.0, nan, -0.5
    ua[6, 0], ua[7, 1] = 1.0, nan
    check(q, p, d, ua, us)


def test_same_sums_whatever_the_alignment():
    """The same rows packed, padded and off the vector grid draw the same tokens."""
    q, p, d, ua, us = make(16, 3, 20001, seed=5)
    want = run(q, p, d, ua, us)
    for pad in (7, 15, 64):
        qq = torch.zeros(16, 4, 20001 + pad)
        pp = torch.zeros(16, 3, 20001 + pad)
        qq[..., :20001], pp[..., :20001] = q, p
        got = run(qq[..., :20001], pp[..., :20001], d, ua, us)
        assert all(np.array_equal(a, b) for a, b in zip(got, want))
    # a storage offset that breaks the 16-byte alignment of the first row
    flat = torch.zeros(16 * 4 * 20001 + 1)
    flat[1:] = q.reshape(-1)
    qs = flat.to(DEV)[1:].view(16, 4, 20001)
    r = sv.verify_chain_probs(qs, p.to(DEV), d.to(DEV), ua.to(DEV), us.to(DEV))
    assert np.array_equal(r["tokens"].cpu().numpy(), want[0])


def test_sliced_and_broadcast_rows():
    """Rows where they are: a part of a longer draft, every other sequence, one
    row for all sequences, one for all positions."""
    q, p, d, ua, us = [t.to(DEV) for t in make(8, 5, 3001, seed=6)]
    want = [run(*[t[::2].contiguous().cpu() for t in (q[:, :4], p[:, :3], d[:, :3], ua[:, :3], us)])]
    r = sv.verify_chain_probs(q[::2, :4], p[::2, :3], *[t[::2].contiguous() for t in (d[:, :3], ua[:, :3], us)])
    assert np.array_equal(r["tokens"].cpu().numpy(), want[0][0])
    for a, b in ((q[:1].expand(8, -1, -1), p[:1].expand(8, -1, -1)),
                 (q[:, :1].expand(-1, 6, -1), p[:, 2:3].expand(-1, 5, -1))):
        r = sv.verify_chain_probs(a, b, d, ua, us)
        want = run(a.contiguous().cpu(), b.contiguous().cpu(), d.cpu(), ua.cpu(), us.cpu())
        for k, x in zip(("tokens", "accept_len", "status"), want):
            assert np.array_equal(r[k].cpu().numpy(), x), k


def test_empty_batch_and_host_memory():
    r = sv.verify_chain_probs(torch.zeros(0, 3, 10, device=DEV), torch.zeros(0, 2, 10, device=DEV),
                              torch.zeros(0, 2, dtype=torch.int32, device=DEV),
                              torch.zeros(0, 2, device=DEV), torch.zeros(0, device=DEV))
    assert r["tokens"].shape == (0, 3)
    a = make(3, 2, 5000, seed=3)
    want = expect(*a)
    r = sv.verify_chain_probs(*[t.pin_memory() for t in a])
    torch.cuda.synchronize()
    assert np.array_equal(r["tokens"].cpu().numpy(), want[0])


def test_two_streams_and_a_captured_graph():
    a = [t.to(DEV) for t in make(32, 3, 9001, seed=11)]
    b = [t.to(DEV) for t in make(32, 3, 9001, seed=12)]
    torch.cuda.synchronize()
    want = [sv.verify_chain_probs(*x)["tokens"].clone() for x in (a, b)]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        ra, rb = sv.verify_chain_probs(*a, stream=s1), sv.verify_chain_probs(*b, stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(ra["tokens"], want[0]) and torch.equal(rb["tokens"], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = sv.verify_chain_probs(*a)
    for x, w in ((a, want[0]), (b, want[1])):
        for t, v in zip(a, [v.clone() for v in x]):
            t.copy_(v)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(r["tokens"], w)


def test_large_batch_against_the_definition():
    """The large-vocabulary chain's shape, a few of its sequences replayed."""
    B, N, V = 256, 7, 128256
    g = torch.Generator(device=DEV).manual_seed(1)
    q = torch.softmax(torch.randn(B, N + 1, V, generator=g, device=DEV) * 3, -1)
    p = torch.softmax(torch.log(q[:, :N]) + 0.4 * torch.randn(B, N, V, generator=g, device=DEV), -1)
    d = torch.multinomial(p.reshape(-1, V), 1, generator=g).view(B, N).to(torch.int32)
    ua, us = torch.rand(B, N, generator=g, device=DEV), torch.rand(B, generator=g, device=DEV)
    r = sv.verify_chain_probs(q, p, d, ua, us)
    pick = [0, 17, 100, 255]
    want = plain.verify_probs(*[t[pick].cpu().numpy() for t in (q, p, d, ua, us)])
    for k, w in zip(("tokens", "accept_len", "status"), want):
        assert np.array_equal(r[k][pick].cpu().numpy(), w), k
    assert int(r["status"].abs().max()) == 0


@pytest.mark.parametrize("V", [5, 300, 40000])
def test_weights_that_sum_to_almost_two(V):
    """Rows need not be normalised: below 2 they are drawn from, at 2 and above
    they are a fault, exactly and wherever the row lies.  Most of these sums round
    to 2 in fp32; from 4 on the integers wrap around."""
    e = 2.0 ** -24
    rows = [(1.0, 1 - e), (1.0, 1.0), (1.5, 0.5 - e / 2), (1 - e, 1 - e, e, e), (1 - e, 1 - e, e, e / 2),
            (1.75, 0.25, 2.0 ** -62), (1.75, 0.25 - e / 4, e / 8), (1.9, 1.9), (1.25,) * 4, (1.0,) * 4, (1.99,) * 5]
    B = len(rows)
    q = torch.zeros(2, B, 2, V)
    for b, row in enumerate(rows):
        at = torch.linspace(0, V - 1, len(row)).long()
        for j, x in enumerate(row):
            q[0, b, 0, at[j]] = x                  # side by side in a warp, or CTAs apart
            q[1, b, 0, V - 1 - j] = x
    us = torch.tensor([0.0, 0.5, 1 - e])
    none = torch.zeros(B, 0, dtype=torch.int32), torch.zeros(B, 0)
    for rows_at in q:
        for u in us:
            for pad in (0, 1, 4):
                wide = torch.zeros(B, 1, V + pad)
                wide[..., :V] = rows_at[:, :1]
                want = check(wide[..., :V], None, *none, u.repeat(B))
                assert want[2].tolist() == [0, 1, 0, 1, 0, 1, 0, 1, 1, 1, 1]
    # after a rejection: q apart from the token that was copied
    d = torch.full((B, 1), 2, dtype=torch.int32)
    one = q[1].clone()
    one[:, 0, 2] = torch.where(one[:, 0, 2] == 0, 0.25, one[:, 0, 2])
    check(one, None, d, torch.full((B, 1), 0.9999), us[1].repeat(B))
