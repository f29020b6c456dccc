"""sv_paged_attention against the plain definition in 64 bits
(tests/plain_serving.py).

Tolerances, from the arithmetic (u = 2^-24, d = relative error of a weight):
a score is an fp32 sum of D exact products, off by at most D u A with
A = scale sum |q_d k_d|, and two more roundings of |s| <= A; the base-2
exponential adds 2^-22; the weights' sum over n slots n u.  So
d <= (D + 4) u A + 2^-22 + n u for a weight relative to its row's largest, and
the same bounds ln l.  The weights enter the product with the values as two
parts of the cache's type, off by eps^2 / 4 <= 2^-18 at most (and fp16 ones by
2^-36 of the row's largest: n u has room for that).  An output is a
weighted mean of values: off by 2 d max|v| + 2^-17 max|v|, and by half a unit
of its own type, 2^-8 (bf16) or 2^-11 (fp16) of its value (fp16: 2^-25 near
zero)."""
import numpy as np
import pytest
import torch

import plain_serving as plain

pytestmark = pytest.mark.gpu

sv = pytest.importorskip("speculative_decoding_verification_vocab_gb300")
DEV = "cuda:0"
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.load_library()


def make(lens, Hq, Hkv, D, page, dtype=torch.bfloat16, seed=0, window=0, sinks=0, spare=2,
         extra_pages=1, sigma=1.5):
    """CPU inputs; NaN in every slot that is not visible, -1 for every table
    entry without one."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    per = max(1, -(-max(lens) // page)) + extra_pages
    P = B * per + spare
    q = (torch.randn(B, Hq, D, generator=g) * sigma).to(dtype)
    full = torch.randn(2, P, page, Hkv, D, generator=g).to(dtype)
    kv = torch.full_like(full, float("nan"))
    table = torch.full((B, per), -1, dtype=torch.int32)
    ids = torch.randperm(P, generator=g)
    for b, n in enumerate(lens):
        j = torch.from_numpy(plain.visible_slots(n, window, sinks))
        own = ids[b * per:(b + 1) * per]
        table[b, j // page] = own[j // page].int()
        kv[:, own[j // page], j % page] = full[:, own[j // page], j % page]
    return q, kv, table, torch.tensor(lens, dtype=torch.int32)


def reference(q, kv, table, lens, scale, window=0, sinks=0):
    return plain.paged_attention(q.double().numpy(), kv.double().numpy(), table.numpy(),
                                 lens.numpy(), scale, window, sinks)


def check(q, kv, table, lens, scale=None, window=0, sinks=0, weights=False, **kw):
    B, Hq, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    page, Hkv = kv.shape[2], kv.shape[3]
    sums = None
    if weights:
        sums = torch.rand(B, Hkv, table.shape[1] * page + 3, generator=torch.Generator().manual_seed(3))
    dev_sums = None if sums is None else sums.to(DEV)
    out, lse, st = sv.paged_attention(q.to(DEV), kv.to(DEV), table.to(DEV), lens.to(DEV), scale,
                                      window, sinks, dev_sums, return_lse=True, **kw)
    torch.cuda.synchronize()
    assert not st.any()
    ref, rlse, got, size = reference(q, kv, table, lens, scale, window, sinks)
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(l), np.isneginf(rlse))
    n = np.maximum(lens.numpy().astype(np.float64), 1)[:, None]
    d = (D + 4) * U * size + 2.0 ** -22 + n * U
    fin = np.isfinite(rlse)
    lerr = np.abs(np.where(fin, l, 0) - np.where(fin, rlse, 0))
    assert (lerr <= d + 4 * U * np.abs(np.where(fin, rlse, 0))).all(), lerr.max()
    vmax = np.nan_to_num(kv[1].double().abs().numpy(), nan=0.0).max()
    half = 2.0 ** -8 if q.dtype == torch.bfloat16 else 2.0 ** -11
    tol = half * np.abs(ref) + (2 * d + 2.0 ** -17)[..., None] * vmax + 2.0 ** -25
    err = np.abs(o - ref)
    assert (err <= tol).all(), (err - tol).max()
    if weights:
        s, before = dev_sums.double().cpu().numpy(), sums.double().numpy()
        cap = table.shape[1] * page
        G = Hq // Hkv
        dk = d.reshape(B, Hkv, G).max(-1)[..., None]
        lmax = np.abs(np.where(fin, rlse, 0)).reshape(B, Hkv, G).max(-1)[..., None]
        bound = got * (2 * dk + 8 * U * lmax + G * U) + U * (before[..., :cap] + got)
        assert (np.abs(s[..., :cap] - before[..., :cap] - got) <= bound).all()
        untouched = got == 0
        assert np.array_equal(s[..., :cap][untouched], before[..., :cap][untouched])
        assert np.array_equal(s[..., cap:], before[..., cap:])
    return out, lse, dev_sums


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,Hq,Hkv,page", [
    ([1], 1, 1, 16),                         # one slot: the value itself
    ([5, 0, 64, 65, 17], 8, 2, 16),          # an empty sequence; tile edges; G = 4
    ([130, 1, 63], 3, 3, 1),                 # G = 1, pages of one slot
    ([200, 333], 14, 2, 24),                 # G = 7, pages that end inside a tile
    ([129, 700], 32, 2, 128),                # G = 16
    ([77, 300], 20, 1, 33),                  # G = 20: two groups of query heads
])
def test_matches_the_definition(lens, Hq, Hkv, page, D, dtype):
    check(*make(lens, Hq, Hkv, D, page, dtype, seed=D + page))


@pytest.mark.parametrize("window,sinks", [(1, 0), (64, 4), (100, 1), (63, 70), (5000, 4), (1, 1)])
def test_window_and_first_tokens(window, sinks):
    lens = [0, 1, 2, 64, 65, 103, 104, 105, 500, 1111]
    check(*make(lens, 8, 2, 64, 16, seed=window, window=window, sinks=sinks), window=window,
          sinks=sinks)
    check(*make(lens, 4, 4, 128, 7, torch.float16, seed=window, window=window, sinks=sinks),
          window=window, sinks=sinks, weights=True)


@pytest.mark.parametrize("lens,Hq,Hkv,D,page", [
    ([40000], 8, 1, 128, 64),                # one long sequence: split and joined
    ([9001, 3], 16, 8, 64, 16),
    ([12000, 1, 5000], 6, 2, 256, 20),
    ([3000] * 9, 4, 4, 128, 32),
])
def test_split_over_the_length(lens, Hq, Hkv, D, page):
    check(*make(lens, Hq, Hkv, D, page, seed=7), weights=True)


@pytest.mark.parametrize("Hq,Hkv,page,window,sinks", [
    (20, 1, 24, 0, 0),       # two groups of heads, rows looked up one by one
    (33, 1, 16, 0, 0),       # three, the last of one head
    (24, 2, 16, 3000, 20),   # G = 12; a window from the middle of a group of 16
    (6, 2, 7, 2500, 37),
])
def test_split_with_groups_and_windows(Hq, Hkv, page, window, sinks):
    lens = [7001, 100, 2530, 4096]
    check(*make(lens, Hq, Hkv, 64, page, torch.float16, seed=Hq, window=window, sinks=sinks),
          window=window, sinks=sinks, weights=True)


@pytest.mark.parametrize("B", [130, 700])
def test_many_sequences(B):
    """More sequences than threads; ragged, with empty ones."""
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(0, 40, B)]
    lens[B // 2] = 3000
    check(*make(lens, 2, 1, 64, 16, seed=B), weights=B == 130)


@pytest.mark.parametrize("Hq,Hkv,D,page", [(4, 1, 64, 16), (20, 2, 128, 33), (6, 3, 256, 16)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 5)])
def test_shares_that_cross_sequences(Hq, Hkv, D, page, window, sinks):
    """A batch in equal shares: sequences of many shares, shares of many
    sequences, empty ones first, last and between."""
    for seed, lens in enumerate(([0, 0, 3000, 1, 0, 64, 65, 5000, 0, 512, 511, 513, 7, 0, 1500, 0] + [20, 0, 300] * 12,
                                 [1] * 39 + [9000],
                                 [2500] + [0] * 40,
                                 [0] * 45,
                                 [640] * 40)):
        check(*make(lens, Hq, Hkv, D, page, seed=seed, window=window, sinks=sinks), window=window, sinks=sinks,
              weights=seed != 1)


def test_faults_among_shares():
    """A sequence with a bad length or page fails alone, wherever it lies in
    the shares."""
    lens = [700, 900, 30, 4000, 2000, 0, 1500, 800] * 6
    q, kv, table, n = make(lens, 4, 2, 128, 16, seed=9)
    want = check(q, kv, table, n)[0]
    n2, table2 = n.clone(), table.clone()
    n2[0], n2[17], n2[47] = -1, table.shape[1] * 16 + 1, 2 ** 31 - 1
    table2[3, 249] = kv.shape[1]
    table2[22, 0] = -1
    sums = torch.zeros(len(lens), 2, table.shape[1] * 16, device=DEV)
    out, lse, st = sv.paged_attention(q.to(DEV), kv.to(DEV), table2.to(DEV), n2.to(DEV), weight_sum=sums,
                                      return_lse=True)
    bad = {0: 256, 17: 256, 47: 256, 3: 512, 22: 512}
    assert st.tolist() == [bad.get(b, 0) for b in range(len(lens))]
    for b in range(len(lens)):
        if b in bad:
            assert torch.isnan(out[b]).all() and torch.isnan(lse[b]).all() and not sums[b].any()
        else:  # two orders of the same sum: half a step of bf16 each, and the sums' own error
            assert torch.allclose(out[b].float(), want[b].float(), rtol=2.0 ** -7, atol=1e-4)


@pytest.mark.parametrize("B", [511, 512, 513])
def test_batches_around_the_largest_that_is_shared(B):
    g = torch.Generator().manual_seed(B)
    lens = [int(x) for x in torch.randint(0, 90, (B,), generator=g)]
    lens[B - 1], lens[3] = 1400, 900
    check(*make(lens, 2, 1, 64, 16, seed=B, extra_pages=0), weights=True)


def test_more_sequences_than_are_split():
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 5, 2100)]
    lens[2099] = 400
    check(*make(lens, 2, 1, 64, 16, seed=5, extra_pages=0))


def test_sharp_scores_and_growing_maxima():
    """Scores that grow along the slots (every tile raises the maximum), and
    one slot that takes all the weight."""
    q, kv, table, lens = make([1500], 4, 1, 128, 16, seed=3)
    base = q[0, 0].float()
    for j in range(1500):
        kv[0, table[0, j // 16], j % 16, 0] = (base * (j / 1500) * 0.2).to(q.dtype)
    q[0] = base.to(q.dtype)
    check(q, kv, table, lens, weights=True)
    check(q, kv, table, lens, scale=2.0)
    kv[0, table[0, 40], 3, 0] = (base * 2).to(q.dtype)
    check(q, kv, table, lens, scale=1.0, weights=True)


@pytest.mark.parametrize("dtype,whole", [(torch.float16, True), (torch.float16, False), (torch.bfloat16, True)])
def test_many_weights_far_below_the_largest(dtype, whole):
    """One slot with weight 1 and value 0, all others with weight 2^-25.5 and
    value 1, in a sequence that one unit goes through (1300 of them, on the same
    pages) or that is cut: out = n w / (1 + n w).  Half the smallest fp16 number
    is 2^-25, so weights held in fp16 against the largest would all be lost.
    Tolerance: each weight of fp16 is off by 2^-36 of the largest (its two
    parts reach down to 2^-24 / 2^11), n of them, and by d of itself; bf16 has
    no such floor."""
    n, D = 20001, 64
    B = 1300 if whole else 1
    k = torch.full((n, D), -2.208984375)  # q.k / 8 = -17.671875
    k[0] = 0
    v = torch.ones(n, D)
    v[0] = 0
    pages = -(-n // 16)
    kv = torch.zeros(2, pages * 16, D)
    kv[0, :n], kv[1, :n] = k, v
    kv = kv.to(dtype).view(2, pages, 16, 1, D)
    q = torch.ones(B, 1, D, dtype=dtype)
    table = torch.arange(pages, dtype=torch.int32).repeat(B, 1)
    out, lse, st = sv.paged_attention(q.to(DEV), kv.to(DEV), table.to(DEV),
                                      torch.full((B,), n, dtype=torch.int32, device=DEV), return_lse=True)
    assert not st.any()
    s = float(kv[0, 1, 0, 0, 0].double()) * D / 8
    w = (n - 1) * np.exp(s)
    ref = w / (1 + w)
    d = (D + 4) * U * abs(s) + 2.0 ** -22 + n * U
    half, floor = (2.0 ** -11, n * 2.0 ** -36 + 2.0 ** -25) if dtype == torch.float16 else (2.0 ** -8, 0.0)
    err = (out.double().cpu() - ref).abs().max()
    assert err <= (half + 2 * d + 2.0 ** -17) * ref + floor, (float(err), ref)
    assert (lse.double().cpu() - np.log1p(w)).abs().max() <= d + 4 * U


def test_infinities_and_nan_in_the_data():
    q, kv, table, lens = make([100, 100, 100, 700], 4, 2, 64, 16, seed=4)
    q = q.abs() + 0.1
    inf = float("inf")
    kv[0, table[0, 2], 5, 0] = -inf            # a score of -inf: weight 0
    kv[0, table[1, :7].long(), :, 1] = -inf    # a head with no finite score
    kv[0, table[2, 0], 0, 0] = float("nan")    # NaN: that head's rows are NaN
    kv[0, table[3, 43], 5, 1] = inf
    sums = torch.zeros(4, 2, table.shape[1] * 16, device=DEV)
    out, lse, st = sv.paged_attention(q.to(DEV), kv.to(DEV), table.to(DEV), lens.to(DEV),
                                      weight_sum=sums, return_lse=True)
    assert not st.any()
    ref, rlse, got, _ = reference(q[:2], kv, table[:2], lens[:2], 64 ** -0.5)
    o = out.double().cpu().numpy()
    assert np.abs(o[:2] - ref).max() < 0.05
    assert (o[1, 2:] == 0).all() and torch.isneginf(lse[1, 2:]).all() and (sums[1, 1] == 0).all()
    assert float(sums[0, 0, 2 * 16 + 5]) == 0.0
    assert np.isnan(o[2, :2]).all() and np.isfinite(o[2, 2:]).all()
    assert np.isnan(o[3, 2:]).all() and np.isfinite(o[3, :2]).all()
    assert torch.isnan(lse[2, :2]).all() and torch.isnan(lse[3, 2:]).all()
    assert torch.isnan(sums[2, 0, :100]).all() and (sums[2, 0, 100:] == 0).all()


@pytest.mark.parametrize("n", [40, 5000])
def test_bad_lengths_and_pages(n):
    """Refused per sequence: NaN rows and a status bit, weight_sum untouched,
    the other sequences as if alone."""
    q, kv, table, lens = make([n] * 6, 4, 2, 128, 16, seed=6)
    cap = table.shape[1] * 16
    want, wlse = [t.clone() for t in sv.paged_attention(
        q.to(DEV), kv.to(DEV), table.to(DEV), lens.to(DEV), return_lse=True)[:2]]
    P = kv.shape[1]
    lens[0], lens[1] = -1, cap + 1
    table[2, 0], table[3, (n - 1) // 16] = P, -1
    table[4, (n - 1) // 16] = 2 ** 31 - 1
    table[5, -1] = -7                          # not needed: anything may stand there
    sums = torch.rand(6, 2, cap, device=DEV)
    before = sums.clone()
    out, lse, st = sv.paged_attention(q.to(DEV), kv.to(DEV), table.to(DEV), lens.to(DEV),
                                      weight_sum=sums, return_lse=True)
    L, G = sv.SV_ROW_BAD_LEN, sv.SV_ROW_BAD_PAGE
    assert st.tolist() == [L, L, G, G, G, 0]
    assert torch.isnan(out[:5]).all() and torch.isnan(lse[:5]).all()
    assert torch.equal(sums[:5], before[:5]) and not torch.equal(sums[5], before[5])
    if n == 40:
        assert torch.equal(out[5], want[5]) and torch.equal(lse[5], wlse[5])
    else:                                      # split otherwise: equal within the output's half unit
        assert torch.allclose(out[5].float(), want[5].float(), rtol=2.0 ** -7, atol=1e-4)


def test_layouts_agree_bit_for_bit():
    """[2][P] and [P][2] orders, a pool inside a larger one, other page ids."""
    q, kv, table, lens = make([300, 777], 8, 2, 128, 16, seed=8)
    d = [t.to(DEV) for t in (q, kv, table, lens)]
    want = sv.paged_attention(*d).clone()
    by_page = d[1].transpose(0, 1).contiguous().transpose(0, 1)
    assert by_page.stride(1) > by_page.stride(0)
    assert torch.equal(sv.paged_attention(d[0], by_page, d[2], d[3]), want)
    wide = torch.full((2, 2 * kv.shape[1], 16, 2, 128), float("nan"), dtype=q.dtype, device=DEV)
    wide[:, ::2] = d[1]
    assert torch.equal(sv.paged_attention(d[0], wide[:, ::2], d[2], d[3]), want)
    layers = torch.zeros(3, *kv.shape, dtype=q.dtype, device=DEV)
    layers[1] = d[1]
    assert torch.equal(sv.paged_attention(d[0], layers[1], d[2], d[3]), want)
    table[1, :10] = table[0, :10]              # shared pages: a common prefix
    check(q, kv, table, lens)


def test_a_contiguous_cache_is_one_page_a_sequence():
    """The library's own cache layout [2][B][S][Hkv][D], any S, slots past the
    sequences holding anything."""
    for S in (256, 300, 7):
        q, kv, table, lens = make([S, S // 2], 8, 2, 64, S, seed=S, spare=0, extra_pages=0)
        check(q, kv, table, lens, weights=True)


def test_a_table_far_longer_than_its_sequences():
    """Room for a million slots a sequence, a few used: the sums too."""
    q, kv, table, lens = make([700, 20, 3001], 8, 2, 64, 16, seed=21, extra_pages=0)
    long = torch.full((3, 60000), -1, dtype=torch.int32)
    long[:, :table.shape[1]] = table
    d = [t.to(DEV) for t in (q, kv)]
    sums = torch.zeros(3, 2, 960000, device=DEV)
    out, lse, st = sv.paged_attention(*d, long.to(DEV), lens.to(DEV), weight_sum=sums, return_lse=True)
    assert not st.any()
    small = torch.zeros(3, 2, table.shape[1] * 16, device=DEV)
    want, wlse, _ = sv.paged_attention(*d, table.to(DEV), lens.to(DEV), weight_sum=small, return_lse=True)
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    assert torch.equal(sums[..., :small.shape[2]], small) and not sums[..., small.shape[2]:].any()


def test_rows_of_the_output_alone_are_written():
    q, kv, table, lens = make([100, 50], 8, 2, 64, 16, seed=9)
    d = [t.to(DEV) for t in (q, kv, table, lens)]
    ws = torch.empty(sv.sv_paged_attention_workspace(2, 8, 2, 64, 16, table.shape[1]),
                     dtype=torch.uint8, device=DEV)
    out = torch.full((4, 8, 64), 7.0, dtype=q.dtype, device=DEV)
    lse = torch.full((4, 8), 7.0, device=DEV)
    st = torch.full((4,), 7, dtype=torch.int32, device=DEV)
    sv.sv_paged_attention(*d, 0, 0, 0.125, None, out[1:3], lse[1:3], st[1:3], ws)
    want, wl, _ = sv.paged_attention(*d, scale=0.125, return_lse=True)
    assert torch.equal(out[1:3], want) and torch.equal(lse[1:3], wl) and st.tolist() == [7, 0, 0, 7]
    for t in (out, lse):
        assert (t[0] == 7).all() and (t[3] == 7).all()


def test_repeats_streams_and_graphs():
    """The same bits from run to run, on two streams at once with a workspace
    each, and from a captured graph whose lengths grow between replays."""
    q, kv, table, lens = make([4000, 9, 2500], 16, 2, 128, 16, seed=10)
    d = [t.to(DEV) for t in (q, kv, table, lens)]
    kv2 = torch.nan_to_num(d[1], nan=0.5)
    table2 = torch.arange(3 * table.shape[1], dtype=torch.int32, device=DEV).view(3, -1)
    args = (d[0], kv2, table2, d[3])
    want = sv.paged_attention(*args).clone()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(4):
        a, b = sv.paged_attention(*args, stream=s1), sv.paged_attention(*args, stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(a, want) and torch.equal(b, want)
    ln = d[3].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = sv.paged_attention(d[0], kv2, table2, ln)
    for step in (0, 1, 16):
        ln.copy_(d[3] + step)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, sv.paged_attention(d[0], kv2, table2, ln)), step


@pytest.mark.parametrize("B,Hkv", [(60, 2), (700, 1)])
def test_streams_and_graphs_of_batches(B, Hkv):
    """As above for a batch in shares and one found by a map, with weight sums:
    every sequence's length changes between replays, some to 0 and back."""
    top = 90000 // B
    g = torch.Generator().manual_seed(B)
    lens = [int(x) for x in torch.randint(0, top, (B,), generator=g)]
    q, kv, table, n = [t.to(DEV) for t in make(lens, 4 * Hkv, Hkv, 64, 16, seed=B)]
    kv = torch.nan_to_num(kv, nan=0.5)
    table = torch.arange(B * table.shape[1], dtype=torch.int32, device=DEV).view(B, -1)
    cap = table.shape[1] * 16
    sums = [torch.zeros(B, Hkv, cap, device=DEV) for _ in range(4)]

    def call(n, w, **kw):
        return sv.paged_attention(q, kv, table, n, weight_sum=w, return_lse=True, **kw)
    want = call(n, sums[0])
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    a, b = call(n, sums[1], stream=s1), call(n, sums[2], stream=s2)
    torch.cuda.synchronize()
    for x, y, z in zip(want, a, b):
        assert torch.equal(x, y) and torch.equal(x, z)
    assert torch.equal(sums[0], sums[1]) and torch.equal(sums[0], sums[2])
    ln = n.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(ln, sums[3])
    sums[3].zero_()
    for seed in range(4):
        ln.copy_(torch.randint(0, top, (B,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32))
        ln[seed::7] = 0
        ln[3] = cap if seed % 2 else 1
        before = sums[3].clone()
        graph.replay()
        torch.cuda.synchronize()
        want = call(ln, before)
        for x, y in zip(want, out):
            assert torch.equal(x, y), seed
        assert torch.equal(before, sums[3]), seed


def test_empty_batch_host_memory_and_refusals():
    q, kv, table, lens = make([150, 90], 8, 2, 64, 16, seed=12)
    d = [t.to(DEV) for t in (q, kv, table, lens)]
    out, lse, st = sv.paged_attention(d[0][:0], d[1], d[2][:0], d[3][:0], return_lse=True)
    assert out.shape == (0, 8, 64) and lse.shape == (0, 8) and st.shape == (0,)
    want = sv.paged_attention(*d)
    got = sv.paged_attention(*[t.pin_memory() for t in (q, kv, table, lens)])
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    n0 = sv.sv_launch_count()
    sums = torch.zeros(2, 2, 40, device=DEV)
    for kw in (dict(scale=0.0), dict(window=-1), dict(weight_sum=sums),
               dict(weight_sum=torch.zeros(2, 2, 400, device=DEV),
                    workspace=torch.empty(8, dtype=torch.uint8, device=DEV))):
        with pytest.raises(sv.SvError):
            sv.paged_attention(*d, **kw)
    flat = torch.zeros(2 * 8 * 64 + 1, dtype=q.dtype, device=DEV)
    with pytest.raises(sv.SvError):                # q off the 16-byte grid
        sv.paged_attention(flat[1:].view(2, 8, 64), *d[1:])
    assert sv.sv_launch_count() == n0


def test_two_host_threads():
    """Calls of two threads at once, each on a stream of its own."""
    import threading
    jobs, results = [], {}
    for i in range(2):
        q, kv, table, lens = make([3000 + 700 * i, 40], 8, 2, 128, 16, seed=30 + i)
        jobs.append([t.to(DEV) for t in (q, kv, table, lens)])
    want = [sv.paged_attention(*j) for j in jobs]
    torch.cuda.synchronize()

    def work(i):
        s = torch.cuda.Stream()
        r = [sv.paged_attention(*jobs[i], stream=s) for _ in range(20)]
        s.synchronize()
        results[i] = r
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in results[i])


def test_offsets_past_32_bits():
    """A pool of more than 2^32 elements whose last pages are the ones used."""
    page, Hkv, D = 64, 8, 128
    P = (1 << 32) // (page * Hkv * D) + 40
    kv = torch.empty(2, P, page, Hkv, D, dtype=torch.bfloat16, device=DEV)
    q, small, table, lens = make([900, 1300], 8, 8, D, page, seed=11)
    n = small.shape[1]
    kv[:, P - n:] = small.to(DEV)
    want = sv.paged_attention(q.to(DEV), small.to(DEV), table.to(DEV), lens.to(DEV))
    moved = torch.where(table >= 0, table + (P - n), table)
    got = sv.paged_attention(q.to(DEV), kv, moved.to(DEV), lens.to(DEV))
    assert torch.equal(got, want)


def test_the_layer_of_the_dynamic_tree_workload():
    """64 query heads on 8 KV heads of 128 over about 4096 tokens, 128
    sequences; a few of them replayed."""
    B, page = 128, 16
    g = torch.Generator(device=DEV).manual_seed(2)
    lens = torch.randint(3585, 4097, (B,), generator=g, device=DEV, dtype=torch.int32)
    kv = torch.empty(2, B * 256, page, 8, 128, dtype=torch.bfloat16, device=DEV)
    kv.normal_(generator=g)
    table = torch.randperm(B * 256, generator=g, device=DEV).to(torch.int32).view(B, 256)
    q = torch.randn(B, 64, 128, generator=g, device=DEV).to(torch.bfloat16)
    sums = torch.zeros(B, 8, 4096, device=DEV)
    out, lse, st = sv.paged_attention(q, kv, table, lens, weight_sum=sums, return_lse=True)
    assert not st.any()
    assert torch.allclose(sums.sum(-1), torch.full((B, 8), 8.0, device=DEV), atol=1e-4)
    for b in (0, 63, 127):
        own = table[b].long()
        small = kv[:, own].cpu()
        t = torch.arange(256, dtype=torch.int32)[None]
        ref, rlse, got, size = reference(q[b:b + 1].cpu(), small, t, lens[b:b + 1].cpu(), 128 ** -0.5)
        d = (128 + 4) * U * size.max() + 2.0 ** -22 + 4096 * U
        tol = 2.0 ** -8 * np.abs(ref) + (2 * d + 2.0 ** -17) * 6
        assert (np.abs(out[b:b + 1].double().cpu().numpy() - ref) <= tol).all()
        assert np.abs(lse[b:b + 1].double().cpu().numpy() - rlse).max() <= d + 60 * U


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("level,lens,Hkv,G", [
    (64, [200, 33, 1, 130], 8, 1),       # scores about 4096, whole sequences
    (128, [200, 64], 4, 3),              # about 16384
    (64, [140, 7], 2, 4),                # four heads' scores in one load
    (128, [2000, 500], 4, 4),            # split and joined
    (128, [1500] + [90] * 59, 2, 1),     # shares
])
def test_weights_of_large_scores_sum_to_one(level, lens, Hkv, G, dtype):
    """Scores c + x, c = level (level + head) thousands and x a multiple of 1/64
    in [-2, 2], scale 1: exact in fp32 whatever the order, so a weight is
    softmax(x) however large c is.  In units of u, relative: fp32 log2 e is off
    by 1, for scores 4 apart 4 log2 e of it; the exponent, one rounding of at most
    2 + 4 log2 e + 15 < 32 (the reference lies within 15 of the largest, and its
    own rounding is common to a row): (6 + 32) ln 2 < 27 and 4 for the base-2
    exponential, in the weight and in the sum alike; n for the sum; 6 for each
    of at most five changes of reference; 1 / sum, the product and G additions."""
    D, page = 64, 16
    q, kv, table, n = make(lens, Hkv * G, Hkv, D, page, dtype, seed=level + G)
    q.zero_()
    q[..., 0] = (level + torch.arange(Hkv * G)).to(dtype)
    q[..., 1] = 1
    x = torch.randint(-128, 129, kv[0, ..., 0].shape, generator=torch.Generator().manual_seed(G)) / 64
    kv[0, ..., 0] = level
    kv[0, ..., 1] = x.to(dtype)
    kv[0, ..., 2:] = 0
    sums = torch.zeros(len(lens), Hkv, table.shape[1] * page, device=DEV)
    _, lse, st = sv.paged_attention(q.to(DEV), kv.to(DEV), table.to(DEV), n.to(DEV), 1.0, weight_sum=sums,
                                    return_lse=True)
    assert not st.any() and lse.min() > level * level
    for b, k in enumerate(lens):
        j = torch.arange(k)
        want = G * torch.softmax(x[table[b, j // page].long(), j % page].double(), 0).T
        d = (2 * (27 + 4) + k + 5 * 6 + 2 + G) * U
        got = sums[b, :, :k].double().cpu()
        assert ((got - want).abs() <= d * want).all(), float(((got - want).abs() / want).max() / d)
        assert not sums[b, :, k:].any()


def test_weights_of_the_most_query_heads():
    """8192 query heads on one KV head: every row's reference and sum wait beside
    one another."""
    check(*make([20, 70], 8192, 1, 64, 16, seed=5), weights=True)
