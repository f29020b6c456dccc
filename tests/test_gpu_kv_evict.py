"""sv_kv_evict against the plain definition (tests/plain_serving.py): kept
slots, moved rows, weights and lengths are copies and whole numbers, so all of
them have to be equal, byte for byte."""
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


def make(L, lens, Hkv, D, page, dtype=torch.bfloat16, seed=0, zeros=0.2, coarse=False):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    per = max(1, -(-max(lens) // page)) + 1
    need = [-(-n // page) for n in lens]
    P = sum(need) + 3
    kv = torch.randint(-100, 100, (L, 2, P, page, Hkv, D), generator=g).to(dtype)
    ids = torch.randperm(P, generator=g).to(torch.int32)
    table = torch.full((B, per), -9, dtype=torch.int32)   # entries nothing needs
    for b, k in enumerate(need):
        table[b, :k] = ids[sum(need[:b]):sum(need[:b]) + k]
    w = torch.randn(L, B, Hkv, per * page + 5, generator=g).exp()
    if coarse:
        w = torch.round(w * 2) / 2                 # many equal weights
    w *= torch.rand(w.shape, generator=g) > zeros
    return kv, table, torch.tensor(lens, dtype=torch.int32), w


def run(kv, table, lens, w, budget, sinks, recent, apart=False, **kw):
    d = [t.to(DEV) for t in (kv, table, lens, w)]
    out = torch.full_like(d[3], 7.0) if apart else None
    kept, n, st = sv.kv_evict(*d, budget, sinks, recent, out_weight_sum=out, **kw)
    torch.cuda.synchronize()
    return d[0].cpu(), (out if apart else d[3]).cpu().numpy(), kept.cpu().numpy(), n.cpu().numpy(), \
        st.cpu().numpy()


def as_bytes(t):
    return t.contiguous().view(torch.uint8).numpy().reshape(*t.shape[:-1], -1)


def check(kv, table, lens, w, budget, sinks, recent):
    want = plain.kv_evict(as_bytes(kv), table.numpy(), lens.numpy(), w.numpy(), budget, sinks, recent)
    for apart in (False, True):
        k, ws, kept, n, st = run(kv, table, lens, w, budget, sinks, recent, apart)
        assert not st.any()
        assert np.array_equal(kept, want[2])
        assert np.array_equal(n, want[3])
        assert np.array_equal(as_bytes(k), want[0])
        ref = want[1].copy()
        if apart:                                  # slots past a sequence stay as they were
            for b, m in enumerate(lens.tolist()):
                ref[:, b, :, m:] = 7.0
        assert np.array_equal(ws, ref, equal_nan=True)


@pytest.mark.parametrize("L,lens,Hkv,D,page,dtype,budget,sinks,recent", [
    (1, [20], 1, 64, 16, torch.bfloat16, 12, 2, 3),
    (2, [100, 0, 1, 64, 65, 129], 2, 128, 16, torch.bfloat16, 64, 4, 16),  # some under the budget
    (1, [300, 299], 3, 64, 24, torch.float16, 100, 0, 0),                  # no first, no recent
    (3, [500], 2, 256, 7, torch.bfloat16, 450, 1, 449),                    # nothing but those
    (1, [700, 350], 8, 32, 33, torch.float32, 1, 0, 0),                    # one slot
    (1, [700], 2, 32, 8, torch.float32, 1, 0, 1),                          # the last slot alone
    (2, [90, 200], 2, 6, 16, torch.bfloat16, 50, 3, 10),                   # rows of 12 bytes
    (1, [200], 2, 20, 16, torch.int8, 70, 3, 10),                          # rows of 20 bytes
    (1, [129, 4000], 1, 128, 1, torch.float16, 128, 5, 60),
])
def test_matches_the_definition(L, lens, Hkv, D, page, dtype, budget, sinks, recent):
    for seed, coarse in ((0, False), (1, True)):
        check(*make(L, lens, Hkv, D, page, dtype, seed, coarse=coarse), budget, sinks, recent)


@pytest.mark.parametrize("budget,recent", [(4096, 512), (20000, 1), (29000, 7000)])
def test_one_long_sequence(budget, recent):
    """Several CTAs choose together; column ranges move apart."""
    check(*make(1, [30011], 2, 64, 64, seed=budget), budget, 4, recent)


@pytest.mark.parametrize("L,lens,Hkv,page,budget", [
    (1, [20000, 9000, 3, 12000, 9001], 4, 64, 5000),     # 20 heads: clusters of 6 that choose together
    (5, [10000], 5, 33, 1000),                           # 25: clusters of 5
    (1, [9500, 200], 17, 16, 333),                       # 34: of 4
    (2, [8300] + [40] * 24, 3, 16, 33),                  # 150: single CTAs
    (2, [9000, 700] + [60] * 18, 4, 32, 50),             # 160: small CTAs, keys read again
    (1, [50000] + [30] * 24, 4, 64, 7),                  # 100, long: large CTAs, keys read again
])
def test_every_arrangement_of_the_work(L, lens, Hkv, page, budget):
    check(*make(L, lens, Hkv, 8, page, seed=budget, coarse=budget % 2 == 1), budget, 1, 3)


def test_equal_weights_keep_the_lower_slots():
    kv, table, lens, w = make(1, [1000], 2, 64, 16, seed=2)
    w.fill_(0.25)
    check(kv, table, lens, w, 300, 4, 100)
    w[0, 0, 0, ::2] = -0.0
    w[0, 0, 0, 1::2] = 0.0                         # equal too
    check(kv, table, lens, w, 300, 4, 100)


def test_odd_weights():
    """NaN below everything, infinities at the ends, negatives, denormals."""
    kv, table, lens, w = make(2, [400, 390], 2, 64, 16, seed=3)
    g = torch.Generator().manual_seed(1)
    w = torch.randn(w.shape, generator=g)
    w[..., 10:300:7] = float("nan")
    w[..., 11:300:13] = float("-inf")
    w[..., 12:300:31] = float("inf")
    w[..., 50:90] *= 1e-41
    check(kv, table, lens, w, 200, 2, 20)
    check(kv, table, lens, w, 360, 2, 20)          # NaN slots have to stay too


@pytest.mark.parametrize("L,lens,Hkv,D,budget", [
    (1, [1000, 77], 2, 8, 60),                           # a few CTAs choose the same
    (1, [12345], 2, 64, 9000),                           # and each a part
    (1, [50003] + [30] * 24, 4, 8, 30000),               # large CTAs, keys read again
    (2, [701, 260] + [90] * 18, 4, 8, 200),              # small CTAs
    (2, [9001, 700] + [60] * 18, 4, 8, 8500),            # keys read again
])
@pytest.mark.parametrize("sinks,recent", [(0, 0), (3, 11)])
def test_so_many_nan_that_some_stay(L, lens, Hkv, D, budget, sinks, recent):
    """NaN ranks below every number, so the lowest limit there is counts the
    slots of NaN, and nothing that lies behind a part's last slot."""
    kv, table, n, w = make(L, lens, Hkv, D, 16, seed=budget)
    g = torch.Generator().manual_seed(5)
    for share, head in ((0.97, 0), (1.0, -1)):
        w[:, :, head][torch.rand(w[:, :, head].shape, generator=g) < share] = float("nan")
    check(kv, table, n, w, budget, sinks, recent)



def test_bad_lengths_and_pages_move_nothing():
    kv, table, lens, w = make(1, [100] * 6, 2, 64, 16, seed=4)
    cap = table.shape[1] * 16
    lens[0], lens[1] = -1, cap + 1
    table[2, 3], table[3, 0], table[4, 6] = kv.shape[2], -1, -1
    k, ws, kept, n, st = run(kv, table, lens, w, 60, 2, 10)
    Ln, Pg = sv.SV_ROW_BAD_LEN, sv.SV_ROW_BAD_PAGE
    assert st.tolist() == [Ln, Ln, Pg, Pg, Pg, 0]
    assert n.tolist() == [-1] * 5 + [60]
    assert (kept[:, :5] == -1).all()
    assert np.array_equal(ws[:, :5], w[:, :5].numpy())
    want = plain.kv_evict(as_bytes(kv), table[5:].numpy(), lens[5:].numpy(), w[:, 5:].numpy(), 60, 2, 10)
    assert np.array_equal(as_bytes(k), want[0]) and np.array_equal(kept[:, 5:], want[2])


def test_layouts():
    """[P][2] order of the page pool, layers apart, pages inside wider ones."""
    kv, table, lens, w = make(2, [150, 90], 2, 64, 16, seed=5)
    d = [t.to(DEV) for t in (table, lens)]
    a, wa = kv.to(DEV), w.to(DEV)
    sv.kv_evict(a, *d, wa, 80, 4, 10)
    b, wb = kv.to(DEV).transpose(1, 2).contiguous().transpose(1, 2), w.to(DEV)
    sv.kv_evict(b, *d, wb, 80, 4, 10)
    wide = torch.zeros(4, 2, 3 * kv.shape[2], *kv.shape[3:], dtype=kv.dtype, device=DEV)
    c, wc = wide[1::2, :, ::3], w.to(DEV)
    c.copy_(kv.to(DEV))
    sv.kv_evict(c, *d, wc, 80, 4, 10)
    assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(wa, wb) and torch.equal(wa, wc)
    assert not wide[::2].any() and not wide[:, :, 1::3].any()


def test_other_sequences_pages_and_other_heads_slots_stay():
    kv, table, lens, w = make(1, [200, 40], 2, 64, 16, seed=6)
    k = run(kv, table, lens, w, 64, 0, 8)[0]
    used = table[0, :-(-200 // 16)].long()
    rest = torch.ones(kv.shape[2], dtype=torch.bool)
    rest[used] = False
    assert torch.equal(k[:, :, rest], kv[:, :, rest])
    tail = used[4:]                                # slots 64.. of the evicted sequence
    assert torch.equal(k[:, :, tail], kv[:, :, tail])


def test_streams_and_graphs():
    kv, table, lens, w = make(2, [3000, 2500, 100], 4, 64, 16, seed=7)
    want = plain.kv_evict(as_bytes(kv), table.numpy(), lens.numpy(), w.numpy(), 1024, 4, 100)
    d = [t.to(DEV) for t in (kv, table, lens, w)]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    kvs = [d[0].clone(), d[0].clone()]
    torch.cuda.synchronize()
    r = [sv.kv_evict(k, d[1], d[2], d[3], 1024, 4, 100, out_weight_sum=torch.zeros_like(d[3]), stream=s)
         for k, s in zip(kvs, (s1, s2))]
    torch.cuda.synchronize()
    for k, x in zip(kvs, r):
        assert np.array_equal(as_bytes(k.cpu()), want[0]) and np.array_equal(x[0].cpu().numpy(), want[2])
    k, n, ws = d[0].clone(), d[2].clone(), d[3].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept, new, _ = sv.kv_evict(k, d[1], n, ws, 1024, 4, 100)
    for _ in range(2):
        k.copy_(d[0])
        ws.copy_(d[3])
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(as_bytes(k.cpu()), want[0]) and np.array_equal(kept.cpu().numpy(), want[2])
        assert np.array_equal(ws.cpu().numpy(), want[1]) and new.tolist() == [1024, 1024, 100]
    n.copy_(new)                                   # under the budget now: the next replay moves nothing
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(as_bytes(k.cpu()), want[0]) and np.array_equal(ws.cpu().numpy(), want[1])


def test_empty_batch_and_host_memory():
    kv, table, lens, w = make(1, [150, 90], 2, 64, 16, seed=12)
    d = [t.to(DEV) for t in (kv, table, lens, w)]
    kept, n, st = sv.kv_evict(d[0], d[1][:0], d[2][:0], d[3][:, :0], 8)
    assert kept.shape == (1, 0, 2, 8) and n.shape == (0,) and torch.equal(d[0].cpu(), kv)
    want = plain.kv_evict(as_bytes(kv), table.numpy(), lens.numpy(), w.numpy(), 64, 4, 8)
    h = [t.pin_memory() for t in (kv, table, lens, w)]
    kept, n, _ = sv.kv_evict(*h, 64, 4, 8)
    torch.cuda.synchronize()
    assert np.array_equal(as_bytes(h[0]), want[0]) and np.array_equal(h[3].numpy(), want[1])
    assert np.array_equal(kept.cpu().numpy(), want[2])


def test_refusals_leave_everything():
    kv, table, lens, w = [t.to(DEV) for t in make(1, [100], 2, 64, 16, seed=13)]
    before = kv.clone(), w.clone()
    n0 = sv.sv_launch_count()
    for kw in (dict(budget=0), dict(budget=20, sinks=15, recent=6), dict(budget=20, sinks=-1)):
        with pytest.raises(sv.SvError):
            sv.kv_evict(kv, table, lens, w, **kw)
    flat = torch.zeros(w.numel() + 4, device=DEV)
    with pytest.raises(sv.SvError):          # a shifted part of the weights themselves
        sv.kv_evict(kv, table, lens, flat[:-4].view(w.shape), 20, out_weight_sum=flat[4:].view(w.shape))
    with pytest.raises(sv.SvError):
        sv.kv_evict(kv, table, lens, w, 20, workspace=torch.empty(8, dtype=torch.uint8, device=DEV))
    assert sv.sv_launch_count() == n0
    assert torch.equal(kv, before[0]) and torch.equal(w, before[1])


def test_offsets_past_32_bits():
    page, Hkv, D = 64, 8, 128
    P = (1 << 32) // (page * Hkv * D) + 40
    small, table, lens, w = make(1, [700, 900], Hkv, D, page, seed=8)
    n = small.shape[2]
    kv = torch.empty(1, 2, P, page, Hkv, D, dtype=torch.bfloat16, device=DEV)
    kv[:, :, P - n:] = small.to(DEV)
    moved = torch.where(table >= 0, table + (P - n), table)
    sv.kv_evict(kv, moved.to(DEV), lens.to(DEV), w.to(DEV), 256, 4, 32)
    want = plain.kv_evict(as_bytes(small), table.numpy(), lens.numpy(), w.numpy(), 256, 4, 32)[0]
    assert np.array_equal(as_bytes(kv[:, :, P - n:].cpu()), want)


def test_a_draft_loop_under_a_budget():
    """The operators as they are used together: a draft head decodes over a
    paged cache and sums its attention weights, the cache is brought back under
    its budget, decoding goes on over what was kept, and the drafts are
    verified from probabilities."""
    B, Hq, Hkv, D, page, budget = 3, 8, 2, 64, 16, 40
    g = torch.Generator().manual_seed(9)
    per, V = 5, 501
    kv = torch.zeros(1, 2, B * per, page, Hkv, D, dtype=torch.bfloat16, device=DEV)
    table = torch.randperm(B * per, generator=g).view(B, per).to(torch.int32).to(DEV)
    lens = torch.tensor([30, 12, 39], dtype=torch.int32, device=DEV)
    sums = torch.zeros(1, B, Hkv, per * page, device=DEV)
    rows = [[torch.randn(2, Hkv, D, generator=g) for _ in range(int(n))] for n in lens]  # what is cached
    head = torch.randn(Hq * D, V, generator=g).to(DEV) * 0.1

    def put(b, j, x):
        kv[0, :, table[b, j // page].long(), j % page] = x.to(torch.bfloat16).to(DEV)
    for b in range(B):
        for j, x in enumerate(rows[b]):
            put(b, j, x)
    probs = []
    kept_rows = [[list(r) for _ in range(Hkv)] for r in rows]     # per head, after evictions
    for step in range(30):
        new = torch.randn(B, 2, Hkv, D, generator=g)
        for b in range(B):
            put(b, int(lens[b]), new[b])
            for h in range(Hkv):
                kept_rows[b][h].append(new[b])
        lens = lens + 1
        q = torch.randn(B, Hq, D, generator=g).to(torch.bfloat16).to(DEV)
        out, lse, st = sv.paged_attention(q, kv[0], table, lens, weight_sum=sums[0], return_lse=True)
        assert not st.any()
        for b in range(B):                                        # against what each head still holds
            for h in range(Hkv):
                x = torch.stack([r[:, h] for r in kept_rows[b][h]]).to(torch.bfloat16).double()
                s = q[b, h * 4:(h + 1) * 4].double().cpu() @ x[:, 0].T * D ** -0.5
                want = torch.softmax(s, -1) @ x[:, 1]
                got = out[b, h * 4:(h + 1) * 4].double().cpu()
                # half a unit of bf16, and the bound of the paged attention's tests
                # with scale sum |q k| <= 16: 2 (68 2^-24 16 + 2^-22) + 2^-17 < 2^-12
                tol = 2.0 ** -8 * want.abs() + 2.0 ** -12 * x[:, 1].abs().max()
                assert ((got - want).abs() <= tol).all()
        probs.append(torch.softmax(out.float().view(B, -1) @ head, -1))
        before = sums.clone()
        kept, lens, st = sv.kv_evict(kv, table, lens, sums, budget, 2, 8)
        assert not st.any() and int(lens.max()) <= budget
        for b in range(B):
            for h in range(Hkv):
                k = [int(j) for j in kept[0, b, h] if j >= 0]
                assert k == plain.kept_slots(before[0, b, h].cpu().numpy(), len(kept_rows[b][h]),
                                             budget, 2, 8)
                kept_rows[b][h] = [kept_rows[b][h][j] for j in k]
    p = torch.stack(probs[-4:], 1)
    q = torch.softmax(torch.log(torch.cat([p, p[:, :1]], 1)) + 0.3 * torch.randn(B, 5, V, generator=g).to(DEV), -1)
    d = torch.multinomial(p.reshape(-1, V).cpu(), 1, generator=g).view(B, 4).to(torch.int32).to(DEV)
    ua, us = torch.rand(B, 4, generator=g).to(DEV), torch.rand(B, generator=g).to(DEV)
    r = sv.verify_chain_probs(q, p, d, ua, us)
    want = plain.verify_probs(*[t.cpu().numpy() for t in (q, p, d, ua, us)])
    for k, x in zip(("tokens", "accept_len", "status"), want):
        assert np.array_equal(r[k].cpu().numpy(), x)
