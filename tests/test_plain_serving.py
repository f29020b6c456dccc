"""CPU pins of the plain definitions the serving operators are tested against,
and the host-side refusals of those operators."""
import numpy as np
import pytest
import torch

import plain_serving as plain


@pytest.fixture(scope="module")
def sv():
    from speculative_decoding_verification_vocab_gb300 import _build
    _build.build()
    import speculative_decoding_verification_vocab_gb300 as m
    m.load_library()
    return m


def test_verification_keeps_the_targets_law():
    """Drafts from p, uniforms on a dense grid: the first emitted token follows
    q, within the grid's step; a walk that swaps the rows does not."""
    q = np.array([[0.5, 0.25, 0.125, 0.125]] * 2, np.float32)
    p = np.array([[0.125, 0.125, 0.5, 0.25]], np.float32)
    G = 64
    u = (np.arange(G, dtype=np.float32) + 0.5) / G

    def law(q, p):
        mass = np.zeros(4)
        for d in range(4):
            for a in u:
                for s in u:
                    t, _, st = plain.verify_one(q, p, np.array([d]), np.array([a]), s)
                    assert st == 0
                    mass[t[0]] += p[0, d] / (G * G)
        return mass
    assert np.abs(law(q, p) - q[0]).max() < 2 / G
    wrong = np.concatenate([p, p])
    assert np.abs(law(wrong, q[:1]) - q[0]).max() > 0.1


def test_one_hot_equals_a_point_mass():
    rng = np.random.default_rng(0)
    for _ in range(50):
        q = rng.dirichlet(np.ones(9), 4).astype(np.float32)
        d = rng.integers(0, 9, 3)
        p = np.zeros((3, 9), np.float32)
        p[np.arange(3), d] = 1
        ua, us = rng.random(3, np.float32) * 0.3, np.float32(rng.random())
        assert plain.verify_one(q, None, d, ua, us) == plain.verify_one(q, p, d, ua, us)


def test_draw_is_the_inverse_cdf():
    rng = np.random.default_rng(1)
    for _ in range(200):
        w = rng.random(50).astype(np.float32)
        u = np.float32(rng.random())
        c = np.cumsum(w.astype(np.float64))
        near = np.abs(c - u * c[-1]).min() < 1e-12
        assert near or plain._draw(w, u) == int((c <= np.float64(u) * c[-1]).sum())


def test_verify_probs_host_checks(sv):
    """Bad arguments are refused before any CUDA call (no GPU here)."""
    f = sv.load_library().sv_verify_chain_probs
    x = 4096  # never looked at: the refusals below come first

    def call(qs=30, qr=10, p=None, ps=20, pr=10, dt=0, d=x, n=None, ua=x, us=x, B=1, N=2, V=10, t=x,
             a=x, s=x, q=x):
        return f(q, qs, qr, p, ps, pr, dt, d, n, ua, us, B, N, V, t, a, s, None)
    assert call(B=-1) == 1 and call(N=-1) == 1 and call(V=0) == 1
    assert call(dt=2) == 1 and b"SV_F32" in sv.load_library().sv_last_error()
    assert call(qs=-1) == 1 and call(qr=-1) == 1 and call(p=x, pr=-8) == 1
    assert b"stride" in sv.load_library().sv_last_error()
    assert call(qr=2 ** 61) == 1 and call(p=x, ps=2 ** 62) == 1
    assert call(V=(1 << 22) + 1) == 2 and call(N=1025) == 2
    assert call(q=None) == 1 and call(us=None) == 1 and call(d=None) == 1 and call(ua=None) == 1
    assert call(t=None) == 1 and call(a=None) == 1 and call(s=None) == 1
    assert b"null" in sv.load_library().sv_last_error()
    assert call(q=x + 2) == 1 and call(us=x + 1) == 1
    assert b"misaligned" in sv.load_library().sv_last_error()
    assert call(B=0, q=None, us=None) == 0


def test_verify_probs_binding_refusals(sv):
    q, p = torch.zeros(2, 3, 8), torch.zeros(2, 2, 8)
    d, ua, us = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2), torch.zeros(2)
    o = (torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
         torch.zeros(2, dtype=torch.int32))

    def call(q=q, p=p, d=d, n=None, ua=ua, us=us, o=o):
        with pytest.raises(ValueError):
            sv.sv_verify_chain_probs(q, p, d, n, ua, us, *o)
    call(p=p.bfloat16())                                   # another type than q
    call(p=torch.zeros(2, 3, 8))                           # another shape
    call(q=torch.zeros(2, 8, 3).transpose(1, 2))           # columns apart
    call(d=d.long()), call(ua=ua.double()), call(us=us[:1])
    call(n=torch.zeros(3, dtype=torch.int32))
    call(d=torch.zeros(2, 4, dtype=torch.int32)[:, ::2])
    call()                                                 # pageable host memory


def test_paged_attention_plain_equals_dense_attention():
    """The plain paged form against torch's dense attention on gathered rows,
    with and without a window."""
    g = torch.Generator().manual_seed(0)
    q = torch.randn(2, 6, 32, generator=g, dtype=torch.float64)
    kv = torch.randn(2, 9, 5, 2, 32, generator=g, dtype=torch.float64)
    table = torch.randperm(9, generator=g)[:8].view(2, 4)
    for window, sinks, lens in ((0, 0, [17, 3]), (6, 2, [20, 7])):
        out, lse, got, _ = plain.paged_attention(q.numpy(), kv.numpy(), table.numpy(),
                                                 np.array(lens), 0.2, window, sinks)
        for b in range(2):
            n = lens[b]
            rows = kv[:, table[b]].reshape(2, 20, 2, 32)[:, :n].repeat_interleave(3, 2)
            seen = torch.tensor([window == 0 or j >= n - window or j < sinks for j in range(n)])
            want = torch.nn.functional.scaled_dot_product_attention(
                q[b][:, None], rows[0].transpose(0, 1), rows[1].transpose(0, 1),
                attn_mask=seen[None, None], scale=0.2)[:, 0]
            assert np.allclose(out[b], want.numpy(), atol=1e-12)
            assert np.allclose(got[b].sum(-1), 3) and not got[b][:, :n][:, ~seen.numpy()].any()


def test_paged_attention_host_checks(sv):
    lib = sv.load_library()
    f, x = lib.sv_paged_attention, 4096

    def call(q=x, kv=x, ks=1 << 20, ps=16 * 2 * 128, dt=1, table=x, lens=x, B=1, Hq=8, Hkv=2, D=128,
             page=16, mp=4, P=8, window=0, sinks=0, scale=1.0, w=None, S=0, out=x, lse=None, st=None,
             ws=x, wb=1 << 30):
        return f(q, kv, ks, ps, dt, table, lens, B, Hq, Hkv, D, page, mp, P, window, sinks, scale, w, S,
                 out, lse, st, ws, wb, None)
    assert call(B=-1) == 1 and call(Hq=9) == 1 and call(page=0) == 1 and call(mp=0) == 1
    assert call(P=0) == 1 and call(window=-1) == 1 and call(sinks=-1) == 1 and call(Hkv=0) == 1
    assert call(dt=0) == 1 and call(D=96) == 2 and b"head dimension" in lib.sv_last_error()
    assert call(scale=0.0) == 1 and call(scale=float("nan")) == 1 and call(scale=float("inf")) == 1
    assert call(scale=3e38) == 1 and call(scale=-1.0) == 1
    assert call(page=1 << 20, mp=1 << 11, ps=1 << 40) == 2
    assert call(ps=16 * 2 * 128 - 8) == 1 and call(ps=16 * 2 * 128 + 4) == 1 and call(ks=-8) == 1
    assert call(w=x, S=63) == 1 and b"weight_sum" in lib.sv_last_error()
    assert call(q=None) == 1 and call(kv=None) == 1 and call(table=None) == 1
    assert call(lens=None) == 1 and call(out=None) == 1
    assert call(q=x + 8) == 1 and call(out=x + 2) == 1 and call(lens=x + 2) == 1
    assert call(mp=400, P=800, wb=16) == 1 and b"workspace" in lib.sv_last_error()
    assert call(B=0, q=None, kv=None) == 0
    ws = sv.sv_paged_attention_workspace
    assert ws(1, 8, 2, 128, 16, 4) == 0 or ws(1, 8, 2, 128, 16, 4) > 0
    assert ws(4, 8, 2, 128, 16, 400, weights=True) > ws(4, 8, 2, 128, 16, 400) > 0
    assert ws(4, 9, 2, 128, 16, 400) == 0 and ws(4, 8, 2, 128, 1 << 20, 1 << 11) == 0
    # a window bounds what is kept aside
    assert ws(4, 8, 2, 128, 16, 4000, 64, 4, True) < ws(4, 8, 2, 128, 16, 4000, 0, 0, True)


def test_paged_attention_binding_refusals(sv):
    bf = torch.bfloat16
    q, kv = torch.zeros(2, 8, 64, dtype=bf), torch.zeros(2, 6, 16, 2, 64, dtype=bf)
    t, n = torch.zeros(2, 3, dtype=torch.int32), torch.ones(2, dtype=torch.int32)

    def call(q=q, kv=kv, t=t, n=n, w=None, out=None, lse=None, st=None):
        with pytest.raises(ValueError):
            sv.sv_paged_attention(q, kv, t, n, 0, 0, 1.0, w, torch.empty_like(q) if out is None else out,
                                  lse, st)
    call(q=q.half()), call(q=q.float(), kv=kv.float()), call(kv=kv[..., :32])
    call(kv=kv.transpose(2, 3)), call(kv=kv[0]), call(kv=kv[:1])
    call(q=torch.zeros(2, 64, 8, dtype=bf).transpose(1, 2))
    call(t=t.long()), call(t=t[0]), call(n=n[:1]), call(n=n.long())
    call(w=torch.zeros(2, 8, 48)), call(w=torch.zeros(2, 2, 48, dtype=torch.float64))
    call(out=torch.zeros(2, 8, 64)), call(lse=torch.zeros(8, 2)), call(st=torch.zeros(2))
    call()                                                 # pageable host memory


def test_kept_slots_by_hand():
    w = np.array([5, 0, 3, 3, 9, 1, 3, 2], np.float32)
    assert plain.kept_slots(w, 8, 8, 1, 1) == list(range(8))
    assert plain.kept_slots(w, 8, 5, 1, 1) == [0, 2, 3, 4, 7]      # the tie at 3: the lower slots
    assert plain.kept_slots(w, 8, 2, 1, 1) == [0, 7]
    assert plain.kept_slots(w, 8, 3, 0, 0) == [0, 2, 4]
    w[4] = np.nan
    assert plain.kept_slots(w, 8, 4, 0, 0) == [0, 2, 3, 6]
    assert plain.kept_slots(w, 8, 8, 0, 0) == list(range(8)) and 4 not in plain.kept_slots(w, 8, 7, 0, 0)


def test_kv_evict_host_checks(sv):
    lib = sv.load_library()
    f, x = lib.sv_kv_evict, 4096

    def call(kv=x, ls=1 << 22, ks=1 << 20, ps=16 * 2 * 64, e=2, t=x, n=x, w=x, ow=x, L=2, B=1, H=2, D=64,
             page=16, mp=4, P=8, S=64, budget=32, sinks=2, recent=4, kept=x, kl=x, st=None, ws=x,
             wb=1 << 30):
        return f(kv, ls, ks, ps, e, t, n, w, ow, L, B, H, D, page, mp, P, S, budget, sinks, recent, kept,
                 kl, st, ws, wb, None)
    assert call(L=0) == 1 and call(B=-1) == 1 and call(H=0) == 1 and call(D=0) == 1 and call(e=0) == 1
    assert call(page=0) == 1 and call(mp=0) == 1 and call(P=0) == 1
    assert call(budget=0) == 1 and call(sinks=-1) == 1 and call(recent=-1) == 1
    assert call(sinks=30, recent=3) == 1 and b"budget" in lib.sv_last_error()
    assert call(sinks=2 ** 31 - 1, recent=2 ** 31 - 1) == 1
    assert call(page=1 << 20, mp=1 << 11, S=2 ** 31 - 1) == 2
    assert call(S=63) == 1 and call(D=3, e=1, ps=1 << 12) == 2
    assert call(ps=16 * 2 * 64 - 1) == 1 and call(ks=0) == 1 and call(ls=0) == 1 and call(ls=-4) == 1
    assert call(ps=2 ** 62) == 1 and call(ls=2 ** 62) == 1
    for name in ("kv", "t", "n", "w", "ow", "kept", "kl", "ws"):
        assert call(**{name: None}) == 1 and b"null" in lib.sv_last_error(), name
    assert call(kv=x + 2) == 1 and call(w=x + 2) == 1 and call(ws=x + 64) == 1
    assert call(ps=16 * 2 * 64 + 1) == 1 and b"misaligned" in lib.sv_last_error()
    assert call(wb=100) == 1 and b"workspace" in lib.sv_last_error()
    y = 1 << 20
    assert call(ow=x + 64, kl=y) == 1 and b"out_weight_sum overlaps" in lib.sv_last_error()
    assert call(ow=x, kl=x) == 1 and b"out_kv_len overlaps" in lib.sv_last_error()
    assert call(D=1025, e=2, ps=1 << 24) == 2 and b"2048" in lib.sv_last_error()
    assert call(B=0, kv=None, w=None) == 0
    assert sv.sv_kv_evict_workspace(2, 3, 4, 100) >= 2 * 3 * 4 * 404
    assert sv.sv_kv_evict_workspace(0, 3, 4, 100) == 0 and sv.sv_kv_evict_workspace(1 << 20, 1 << 10, 8, 9) == 0


def test_kv_evict_binding_refusals(sv):
    kv = torch.zeros(1, 2, 6, 16, 2, 64, dtype=torch.bfloat16)
    t, n, w = torch.zeros(2, 3, dtype=torch.int32), torch.ones(2, dtype=torch.int32), torch.zeros(1, 2, 2, 48)
    kept, kl = torch.zeros(1, 2, 2, 8, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)

    def call(kv=kv, t=t, n=n, w=w, ow=w, budget=8, kept=kept, kl=kl, st=None):
        with pytest.raises(ValueError):
            sv.sv_kv_evict(kv, t, n, w, ow, budget, 1, 1, kept, kl, st)
    call(kv=kv[0]), call(kv=kv.transpose(3, 4)), call(t=t.long()), call(t=t[:1]), call(n=n.float())
    call(w=w.double()), call(w=w[..., ::2], ow=w), call(ow=w[..., :40]), call(budget=9)
    call(kept=kept.long()), call(kl=kl[:1]), call(st=torch.zeros(3, dtype=torch.int32))
    call()                                                 # pageable host memory


def test_kv_evict_sizes_whose_products_pass_63_bits(sv):
    lib, x, most = sv.load_library(), 4096, 2 ** 31 - 1

    def call(L=1, B=1, H=1, page=16, ps=16 * 2048, ls=1 << 30):
        return lib.sv_kv_evict(None, ls, 1 << 20, ps, 2, x, x, x, x, L, B, H, 1024, page, 1, 8, 1 << 30, 32, 2, 4,
                               x, x, None, x, 1 << 62, None)
    for shape in ((most, most, 4), (most, 2, most), (1, most, most), (1 << 20, 1 << 20, 1 << 25)):
        assert sv.sv_kv_evict_workspace(*shape, 9) == 0
        assert call(*shape, ps=1 << 50, ls=4) == 2 and b"2^24" in lib.sv_last_error()
    # a page of 2^30 slots of 2^24 heads of 2 KB: 2^65 bytes, which no stride covers
    assert call(H=1 << 24, page=1 << 30) == 1 and b"page_stride" in lib.sv_last_error()
    assert call(ps=-(2 ** 63)) == 1 and b"page_stride" in lib.sv_last_error()
    assert call(ps=16 * 1024) == 1 and b"null" in lib.sv_last_error()
    assert call(ps=16 * 1024 - 1) == 1 and b"page_stride" in lib.sv_last_error()


def test_numbers_beyond_32_bits_are_refused(sv):
    """They would reach the library without their upper bits: another window, or
    a far smaller budget."""
    bf, i32 = torch.bfloat16, torch.int32
    q, kv = torch.zeros(2, 8, 64, dtype=bf), torch.zeros(1, 2, 6, 16, 2, 64, dtype=bf)
    t, n = torch.zeros(2, 3, dtype=i32), torch.ones(2, dtype=i32)
    w = torch.zeros(1, 2, 2, 48)
    for window, sinks in ((2 ** 32 + 5, 0), (2 ** 31, 0), (0, 2 ** 32 + 4), (-2 ** 32, 0)):
        with pytest.raises(ValueError, match="32 bits"):
            sv.sv_paged_attention(q, kv[0], t, n, window, sinks, 1.0, None, torch.empty_like(q))
        with pytest.raises(ValueError, match="32 bits"):
            sv.sv_paged_attention_workspace(2, 8, 2, 64, 16, 3, window, sinks)
    for sinks, recent in ((2 ** 32 + 1, 1), (1, 2 ** 40)):
        with pytest.raises(ValueError, match="32 bits"):
            sv.sv_kv_evict(kv, t, n, w, w, 8, sinks, recent, torch.zeros(1, 2, 2, 8, dtype=i32), n.clone())
    with pytest.raises(ValueError, match="32 bits"):
        sv.sv_kv_evict(kv, t, n, w, w, 2 ** 32 + 8, 1, 1, torch.zeros(1, 2, 2, 8, dtype=i32), n.clone())
    with pytest.raises(ValueError, match="32 bits"):
        sv.sv_kv_evict_workspace(1, 2, 2, 2 ** 32 + 8)
    assert sv.sv_kv_evict_workspace(1, 2, 2, 2 ** 31 - 1) == 0    # beyond the library's own limit
    # more slots a head than an int holds: a view, no such memory
    far = torch.zeros(1).expand(1, 2, 2, 2 ** 32 + 48)
    with pytest.raises(ValueError, match="32 bits"):
        sv.sv_kv_evict(kv, t, n, far, far, 8, 1, 1, torch.zeros(1, 2, 2, 8, dtype=i32), n.clone())
    with pytest.raises(ValueError, match="32 bits"):
        sv.sv_paged_attention(q, kv[0], t, n, 0, 0, 1.0, far[0], torch.empty_like(q))


def test_paged_attention_workspace_sizes(sv):
    """A table of 4 pages of 16 leaves no room for two units: nothing to join, and
    with sums a score for each query head and slot, a reference and sum for each
    head and a flag for each KV head, each from a multiple of 256 bytes.  The scores
    are what a long table costs."""
    ws = sv.sv_paged_attention_workspace
    assert ws(1, 8, 2, 128, 16, 4) == 0
    assert ws(1, 8, 2, 128, 16, 4, weights=True) == 256 + 256 + 8 * 64 * 4
    long, sums = ws(128, 64, 8, 128, 16, 8192), ws(128, 64, 8, 128, 16, 8192, weights=True)
    assert sums - long == 128 * 64 * 131072 * 4
    assert ws(128, 64, 8, 128, 16, 8192, 4096, 4, True) < sums // 16
