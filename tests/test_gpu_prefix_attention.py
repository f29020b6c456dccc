"""sv_prefix_attention against the plain definition in 64 bits
(tests/plain_target.py).

Tolerances as derived in test_gpu_paged_attention.py, with u = 2^-24 and d the
relative error of a weight: scores (D + 4) u A, the base-2 exponential 2^-22, a
sum over n slots n u.  The prefix's weights go into the product as one number of
the cache's type: half a step of each, h = eps / 2 = 2^-8 or 2^-11, so an output
is off by h max|v| more, and by half a step of its own."""
import numpy as np
import pytest
import torch

import plain_target as plain

pytestmark = pytest.mark.gpu

sv = pytest.importorskip("speculative_decoding_verification_vocab_gb300")
DEV = "cuda:0"
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.load_library()


def make(plens, lens, Hq, Hkv, D, page, dtype=torch.bfloat16, seed=0, sigma=1.5, extra=1, spare=3):
    """CPU inputs; NaN in every slot that is not visible, an entry out of range
    for every page without one."""
    g = torch.Generator().manual_seed(seed)
    N, B = len(plens), len(lens)
    per_p = max(1, -(-max(plens) // page)) + extra
    per = max(1, -(-max(lens) // page)) + extra
    P = N * per_p + B * per + spare
    ids = torch.randperm(P, generator=g).to(torch.int32)
    q = (torch.randn(B, Hq, D, generator=g) * sigma).to(dtype)
    full = torch.randn(2, P, page, Hkv, D, generator=g).to(dtype)
    kv = torch.full_like(full, float("nan"))
    tables = []
    at = 0
    for ns, width in ((plens, per_p), (lens, per)):
        t = torch.full((len(ns), width), -7, dtype=torch.int32)
        for i, n in enumerate(ns):
            j = torch.arange(n)
            own = ids[at:at + width]
            at += width
            t[i, j // page] = own[j // page]
            kv[:, own[j // page].long(), j % page] = full[:, own[j // page].long(), j % page]
        tables.append(t)
    i32 = torch.int32
    return q, kv, tables[0], torch.tensor(plens, dtype=i32), tables[1], torch.tensor(lens, dtype=i32)


def close(out, lse, status, q, kv, pt, pl, t, n, scale):
    """The device's answer against the definition, sequence by sequence."""
    B, Hq, D = q.shape
    Hkv, W = kv.shape[3], B // len(pl)
    ref, rlse, rst = plain.prefix_attention(q.double().numpy(), kv.double().numpy(), pt.numpy(), pl.numpy(),
                                            t.numpy(), n.numpy(), scale)
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert status.cpu().numpy().tolist() == rst.tolist()
    bad = rst != 0
    assert np.isnan(o[bad]).all() and np.isnan(l[bad]).all()
    assert np.array_equal(np.isneginf(l), np.isneginf(rlse))
    total = (pl.numpy()[np.arange(B) // W] + n.numpy()).astype(np.float64)[:, None]
    kmax = np.nan_to_num(np.abs(kv[0].double().numpy()), nan=0.0, posinf=0.0).max((0, 1))  # [Hkv][D]
    size = scale * np.einsum("bhgd,hd->bhg", np.abs(q.double().numpy()).reshape(B, Hkv, -1, D), kmax).reshape(B, Hq)
    d = (D + 4) * U * size + 2.0 ** -22 + total * U
    fin = np.isfinite(rlse)
    lerr = np.abs(np.where(fin, l, 0) - np.where(fin, rlse, 0))
    assert (lerr <= d + 4 * U * np.abs(np.where(fin, rlse, 0))).all(), lerr.max()
    vmax = np.nan_to_num(kv[1].double().abs().numpy(), nan=0.0).max()
    half = torch.finfo(q.dtype).eps / 2
    tol = half * np.abs(ref) + (2 * d + half + 2.0 ** -17)[..., None] * vmax + 2.0 ** -25
    err = np.where(bad[:, None, None], 0, np.abs(o - ref))
    assert (err <= tol)[~bad].all(), (err - tol)[~bad].max()


def check(q, kv, pt, pl, t, n, scale=None, **kw):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    out, lse, st = sv.prefix_attention(q.to(DEV), kv.to(DEV), pt.to(DEV), pl.to(DEV), t.to(DEV), n.to(DEV), scale,
                                       return_lse=True, **kw)
    torch.cuda.synchronize()
    close(out, lse, st, q, kv, pt, pl, t, n, scale)
    return out, lse, st


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("plens,lens,Hq,Hkv,page", [
    ([1], [0], 1, 1, 16),                                  # one slot: the value itself
    ([0], [1, 0, 5], 2, 1, 16),                            # no prefix; nothing at all
    ([128], [1, 2], 8, 2, 16),                             # a whole tile
    ([129, 0, 127], [3, 0, 20, 64, 0, 65], 8, 8, 32),      # edges, an empty prefix between
    ([300], [7] * 5, 14, 2, 24),                           # G = 7, pages that end inside a tile
    ([1000, 513], [0, 33, 1, 100], 32, 2, 1),              # G = 16, pages of one slot
    ([700], [9] * 40, 16, 4, 33),                          # 160 rows: two query tiles, one ragged
    ([257, 640], [1] * 64, 48, 6, 128),                    # 32 sequences of 8: two full tiles
    ([90], [200] * 3, 20, 1, 8),                           # more of their own than shared
])
def test_matches_the_definition(plens, lens, Hq, Hkv, page, D, dtype):
    check(*make(plens, lens, Hq, Hkv, D, page, dtype))


@pytest.mark.parametrize("D", [64, 128])
def test_long_prefix_split_over_the_card(D):
    check(*make([20011], [17, 0, 300, 1], 16, 2, D, 64, seed=1))


@pytest.mark.parametrize("N", [33, 150])
def test_many_prefixes(N):
    g = torch.Generator().manual_seed(N)
    plens = torch.randint(0, 700, (N,), generator=g).tolist()
    plens[5] = plens[31] = plens[32] = 0
    lens = torch.randint(0, 40, (2 * N,), generator=g).tolist()
    check(*make(plens, lens, 4, 2, 64, 16, torch.float16, seed=N))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_equal_to_one_cache(dtype):
    """The same slots through sv_paged_attention, a table for each sequence: the
    prefix ends with a page."""
    page, W = 32, 6
    q, kv, pt, pl, t, n = make([20 * page], [50, 1, 0, 33, 64, 100], 32, 4, 128, page, dtype, extra=0)
    both = torch.cat([pt.expand(W, -1), t], 1).contiguous()
    scale = 128 ** -0.5
    a = sv.prefix_attention(*(x.to(DEV) for x in (q, kv, pt, pl, t, n)), return_lse=True)
    b = sv.paged_attention(q.to(DEV), kv.to(DEV), both.to(DEV), (n + pl[0]).to(DEV), return_lse=True)
    torch.cuda.synchronize()
    half = torch.finfo(dtype).eps / 2
    assert float((a[0].double() - b[0].double()).abs().max()) <= 4 * half * float(kv[1].double().nan_to_num().abs().max())
    assert float((a[1] - b[1]).abs().max()) <= 1e-4
    close(*a, q, kv, pt, pl, t, n, scale)


def test_scores_that_grow_and_fall_far():
    """Keys sorted so that the maximum rises with every tile (each moves the
    reference), falls, or stands at one slot far above the others."""
    for dtype in (torch.bfloat16, torch.float16):
        q, kv, pt, pl, t, n = make([1500], [3, 0], 4, 2, 128, 16, dtype, seed=3)
        q[:] = 0
        q[..., 0] = 8.0
        j = torch.arange(1500)
        for ramp in (j / 15.0 - 50, 50 - j / 15.0, torch.where(j == 777, 60.0, 0.0), torch.where(j == 1499, 100.0, -100.0)):
            kv[0, pt[0, j // 16].long(), j % 16, :, 0] = ramp[:, None].to(dtype)
            check(q, kv, pt, pl, t, n, 1.0)


def test_infinite_scores_and_values():
    q, kv, pt, pl, t, n = make([300, 300], [2, 1, 0, 4], 4, 2, 64, 16, seed=5)
    q[..., 0] = 1.0
    kv[0, pt[0, :18].long(), :, :, 0] = float("-inf")      # some scores of -inf in prefix 0
    out, lse, st = sv.prefix_attention(*(x.to(DEV) for x in (q, kv, pt, pl, t, n)), return_lse=True)
    torch.cuda.synchronize()
    close(out[:2], lse[:2], st[:2], q[:2], kv, pt[:1], pl[:1], t[:2], n[:2], 64 ** -0.5)
    kv[0, pt[0, :19].long(), :, :, 0] = float("-inf")      # all of them: as if it were not there
    out, lse, st = sv.prefix_attention(*(x.to(DEV) for x in (q, kv, pt, pl, t, n)), return_lse=True)
    alone = sv.paged_attention(q.to(DEV), kv.to(DEV), t.to(DEV), n.to(DEV), return_lse=True)
    torch.cuda.synchronize()
    assert not bool(st.any())
    assert torch.allclose(out[:2].float(), alone[0][:2].float(), atol=2e-2) and torch.allclose(lse[:2], alone[1][:2], atol=1e-4)
    kv[1, pt[1, 3].long(), 2] = float("nan")               # a NaN that is visible stays in its group
    out, lse, st = sv.prefix_attention(*(x.to(DEV) for x in (q, kv, pt, pl, t, n)), return_lse=True)
    torch.cuda.synchronize()
    assert bool(out[2:].isnan().all()) and not bool(out[:2].isnan().any())


def test_faults():
    q, kv, pt, pl, t, n = make([300, 200, 100, 64], [5, 0, 9, 1, 2, 3, 4, 5], 8, 2, 128, 16, seed=7)
    P = kv.shape[1]
    pl[0] = -1
    pt[1, 12] = P                    # the page of slots 192..199
    n[5] = 10 ** 6
    t[7, 0] = -1
    out, lse, st = check(q, kv, pt, pl, t, n)
    assert st.tolist() == [256, 256, 512, 512, 0, 256, 0, 512]
    pl[0] = pt.shape[1] * 16 + 1
    out, lse, st = check(q, kv, pt, pl, t, n)
    assert st.tolist()[:2] == [256, 256]


def test_layouts_and_a_given_workspace():
    q, kv, pt, pl, t, n = make([333], [9, 70, 0], 12, 2, 64, 20, seed=2)
    want = check(q, kv, pt, pl, t, n)
    swapped = kv.transpose(0, 1).contiguous().transpose(0, 1)    # [pages][2][page][Hkv][D]
    size = sv.sv_prefix_attention_workspace(3, 1, 12, 2, 64, 20, pt.shape[1], t.shape[1])
    guard = 4096
    buf = torch.full((size + 2 * guard,), 0xA5, dtype=torch.uint8, device=DEV)
    ws = buf[guard:guard + size]
    dev = [x.to(DEV) for x in (q, swapped, pt, pl, t, n)]
    dev[1] = dev[1].transpose(0, 1).contiguous().transpose(0, 1)
    got = sv.prefix_attention(*dev, return_lse=True, workspace=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert bool((buf[:guard] == 0xA5).all()) and bool((buf[guard + size:] == 0xA5).all())
    # again with other lengths, over what the first call left
    dev[3], dev[5] = torch.tensor([40], dtype=torch.int32, device=DEV), torch.tensor([0, 3, 0], dtype=torch.int32, device=DEV)
    got = sv.prefix_attention(*dev, return_lse=True, workspace=ws)
    torch.cuda.synchronize()
    close(*got, q, kv, pt, dev[3].cpu(), t, dev[5].cpu(), 64 ** -0.5)
    with pytest.raises(sv.SvError, match="workspace"):
        sv.prefix_attention(*dev, workspace=ws[:-256])


def test_captured_launch_follows_growing_lengths():
    q, kv, pt, pl, t, n = make([900, 700], [60] * 6, 8, 2, 128, 16, seed=4)
    dev = [x.to(DEV) for x in (q, kv, pt, pl, t, n)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = sv.prefix_attention(*dev, return_lse=True)
    for pn, on in (([1, 700], [1, 2, 3, 4, 5, 6]), ([900, 0], [60, 0, 0, 1, 60, 33]), ([128, 129], [16] * 6)):
        dev[3].copy_(torch.tensor(pn)), dev[5].copy_(torch.tensor(on))
        graph.replay()
        torch.cuda.synchronize()
        close(*got, q, kv, pt, dev[3].cpu(), t, dev[5].cpu(), 128 ** -0.5)


def test_streams_and_two_calls_at_once():
    q, kv, pt, pl, t, n = make([5000], [40] * 32, 32, 4, 128, 64, seed=6)
    dev = [x.to(DEV) for x in (q, kv, pt, pl, t, n)]
    want = sv.prefix_attention(*dev, return_lse=True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [sv.prefix_attention(*dev, return_lse=True, stream=s) for _ in range(4) for s in streams]
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want))


def test_offsets_that_pass_32_bits():
    """Pages more than 2^31 elements apart."""
    page, H, D = 16, 2, 64
    stride = (1 << 31) // 3 // 8 * 8
    buf = torch.zeros(5 * stride, dtype=torch.bfloat16, device=DEV)
    kv = buf.as_strided((2, 4, page, H, D), (page * H * D, stride, H * D, D, 1))
    kv.copy_(torch.randn(2, 4, page, H, D, device=DEV))
    q = torch.randn(2, 4, D, device=DEV).to(torch.bfloat16)
    i32 = dict(dtype=torch.int32, device=DEV)
    args = (torch.tensor([[3, 0]], **i32), torch.tensor([27], **i32), torch.tensor([[2], [1]], **i32),
            torch.tensor([5, 16], **i32))
    got = sv.prefix_attention(q, kv, *args, return_lse=True)
    want = sv.prefix_attention(q, kv.contiguous(), *args, return_lse=True)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
