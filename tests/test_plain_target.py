"""CPU pins of the plain definitions that the target's side of a round is tested
against, and the host-side refusals of those operators."""
import math

import numpy as np
import pytest
import torch

import plain_target as plain


@pytest.fixture(scope="module")
def sv():
    from speculative_decoding_verification_vocab_gb300 import _build
    _build.build()
    import speculative_decoding_verification_vocab_gb300 as m
    m.load_library()
    return m


def test_token_logprobs_pin():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(50, generator=g, dtype=torch.float64) * 3
    lp = torch.log_softmax(x / 0.5, -1)
    given, H, top, top_lp, st = plain.token_logprobs(x.numpy(), 7, 5, 0.5)
    assert st == 0 and abs(given - float(lp[7])) < 1e-12
    assert abs(H - float(torch.distributions.Categorical(logits=lp).entropy())) < 1e-12
    assert top == lp.topk(5).indices.tolist() and np.allclose(top_lp, lp.topk(5).values, atol=1e-12)
    assert plain.token_logprobs(np.zeros(8), 3, 3, 1.0)[2] == [0, 1, 2]
    assert abs(plain.token_logprobs(np.zeros(8), 3, 3, 1.0)[1] - math.log(8)) < 1e-12
    x[3:] = -math.inf
    assert plain.token_logprobs(x.numpy(), 7, 5, 1.0)[2][3:] == [-1, -1]
    assert plain.token_logprobs([math.nan, 1.0], 0, 1, 1.0)[4] == plain.ROW_NAN


@pytest.mark.parametrize("tail", [True, False])
def test_distill_pin(tail):
    """The loss is torch's KL divergence of the two distributions over the list
    and the rest; the gradient is autograd's."""
    g = torch.Generator().manual_seed(1)
    V, K, T = 30, 6, 1.7
    T = float(np.float32(T))
    x = (torch.randn(V, generator=g, dtype=torch.float64) * 2).requires_grad_()
    y = torch.log_softmax(torch.randn(V, generator=g, dtype=torch.float64) * 2, -1).topk(K)
    lp = torch.log_softmax(x / T, -1)
    rest = torch.ones(V, dtype=torch.bool)
    rest[y.indices] = False
    t, ls = y.values.exp(), lp[y.indices]
    if tail:
        t = torch.cat([t, (1 - t.sum())[None]])
        ls = torch.cat([ls, torch.logsumexp(lp[rest], 0)[None]])
    else:
        t = t / t.sum()
    loss = torch.nn.functional.kl_div(ls, t, reduction="sum")
    loss.backward()
    got, grad, st = plain.distill(x.detach().numpy(), y.indices.numpy(), y.values.numpy(), T, tail)
    assert st == 0 and abs(got - float(loss.detach())) < 1e-12
    assert np.abs(grad - x.grad.numpy()).max() < 1e-12
    # a student equal to its teacher over the whole vocabulary: nothing to learn
    full = torch.log_softmax(x.detach(), -1)
    got, grad, _ = plain.distill(x.detach().numpy(), np.arange(V), full.numpy(), 1.0, tail)
    assert abs(got) < 1e-12 and np.abs(grad).max() < 1e-12
    assert plain.distill(x.detach().numpy(), [-1, -1], [0.0, 0.0], 1.0, tail)[::2] == (0.0, 0)
    assert plain.distill(x.detach().numpy(), [4, 4], [-1.0, -1.0], 1.0, tail)[2] == plain.BAD_TOKEN


def test_token_logprobs_refusals(sv):
    lib, x = sv.load_library(), 4096

    def call(logits=x, ss=1000, rs=100, dt=1, rows=None, tok=x, B=2, T=3, P=3, V=100, K=4, temp=1.0, lp=x, H=x,
             tt=x, tl=x, st=x):
        return lib.sv_token_logprobs(logits, ss, rs, dt, rows, tok, B, T, P, V, K, temp, lp, H, tt, tl, st, None)
    for bad in (dict(B=-1), dict(T=0), dict(P=-1), dict(V=0), dict(K=-1), dict(dt=3), dict(P=4), dict(K=101),
                dict(temp=0.0), dict(temp=-1.0), dict(temp=math.inf), dict(temp=math.nan), dict(temp=1e-45),
                dict(ss=-1), dict(rs=-1), dict(ss=2 ** 62), dict(rs=2 ** 60),
                dict(logits=None), dict(H=None), dict(st=None), dict(lp=None), dict(tt=None), dict(tl=None),
                dict(logits=x + 1), dict(tok=x + 2), dict(rows=x + 2), dict(lp=x + 2), dict(H=x + 1), dict(tt=x + 2),
                dict(tl=x + 2), dict(st=x + 2), dict(dt=0, logits=x + 2)):
        assert call(**bad) == 1, bad
        assert lib.sv_last_error(), bad
    assert call(V=1000, K=129) == 2 and b"K >" in lib.sv_last_error()
    assert call(V=(1 << 22) + 1) == 2 and call(B=1 << 27, ss=0) == 2
    assert call(B=0, logits=None) == 0 and call(P=0, logits=None) == 0
    # what is left is the pointers themselves, which are no device's
    assert call() == 1 and b"logits" in lib.sv_last_error()
    assert call(rows=x, P=9) == 1 and b"logits" in lib.sv_last_error()


def test_distill_refusals(sv):
    lib, x = sv.load_library(), 4096

    def loss(logits=x, rs=100, dt=1, tok=x, lp=x, w=None, R=3, V=100, K=4, temp=1.0, tail=1, loss=x, stat=x, grad=x,
             gs=100, st=x):
        return lib.sv_distill_loss(logits, rs, dt, tok, lp, w, R, V, K, temp, tail, loss, stat, grad, gs, st, None)

    def grad(logits=x, rs=100, dt=1, tok=x, lp=x, w=None, R=3, V=100, K=4, temp=1.0, tail=1, stat=x, grad=x, gs=100,
             st=x):
        return lib.sv_distill_grad(logits, rs, dt, tok, lp, stat, w, R, V, K, temp, tail, grad, gs, st, None)
    for call in (loss, grad):
        for bad in (dict(R=-1), dict(V=0), dict(K=0), dict(K=101), dict(dt=3), dict(tail=2), dict(temp=0.0),
                    dict(temp=math.nan), dict(temp=math.inf), dict(rs=-1), dict(rs=2 ** 60), dict(gs=99),
                    dict(gs=2 ** 60), dict(gs=101), dict(logits=None), dict(tok=None), dict(lp=None), dict(st=None),
                    dict(logits=x + 1), dict(tok=x + 2), dict(lp=x + 2), dict(w=x + 2), dict(st=x + 2),
                    dict(grad=x + 1), dict(stat=x + 8), dict(dt=0, logits=x + 2)):
            assert call(**bad) == 1, bad
        assert call(V=1000, rs=1000, gs=1000, K=129) == 2 and call(R=(1 << 22) + 1) == 2
        assert call(V=(1 << 22) + 1) == 2
        assert call(R=0, logits=None) == 0
        assert call() == 1 and b"logits" in lib.sv_last_error()
    assert grad(stat=None) == 1 and grad(grad=None) == 1
    assert loss(loss=None, grad=None, stat=None) == 1


def test_binding_refusals(sv):
    x, i32 = torch.zeros(2, 3, 50), torch.int32
    tok, e, t2 = torch.zeros(2, 3, dtype=i32), torch.zeros(2, 3), torch.zeros(2, 3, 4, dtype=i32)
    ok = dict(logits=x, rows=None, tokens=tok, temperature=1.0, out_logprob=e, out_entropy=e, out_top_token=t2,
              out_top_logprob=torch.zeros(2, 3, 4), out_status=tok)
    for bad in (dict(logits=x[0]), dict(logits=x.double()), dict(logits=x.transpose(1, 2)), dict(tokens=tok.long()),
                dict(tokens=tok[:1]), dict(rows=tok[:, :2].contiguous()), dict(tokens=tok[:, ::2]),
                dict(out_logprob=e.double()), dict(out_entropy=e[:1]), dict(out_status=e),
                dict(out_top_logprob=torch.zeros(2, 3, 5)), dict(out_top_token=t2.long()),
                dict()):                                   # pageable host memory
        with pytest.raises(ValueError):
            sv.sv_token_logprobs(**{**ok, **bad})
    x, t, v = torch.zeros(4, 50), torch.zeros(4, 5, dtype=i32), torch.zeros(4, 5)
    ok = dict(logits=x, teacher_token=t, teacher_logprob=v, weight=None, temperature=1.0, tail=True,
              out_grad=torch.zeros(4, 50), out_status=t[:, 0].contiguous())
    for bad in (dict(logits=x[None]), dict(logits=x.double()), dict(logits=x.t()), dict(teacher_token=t.long()),
                dict(teacher_logprob=v.double()), dict(teacher_token=t[:3]), dict(teacher_logprob=v[:, :4]),
                dict(weight=torch.zeros(3)), dict(weight=torch.zeros(4).double()), dict(out_grad=x.half()),
                dict(out_grad=x[:, :49]), dict(out_grad=torch.zeros(50, 4).t()), dict(out_grad=x[None]),
                dict(out_status=torch.zeros(4)), dict()):
        with pytest.raises(ValueError):
            sv.sv_distill_loss(out_loss=torch.zeros(4), out_stat=torch.zeros(4, 4), **{**ok, **bad})
        with pytest.raises(ValueError):
            sv.sv_distill_grad(stat=torch.zeros(4, 4), **{**ok, **bad})
    with pytest.raises(ValueError):
        sv.sv_distill_grad(stat=torch.zeros(4, 3), **ok)
    with pytest.raises(ValueError):
        sv.sv_distill_loss(out_loss=torch.zeros(5), out_stat=None, **ok)


def test_prefix_attention_pin():
    """Torch's dense attention over the two parts of each sequence, laid out as
    one; with the parts of another sequence it differs."""
    g = torch.Generator().manual_seed(3)
    page, Hkv, G, D = 4, 2, 3, 8
    q = torch.randn(4, Hkv * G, D, generator=g, dtype=torch.float64)
    kv = torch.randn(2, 12, page, Hkv, D, generator=g, dtype=torch.float64)
    pt, pl = np.array([[3, 7, 0], [5, 1, -1]]), np.array([11, 8])
    t, n = np.array([[2], [4], [6], [8]]), np.array([1, 4, 0, 3])
    out, lse, st = plain.prefix_attention(q.numpy(), kv.numpy(), pt, pl, t, n, 0.5)
    assert not st.any()
    for b in range(4):
        rows = [(pt[b // 2][j // page], j % page) for j in range(pl[b // 2])]
        rows += [(t[b][j // page], j % page) for j in range(n[b])]
        i, r = torch.tensor([x for x, _ in rows]), torch.tensor([x for _, x in rows])
        k, v = kv[0, i, r].transpose(0, 1), kv[1, i, r].transpose(0, 1)
        want = torch.nn.functional.scaled_dot_product_attention(
            q[b].view(Hkv, G, D), k, v, scale=0.5).reshape(Hkv * G, D)
        assert np.abs(out[b] - want.numpy()).max() < 1e-12
        x = torch.einsum("hgd,hjd->hgj", q[b].view(Hkv, G, D), k) * 0.5
        assert np.abs(lse[b] - torch.logsumexp(x, -1).reshape(-1).numpy()).max() < 1e-12
    assert np.abs(out - plain.prefix_attention(q.numpy(), kv.numpy(), pt[::-1], pl[::-1], t, n, 0.5)[0]).max() > 0.01
    st = plain.prefix_attention(q.numpy(), kv.numpy(), pt, np.array([13, 9]), t, n, 0.5)[2]
    assert st.tolist() == [plain.BAD_LEN] * 2 + [plain.BAD_PAGE] * 2


def test_prefix_attention_refusals(sv):
    lib, x = sv.load_library(), 4096
    need = sv.sv_prefix_attention_workspace(6, 2, 8, 2, 128, 16, 4, 3)
    assert need > 0

    def call(q=x, kv=x, ks=1 << 20, ps=16 * 2 * 128, dt=1, pt=x, pl=x, t=x, n=x, B=6, N=2, Hq=8, Hkv=2, D=128, page=16,
             mp=4, m=3, P=40, scale=0.1, out=x, lse=x, st=x, ws=x, wb=need):
        return lib.sv_prefix_attention(q, kv, ks, ps, dt, pt, pl, t, n, B, N, Hq, Hkv, D, page, mp, m, P, scale, out,
                                       lse, st, ws, wb, None)
    for bad in (dict(B=-2), dict(N=0), dict(N=4), dict(Hq=7), dict(Hkv=0), dict(D=0), dict(page=0), dict(mp=0),
                dict(m=0), dict(P=0), dict(dt=0), dict(scale=0.0), dict(scale=math.inf), dict(scale=math.nan),
                dict(ps=16 * 2 * 128 - 8), dict(ps=16 * 2 * 128 + 1), dict(ks=0), dict(ks=12), dict(ks=2 ** 62),
                dict(ps=2 ** 62), dict(q=None), dict(kv=None), dict(pt=None), dict(pl=None), dict(t=None),
                dict(n=None), dict(out=None), dict(ws=None), dict(q=x + 8), dict(kv=x + 8), dict(out=x + 8),
                dict(pt=x + 2), dict(pl=x + 2), dict(t=x + 1), dict(n=x + 2), dict(lse=x + 2), dict(st=x + 2),
                dict(ws=x + 64), dict(wb=need - 1)):
        assert call(**bad) == 1, bad
    for far in (dict(D=256, ps=16 * 2 * 256), dict(mp=1 << 27), dict(m=1 << 27), dict(B=1 << 26, N=1 << 26)):
        assert call(**far) == 2, far
    assert call(B=0, q=None) == 0
    assert call() == 1 and b"q" in lib.sv_last_error()
    size = sv.sv_prefix_attention_workspace
    for bad in ((6, 4, 8, 2, 128, 16, 4, 3), (0, 2, 8, 2, 128, 16, 4, 3), (6, 0, 8, 2, 128, 16, 4, 3),
                (6, 2, 7, 2, 128, 16, 4, 3)):
        assert size(*bad) == 0
    with pytest.raises(ValueError, match="32 bits"):
        size(6, 2, 8, 2, 128, 16, 2 ** 32 + 4, 3)
    # rows that are not there are not stored: 4 rows to a part, not 128
    assert size(1, 1, 4, 1, 128, 16, 4, 3) * 16 < size(32, 1, 4, 1, 128, 16, 4, 3)


def test_prefix_attention_binding_refusals(sv):
    bf, i32 = torch.bfloat16, torch.int32
    q, kv = torch.zeros(6, 8, 64, dtype=bf), torch.zeros(2, 9, 16, 2, 64, dtype=bf)
    ok = dict(q=q, kv=kv, prefix_table=torch.zeros(2, 3, dtype=i32), prefix_len=torch.zeros(2, dtype=i32),
              block_table=torch.zeros(6, 2, dtype=i32), seq_len=torch.zeros(6, dtype=i32), scale=1.0,
              out=torch.zeros_like(q))
    for bad in (dict(q=q.float()), dict(kv=kv.half()), dict(kv=kv[..., :32]), dict(kv=kv[0]),
                dict(kv=kv.transpose(2, 3)), dict(prefix_len=torch.zeros(4, dtype=i32)),
                dict(prefix_len=torch.zeros(0, dtype=i32)), dict(prefix_len=torch.zeros(2)),
                dict(prefix_table=torch.zeros(3, 3, dtype=i32)), dict(prefix_table=torch.zeros(6, dtype=i32)),
                dict(block_table=torch.zeros(5, 2, dtype=i32)), dict(block_table=torch.zeros(6, 2)),
                dict(seq_len=torch.zeros(6, 1, dtype=i32)), dict(out=q.float()), dict(out=q[:5]),
                dict(out_lse=torch.zeros(6, 7)), dict(out_status=torch.zeros(6)),
                dict(workspace=torch.zeros(8, 8)[:, ::2]), dict()):   # the last: pageable host memory
        with pytest.raises(ValueError):
            sv.sv_prefix_attention(**{**ok, **bad})
