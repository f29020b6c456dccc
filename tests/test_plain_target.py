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
