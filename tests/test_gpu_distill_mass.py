"""sv_distill_loss and sv_distill_grad where a mask leaves the student's rest
nothing or the list is the whole vocabulary, against tests/plain_distill_mass.py."""
import math

import numpy as np
import pytest
import torch

import plain_distill_mass as mass

pytestmark = pytest.mark.gpu

sv = pytest.importorskip("speculative_decoding_verification_vocab_gb300")
DEV = "cuda:0"
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.load_library()


def calls(x, token, value, T=1.0, tail=True):
    """Loss, gradient and status by every way there is: the loss alone and the
    gradient from its statistics, both at once, both in the logits' place."""
    one = sv.distill_loss(x, token, value, temperature=T, tail=tail)
    later, st = sv.distill_grad(x, token, value, one["stat"], temperature=T, tail=tail)
    yield one["loss"], later, one["status"]
    assert torch.equal(st, one["status"])
    r = sv.distill_loss(x, token, value, temperature=T, tail=tail, grad=True)
    yield r["loss"], r["grad"], r["status"]
    at, at2 = x.clone(), x.clone()
    a = sv.distill_loss(at, token, value, temperature=T, tail=tail, out_grad=at)
    sv.distill_grad(at2, token, value, one["stat"], temperature=T, tail=tail, out_grad=at2)
    assert a["grad"] is at and torch.equal(at, r["grad"]) and torch.equal(at2, later)
    assert torch.equal(a["loss"].nan_to_num(7.0), r["loss"].nan_to_num(7.0)) and torch.equal(a["status"], r["status"])


def hold(x, token, value, T=1.0, tail=True):
    """Every row against the definition.  Errors of 32 bits, u = 2^-24 each, as in
    test_gpu_distill.py: an exponent y of up to 48 counts (40, and the reference's
    slack) three roundings of itself, its power 4, V / 512 + 24 additions: `rel` of a
    student's share; 8 + K of a teacher's weight and of t_r.  A loss adds the weights
    times logs of up to `big`, of the entries that have a weight, and t_r (ln t_r - ln
    s_r): t_r's error times both logs and 1, and t_r times the share's."""
    V, K = x.shape[1], token.shape[1]
    u = 2.0 ** -24
    rel, rel_t = u * (3 * 48 + 4 + V / 512 + 24), u * (8 + K)
    half = torch.finfo(x.dtype).eps / 2
    tiny = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -24}[x.dtype]
    xs, toks, vals = x.double().cpu().numpy(), token.cpu().numpy(), value.double().cpu().numpy()
    want = [mass.definition(xs[r], toks[r], vals[r], T, tail) for r in range(len(xs))]
    for loss, grad, status in calls(x, token, value, T, tail):
        loss, grad, status = loss.double().cpu().numpy(), grad.double().cpu().numpy(), status.cpu().numpy()
        for r, (wl, wg, st) in enumerate(want):
            assert status[r] == st, r
            if st:
                assert math.isnan(loss[r]) and not grad[r].any(), r
                continue
            if not math.isfinite(wl):
                assert loss[r] == wl, (r, loss[r], wl)
            live = toks[r] != -1
            z = (xs[r] - xs[r].max()) / T
            lp = z - np.log(np.exp(z).sum())
            if not live.any():
                assert loss[r] == 0 and not grad[r].any()
                continue
            t, tr = mass.masses(vals[r][live], tail)
            of = lp[toks[r][live]]
            weighty = (t > 2.0 ** -126) & np.isfinite(of)
            big = (np.abs(of) + np.abs(vals[r][live]))[weighty].max(initial=0.0)
            s = np.exp(lp)
            weight = np.zeros(V)
            weight[toks[r][live]] = t
            rest = np.ones(V, bool)
            rest[toks[r][live]] = False
            top = lp[rest].max(initial=-np.inf)
            e = np.where(rest & (lp > -np.inf), np.exp(np.minimum(lp - (top if top > -np.inf else 0), 0)), 0)
            share = e / max(e.sum(), 1e-300)
            # (t_r is off by rel_t even where it is 0, but not where it does not count)
            lsr = top + math.log(e.sum()) if top > -np.inf else -np.inf
            counts = tail and not (lsr < math.log(mass.NO_SHARE) and tr < mass.ROUNDING)
            if math.isfinite(wl):
                logs = abs(lsr) + abs(math.log(max(tr, 2.0 ** -24))) + 1 if counts else 0.0
                tol = (rel + 2 * rel_t) * (2 + big) + logs * rel_t + tr * rel + 2.0 ** -22 * abs(wl)
                assert abs(loss[r] - wl) <= tol, (r, loss[r], wl, tol)
            tol = (3 * s * rel + weight * rel_t + share * (tr * rel + rel_t * counts)) / T
            off = np.abs(grad[r] - wg) - tol - (half + 2.0 ** -23) * np.abs(wg) - tiny
            assert (off <= 0).all(), (r, off.max(), int(off.argmax()))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lowest", [False, True])
@pytest.mark.parametrize("V,K", [(130, 128), (3001, 64), (40000, 20)])
def test_teacher_and_student_under_one_mask(V, K, lowest, dtype):
    """A mask leaves up to K tokens, the same for both; the list comes from the
    teacher's log probabilities as it is.  Their sum is 1 but for rounding, and the
    student's rest has no mass: the loss is that of the tokens that are left."""
    g = torch.Generator(device=DEV).manual_seed(V)
    R = 60
    masked = torch.finfo(dtype).min if lowest else -math.inf
    n = torch.randint(1, K + 1, (R,), generator=g, device=DEV)
    n[:4] = torch.tensor([1, 2, K - 1, K])
    rank = torch.rand(R, V, generator=g, device=DEV).argsort(1).argsort(1)
    gone = rank >= n[:, None]
    x = (torch.randn(R, V, generator=g, device=DEV) * 3).to(dtype).masked_fill(gone, masked)
    y = (torch.randn(R, V, generator=g, device=DEV) * 3).to(dtype).masked_fill(gone, masked)
    for T in (1.0, 0.7):
        t = sv.token_logprobs(y[:, None], top_k=K, temperature=T)
        token, value = t["top_token"][:, 0].contiguous(), t["top_logprob"][:, 0].contiguous()
        assert not bool(t["status"].any())
        if not lowest:
            assert torch.equal((token != -1).sum(1), n)
        r = sv.distill_loss(x, token, value, temperature=T, grad=True)
        assert not bool(r["status"].any()) and bool((r["loss"] < 100).all())
        # nothing but the tokens that are left has a gradient
        assert not bool(r["grad"][gone].any())
        hold(x, token, value, T)
        hold(x, token, value, T, tail=False)
        # and none at all where the student is its teacher, but for rounding: that of the
        # weights and of the student's shares, up to 1
        own = sv.distill_loss(y, token, value, temperature=T, grad=True)
        assert float(own["loss"].abs().max()) <= 2.0 ** -24 * (8 + K + 172 + V / 512) * 40
        assert float(own["grad"].float().abs().max()) <= 2.0 ** -24 * (8 + K + 172 + V / 512) / T


@pytest.mark.parametrize("low", [-math.inf, -3.4028234663852886e38, -80.0, -50.0])
def test_what_the_teacher_leaves_of_a_masked_rest(low):
    """Less than 2^-16 counts as nothing where the student's rest has no share (below
    2^-100: 200 tokens at -80 have 2^-107, at -50 2^-64), more does not."""
    V, K = 205, 5
    g = torch.Generator().manual_seed(4)
    totals = torch.tensor([1 - 2.0 ** -18, 1 - 2.0 ** -14, 1 - 2.0 ** -20, 1.0, 0.9], dtype=torch.float64)
    R = len(totals)
    x = torch.full((R, V), low)
    token = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(R)]).to(torch.int32)
    x.scatter_(1, token.long(), torch.randn(R, K, generator=g))
    value = torch.log_softmax(torch.randn(R, K, generator=g, dtype=torch.float64), 1) + totals.log()[:, None]
    hold(x.to(DEV), token.to(DEV), value.float().to(DEV))
    loss = sv.distill_loss(x.to(DEV), token.to(DEV), value.float().to(DEV))["loss"].tolist()
    if low == -math.inf:
        assert [math.isinf(v) for v in loss] == [False, True, False, False, True]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [1, 7, 40, 128])
def test_the_whole_vocabulary_listed(V, dtype):
    """No rest at all: what the teacher's weights lack of 1 beyond rounding has
    nowhere to go."""
    g = torch.Generator(device=DEV).manual_seed(V)
    R = 3
    x = (torch.randn(R, V, generator=g, device=DEV) * 2).to(dtype)
    value = torch.log_softmax(torch.randn(R, V, generator=g, device=DEV).double() * 2, -1).float()
    token = torch.arange(V, dtype=torch.int32, device=DEV).expand(R, V).contiguous()
    value[1] -= math.log(2.0)
    hold(x, token, value)
    loss = sv.distill_loss(x, token, value)["loss"]
    assert loss.isinf().tolist() == [False, True, False]
    hold(x, token, value, tail=False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V,K", [(50, 4), (50, 50), (3001, 20), (128256, 128)])
def test_weights_that_add_up_to_more_than_one(V, K, dtype):
    """Up to 1 + 2^-8 is taken: the loss's gradient is s_v sum t - t_v then."""
    g = torch.Generator(device=DEV).manual_seed(V + K)
    totals = torch.tensor([1 + 2.0 ** -9, 1 + 2.0 ** -8.1, 1 + 2.0 ** -12, 1.0], dtype=torch.float64, device=DEV)
    R = len(totals)
    x = (torch.randn(R, V, generator=g, device=DEV) * 2).to(dtype)
    top = (x.double() + torch.randn(R, V, generator=g, device=DEV)).topk(K, -1)
    value = (torch.log_softmax(top.values, -1) + totals.log()[:, None]).float()
    for T in (1.0, 0.7):
        hold(x, top.indices.to(torch.int32), value, T)


def test_the_gradient_of_more_than_one_against_differences():
    """Central differences of the loss, per element: the loss is off by d = 1e-5 at most
    here (V = 50, logs below 12), a step of h = 0.03 by h^2 / 6 of third derivatives,
    which are below 1.  A student sure of a token has s_v = 0.8 there: 2^-8.1 of it is
    five times what these leave."""
    V, K, h = 50, 4, 0.03
    g = torch.Generator().manual_seed(8)
    x = torch.randn(1, V, generator=g)
    x[0, 7] = 5.5
    token = torch.tensor([[3, 7, 20, 41]], dtype=torch.int32)
    value = (torch.log_softmax(torch.randn(1, K, generator=g, dtype=torch.float64), 1) + math.log(1 + 2.0 ** -8.1)).float()
    grad = sv.distill_loss(x.to(DEV), token.to(DEV), value.to(DEV), grad=True)["grad"].double().cpu()[0]
    rows = torch.cat([x + torch.eye(V) * h, x - torch.eye(V) * h]).to(DEV)
    loss = sv.distill_loss(rows, token.expand(2 * V, K).contiguous().to(DEV),
                           value.expand(2 * V, K).contiguous().to(DEV))["loss"].double().cpu()
    # the steps as they were taken
    step = (rows[:V].double() - rows[V:].double()).diagonal().cpu()
    assert float(((loss[:V] - loss[V:]) / step - grad).abs().max()) <= 1e-5 / h + h * h / 6
