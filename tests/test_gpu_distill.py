"""sv_distill_loss and sv_distill_grad against the plain definition in 64 bits
(tests/plain_target.py), element by element, and against differences of the
loss."""
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


def make(R, V, K, dtype, seed, pad=0, noise=1.0, T=1.0, sigma=3.0):
    """CPU inputs: rows with NaN between them, a teacher near its student."""
    g = torch.Generator().manual_seed(seed)
    full = torch.full((R, V + pad), float("nan"), dtype=dtype)
    x = torch.randn(R, V, generator=g) * sigma
    full[:, :V] = x.to(dtype)
    y = torch.log_softmax((x + noise * torch.randn(R, V, generator=g)).double() / T, -1)
    top = y.topk(K, -1)
    return full[:, :V], top.indices.to(torch.int32), top.values.float()


def put(t):
    if t is None:
        return None
    d = torch.empty_strided(t.size(), t.stride(), dtype=t.dtype, device=DEV)
    return d.copy_(t)


def near(name, got, want, tol, at):
    """Infinities and NaN equal, the rest within tol (elementwise)."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine], want[~fine], equal_nan=True), (name, at)
    off = np.abs(got - want)[fine] - np.broadcast_to(tol, want.shape)[fine]
    assert np.isfinite(got[fine]).all() and (off <= 0).all(), (name, at, off.max(), int(off.argmax()))


def compare(logits, token, value, weight, T, tail, loss, grad, status):
    R, V = logits.shape
    K = token.shape[1]
    x = logits.float().numpy()
    w = np.ones(R) if weight is None else weight.double().numpy()
    half = torch.finfo(logits.dtype).eps / 2
    tiny = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -24}[logits.dtype]
    for r in range(R):
        want_l, want_g, st = plain.distill(x[r], token[r].numpy(), value[r].numpy(), T, tail)
        assert status[r] == st, (r, status[r], st)
        # An exponent y is off by 3 roundings of itself (|y| <= 40 counts, 8 of it the
        # reference's slack), the exponential by 2^-22, a sum by its additions (V / 512
        # of a thread, 24 joins); a teacher's weight by expf's 2 ulp and, normalised, by
        # its list's sum; t_r by K of those and its own additions.
        rel = 2.0 ** -24 * (3 * 48 + 4 + V / 512 + 24)
        rel_t = 2.0 ** -24 * (8 + K)
        entries = [(int(t), float(a)) for t, a in zip(token[r], value[r]) if t != -1]
        if st or not entries:
            assert (math.isnan(want_l) and math.isnan(loss[r])) or loss[r] == 0
            assert grad is None or not grad[r].any()
            continue
        lp = plain.log_softmax(x[r], T)
        big = np.abs(lp[[t for t, _ in entries]])
        big = float(big[np.isfinite(big)].max(initial=0.0)) + max(
            [abs(a) for _, a in entries if a > -math.inf], default=0.0)
        # logs of up to `big`, of weights that add up to 1, and the rest's: ln of t_r
        # off by rel_t / t_r of itself times t_r
        if loss is not None:
            near("loss", loss[r], want_l, (rel + 2 * rel_t) * (2 + big) + 40 * rel_t + 2.0 ** -22 * abs(want_l), r)
        if grad is not None:
            s = np.exp(lp)
            listed = np.zeros(V)
            a = np.array([v for _, v in entries])
            t = np.exp(a) if tail else np.exp(a - a.max()) / np.exp(a - a.max()).sum()
            listed[[i for i, _ in entries]] = t
            rest = np.ones(V, bool)
            rest[[i for i, _ in entries]] = False
            sr = s[rest].sum()
            share = np.where(rest & (sr > 0), s / (sr if sr > 0 else 1), 0.0)
            tr = max(0.0, 1 - t.sum()) if tail else 0.0
            tol = np.abs(w[r]) / T * (2 * s * rel + listed * rel_t + share * (tr * rel + rel_t))
            want = want_g * w[r]
            near("grad", grad[r], want, tol + (half + 2.0 ** -23) * np.abs(want) + tiny, r)


def check(logits, token, value, weight=None, T=1.0, tail=True):
    """Loss alone, loss and gradient, gradient from the statistics, in place."""
    x, tok, val, w = put(logits), put(token), put(value), put(weight)
    one = sv.distill_loss(x, tok, val, weight=w, temperature=T, tail=tail)
    both = sv.distill_loss(x, tok, val, weight=w, temperature=T, tail=tail, grad=True)
    later, st = sv.distill_grad(x, tok, val, one["stat"], weight=w, temperature=T, tail=tail)
    torch.cuda.synchronize()
    f = lambda t: t.float().cpu().numpy()  # noqa: E731
    compare(logits, token, value, weight, T, tail, f(one["loss"]), None, one["status"].cpu().numpy())
    compare(logits, token, value, weight, T, tail, f(both["loss"]), f(both["grad"]), both["status"].cpu().numpy())
    compare(logits, token, value, weight, T, tail, f(one["loss"]), f(later), st.cpu().numpy())
    x2, x3 = put(logits), put(logits)
    a = sv.distill_loss(x2, tok, val, weight=w, temperature=T, tail=tail, out_grad=x2)
    b, _ = sv.distill_grad(x3, tok, val, one["stat"], weight=w, temperature=T, tail=tail, out_grad=x3)
    torch.cuda.synchronize()
    assert a["grad"] is x2 and torch.equal(a["loss"], both["loss"]) or bool(a["loss"].isnan().any())
    assert torch.equal(x2, both["grad"]) and torch.equal(x3, later)
    return both


@pytest.mark.parametrize("tail", [True, False])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R,V,K,pad", [
    (1, 1, 1, 0),
    (2, 7, 7, 0),            # the whole vocabulary listed
    (3, 7, 3, 0),
    (2, 129, 128, 1),
    (5, 1000, 8, 0),
    (3, 1001, 5, 0),         # rows off the 16-byte grid
    (2, 8192, 20, 8),
    (3, 32000, 64, 0),
    (2, 40001, 100, 63),
    (2, 128256, 64, 0),
])
def test_matches_the_definition(R, V, K, pad, dtype, tail):
    logits, token, value = make(R, V, K, dtype, R * V + K, pad)
    check(logits, token, value, tail=tail)


@pytest.mark.parametrize("T", [0.3, 2.5])
@pytest.mark.parametrize("tail", [True, False])
def test_temperature_and_weights(T, tail):
    logits, token, value = make(4, 5003, 16, torch.float32, 7, T=T)
    weight = torch.tensor([1.0, 0.0, -2.5, 1e-3])
    check(logits, token, value, weight, T, tail)


@pytest.mark.parametrize("R", [700, 2500])
def test_many_rows(R):
    """Fewer CTAs to a row, for the loss alone and for the gradient."""
    V, K = 33001, 12
    g = torch.Generator(device=DEV).manual_seed(R)
    x = (torch.randn(R, V, generator=g, device=DEV) * 3).to(torch.bfloat16)
    lt = torch.log_softmax(x.double() + torch.randn(R, V, generator=g, device=DEV), -1).topk(K, -1)
    tok, val = lt.indices.to(torch.int32), lt.values.float()
    lp = torch.log_softmax(x.double(), -1)
    t = val.double().exp()
    rest = lp.scatter(1, tok.long(), -math.inf)
    lsr = torch.logsumexp(rest, 1)
    tr = 1 - t.sum(1)
    loss = (t * (val.double() - lp.gather(1, tok.long()))).sum(1) + tr * (tr.log() - lsr)
    grad = (rest - lsr[:, None]).exp() * (lsr.exp() - tr)[:, None]
    grad.scatter_(1, tok.long(), lp.gather(1, tok.long()).exp() - t)
    one = sv.distill_loss(x, tok, val)
    both = sv.distill_loss(x, tok, val, grad=True)
    later, _ = sv.distill_grad(x, tok, val, one["stat"])
    for r in (one, both):
        assert float((r["loss"] - loss).abs().max()) <= 1e-4
        assert int(r["status"].count_nonzero()) == 0
    for got in (both["grad"], later):
        # a bf16 step of each and what 32 bits lose of numbers up to 1
        assert float(((got.double() - grad).abs() - 2.0 ** -8 * grad.abs()).max()) <= 1e-4


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [130, 5003, 20011, 70001])
def test_many_rows_with_faults_and_short_lists(V, dtype):
    """More rows than clusters run at once, each CTA going from row to row: rows
    without a list, faulty ones and ordinary ones after each other."""
    R, K = 1000 if V < 6000 else 950, 128 if V < 6000 else 33
    g = torch.Generator(device=DEV).manual_seed(V)
    x = (torch.randn(R, V, generator=g, device=DEV) * 3).to(dtype)
    top = torch.log_softmax(x.double() + torch.randn(R, V, generator=g, device=DEV), -1).topk(K, -1)
    token, value = top.indices.to(torch.int32), top.values.float()
    r = torch.arange(R, device=DEV)
    token[r % 7 == 1, 5:] = -1
    token[r % 11 == 2] = -1
    token[r % 13 == 3, 1] = token[r % 13 == 3, 4]
    token[r % 17 == 4, 2] = V
    x[r % 19 == 5, V // 2] = math.nan
    value[r % 23 == 6, 3] = math.inf
    x[r % 29 == 7, V // 3:] = -math.inf
    weight = torch.rand(R, generator=g, device=DEV) + 0.5
    for tail in (True, False):
        both = sv.distill_loss(x, token, value, weight=weight, tail=tail, grad=True)
        at = x.clone()
        again = sv.distill_loss(at, token, value, weight=weight, tail=tail, out_grad=at)
        assert torch.equal(at, both["grad"]) and torch.equal(again["status"], both["status"])
        some = torch.cat([torch.arange(0, 60), torch.arange(R - 60, R)])
        f = lambda t: t[some.to(DEV)].float().cpu().numpy()  # noqa: E731
        compare(x.cpu()[some], token.cpu()[some], value.cpu()[some], weight.cpu()[some], 1.0, tail, f(both["loss"]),
                f(both["grad"]), both["status"].cpu().numpy()[some])
        few = sv.distill_loss(x[:100].contiguous(), token[:100], value[:100], weight=weight[:100], tail=tail, grad=True)
        assert torch.equal(few["status"], both["status"][:100])
        ok = few["loss"].isfinite()
        assert float((few["loss"] - both["loss"][:100])[ok].abs().max()) <= 1e-4


def test_slices_beyond_shared_memory():
    """Rows so long that the gradient reads them a second time."""
    for V, dtype in ((1 << 21, torch.float32), (sv.SV_MAX_VOCAB, torch.bfloat16), (900001, torch.float32)):
        K = 128
        g = torch.Generator(device=DEV).manual_seed(V % 1000)
        x = (torch.randn(2, V, generator=g, device=DEV) * 2).to(dtype)
        lt = torch.log_softmax(x.double() + torch.randn(2, V, generator=g, device=DEV), -1).topk(K, -1)
        tok, val = lt.indices.to(torch.int32), lt.values.float()
        both = sv.distill_loss(x, tok, val, grad=True)
        one = sv.distill_loss(x, tok, val)
        later, _ = sv.distill_grad(x, tok, val, one["stat"])
        compare(x.cpu(), tok.cpu(), val.cpu(), None, 1.0, True, both["loss"].cpu().numpy(),
                both["grad"].float().cpu().numpy(), both["status"].cpu().numpy())
        assert float((one["loss"] - both["loss"]).abs().max()) <= 1e-4
        # both read the same statistics but for how the sums were split
        assert float((later.double() - both["grad"].double()).abs().max()) <= 2.0 ** -7
        at = x.clone()
        sv.distill_loss(at, tok, val, out_grad=at)
        assert torch.equal(at, both["grad"])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [40, 9001, 128256])
def test_masked_and_extreme_rows(V, dtype):
    lowest = torch.finfo(dtype).min
    R, K = 14, 6
    logits, token, value = make(R, V, K, dtype, V)
    x = logits.clone()
    x[0, token[0, 0]] = -math.inf            # a token the teacher wants and the student excludes: +inf
    x[1] = -math.inf                         # a fault
    x[2] = lowest                            # uniform
    x[3, V // 2] = math.nan
    x[4, int(token[4, 1])] = math.inf
    keep = x[5, token[5].long()].clone()
    x[5] = -math.inf                         # nothing but the list: the rest has no mass
    x[5, token[5].long()] = keep
    x[6] = -50.0                             # a student sure of its list, the rest far below
    x[6, token[6].long()] = 50.0
    x[7, V // 2:] = -math.inf
    token[7] = torch.arange(K)
    value[8, 3:] = -math.inf                 # weights of 0
    token[9, 2:] = -1                        # a short list
    value[9, 2:] = math.nan                  # of unused entries nothing is looked at
    token[10] = -1                           # no list
    value[11] = torch.tensor([-1e-7] + [-17.0] * 5)    # a teacher who is almost sure
    value[12] = torch.tensor([0.0] + [-math.inf] * 5)  # one who is sure
    x[13] = torch.finfo(dtype).max
    check(x, token, value)
    check(x, token, value, tail=False)


def test_faults_of_the_teacher():
    logits, token, value = make(9, 3001, 4, torch.float32, 1)
    token[0, 1] = 3001
    token[1, 2] = -2
    token[2, 3] = token[2, 0]                 # listed twice
    value[3, 0] = math.nan
    value[4, 1] = math.inf
    value[5] = -0.5                           # adds up to 2.4
    value[6] = -math.inf
    token[7, 0], token[7, 1] = 3000, 0        # the row's ends
    token[8, :2] = token[8, 2]                # three times
    got = check(logits, token, value)
    assert got["status"].tolist() == [2, 2, 2, 1, 1, 1, 0, 0, 2]
    got = check(logits, token, value, tail=False)
    assert got["status"].tolist() == [2, 2, 2, 1, 1, 0, 1, 0, 2]


@pytest.mark.parametrize("V", [37, 1001])
@pytest.mark.parametrize("dtype", TYPES)
def test_listed_twice_anywhere(V, dtype):
    """The same token at every place of the row: before the first 16-byte border,
    in a piece, behind the last."""
    logits, _, _ = make(1, V, 2, dtype, 3)
    x = logits.expand(V, V).contiguous()
    token = torch.arange(V, dtype=torch.int32)[:, None].expand(V, 2).contiguous()
    value = torch.full((V, 2), -1.0)
    r = sv.distill_loss(put(x), put(token), put(value), grad=True)
    assert bool((r["status"] == 2).all()) and bool(r["loss"].isnan().all()) and not bool(r["grad"].any())


@pytest.mark.parametrize("dtype", TYPES)
def test_gradient_rows_elsewhere(dtype):
    """Rows of the gradient off the logits' place on the 16-byte grid; what lies
    between them stays."""
    logits, token, value = make(4, 5001, 9, dtype, 5, pad=3)
    x, tok, val = put(logits), put(token), put(value)
    want = sv.distill_loss(x, tok, val, grad=True)["grad"]
    stat = sv.distill_loss(x, tok, val)["stat"]
    later, _ = sv.distill_grad(x, tok, val, stat)
    for pad, at in ((0, 0), (1, 1), (7, 3), (3, 8)):
        buf = torch.full((4 * (5001 + pad) + at,), 77.0, dtype=dtype, device=DEV)
        out = buf[at:].view(4, 5001 + pad)[:, :5001]
        sv.distill_loss(x, tok, val, out_grad=out)
        assert torch.equal(out, want)
        if pad:
            assert bool((buf[at:].view(4, 5001 + pad)[:, 5001:] == 77).all())
        sv.distill_grad(x, tok, val, stat, out_grad=out)
        assert torch.equal(out, later)


@pytest.mark.parametrize("tail", [True, False])
def test_gradient_against_differences(tail):
    """Central differences of the loss, per element: the loss is off by d = 1e-5 at
    most here (V = 200, logs below 12), a step of h = 0.1 by h^2 / 6 of third
    derivatives, which are below 1."""
    V, K, h = 200, 10, 0.1
    logits, token, value = make(1, V, K, torch.float32, 11, T=0.8)
    grad = sv.distill_loss(put(logits), put(token), put(value), temperature=0.8, tail=tail, grad=True)["grad"]
    step = torch.eye(V) * h
    rows = torch.cat([logits + step, logits - step])
    loss = sv.distill_loss(put(rows), put(token.expand(2 * V, K).contiguous()),
                           put(value.expand(2 * V, K).contiguous()), temperature=0.8, tail=tail)["loss"].double()
    diff = (loss[:V] - loss[V:]) / (2 * h)
    assert float((diff - grad[0].double()).abs().max()) <= 1e-5 / h + h * h / 6 / 0.8 ** 3


def test_autograd_graph_takes_the_gradient():
    """The gradient of a draft's output layer through torch, from the row
    gradients, against torch's own of the same loss in 64 bits."""
    g = torch.Generator(device=DEV).manual_seed(2)
    V, D, R, K = 3001, 32, 24, 16
    h = torch.randn(R, D, generator=g, device=DEV)
    W = (torch.randn(V, D, generator=g, device=DEV) * 0.3).requires_grad_()
    teacher = torch.randn(1, R, V, generator=g, device=DEV) * 2
    t = sv.token_logprobs(teacher, top_k=K)
    tok, val = t["top_token"][0], t["top_logprob"][0]
    x = h @ W.t()
    r = sv.distill_loss(x.detach(), tok, val, weight=torch.full((R,), 1.0 / R, device=DEV), grad=True)
    x.backward(r["grad"])
    W2 = W.detach().double().requires_grad_()
    lp = torch.log_softmax(h.double() @ W2.t(), -1)
    tt = val.double().exp()
    tr = (1 - tt.sum(1)).clamp(min=1e-300)
    lsr = torch.logsumexp(lp.scatter(1, tok.long(), -math.inf), 1)
    loss = ((tt * (val.double() - lp.gather(1, tok.long()))).sum(1) + tr * (tr.log() - lsr)).mean()
    loss.backward()
    assert abs(float(r["loss"].mean()) - float(loss)) <= 1e-4
    # 2^-10: the products run in fp32, or less where torch is told so
    assert float((W.grad.double() - W2.grad).abs().max()) <= 2.0 ** -10 * float(W2.grad.abs().max())


def test_streams_capture_and_two_calls_at_once():
    logits, token, value = make(40, 32000, 20, torch.bfloat16, 6)
    x, tok, val = put(logits), put(token), put(value)
    want = sv.distill_loss(x, tok, val, grad=True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [sv.distill_loss(x, tok, val, grad=True, stream=s) for _ in range(4) for s in streams]
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(r[k], want[k]) for k in want)
    static = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = sv.distill_loss(static, tok, val, grad=True)
        later, st = sv.distill_grad(static, tok, val, r["stat"])
    for seed in (7, 8):
        static.copy_(make(40, 32000, 20, torch.bfloat16, seed)[0])
        graph.replay()
        want = sv.distill_loss(static, tok, val, grad=True)
        torch.cuda.synchronize()
        assert all(torch.equal(r[k], want[k]) for k in want)
        # the same statistics: equal gradients
        assert torch.equal(later, want["grad"]) and not bool(st.any())
    host = sv.distill_loss(static.cpu().pin_memory(), tok, val, grad=True)
    torch.cuda.synchronize()
    assert all(torch.equal(host[k].to(DEV), want[k]) for k in want)


@pytest.mark.parametrize("V,dtype", [(1 << 20, torch.float32), (1 << 22, torch.float32), (1 << 21, torch.bfloat16)])
def test_many_rows_of_large_vocabularies(V, dtype):
    """More rows than the card has CTAs, all of them one row of memory: the same loss
    as alone, but for the order of its sums (`rel` of compare, for each of them)."""
    logits, token, value = make(1, V, 100, dtype, 4)
    x, tok, val = put(logits), put(token), put(value)
    alone = sv.distill_loss(x, tok, val)
    R = 1300
    many = sv.distill_loss(x.expand(R, V), tok.expand(R, -1).contiguous(), val.expand(R, -1).contiguous())
    torch.cuda.synchronize()
    f = lambda t: t.float().cpu().numpy()  # noqa: E731
    compare(logits, token, value, None, 1.0, True, f(alone["loss"]), None, alone["status"].cpu().numpy())
    compare(logits, token, value, None, 1.0, True, f(many["loss"][:1]), None, many["status"][:1].cpu().numpy())
    assert torch.equal(many["loss"], many["loss"][:1].expand(R)) and not bool(many["status"].any())
