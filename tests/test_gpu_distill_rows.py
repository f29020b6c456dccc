"""Faulty, listless and ordinary rows in one batch, each held to its own answer; the
later gradient of the longest rows element by element."""
import math

import pytest
import torch

import test_gpu_distill as distill
from test_gpu_distill_mass import calls

pytestmark = pytest.mark.gpu

sv = pytest.importorskip("speculative_decoding_verification_vocab_gb300")
DEV = "cuda:0"
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.load_library()


@pytest.mark.parametrize("tail", [True, False])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R,V,K", [(1000, 130, 128), (20, 5003, 16), (600, 70001, 8)])
def test_every_row_has_its_own_answer(R, V, K, dtype, tail):
    """By every way (and the same ones in place): NaN and a gradient of zeros exactly
    where the status is not 0, zeros exactly where there is no list."""
    g = torch.Generator(device=DEV).manual_seed(R)
    x = (torch.randn(R, V, generator=g, device=DEV) * 3).to(dtype)
    top = torch.log_softmax(x.double() + torch.randn(R, V, generator=g, device=DEV), -1).topk(K, -1)
    token, value = top.indices.to(torch.int32), top.values.float()
    r = torch.arange(R, device=DEV)
    token[r % 5 == 1] = -1                                # no list
    token[r % 7 == 2, 1] = token[r % 7 == 2, 4]           # listed twice, or an entry not used
    x[r % 9 == 3, V - 1] = math.nan
    value[r % 11 == 4, 2] = math.nan
    token[r % 13 == 6, 0] = V
    listless = (token == -1).all(1)
    twice = token.sort(1).values
    twice = ((twice[:, 1:] == twice[:, :-1]) & (twice[:, 1:] != -1)).any(1)
    want = torch.zeros(R, dtype=torch.int32, device=DEV)
    want[x.isnan().any(1) | (value.isnan() & (token != -1)).any(1)] |= sv.SV_ROW_NAN
    want[twice | (token == V).any(1)] |= sv.SV_ROW_BAD_TOKEN
    want[listless] = 0
    assert 0 < int(listless.sum()) < R and 0 < int((want != 0).sum()) < R
    ways = list(calls(x, token, value, tail=tail))
    for loss, grad, status in ways:
        assert torch.equal(status, want)
        assert torch.equal(loss.isnan(), want != 0)
        assert bool((loss[listless] == 0).all()) and bool((loss[(want == 0) & ~listless] != 0).all())
        assert torch.equal(grad.any(1), (want == 0) & ~listless)
    # an ordinary row is not another's neighbour: alone it is what it is in the batch, but
    # for the order of its sums (a clone: where a row lies on the 16-byte grid is part of
    # that order)
    rel = 2.0 ** -24 * (3 * 48 + 4 + V / 512 + 24 + 8 + K)
    at = int(((want == 0) & ~listless).nonzero()[-1])
    alone = list(calls(x[at:at + 1].clone(), token[at:at + 1], value[at:at + 1], tail=tail))
    for (loss, grad, _), (one, g1, _) in zip(ways, alone):
        assert abs(float(loss[at] - one[0])) <= 4 * rel * 40
        off = (grad[at].double() - g1[0].double()).abs()
        assert bool((off <= 4 * rel + torch.finfo(dtype).eps * g1[0].double().abs()).all())


@pytest.mark.parametrize("tail", [True, False])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [3, 130, 9001, 128256])
def test_a_fault_wherever_it_stands(V, dtype, tail):
    """NaN or +inf at a listed token, at all of them, beside them, beside a list of
    logits of -inf: the row is faulty.  -inf alone is no fault."""
    g = torch.Generator(device=DEV).manual_seed(V)
    for K in (1, 2, min(V, 40)):
        R = 8
        x = (torch.randn(R, V, generator=g, device=DEV) * 2).to(dtype)
        token = torch.rand(R, V, generator=g, device=DEV).argsort(1)[:, :K].to(torch.int32)
        value = torch.log_softmax(torch.randn(R, K, generator=g, device=DEV), 1) - (0.1 if K < V else 0.0)
        at = token.long()
        x[0].scatter_(0, at[0, -1:], math.nan)
        x[1].scatter_(0, at[1], math.nan)
        x[2].scatter_(0, at[2, :1], math.inf)
        x[3].scatter_(0, at[3], math.inf)
        x[4].scatter_(0, at[4], -math.inf)
        if K < V:
            other = torch.tensor([sorted(set(range(V)) - set(row.tolist()))[-1] for row in at.cpu()], device=DEV)
            x[4, other[4]] = math.nan
            x[5, other[5]] = math.nan
            x[6].scatter_(0, at[6], -math.inf)
        faulty = [0, 1, 2, 3, 4, 5] if K < V else [0, 1, 2, 3, 4]
        for loss, grad, status in calls(x, token, value, tail=tail):
            assert status.tolist() == [sv.SV_ROW_NAN if r in faulty else 0 for r in range(R)]
            assert bool(loss[faulty].isnan().all()) and not bool(grad[faulty].any())
            assert not bool(loss.isnan()[[6, 7]].any()) and not bool(grad.isnan().any())
            assert math.isinf(float(loss[6])) == (K < V)


@pytest.mark.parametrize("V,dtype", [(1 << 21, torch.float32), (sv.SV_MAX_VOCAB, torch.bfloat16), (900001, torch.float16)])
def test_later_gradient_of_the_longest_rows(V, dtype):
    K = 128
    g = torch.Generator(device=DEV).manual_seed(V % 1000)
    x = (torch.randn(2, V, generator=g, device=DEV) * 2).to(dtype)
    top = torch.log_softmax(x.double() + torch.randn(2, V, generator=g, device=DEV), -1).topk(K, -1)
    token, value = top.indices.to(torch.int32), top.values.float()
    weight = torch.tensor([1000.0, -3.0])                 # (fp16 begins at 6e-8)
    one = sv.distill_loss(x, token, value, weight=weight.to(DEV))
    later, status = sv.distill_grad(x, token, value, one["stat"], weight=weight.to(DEV))
    torch.cuda.synchronize()
    distill.compare(x.cpu(), token.cpu(), value.cpu(), weight, 1.0, True, one["loss"].cpu().numpy(),
                    later.float().cpu().numpy(), status.cpu().numpy())
    # some of its elements are far above what compare allows beside them
    assert float(later.float().abs().max()) > 2.0 ** -7
