"""The target's operators as a serving and training program runs them: candidates
of a few prompts decode behind their shared prefixes, a round of verification
answers with tokens and their log probabilities, and the alternatives train the
draft.  Each step is held against its plain definition on the very numbers that
the step before left; then the whole is captured and replayed."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import test_gpu_distill as distill
import test_gpu_prefix_attention as prefix
import test_gpu_token_logprobs as logprobs

pytestmark = pytest.mark.gpu

sv = pytest.importorskip("speculative_decoding_verification_vocab_gb300")
DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.load_library()


class Target:
    """One attention layer and a vocabulary: B = N W sequences, a cache of pages of
    16, room for `steps` tokens behind the first `own` of each sequence's own."""
    def __init__(self, seed, plens=(700, 45), W=3, Hq=8, Hkv=2, D=64, V=4099, steps=4, own=13, K=12):
        g = torch.Generator().manual_seed(seed)
        N, B, page = len(plens), len(plens) * W, 16
        q, kv, pt, pl, t, n = prefix.make(list(plens), [own + steps] * B, Hq, Hkv, D, page, seed=seed)
        self.shape, self.K = (B, N, Hq, Hkv, D, V, steps, page), K
        # the newest slots are written as they are decoded
        self.new = torch.randn(steps, 2, B, Hkv, D, generator=g).to(torch.bfloat16)
        for i in range(steps):
            at = own + i
            kv[:, t[:, at // page].long(), at % page] = float("nan")
        self.q = torch.randn(steps, B, Hq, D, generator=g).to(torch.bfloat16).to(DEV)
        head = torch.randn(Hq * D, V, generator=g) * 2
        self.cpu = (kv, pt, pl, t)
        self.kv, self.pt, self.pl, self.t = (x.to(DEV) for x in self.cpu)
        self.head = head.to(DEV)
        self.newd, self.own = self.new.to(DEV), own
        self.slots = [(self.t[:, (own + i) // page].long(), (own + i) % page) for i in range(steps)]
        self.lens = [torch.full((B,), own + i + 1, dtype=torch.int32, device=DEV) for i in range(steps)]
        self.ws = torch.empty(sv.sv_prefix_attention_workspace(B, N, Hq, Hkv, D, page, pt.shape[1], t.shape[1]),
                              dtype=torch.uint8, device=DEV)
        self.dlogits = (torch.randn(B, steps - 1, V, generator=g) * 2).to(torch.bfloat16).to(DEV)
        self.drafts = torch.randint(0, V, (B, steps - 1), generator=g, dtype=torch.int32).to(DEV)
        self.weight = torch.rand(B * (steps - 1), generator=g).to(DEV)

    def run(self):
        B, N, Hq, Hkv, D, V, steps, page = self.shape
        att, rows = [], []
        for i in range(steps):
            page_of, at = self.slots[i]
            self.kv[:, page_of, at] = self.newd[i]
            att.append(sv.prefix_attention(self.q[i], self.kv, self.pt, self.pl, self.t, self.lens[i], return_lse=True,
                                           workspace=self.ws))
            rows.append((att[-1][0].view(B, Hq * D, 1).float() * self.head).sum(1).to(torch.bfloat16))
        logits = torch.stack(rows, 1)                                        # [B][steps][V]
        told = sv.verify_chain(logits, self.dlogits, self.drafts, seed=3, step=1)
        said = sv.token_logprobs(logits, told["tokens"], top_k=self.K)
        # the draft's positions 0 .. steps - 2, the round's emitted ones; an entry that is
        # not asked for comes with -1 for its tokens, and has neither loss nor gradient
        R = B * (steps - 1)
        x = self.dlogits.view(R, V)
        token = said["top_token"][:, :steps - 1].reshape(R, self.K)
        value = said["top_logprob"][:, :steps - 1].reshape(R, self.K)
        lost = sv.distill_loss(x, token, value, weight=self.weight, grad=True)
        alone = sv.distill_loss(x, token, value, weight=self.weight)
        later, st = sv.distill_grad(x, token, value, alone["stat"], weight=self.weight)
        return dict(logits=logits, tokens=told["tokens"], x=x, token=token, value=value, later=later, later_status=st,
                    att=torch.stack([a[0] for a in att]), lse=torch.stack([a[1] for a in att]),
                    att_status=torch.stack([a[2] for a in att]), **{"said_" + k: v for k, v in said.items()},
                    **{"lost_" + k: v for k, v in lost.items()})


def same(a, b):
    return all(torch.equal(a[k].nan_to_num(7.0), b[k].nan_to_num(7.0)) if a[k].is_floating_point()
               else torch.equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("seed", [0, 1])
def test_candidates_to_training(seed):
    target = Target(seed)
    B, N, Hq, Hkv, D, V, steps, page = target.shape
    got = target.run()
    torch.cuda.synchronize()
    kv, pt, pl, t = target.cpu
    for i in range(steps):
        at = target.own + i
        kv[:, t[:, at // page].long(), at % page] = target.new[i]
        prefix.close(got["att"][i], got["lse"][i], got["att_status"][i], target.q[i].cpu(), kv, pt, pl, t,
                     target.lens[i].cpu(), D ** -0.5)
    again = logprobs.check(got["logits"].cpu(), got["tokens"].cpu(), K=target.K)
    assert all(np.array_equal(again[k], got["said_" + k].cpu().numpy()) for k in again)
    f = lambda t: t.float().cpu().numpy()  # noqa: E731
    args = (got["x"].cpu(), got["token"].cpu(), got["value"].cpu(), target.weight.cpu(), 1.0, True)
    distill.compare(*args, f(got["lost_loss"]), f(got["lost_grad"]), got["lost_status"].cpu().numpy())
    distill.compare(*args, f(got["lost_loss"]), f(got["later"]), got["later_status"].cpu().numpy())
    ended = (got["tokens"][:, :steps - 1].reshape(-1) == -1).cpu()
    assert bool(ended.any()) and not bool(ended.all())        # rounds that stop before the last draft
    assert bool((got["lost_loss"].cpu()[ended] == 0).all()) and not bool(got["lost_grad"].cpu()[ended].any())
    # captured and replayed, twice, on new inputs
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = target.run()
    for s in (seed + 10, seed + 20):
        other = Target(s)
        for name in ("q", "head", "dlogits", "drafts", "weight", "newd"):
            getattr(target, name).copy_(getattr(other, name))
        graph.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in out.items()}
        want = target.run()
        torch.cuda.synchronize()
        assert same(got, want)


def test_two_graphs_with_workspaces_of_their_own():
    """Two captured rounds replayed at once, on two streams."""
    targets = [Target(5), Target(6, plens=(90, 1400, 3), W=2)]
    graphs, outs, wants = [], [], []
    for target in targets:
        target.run()
        torch.cuda.synchronize()
        wants.append({k: v.clone() for k, v in target.run().items()})
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            outs.append(target.run())
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert all(same(o, w) for o, w in zip(outs, wants))


PROGRAM = """
import sys
sys.path.insert(0, {root!r})
import torch
import speculative_decoding_verification_vocab_gb300 as sv
g = torch.Generator(device="cuda").manual_seed(1)
N, W, Hq, Hkv, D, page, n, V = 2, 3, 8, 2, 128, 16, {n}, {V}
B, per, own = N * W, -(-n // 16), 4
i32 = dict(dtype=torch.int32, device="cuda")
kv = torch.randn(2, N * per + B * own, page, Hkv, D, generator=g, device="cuda").to(torch.bfloat16)
pt = torch.arange(N * per, **i32).view(N, per)
t = torch.arange(N * per, N * per + B * own, **i32).view(B, own)
pl, lens = torch.full((N,), n, **i32), torch.arange(B, **i32) * 9
q = torch.randn(B, Hq, D, generator=g, device="cuda").to(torch.bfloat16)
x = (torch.randn(B, 1, V, generator=g, device="cuda") * 3).to(torch.bfloat16)
y = (torch.randn(B, V, generator=g, device="cuda") * 3).to(torch.bfloat16)
tok = torch.randint(0, V, (B, 1), generator=g, **i32)

def run():
    out = sv.prefix_attention(q, kv, pt, pl, t, lens, return_lse=True)
    r = sv.token_logprobs(x, tok, top_k=20)
    a = sv.distill_loss(y, r["top_token"][:, 0], r["top_logprob"][:, 0], grad=True)
    b = sv.distill_loss(y, r["top_token"][:, 0], r["top_logprob"][:, 0], tail=False)
    c = sv.distill_grad(y, r["top_token"][:, 0], r["top_logprob"][:, 0], b["stat"], tail=False)
    return [*out, *r.values(), *a.values(), *b.values(), *c]

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in got]
want = run()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want))
print("same")
"""


@pytest.mark.parametrize("n,V", [(40, 1000), (9000, 128256)])
def test_first_call_inside_a_capture(n, V):
    r = subprocess.run([sys.executable, "-c", PROGRAM.format(root=ROOT, n=n, V=V)], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]
